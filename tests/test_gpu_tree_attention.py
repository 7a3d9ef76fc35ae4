"""GPU tests of tree attention over the paged cache against the plain fp64 definition.

Tolerances (derived, per element; as for one-token attention): with w = sum_j p_j |v_j|, a
weight kept to 16 bits is off by up to 2^-17 of itself and the bf16 output rounded by up to 2^-8 of |o| <= w.  Sums over the keys run
on the matrix instructions, which cut each step off: up to 2^-23 of w for every 16 keys of a
part, and a part has at most 4096 of these tests' keys: 2^-15.  Scores are fp32
sums of exact products in steps of at least 8 terms: off by (D / 8 + 8) 2^-23 of
S = max_j scale sum_d |q_d k_jd|, and ex2 and the sums by some 2^-21; a score's error reaches a
weight and the normalisation, so twice.  lse carries the score error once.
"""
import numpy as np
import pytest
import torch

from oracle import paged, tree
from parity_utils import DEV, f64
from test_gpu_paged import as_device, make_cache

pytestmark = pytest.mark.gpu


def signed(words):
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64)


def random_tree(n, rng, chain=False):
    return tree.words([-1] + [i - 1 if chain or rng.random() < 0.5 else int(rng.integers(-1, i))
                              for i in range(1, n)]) if n else []


def tree_case(shapes, H, G, D, page, cache="bf16", order="token", seed=0, peak=1.0, words=None):
    """shapes: (nodes, keys before them) of every request."""
    gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    lens = [n + c for n, c in shapes]
    held = [paged.pages(x, page) for x in lens]
    num_pages = sum(held) + 3
    perm = torch.randperm(num_pages, generator=gen)
    table = torch.full((len(shapes), max(held + [1]) + 1), 2 ** 30, dtype=torch.int32)  # never read
    k, v = make_cache(num_pages, page, H, D, cache, order, gen)
    at = 0
    for b, x in enumerate(lens):
        table[b, :held[b]] = perm[at:at + held[b]].to(torch.int32)
        for i in range(held[b]):
            m = min(page, x - i * page)
            for t in (k, v):
                y = torch.randn(m, H, D, generator=gen) * (40.0 if cache == "fp8" else 1.0)
                t[int(perm[at + i]), :m] = y.to(t.dtype)
        at += held[b]
    cu = np.concatenate([[0], np.cumsum([n for n, _ in shapes])]).astype(np.int64)
    if words is None:
        words = [w for n, _ in shapes for w in random_tree(n, rng)]
    q = (torch.randn(int(cu[-1]), H * G, D, generator=gen) * peak).to(torch.bfloat16)
    scales = (None, None)
    if cache == "fp8":
        scales = tuple(torch.rand(H, generator=gen) * 0.03 + 0.01 for _ in range(2))
    return dict(q=q, k=k, v=v, table=table, lens=torch.tensor(lens, dtype=torch.int32), cu=cu,
                words=words, scales=scales, scale=D ** -0.5, D=D,
                most=max([n for n, _ in shapes] + [1]))


def on_device(lib, x):
    ks, vs = (None if s is None else s.to(DEV) for s in x["scales"])
    cache = lib.PagedCache(as_device(x["k"]), as_device(x["v"]), ks, vs)
    return cache, (x["table"].to(DEV), x["lens"].to(DEV),
                   torch.tensor(x["cu"], dtype=torch.int32, device=DEV), signed(x["words"]).to(DEV))


def run(lib, x, **kw):
    cache, args = on_device(lib, x)
    return lib.paged_tree_decode(x["q"].to(DEV), cache, *args, x["most"], x["scale"], want_lse=True, **kw)


def expected(x, **kw):
    ks, vs = (None if s is None else s.numpy() for s in x["scales"])
    a = dict(q=f64(x["q"]), k_cache=x["k"].float().double().numpy(),
             v_cache=x["v"].float().double().numpy(), table=x["table"].numpy(),
             seq_lens=x["lens"].numpy(), cu=x["cu"], words_=x["words"], scale=x["scale"], k_scale=ks,
             v_scale=vs)
    a.update(kw)
    return tree.attend(**a)


def check(x, o, lse, ref=None):
    o_ref, lse_ref, w, spread = expected(x) if ref is None else ref
    es = (x["D"] / 8 + 8) * 2.0 ** -23 * spread + 2.0 ** -21
    err = np.abs(f64(o) - o_ref)
    tol = (2.0 ** -8 + 2.0 ** -17 + 2.0 ** -15 + 2 * es[..., None]) * w
    assert np.isfinite(f64(o)).all()
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()
    got, none = f64(lse), np.isneginf(lse_ref)
    assert np.isneginf(got[none]).all()
    assert (np.abs(got[~none] - lse_ref[~none])
            <= es[~none] + 2.0 ** -22 * np.abs(lse_ref[~none])).all()


SHAPES = [(1, 0), (0, 5), (3, 61), (64, 0), (17, 111), (5, 127), (1, 128), (33, 300), (64, 1), (2, 255)]


@pytest.mark.parametrize("cache,order", [("bf16", "token"), ("bf16", "head"), ("fp8", "token"),
                                         ("fp8", "head")])
@pytest.mark.parametrize("H,G,D,page", [(2, 4, 128, 16), (1, 1, 64, 24), (2, 12, 128, 64), (1, 3, 64, 1),
                                        (1, 6, 256, 7), (2, 2, 256, 128), (1, 24, 64, 33)])
def test_trees(lib, H, G, D, page, cache, order):
    x = tree_case(SHAPES, H, G, D, page, cache, order, seed=H * 100 + G)
    o, lse = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    check(x, o, lse)


@pytest.mark.parametrize("shapes", [[(7, 9000)], [(1, 4000), (12, 0), (64, 5000)], [(3, 700)] * 9,
                                    [(0, 0), (2, 3)], [(16, 1000), (40, 1)]])
@pytest.mark.parametrize("cache,D,G", [("bf16", 128, 8), ("fp8", 128, 4), ("bf16", 64, 1),
                                       ("bf16", 256, 3), ("fp8", 256, 2), ("fp8", 64, 9)])
def test_long(lib, shapes, cache, D, G):
    """Lengths that are split over many blocks and joined."""
    x = tree_case(shapes, 2, G, D, 64, cache, seed=len(shapes), peak=3.0)
    o, lse = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    check(x, o, lse)


@pytest.mark.parametrize("cache,D,H,G,shapes", [("bf16", 128, 8, 2, [(3, 30000), (1, 9000)]),
                                                ("fp8", 128, 6, 3, [(2, 41003)]),
                                                ("bf16", 64, 8, 1, [(4, 35000)]),
                                                ("bf16", 256, 5, 2, [(2, 25000), (3, 1)]),
                                                ("bf16", 128, 2, 48, [(3, 40000)]),
                                                ("fp8", 64, 2, 70, [(2, 60000)])])
def test_many_tiles_of_a_block(lib, cache, D, H, G, shapes):
    """Pieces of many tiles, whose references grow on the way: the last keys score highest.  (A
    part has at most 1500 keys.)"""
    x = tree_case(shapes, H, G, D, 64, cache, seed=D + G, peak=2.0)
    for b in range(len(shapes)):                           # keys grow towards the end
        n = int(x["lens"][b])
        for i in range(paged.pages(n, 64)):
            p = int(x["table"][b, i])
            up = 0.2 + 2.0 * i * 64 / n
            x["k"][p] = (x["k"][p].float() * up).to(x["k"].dtype)
    o, lse = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    check(x, o, lse)


def test_many_requests(lib):
    """More requests than blocks, of no, one or a few nodes."""
    rng = np.random.default_rng(3)
    shapes = [(int(rng.integers(0, 5)), int(rng.integers(0, 40))) for _ in range(700)]
    x = tree_case(shapes, 1, 2, 64, 16, seed=9)
    o, lse = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    check(x, o, lse)


@pytest.mark.parametrize("D,G,cache", [(128, 4, "bf16"), (128, 2, "fp8"), (64, 16, "bf16"), (256, 1, "bf16")])
def test_words_are_taken_as_they_are(lib, D, G, cache):
    """Any set of drafted keys, none at all among them; bits past the request's nodes mean nothing."""
    rng = np.random.default_rng(D + G)
    shapes = [(9, 0), (64, 0), (31, 200), (64, 63), (2, 0)]
    words = []
    for n, _ in shapes:
        for _ in range(n):
            w = int(rng.integers(0, 2 ** 63)) * 2 + int(rng.integers(0, 2))
            words.append(int(rng.choice([0, w, w & 0xff, 2 ** 64 - 1, 1 << (n - 1)])))
    x = tree_case(shapes, 2, G, D, 24, cache, seed=5, words=words)
    x["words"][0] = x["words"][-1] = 0
    x["words"][1] = 2 ** 64 - (1 << 9)                     # only bits past the nodes
    o, lse = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    ref = expected(x)
    assert np.isneginf(ref[1][0]).all() and np.isneginf(ref[1][1]).all()
    check(x, o, lse, ref)
    assert not o[0].any() and not o[1].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v", "both"])
@pytest.mark.parametrize("D,G", [(128, 4), (64, 12), (256, 2)])
def test_what_a_node_does_not_see_has_no_part(lib, D, G, where, bad):
    """One drafted node's key and value are not finite: the nodes that see it are the only ones
    to be changed."""
    shapes = [(40, 77), (6, 0), (20, 300)]
    x = tree_case(shapes, 2, G, D, 16, seed=4)
    ref = expected(x)
    b, node = 0, 3
    pos = 77 + node
    p, r = int(x["table"][b, pos // 16]), pos % 16
    for name in ("k", "v") if where == "both" else (where,):
        x[name][p, r] = bad
    o, lse = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    sees = np.array([x["words"][i] >> node & 1 if i < 40 else 0 for i in range(66)], bool)
    assert sees.sum() > 1 and (~sees).sum() > 1
    keep = dict(x, q=x["q"][~sees])
    check(keep, o[torch.tensor(~sees)], lse[torch.tensor(~sees)], tuple(t[~sees] for t in ref))
    got, l = f64(o)[sees], f64(lse)[sees]
    if where == "v":                                       # the weights are as they were
        assert (np.isnan(got) if np.isnan(bad) else got == bad).all()
        assert np.abs(l - ref[1][sees]).max() < 1e-4
    elif np.isnan(bad):
        assert np.isnan(got).all() and np.isnan(l).all()
    else:                                                  # a score of +inf, -inf or inf - inf
        assert not np.isinf(got).any() or where == "both"


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_infinite_value_of_the_context(lib, cache):
    """An infinite (NaN in 8 bits) value reaches every output of its channel, no other."""
    x = tree_case([(12, 500)], 1, 4, 128, 16, cache, seed=8)
    p, r = int(x["table"][0, 10]), 3
    val = float("inf") if cache == "bf16" else float("nan")
    ref = expected(x)
    raw = x["v"].float()
    raw[p, r, 0, 5] = val
    x["v"] = raw.to(x["v"].dtype)
    o, lse = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    got = f64(o)
    assert (np.isnan(got[..., 5]) if cache == "fp8" else np.isposinf(got[..., 5])).all()
    o[..., 5] = torch.tensor(ref[0][..., 5]).to(o)
    check(x, o, lse, ref)


def test_large_values_stay_finite(lib):
    """Values near the end of bf16's range: averages of them are finite."""
    x = tree_case([(9, 400)], 2, 4, 64, 16, seed=2)
    x["v"] = torch.where(torch.isnan(x["v"]), x["v"], torch.full_like(x["v"], 3.0e38))
    o, _ = run(lib, x)
    top = float(torch.tensor(3.0e38).to(torch.bfloat16))
    assert (np.abs(f64(o) / top - 1) <= 2.0 ** -8 + 2.0 ** -15).all()


def test_negative_and_zero_scale(lib):
    for scale in (-0.3, 0.0):
        x = dict(tree_case([(10, 200), (3, 0)], 2, 4, 128, 16, seed=6), scale=scale)
        o, lse = run(lib, x)
        check(x, o, lse)


def test_rows_apart_and_rows_behind(lib):
    """q as a slice of a fused projection; rows behind the last request stay as they were."""
    x = tree_case([(5, 90), (11, 30)], 2, 4, 128, 16, seed=11)
    cache, (table, lens, cu, words) = on_device(lib, x)
    N, Hq = 16, 8
    wide = torch.full((N + 3, 3 * Hq * 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:N, 256:256 + Hq * 128] = x["q"].to(DEV).view(N, -1)
    q = wide[:, 256:256 + Hq * 128].view(N + 3, Hq, 128)
    o = torch.full((N + 3, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((N + 3, Hq), 7.0, device=DEV)
    more = torch.cat([words, torch.full((3,), -1, device=DEV)])
    ws = torch.empty(lib.kda_paged_tree_decode_workspace_size(2, 11, Hq, 2, 128), dtype=torch.uint8,
                     device=DEV)
    lib.kda_paged_tree_decode(q, cache, table, lens, cu, more, 11, x["scale"], o, lse, ws)
    assert lib.kda_get_last_device_error() == 0
    check(x, o[:N], lse[:N])
    assert (o[N:] == 7).all() and (lse[N:] == 7).all()
    o2 = torch.full_like(o, 7.0)
    lib.kda_paged_tree_decode(q, cache, table, lens, cu, more, 64, x["scale"], o2, None,
                              torch.empty(lib.kda_paged_tree_decode_workspace_size(2, 64, Hq, 2, 128),
                                          dtype=torch.uint8, device=DEV))
    check(x, o2[:N], lse[:N])


def test_refusals_on_the_device(lib):
    x = tree_case([(4, 50), (6, 20), (3, 10)], 2, 2, 64, 16, seed=1)
    cache, (table, lens, cu, words) = on_device(lib, x)
    ref, q = expected(x), x["q"].to(DEV)
    assert lib.kda_get_last_device_error() == 0

    def call(table=table, lens=lens, cu=cu, most=6):
        o = torch.full((13, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((13, 4), 7.0, device=DEV)
        ws = torch.empty(lib.kda_paged_tree_decode_workspace_size(3, most, 4, 2, 64), dtype=torch.uint8,
                         device=DEV)
        lib.kda_paged_tree_decode(q, cache, table, lens, cu, words, most, x["scale"], o, lse, ws)
        assert lib.kda_get_last_device_error() == 1
        return o, lse

    def good(o, lse, rows):
        at = np.array(rows)
        check(x, o[torch.tensor(at)], lse[torch.tensor(at)], tuple(t[at] for t in ref))
    rest = list(range(4)) + list(range(10, 13))
    for bad in (5, -1, table.shape[1] * 16 + 1, 2 ** 31 - 1):      # a length below the nodes, past the table
        wrong = lens.clone()
        wrong[1] = bad
        o, lse = call(lens=wrong)
        good(o, lse, rest)
        assert not o[4:10].any() and torch.isneginf(lse[4:10]).all()
    o, lse = call(most=5)                                          # more rows than max_nodes
    good(o, lse, rest)
    assert not o[4:10].any() and torch.isneginf(lse[4:10]).all()
    for bad in ([0, 4, 10, 14], [-1, 4, 10, 13], [0, 4, 3, 13]):   # offsets outside, or going back
        o, lse = call(cu=torch.tensor(bad, dtype=torch.int32, device=DEV))
        if bad[3] == 14:
            good(o, lse, range(10))
            assert (o[10:] == 7).all() and (lse[10:] == 7).all()
    for bad in (-1, cache.num_pages, 2 ** 31 - 1, -2 ** 31):       # a page that is not one: its keys are left out
        wrong = table.clone()
        wrong[0, 1] = bad
        o, lse = call(table=wrong)
        good(o, lse, range(4, 13))
        gone = dict(x, k=x["k"].clone())
        seen = [j for j in range(54) if not 16 <= j < 32]
        k, v = (t[x["table"][0, :4].long()].flatten(0, 1)[:54][seen].float().double().numpy()
                for t in (x["k"], x["v"]))
        pad = paged.pages(len(seen), 16) * 16 - len(seen)
        k, v = (np.concatenate([t, np.zeros((pad,) + t.shape[1:])]).reshape(-1, 16, 2, 64) for t in (k, v))
        sub = tree.attend(f64(x["q"][:4]), k, v, [list(range(len(k)))], [len(seen)], [0, 4],
                          x["words"][:4], x["scale"])
        check(gone, o[:4], lse[:4], sub)


def test_same_bits_streams_and_graph(lib):
    """Twice the same bits, on another stream and from a captured graph too, whose inputs change."""
    x = tree_case([(16, 3000), (9, 100), (64, 700)], 4, 8, 128, 16, seed=21)
    cache, args = on_device(lib, x)
    q = x["q"].to(DEV)
    o1, l1 = lib.paged_tree_decode(q, cache, *args, x["most"], x["scale"], want_lse=True)
    o2, l2 = lib.paged_tree_decode(q, cache, *args, x["most"], x["scale"], want_lse=True)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o3, l3 = lib.paged_tree_decode(q, cache, *args, x["most"], x["scale"], want_lse=True, stream=side)
    side.synchronize()
    assert torch.equal(o1, o3) and torch.equal(l1, l3)
    o, lse = torch.zeros_like(o1), torch.zeros_like(l1)
    ws = torch.empty(lib.kda_paged_tree_decode_workspace_size(3, x["most"], 32, 4, 128),
                     dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            lib.kda_paged_tree_decode(q, cache, *args, x["most"], x["scale"], o, lse, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o1) and torch.equal(lse, l1)
    q2 = torch.flip(q, [0]).contiguous()
    want, wl = lib.paged_tree_decode(q2, cache, *args, x["most"], x["scale"], want_lse=True)
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wl)
    assert lib.kda_get_last_device_error() == 0


def test_one_node_is_one_token_attention(lib):
    """A single drafted token that sees itself: what one-token attention gives, to its rounding."""
    x = tree_case([(1, 40), (1, 1000), (1, 0)], 4, 8, 128, 16, seed=13)
    cache, (table, lens, cu, words) = on_device(lib, x)
    o, lse = lib.paged_tree_decode(x["q"].to(DEV), cache, table, lens, cu, words, 1, x["scale"], want_lse=True)
    one, one_lse = lib.paged_decode(x["q"].to(DEV), cache, table, lens, x["scale"], want_lse=True)
    _, _, w, _ = expected(x)
    assert (np.abs(f64(o) - f64(one)) <= 2.0 ** -7 * w).all()
    assert (np.abs(f64(lse) - f64(one_lse)) < 1e-4).all()


def test_offsets_past_32_bits(lib):
    """A cache of more than 4 GB a half: pages far apart in memory."""
    pages, page, H, D = 9000, 64, 32, 128
    k = torch.empty(pages, page, H, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    at = torch.tensor([[8999, 4097, 0, 8500]], dtype=torch.int32, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(0)
    for t in (k, v):
        t[at[0].long()] = torch.randn(4, page, H, D, device=DEV, generator=gen).to(torch.bfloat16)
    q = torch.randn(5, H, D, device=DEV, generator=gen).to(torch.bfloat16)
    words = signed(tree.words([-1, 0, 0, 1, 3])).to(DEV)
    lens, cu = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([250], [0, 5]))
    o, lse = lib.paged_tree_decode(q, lib.PagedCache(k, v), at, lens, cu, words, 5, 0.1, want_lse=True)
    small_k, small_v = (t[at[0].long()].contiguous() for t in (k, v))
    near = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    o2, lse2 = lib.paged_tree_decode(q, lib.PagedCache(small_k, small_v), near, lens, cu, words, 5, 0.1,
                                     want_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.isfinite(o.float()).all()
