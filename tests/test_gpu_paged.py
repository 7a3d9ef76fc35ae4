"""GPU tests of the paged key-value cache: plan, append and one-token attention
against the oracle's plain fp64 definitions.

Tolerances (derived, per element).  The plan is exact; a bf16 append is a copy;
an 8-bit append rounds the fp32 quotient to nearest: exact.  Attention: with
w = sum_j p_j |v_j|, a bf16 output is rounded by up to 2^-8 of |o| <= w, which
leaves next to nothing for the weights; for fp32 outputs they may be off by
2^-17 of themselves (two words of 8 bits), which the sum carries to w.  Scores are fp32 sums of exact
products in steps of at least 8 terms: off by (D / 8 + 8) 2^-23 of
S = max_j scale sum_d |q_d k_jd|, and ex2 and the sums by some 2^-21; a score's
error reaches a weight and the normalisation, so twice.  lse carries the score
error once.
"""
import numpy as np
import pytest
import torch

from oracle import paged
from parity_utils import DEV, f64

pytestmark = pytest.mark.gpu

ERR_INVALID = 1


def make_cache(num_pages, page, H, D, cache, order, gen, sigma=1.0):
    """A cache full of NaN (what no call may read) and the fp64 values of its two halves."""
    dtype = torch.float8_e4m3fn if cache == "fp8" else torch.bfloat16
    out = []
    for _ in range(2):
        shape = (num_pages, H, page, D) if order == "head" else (num_pages, page, H, D)
        t = torch.full(shape, float("nan")).to(dtype)
        out.append(t.permute(0, 2, 1, 3) if order == "head" else t)
    return out


def as_device(t):
    """The same strides on the device (a permuted view stays one)."""
    d = torch.empty_strided(t.size(), t.stride(), dtype=t.dtype, device=DEV)
    raw = torch.uint8 if t.element_size() == 1 else t.dtype
    d.view(raw).copy_(t.view(raw))
    return d


def attention_case(lens, H, G, D, page, cache="bf16", order="token", seed=0, peak=1.0):
    gen = torch.Generator().manual_seed(seed)
    B = len(lens)
    held = [paged.pages(n, page) for n in lens]
    num_pages = sum(held) + 3
    perm = torch.randperm(num_pages, generator=gen)
    width = max(held + [1]) + 1
    table = torch.full((B, width), 2 ** 30, dtype=torch.int32)     # never read
    k, v = make_cache(num_pages, page, H, D, cache, order, gen)
    at = 0
    for b, n in enumerate(lens):
        table[b, :held[b]] = perm[at:at + held[b]].to(torch.int32)
        for i in range(held[b]):
            p = int(perm[at + i])
            m = min(page, n - i * page)
            for t in (k, v):
                x = torch.randn(m, H, D, generator=gen) * (40.0 if cache == "fp8" else 1.0)
                t[p, :m] = x.to(t.dtype)
        at += held[b]
    q = (torch.randn(B, H * G, D, generator=gen) * peak).to(torch.bfloat16)
    scales = (None, None)
    if cache == "fp8":
        scales = tuple(torch.rand(H, generator=gen) * 0.03 + 0.01 for _ in range(2))
    return dict(q=q, k=k, v=v, table=table, lens=torch.tensor(lens, dtype=torch.int32),
                scales=scales, scale=D ** -0.5, H=H, G=G, D=D)


def run_decode(lib, x, o_dtype, want_lse=True, stream=None):
    ks, vs = (None if s is None else s.to(DEV) for s in x["scales"])
    cache = lib.PagedCache(as_device(x["k"]), as_device(x["v"]), ks, vs)
    o, lse = lib.paged_decode(x["q"].to(DEV), cache, x["table"].to(DEV), x["lens"].to(DEV),
                              x["scale"], o_dtype=o_dtype, want_lse=want_lse, stream=stream)
    return o, lse


def check_decode(x, o, lse, lens=None):
    ks, vs = (None if s is None else s.numpy() for s in x["scales"])
    o_ref, lse_ref, w, spread = paged.decode(
        f64(x["q"]), x["k"].float().double().numpy(), x["v"].float().double().numpy(),
        x["table"].numpy(), x["lens"].numpy() if lens is None else lens, x["scale"], ks, vs)
    es = (x["D"] / 8 + 8) * 2.0 ** -23 * spread + 2.0 ** -21
    rounding = 2.0 ** -8 if o.dtype == torch.bfloat16 else 2.0 ** -17 + 2.0 ** -22
    err = np.abs(f64(o) - o_ref)
    tol = (rounding + 2 * es[..., None]) * w
    assert np.isfinite(f64(o)).all()
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()
    if lse is not None:
        got = f64(lse)
        empty = np.isneginf(lse_ref)
        assert np.isneginf(got[empty]).all()
        got, ref, es = got[~empty], lse_ref[~empty], es[~empty]
        assert (np.abs(got - ref) <= es + 2.0 ** -22 * np.abs(ref)).all()


LENS = [0, 1, 15, 16, 17, 2, 63, 64, 65, 0, 127, 129, 300, 1023, 1]


@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cache,order", [("bf16", "token"), ("bf16", "head"), ("fp8", "token"),
                                         ("fp8", "head")])
@pytest.mark.parametrize("H,G,D,page", [(2, 4, 128, 16), (1, 1, 64, 24), (3, 12, 128, 64),
                                        (2, 16, 64, 1), (1, 20, 256, 7), (4, 8, 256, 128),
                                        (2, 2, 128, 33)])
def test_decode(lib, H, G, D, page, cache, order, o_dtype):
    x = attention_case(LENS, H, G, D, page, cache, order, seed=H * 100 + G)
    o, lse = run_decode(lib, x, o_dtype)
    assert lib.kda_get_last_device_error() == 0
    check_decode(x, o, lse)


@pytest.mark.parametrize("lens", [[20011], [5000, 1, 0, 9999], [4096] * 5 + [3], [0, 0], [1]])
@pytest.mark.parametrize("cache,D,G", [("bf16", 128, 8), ("fp8", 128, 4), ("bf16", 64, 1),
                                       ("bf16", 256, 6), ("bf16", 128, 24), ("fp8", 64, 32),
                                       ("fp8", 128, 30), ("bf16", 256, 20), ("bf16", 64, 13),
                                       ("bf16", 128, 48), ("fp8", 64, 70), ("bf16", 256, 40)])
def test_decode_long(lib, lens, cache, D, G):
    """Lengths that are split over many blocks and joined."""
    x = attention_case(lens, 2, G, D, 64, cache, "token", seed=len(lens), peak=3.0)
    for dt in (torch.bfloat16, torch.float32):
        o, lse = run_decode(lib, x, dt)
        assert lib.kda_get_last_device_error() == 0
        check_decode(x, o, lse)


@pytest.mark.parametrize("H,G,D,cache,lens", [(32, 2, 64, "fp8", [9001, 20000, 0, 1, 11111]),
                                               (6, 1, 64, "bf16", [40000, 77, 41003]),
                                               (8, 8, 128, "fp8", [30001, 33333]),
                                               (32, 9, 64, "bf16", [100] * 190 + [3]),
                                               (2, 40, 128, "bf16", [40000, 30000]),
                                               (1, 100, 128, "bf16", [60000, 5, 500]),
                                               (2, 70, 256, "fp8", [25000, 1]),
                                               (1, 200, 64, "bf16", [70000, 200])])
def test_decode_heads_side_by_side(lib, H, G, D, cache, lens):
    """Lists long enough that neighbouring heads of short rows are walked together, and
    groups of several units."""
    x = attention_case(lens, H, G, D, 64, cache, "token", seed=H)
    for dt in (torch.bfloat16, torch.float32):
        o, lse = run_decode(lib, x, dt)
        assert lib.kda_get_last_device_error() == 0
        check_decode(x, o, lse)


def test_decode_many_short(lib):
    """More sequences than blocks, most of them of a few keys."""
    gen = np.random.default_rng(5)
    lens = [int(n) for n in gen.integers(0, 40, 700)]
    x = attention_case(lens, 4, 3, 64, 16, "bf16", "head", seed=5)
    o, lse = run_decode(lib, x, torch.bfloat16)
    check_decode(x, o, lse)
    o2, _ = run_decode(lib, x, torch.bfloat16, want_lse=False)
    assert torch.equal(o, o2)


def test_decode_same_bits_strides_streams_and_graph(lib):
    """Rows of a fused projection, another stream and a captured graph give the same bits; a
    graph follows lengths that change on the device."""
    x = attention_case([900, 33, 0, 2500], 4, 4, 128, 16, seed=8)
    o, lse = run_decode(lib, x, torch.float32)
    cache = lib.PagedCache(as_device(x["k"]), as_device(x["v"]))
    wide = torch.randn(4, 3 * 16 * 128, device=DEV).to(torch.bfloat16)
    q = wide[:, 16 * 128:2 * 16 * 128].view(4, 16, 128)
    q.copy_(x["q"].to(DEV))
    table, lens = x["table"].to(DEV), x["lens"].to(DEV)
    o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    ws = torch.full((lib.kda_paged_decode_workspace_size(4, 16, 4, 128),), 255, dtype=torch.uint8,
                    device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lib.kda_paged_decode(q, cache, table, lens, x["scale"], o2, lse2, ws, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.kda_paged_decode(q, cache, table, lens, x["scale"], o2, lse2, ws)
    o2.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    fewer = torch.tensor([17, 33, 0, 1200], dtype=torch.int32)
    lens.copy_(fewer)
    g.replay()
    torch.cuda.synchronize()
    check_decode(x, o2, lse2, lens=fewer.numpy())
    assert lib.kda_get_last_device_error() == 0


def test_decode_bad_lengths_and_pages(lib):
    """A bad length counts as empty, keys on a bad page are left out; both are reported."""
    x = attention_case([40, 50, 60, 70], 2, 4, 64, 16, seed=3)
    good, _ = run_decode(lib, x, torch.float32)
    x["lens"][1] = -5
    x["lens"][2] = x["table"].shape[1] * 16 + 1
    o, lse = run_decode(lib, x, torch.float32)
    assert lib.kda_get_last_device_error() == ERR_INVALID
    assert lib.kda_get_last_device_error() == 0
    assert torch.equal(o[0], good[0]) or float((o[0] - good[0]).abs().max()) < 1e-5
    assert float(o[1:3].abs().max()) == 0.0 and bool(torch.isneginf(lse[1:3]).all())
    # keys 16..31 of sequence 0 are on a page that does not exist
    x = attention_case([40, 50, 60, 70], 2, 4, 64, 16, seed=3)
    whole = x["table"].clone()
    for bad in (-1, x["k"].shape[0], 2 ** 31 - 1):
        x["table"][0, 1] = bad
        o, lse = run_decode(lib, x, torch.float32)
        assert lib.kda_get_last_device_error() == ERR_INVALID
        cut = dict(x, table=whole.clone())
        cut["table"][0, :2] = whole[0, [0, 2]]
        cut["lens"] = torch.tensor([24, 50, 60, 70], dtype=torch.int32)
        check_decode(cut, o, lse)


def test_decode_extreme_scores(lib):
    """Scores of both signs up to some thousands (one key takes all), equal scores, zero scale,
    and infinite or NaN values in keys that a sequence does not hold."""
    x = attention_case([33, 200, 1000, 5], 2, 4, 128, 16, seed=4, peak=1000.0)
    for scale in (1.0, -1.0, 0.0):
        x["scale"] = scale
        o, lse = run_decode(lib, x, torch.float32)
        check_decode(x, o, lse)
    # an infinite key component: its keys' weights are 1 / 0 (score -inf) where q is negative
    x = attention_case([50], 1, 1, 64, 16, seed=6)
    x["q"][:] = -1.0
    x["k"][x["table"][0, 1], 3, 0, 5] = float("inf")
    o, lse = run_decode(lib, x, torch.float32)
    gone = dict(x, k=x["k"].clone(), v=x["v"].clone(), table=x["table"].clone())
    p, last = x["table"][0, 1], x["table"][0, 3]
    for t in ("k", "v"):                                   # the same keys without that one
        gone[t][p, 3] = x[t][last, 1]
    gone["lens"] = torch.tensor([49], dtype=torch.int32)
    check_decode(gone, o, lse)
    x["v"][x["table"][0, 0], 2, 0, 9] = float("nan")
    o, _ = run_decode(lib, x, torch.float32)
    nan = torch.isnan(o)
    assert bool(nan[..., 9].all()) and int(nan.sum()) == nan[..., 9].numel()


def test_decode_far_pages(lib):
    """Pages past 2^31 values: offsets of more than 32 bits."""
    H, D, page = 8, 128, 64
    num_pages = 2 ** 32 // (H * D * page) + 40             # 4 Gi values, 8.6 GB each
    k = torch.empty(num_pages, page, H, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    x = attention_case([200, 513], H, 2, D, page, seed=9)
    small = x["k"].shape[0]
    far = torch.arange(small, dtype=torch.int64) * 37 % 40 + (num_pages - 40)
    far[0] = num_pages // 2 + 1
    assert far.unique().numel() == small
    k[far.to(DEV)] = x["k"].to(DEV)
    v[far.to(DEV)] = x["v"].to(DEV)
    table = torch.where(x["table"] < small, far[x["table"].clamp(max=small - 1).long()].int(),
                        x["table"])
    cache = lib.PagedCache(k, v)
    o, lse = lib.paged_decode(x["q"].to(DEV), cache, table.to(DEV), x["lens"].to(DEV), x["scale"],
                              want_lse=True)
    check_decode(x, o, lse)
    new = torch.randn(3, H, D).to(torch.bfloat16)
    slots = [num_pages * page - 1, -1, (num_pages - 1) * page + 5]
    lib.kda_paged_append(new.to(DEV), -new.to(DEV), torch.tensor(slots, dtype=torch.int32).to(DEV),
                         cache)
    assert torch.equal(k[-1, page - 1].cpu(), new[0]) and torch.equal(v[-1, 5].cpu(), -new[2])
    assert lib.kda_get_last_device_error() == 0


@pytest.mark.parametrize("H,D", [(1, 64), (4, 128), (3, 256), (32, 64)])
@pytest.mark.parametrize("cache,order", [("bf16", "token"), ("bf16", "head"), ("fp8", "token"),
                                         ("fp8", "head")])
@pytest.mark.parametrize("N", [1, 7, 300])
def test_append(lib, H, D, cache, order, N):
    gen = torch.Generator().manual_seed(N + H)
    page, num_pages = 12, 40
    rows = (torch.randn(N, 2 * H * D + 24, generator=gen) * 3).to(torch.bfloat16)
    k, v = rows[:, :H * D].view(N, H, D), rows[:, H * D + 8:2 * H * D + 8].view(N, H, D)
    if cache == "fp8":                                     # limits, subnormals and zeros too
        k[0, 0, :6] = torch.tensor([1e30, -1e30, 1e-5, -1e-5, 0.0, 1e-30])
    slots = torch.randperm(num_pages * page, generator=gen)[:N].to(torch.int32)
    if N > 4:
        slots[3] = -1
    kc, vc = make_cache(num_pages, page, H, D, cache, order, gen)
    scales = (None, None)
    if cache == "fp8":
        scales = tuple(torch.rand(H, generator=gen) * 0.05 + 0.003 for _ in range(2))
    kd, vd = as_device(kc), as_device(vc)
    c = lib.PagedCache(kd, vd, *(None if s is None else s.to(DEV) for s in scales))
    dev = rows.to(DEV)
    lib.kda_paged_append(dev[:, :H * D].view(N, H, D), dev[:, H * D + 8:2 * H * D + 8].view(N, H, D),
                         slots.to(DEV), c)
    assert lib.kda_get_last_device_error() == 0
    for got, was, x, s in ((kd, kc, k, scales[0]), (vd, vc, v, scales[1])):
        ref = paged.append(was.float().double().numpy(), f64(x), slots.tolist(),
                           None if s is None else s.numpy())
        np.testing.assert_array_equal(got.float().cpu().double().numpy(), ref)


def test_append_every_bf16_to_8_bits(lib):
    """Every finite bf16 value over an awkward scale, and NaN and infinities."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits.view(512, 1, 128)
    s = torch.tensor([0.0137])
    cache = torch.zeros(32, 16, 1, 128, dtype=torch.float8_e4m3fn, device=DEV)
    c = lib.PagedCache(cache, torch.zeros_like(cache), s.to(DEV), torch.ones(1, device=DEV))
    lib.kda_paged_append(x.to(DEV), x.to(DEV), torch.arange(512, dtype=torch.int32, device=DEV), c)
    for got, scale in ((c.k_cache, s), (c.v_cache, torch.ones(1))):
        got = got.float().cpu().flatten()
        quotient = (bits.float() / scale).double().numpy()
        fine = np.isfinite(quotient)
        np.testing.assert_array_equal(got.double().numpy()[fine], paged.e4m3(quotient[fine]))
        inf = np.isinf(quotient)
        np.testing.assert_array_equal(got.numpy()[inf], np.sign(quotient[inf]) * 448)
        assert torch.isnan(got)[np.isnan(quotient)].all()


def test_append_slot_past_the_cache(lib):
    k = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device=DEV)
    c = lib.PagedCache(k, torch.zeros_like(k))
    x = torch.ones(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    lib.kda_paged_append(x, x, torch.tensor([8, 2, 2 ** 31 - 1], dtype=torch.int32, device=DEV), c)
    assert lib.kda_get_last_device_error() == ERR_INVALID
    assert float(k.float().sum()) == 64 and float(k[0, 2].float().sum()) == 64


def run_plan(lib, cached, new, free, table, page, num_pages, N):
    t = torch.tensor(table, dtype=torch.int32, device=DEV).view(len(cached), -1)
    out = lib.page_plan(*(torch.tensor(a, dtype=torch.int32, device=DEV)
                          for a in (cached, new, free)), t, page, num_pages, N)
    return (t, *out)


def check_plan(got, ref):
    t, seq, cu, slots, used = (x.cpu().numpy() for x in got)
    np.testing.assert_array_equal(t, ref[0])
    np.testing.assert_array_equal(seq, ref[1])
    np.testing.assert_array_equal(cu, ref[2])
    np.testing.assert_array_equal(slots, ref[3])
    assert int(used[0]) == ref[4]


@pytest.mark.parametrize("B,hi_cached,hi_new,page", [(1, 0, 1, 16), (1, 100, 9000, 16),
                                                     (7, 50, 3, 1), (300, 70, 40, 24),
                                                     (1500, 33, 2, 64), (2500, 5, 1, 16),
                                                     (64, 0, 2048, 128)])
def test_plan(lib, B, hi_cached, hi_new, page):
    gen = np.random.default_rng(B)
    cached = gen.integers(0, hi_cached + 1, B)
    new = gen.integers(0, hi_new + 1, B)
    new[0] = hi_new
    held = [paged.pages(c, page) for c in cached]
    width = max(paged.pages(c + n, page) for c, n in zip(cached, new)) + 1
    num_pages = int(sum(paged.pages(c + n, page) for c, n in zip(cached, new))) + 2
    perm = gen.permutation(num_pages)
    table = np.full((B, width), -7)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    N = int(new.sum())
    for extra in (0, 1, 1500):
        ref = paged.plan(cached, new, perm[at:], table, page, num_pages, N + extra)
        got = run_plan(lib, cached, new, perm[at:], table, page, num_pages, N + extra)
        assert lib.kda_get_last_device_error() == 0 and not ref[5]
        check_plan(got, ref)


@pytest.mark.parametrize("seed", range(6))
def test_plan_refusals(lib, seed):
    """Bad lengths, too few pages, too few rows and bad page numbers, in any mixture."""
    gen = np.random.default_rng(seed)
    B, page, width, num_pages = 1100, 8, 5, 500
    cached = gen.integers(-1 if seed % 2 else 0, 42, B)
    new = gen.integers(-1 if seed % 3 else 0, 20, B)
    cached[5], new[5] = 2 ** 31 - 1, 2 ** 31 - 1
    new[9] = 2 ** 31 - 1 if seed == 5 else 3
    table = gen.integers(-2 if seed == 4 else 0, num_pages + (2 if seed == 4 else 0), (B, width))
    free = gen.integers(0, num_pages + (3 if seed == 4 else 0), 700 if seed < 3 else 4000)
    N = [30000, 4000, 0, 2500, 30000, 9000][seed]
    ref = paged.plan(cached, new, free, table, page, num_pages, N)
    got = run_plan(lib, cached, new, free, table, page, num_pages, N)
    assert (lib.kda_get_last_device_error() == ERR_INVALID) == ref[5]
    check_plan(got, ref)


def test_plan_of_nothing(lib):
    t = torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    seq, cu, slots, used = lib.page_plan(e, e, e, t, 16, 4, 5)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 5 and used.tolist() == [0]
    assert lib.kda_get_last_device_error() == 0
