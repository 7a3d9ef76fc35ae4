"""GPU tests of the KDA recurrence over trees: every node's output and update, and the state after a
path, against the fp64 recurrence.

Tolerances (derived, per element): every product is relative to magnitudes that the oracle carries
along (sum |S_0| |E k|, |E k . k_j| |u_j|, ..).  A sum of 128 products, in any order, is off by at
most 128 x 2^-24 of its magnitude; a decay is a product of at most 64 factors, each expf within
2 x 2^-23 and rounded once: 64 x 5 x 2^-24; the operands and the last steps some 8 x 2^-24.  Sums that the
matrix instructions cut off instead of rounding lose 2^-23 at each of at most 48 steps: 96 x 2^-24.
All together GAMMA of the magnitude.  A bf16 output or state is rounded by up to 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from oracle import tree
from parity_utils import DEV, f64
from test_gpu_tree_attention import random_tree, signed

pytestmark = pytest.mark.gpu

GAMMA = (128 + 320 + 8 + 96) * 2.0 ** -24


def case(counts, H, state="fp32", chain=False, seed=0, spare=2, decay=2.0):
    gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    B, N = len(counts), sum(counts)

    def normal(*shape):
        return torch.randn(*shape, generator=gen)
    q, k = (torch.nn.functional.normalize(normal(N, H, 128), dim=-1).to(torch.bfloat16) for _ in range(2))
    x = dict(q=q, k=k, v=normal(N, H, 128).to(torch.bfloat16),
             g=-torch.nn.functional.softplus(decay * normal(N, H, 128) - 3), beta=torch.sigmoid(normal(N, H)),
             pool=(0.3 * normal(B + spare, H, 128, 128)).to(torch.float32 if state == "fp32"
                                                           else torch.bfloat16),
             slots=torch.tensor(rng.permutation(B + spare)[:B], dtype=torch.int32),
             cu=torch.tensor([sum(counts[:b]) for b in range(B + 1)], dtype=torch.int32),
             words=[w for n in counts for w in random_tree(n, rng, chain)], counts=counts,
             most=max(counts + [1]))
    return x


def run(lib, x, o_dtype=torch.float32, scale=0.25, slots="slots", **kw):
    d = {n: x[n].to(DEV) for n in ("q", "k", "v", "g", "beta", "pool", "cu")}
    idx = None if slots is None else x[slots].to(DEV)
    words = signed(x["words"]).to(DEV) if x["words"] else torch.zeros(0, dtype=torch.int64, device=DEV)
    o, u = lib.recurrent_tree_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], d["pool"], d["cu"], words,
                                     x["most"], state_indices=idx, scale=scale, o_dtype=o_dtype, **kw)
    assert torch.equal(d["pool"], x["pool"].to(DEV))           # read only
    return o, u, d, words


def expected(x, b, scale=0.25):
    lo, hi = int(x["cu"][b]), int(x["cu"][b + 1])
    a = [f64(x[n][lo:hi]) for n in ("q", "k", "v", "g", "beta")]
    return tree.recurrent(*a, f64(x["pool"][int(x["slots"][b])]), x["words"][lo:hi], scale)


def check(x, o, u, scale=0.25):
    for b in range(len(x["counts"])):
        lo, hi = int(x["cu"][b]), int(x["cu"][b + 1])
        if lo == hi:
            continue
        o_ref, u_ref, mag_o, mag_u, _ = expected(x, b, scale)
        rounding = 2.0 ** -8 * np.abs(o_ref) if o.dtype == torch.bfloat16 else 0
        for got, ref, tol in ((o, o_ref, GAMMA * (1 + 2.0 ** -8) * mag_o + rounding), (u, u_ref, GAMMA * mag_u)):
            err = np.abs(f64(got[lo:hi]) - ref)
            assert (err <= tol).all(), (err / tol).max()


COUNTS = [[5], [1, 0, 3, 8], [16, 7, 2], [17, 33], [64, 1, 50], [9] * 20]


@pytest.mark.parametrize("state,o_dtype", [("fp32", torch.float32), ("fp32", torch.bfloat16),
                                           ("bf16", torch.float32), ("bf16", torch.bfloat16)])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("chain", [False, True])
def test_every_node(lib, counts, chain, state, o_dtype):
    x = case(counts, 3, state, chain, seed=len(counts))
    o, u, _, _ = run(lib, x, o_dtype)
    assert lib.kda_get_last_device_error() == 0
    check(x, o, u)


def test_decays_of_every_strength(lib):
    """From none to ones that leave nothing (below -160, where fp32 ends), side by side."""
    x = case([12, 40], 2, chain=True, seed=3)
    x["g"][..., ::3] = 0
    x["g"][..., 1::7] = -40.0
    x["g"][..., 2::11] = -200.0
    x["g"][3, :, 5] = -float("inf")
    o, u, _, _ = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    assert torch.isfinite(o).all() and torch.isfinite(u).all()
    check(x, o, u)


@pytest.mark.parametrize("state", ["fp32", "bf16"])
@pytest.mark.parametrize("counts", [[6, 1, 3], [16, 30, 64], [2] * 30], ids=str)
def test_commit(lib, counts, state):
    x = case(counts, 2, state, seed=7)
    rng = np.random.default_rng(1)
    last = torch.tensor([int(rng.integers(-1, n)) for n in counts], dtype=torch.int32)
    last[0] = counts[0] - 1
    _, u, d, words = run(lib, x)
    lib.kda_recurrent_tree_commit(d["k"], d["g"], u, d["pool"], x["slots"].to(DEV), d["cu"], words,
                                  last.to(DEV), x["most"])
    assert lib.kda_get_last_device_error() == 0
    pool = d["pool"].cpu()
    for b, n in enumerate(counts):
        lo, slot = int(x["cu"][b]), int(x["slots"][b])
        if last[b] < 0:
            assert torch.equal(pool[slot], x["pool"][slot])
            continue
        ref, mag = tree.commit(f64(x["pool"][slot]), f64(x["k"][lo:lo + n]), f64(x["g"][lo:lo + n]),
                               f64(u[lo:lo + n]), x["words"][lo:lo + n], int(last[b]))
        tol = GAMMA * mag + (2.0 ** -8 * np.abs(ref) if state == "bf16" else 0)
        assert (np.abs(f64(pool[slot]) - ref) <= tol).all()
    spare = [s for s in range(len(pool)) if s not in x["slots"].tolist()]
    assert torch.equal(pool[spare], x["pool"][spare])


def test_step_and_commit_are_the_chain_of_tokens(lib):
    """A path through a tree gives what decoding its tokens one by one does."""
    x = case([24], 4, seed=5)
    o, u, d, words = run(lib, x)
    pool = x["pool"].to(DEV)
    slot = x["slots"].to(DEV)
    e = 23
    at = tree.path(x["words"], e)
    for j in at:
        one = lib.decode_indexed(d["q"][j:j + 1].contiguous(), d["k"][j:j + 1].contiguous(),
                                 d["v"][j:j + 1].contiguous(), d["g"][j:j + 1].contiguous(),
                                 d["beta"][j:j + 1].contiguous(), pool, slot, 0.25, torch.float32)
        assert (one[0] - o[j]).abs().max() < 1e-4
    lib.kda_recurrent_tree_commit(d["k"], d["g"], u, d["pool"], slot, d["cu"], words,
                                  torch.tensor([e], dtype=torch.int32, device=DEV), 24)
    assert (pool - d["pool"]).abs().max() < 1e-4


def test_inactive_and_refused(lib):
    x = case([3, 5, 2, 4], 2, seed=2)
    x["slots"][1], x["slots"][3] = -1, x["pool"].shape[0]
    o, u, d, words = run(lib, x)
    assert lib.kda_get_last_device_error() == 1                # the slot past the pool
    assert not o[3:8].any() and not u[3:8].any() and not o[10:].any() and not u[10:].any()
    keep = dict(x, counts=[3])
    check(keep, o, u)
    before = d["pool"].clone()
    lib.kda_recurrent_tree_commit(d["k"], d["g"], u, d["pool"], x["slots"].to(DEV), d["cu"], words,
                                  torch.tensor([3, 1, -5, 1], dtype=torch.int32, device=DEV), 5)
    assert lib.kda_get_last_device_error() == 1
    assert torch.equal(before, d["pool"])                      # 3 is past the nodes, the others inactive

    x = case([3, 5, 2], 2, seed=2)
    x["most"] = 4                                              # the second has more
    o, u, _, _ = run(lib, x)
    assert lib.kda_get_last_device_error() == 1
    assert not o[3:8].any() and not u[3:8].any()
    check(dict(x, counts=[3]), o, u)
    for bad in ([0, 3, 8, 11], [-1, 3, 8, 10], [0, 3, 2, 10]):
        x = case([3, 5, 2], 2, seed=2)
        x["cu"] = torch.tensor(bad, dtype=torch.int32)
        run(lib, x)
        assert lib.kda_get_last_device_error() == 1


def test_rows_behind_shared_slots_and_no_indices(lib):
    x = case([4, 6], 2, seed=4, spare=0)
    o = torch.full((12, 2, 128), 7.0, device=DEV)
    u = o.clone()
    ext = {n: torch.cat([x[n], x[n][:2]]).to(DEV) for n in ("q", "k", "v", "g", "beta")}
    words = torch.cat([signed(x["words"]), torch.tensor([-1, -1])]).to(DEV)
    lib.kda_recurrent_tree_decode(ext["q"], ext["k"], ext["v"], ext["g"], ext["beta"], x["pool"].to(DEV), None,
                                  x["cu"].to(DEV), words, 64, 0.25, o, u)
    x["slots"] = torch.tensor([0, 1], dtype=torch.int32)
    check(x, o, u)
    assert (o[10:] == 7).all() and (u[10:] == 7).all()
    x["slots"] = torch.tensor([1, 1], dtype=torch.int32)       # two requests read one state
    o2 = torch.empty_like(o)
    lib.kda_recurrent_tree_decode(ext["q"], ext["k"], ext["v"], ext["g"], ext["beta"], x["pool"].to(DEV),
                                  x["slots"].to(DEV), x["cu"].to(DEV), words, 6, 0.25, o2, None)
    check(x, o2, u=torch.tensor(np.concatenate([expected(x, b)[1] for b in range(2)] + [np.zeros((2, 2, 128))])))
    assert lib.kda_get_last_device_error() == 0


def test_nothing_to_do(lib):
    x = case([0, 0], 1, seed=1)
    o, u, d, words = run(lib, x)
    lib.kda_recurrent_tree_commit(d["k"], d["g"], u, d["pool"], None, d["cu"], words,
                                  torch.tensor([-1, -1], dtype=torch.int32, device=DEV), 1)
    assert o.numel() == 0 and lib.kda_get_last_device_error() == 0


def test_a_state_that_is_not_finite_stays_with_its_request(lib):
    x = case([5, 4], 2, seed=9)
    x["pool"][int(x["slots"][0]), 1, 7, 9] = float("inf")
    o, u, _, _ = run(lib, x)
    assert not torch.isfinite(u[:5, 1]).all()
    assert torch.isfinite(u[:5, 0]).all() and torch.isfinite(o[5:]).all()
    b = dict(x, counts=[5, 4])
    o_ref, u_ref, mag_o, mag_u, _ = expected(b, 1)
    assert (np.abs(f64(u[5:]) - u_ref) <= GAMMA * mag_u).all()


def test_same_bits_streams_and_graph(lib):
    x = case([16] * 6 + [40], 8, seed=12)
    o, u, d, words = run(lib, x)
    o2, u2, _, _ = run(lib, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o3, u3, _, _ = run(lib, x, stream=side)
    side.synchronize()
    for a, b in ((o, o2), (u, u2), (o, o3), (u, u3)):
        assert torch.equal(a, b)
    og, ug, slots = torch.zeros_like(o), torch.zeros_like(u), x["slots"].to(DEV)
    last = torch.full((7,), 3, dtype=torch.int32, device=DEV)
    pool = d["pool"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.kda_recurrent_tree_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], pool, slots, d["cu"], words,
                                      40, 0.25, og, ug)
        lib.kda_recurrent_tree_commit(d["k"], d["g"], ug, pool, slots, d["cu"], words, last, 40)
    want = d["pool"].clone()
    for _ in range(2):                                         # each replay is the next step
        graph.replay()
        ow, uw = lib.recurrent_tree_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], want, d["cu"], words, 40,
                                           state_indices=slots, scale=0.25, o_dtype=torch.float32)
        lib.kda_recurrent_tree_commit(d["k"], d["g"], uw, want, slots, d["cu"], words, last, 40)
        torch.cuda.synchronize()
        assert torch.equal(og, ow) and torch.equal(ug, uw) and torch.equal(pool, want)
    assert lib.kda_get_last_device_error() == 0
