"""The KDA recurrence over trees where values are not finite: what a node does not see has no part in
its output and update, so a draft that is dropped leaves nothing behind, and a state's infinite or
largest values act as in fp32 arithmetic."""
import numpy as np
import pytest
import torch

from oracle import tree
from parity_utils import DEV, f64
from test_gpu_tree_recurrent import GAMMA, case, expected, run

pytestmark = pytest.mark.gpu


def commit(lib, x, d, u, words, last):
    pool = d["pool"].clone()
    lib.kda_recurrent_tree_commit(d["k"], d["g"], u, pool, x["slots"].to(DEV), d["cu"], words,
                                  torch.tensor(last, dtype=torch.int32, device=DEV), x["most"])
    return pool


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("n,state,o_dtype", [(12, "fp32", torch.float32), (12, "bf16", torch.bfloat16),
                                             (24, "fp32", torch.bfloat16), (24, "bf16", torch.float32),
                                             (50, "fp32", torch.float32), (50, "bf16", torch.bfloat16)])
def test_what_a_node_does_not_see_has_no_part(lib, n, state, o_dtype, where, bad):
    H, node, head, c = 3, 2, 1, 77
    if where == "g" and bad == -float("inf"):
        bad = float("nan")                                 # (such a decay is an ordinary 0)
    x = case([5, n, 3], H, state, seed=n, decay=1.0)
    rng = np.random.default_rng(n)                         # node 3 is below the bad one, node 4 is not
    x["words"][5:5 + n] = tree.words([-1, -1, 0, 2, 1] + [int(rng.integers(-1, i)) for i in range(5, n)])
    clean = {m: t.clone() if torch.is_tensor(t) else t for m, t in x.items()}
    o0, u0, _, _ = run(lib, x, o_dtype)
    sees = np.array([bool(w >> node & 1) for w in x["words"][5:5 + n]])
    assert sees.sum() > 1 and (~sees).sum() > 2
    if where == "beta":
        x[where][5 + node, head] = bad
    else:
        x[where][5 + node, head, c] = bad
    o, u, d, words = run(lib, x, o_dtype)
    assert lib.kda_get_last_device_error() == 0
    others = [h for h in range(H) if h != head]            # other heads and requests: the same bits
    for got, before in ((o, o0), (u, u0)):
        assert torch.equal(got[:, others], before[:, others])
        assert torch.equal(got[:5], before[:5]) and torch.equal(got[5 + n:], before[5 + n:])
    mine, node_of = slice(5, 5 + n), np.arange(n)
    if where == "q":                                       # of this node's output alone
        assert torch.equal(u, u0)
        sees = node_of == node
    # (what a kernel's sums had spoiled is solved again in fp32 sums of its own: the tolerance, not the bits)
    o_ref, u_ref, mag_o, mag_u, _ = expected(clean, 1)
    rounding = 2.0 ** -8 * np.abs(o_ref) if o_dtype == torch.bfloat16 else 0
    for got, ref, tol in ((o, o_ref, GAMMA * (1 + 2.0 ** -8) * mag_o + rounding), (u, u_ref, GAMMA * mag_u)):
        err = np.abs(f64(got[mine]) - ref)
        assert (err[~sees] <= tol[~sees]).all(), (err / tol)[~sees].max()
    cols = [i for i in range(128) if i != c]
    if where == "v":                                       # of this column alone
        assert torch.equal(o[:, :, cols], o0[:, :, cols]) and torch.equal(u[:, :, cols], u0[:, :, cols])
        hit = (o[mine, head, c], u[mine, head, c])
    else:
        hit = (o[mine, head], u[mine, head]) if where != "q" else (o[mine, head],)
    for t in hit:
        assert not torch.isfinite(t[torch.tensor(sees)]).any()
    # a path without the bad node leaves its own state behind
    last = [4, 4, 2]
    pool = commit(lib, x, d, u, words, last)
    assert lib.kda_get_last_device_error() == 0
    for b, (lo, m) in enumerate(((0, 5), (5, n), (5 + n, 3))):
        slot = int(x["slots"][b])
        ref, mag = tree.commit(f64(x["pool"][slot]), *(f64(clean[t][lo:lo + m]) for t in ("k", "g")),
                               f64(u[lo:lo + m]), x["words"][lo:lo + m], last[b])
        tol = GAMMA * mag + (2.0 ** -8 * np.abs(ref) if state == "bf16" else 0)
        assert (np.abs(f64(pool[slot]) - ref) <= tol).all()


@pytest.mark.parametrize("state", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [9, 20, 40])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_infinite_states(lib, n, state, value):
    """Nodes without ancestors, so that every output is one token's: the class of every value is what
    one-token decoding gives, the updates' what the definition does; other columns keep their bits."""
    x = case([n], 2, state, seed=n, decay=0.5)
    x["words"] = [1 << i for i in range(n)]
    o0, u0, _, _ = run(lib, x)
    row, c = 7, 9
    x["pool"][int(x["slots"][0]), 1, row, c] = value
    o, u, d, _ = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    cols = [i for i in range(128) if i != c]
    assert torch.equal(o[:, 0], o0[:, 0]) and torch.equal(u[:, 0], u0[:, 0])
    assert torch.equal(o[:, 1, cols], o0[:, 1, cols]) and torch.equal(u[:, 1, cols], u0[:, 1, cols])
    with np.errstate(all="ignore"):
        u_ref = expected(x, 0)[1][:, 1, c]
    got = f64(u)[:, 1, c]
    assert np.isinf(u_ref).all() and (got == u_ref).all()
    for i in range(n):
        one = lib.decode_indexed(*(d[m][i:i + 1].clone() for m in ("q", "k", "v", "g", "beta")),
                                 x["pool"].to(DEV), x["slots"].to(DEV), 0.25, torch.float32)[0, 1, c]
        a, b = float(one), float(o[i, 1, c])
        assert np.isnan(a) and np.isnan(b) or a == b, i


@pytest.mark.parametrize("n", [9, 20, 40])
def test_largest_states(lib, n):
    """Values next to fp32's end, whose updates and outputs are finite."""
    x = case([n], 2, seed=n)
    slot = int(x["slots"][0])
    x["pool"][slot, 1, 3, :64] = 3.4028e38
    x["pool"][slot, 0, 100, 5] = -3.4028e38
    o, u, _, _ = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    o_ref, u_ref, mag_o, mag_u, _ = expected(x, 0)
    for got, ref, mag in ((o, o_ref, mag_o), (u, u_ref, mag_u)):
        assert np.isfinite(f64(got)).all() and (np.abs(f64(got) - ref) <= GAMMA * mag).all()


def test_many_requests_some_not_finite(lib):
    """Blocks that walk over units: those before and behind a bad one keep their bits; without u too."""
    rng = np.random.default_rng(0)
    counts = [int(t) for t in rng.integers(1, 9, 300)]
    x = case(counts, 4, seed=6)
    o0, u0, _, _ = run(lib, x)
    bad = rng.choice(300, 40, replace=False)
    hit = np.zeros((sum(counts), 4), bool)
    for b in bad:
        h = int(rng.integers(0, 4))
        lo = int(x["cu"][b])
        x["v"][lo, h, 3] = float("nan")
        for i in range(counts[b]):
            hit[lo + i, h] = x["words"][lo + i] & 1
    o, u, d, words = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    part = np.zeros_like(hit)                              # rows that come after a bad one in its unit
    for b in bad:
        lo, hi = int(x["cu"][b]), int(x["cu"][b + 1])
        part[lo:hi] = hit[lo:hi].any(0)
    keep = torch.tensor(~part)
    assert torch.equal(o[keep], o0[keep]) and torch.equal(u[keep], u0[keep])
    assert torch.equal(o[:, :, 4:], o0[:, :, 4:])
    near = torch.tensor(part & ~hit)                       # beside a bad branch: to rounding
    if near.any():
        assert (u[near] - u0[near]).abs().max() < 1e-4 and (o[near] - o0[near]).abs().max() < 1e-4
    at = torch.tensor(hit)
    assert torch.isnan(o[at][:, 3]).all() and torch.isnan(u[at][:, 3]).all()
    assert torch.equal(o[at][:, 4:], o0[at][:, 4:])
    alone = torch.empty_like(o)
    lib.kda_recurrent_tree_decode(d["q"], d["k"], d["v"], d["g"], d["beta"], d["pool"], x["slots"].to(DEV),
                                  d["cu"], words, x["most"], 0.25, alone, None)
    assert torch.equal(alone[keep], o0[keep]) and torch.isnan(alone[at][:, 3]).all()
