"""GPU tests of tree attention where a block goes from unit to unit (a sequence's rows of a key head)
many times in a call: several hundred units of few and of many tiles, rows for one and for two products
side by side, references that grow from tile to tile.  Against the fp64 definition (tolerances:
test_gpu_tree_attention.py), and the same bits in every one of many calls."""
import numpy as np
import pytest
import torch

from oracle import paged
from parity_utils import DEV
from test_gpu_tree_attention import check, on_device, run, tree_case

pytestmark = pytest.mark.gpu


def expected(x):
    """oracle.tree.attend in fp64 torch products (the cases are large for loops); all pages are good."""
    k, v = (t.to(DEV).double() for t in (x["k"], x["v"]))
    for t, s in zip((k, v), x["scales"]):
        if s is not None:
            t *= s.to(DEV).double()[:, None]
    N, Hq, D = x["q"].shape
    page, H = k.shape[1:3]
    G = Hq // H
    o, w = (torch.zeros(N, Hq, D, dtype=torch.float64, device=DEV) for _ in range(2))
    lse, spread = (torch.zeros(N, Hq, dtype=torch.float64, device=DEV) for _ in range(2))
    for b, L in enumerate(x["lens"].tolist()):
        lo, hi = int(x["cu"][b]), int(x["cu"][b + 1])
        n = hi - lo
        if n == 0:
            continue
        at = x["table"][b, :paged.pages(L, page)].long().to(DEV)
        kb, vb = (t[at].flatten(0, 1)[:L].transpose(0, 1) for t in (k, v))             # [H, L, D]
        q = x["q"][lo:hi].to(DEV).double().view(n, H, G, D).permute(1, 0, 2, 3).reshape(H, n * G, D)
        s = (q @ kb.transpose(1, 2) * x["scale"]).view(H, n, G, L)
        seen = torch.ones(n, L, dtype=torch.bool)
        for i in range(n):
            seen[i, L - n:] = torch.tensor([bool(x["words"][lo + i] >> j & 1) for j in range(n)])
        s = s.masked_fill(~seen.to(DEV)[None, :, None, :], -float("inf"))
        p, l = torch.softmax(s, -1).view(H, n * G, L), torch.logsumexp(s, -1)
        top = (q.abs() @ kb.abs().transpose(1, 2) * abs(x["scale"])).view(H, n, G, L)
        top = top.masked_fill(~seen.to(DEV)[None, :, None, :], 0).amax(-1)

        def rows(t, *last):                                    # [H, n, G, ..] -> [n, Hq, ..]
            return t.reshape(H, n, G, *last).transpose(0, 1).reshape(n, Hq, *last)
        o[lo:hi], w[lo:hi] = rows(p @ vb, D), rows(p @ vb.abs(), D)
        lse[lo:hi], spread[lo:hi] = rows(l), rows(top)
    return tuple(t.cpu().numpy() for t in (o, lse, w, spread))


def many_units(D, H, G, wide, cache, longest, seed):
    """One request in `wide` has more than 128 rows to a key head, where there is one."""
    rng = np.random.default_rng(seed)
    few, many = min(64, 128 // G), min(64, 256 // G)
    shapes = []
    for b in range(60):
        n = int(rng.integers(few + 1, many + 1)) if wide and b % wide == 0 else int(rng.integers(1, few + 1))
        shapes.append((n, int(np.exp(rng.uniform(np.log(130), np.log(longest - n))))))
    x = tree_case(shapes, H, G, D, 64, cache, seed=seed, peak=2.0)
    for b, n in enumerate(x["lens"].tolist()):                 # keys grow towards the end
        for i in range(paged.pages(n, 64)):
            p = int(x["table"][b, i])
            x["k"][p] = (x["k"][p].float() * (0.2 + 2.0 * i * 64 / n)).to(x["k"].dtype)
    return x


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
@pytest.mark.parametrize("D,H,G,wide", [(128, 8, 8, 4), (64, 8, 8, 4), (256, 8, 8, 4), (128, 8, 8, 0),
                                        (64, 6, 12, 3), (256, 10, 1, 0)])
def test_units_one_after_another(lib, D, H, G, wide, cache):
    x = many_units(D, H, G, wide, cache, 4000 if D < 256 else 2000, seed=D + G + wide)
    o, lse = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    check(x, o, lse, expected(x))
    c, args = on_device(lib, x)
    q = x["q"].to(DEV)
    for _ in range(50):
        o2, lse2 = lib.paged_tree_decode(q, c, *args, x["most"], x["scale"], want_lse=True)
        same = torch.equal(o, o2) and torch.equal(lse, lse2)
        assert same
    assert lib.kda_get_last_device_error() == 0


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bits_do_not_depend_on_the_call_before(lib, D, cache):
    """Requests of a few rows, after a call with large queries in every row of a block and after one
    with none: what lies where a unit has no rows has no part."""
    x = many_units(D, 4, 3, 0, cache, 1500, seed=D)
    big = tree_case([(64, 900)] * 12, 4, 4, D, 64, cache, seed=D + 1)
    c, args = on_device(lib, x)
    cb, args_b = on_device(lib, big)
    q, qb = x["q"].to(DEV), big["q"].to(DEV)
    got = []
    for up in (1e4, 0.0, -1e4, 1.0):
        lib.paged_tree_decode((qb.float() * up).to(torch.bfloat16), cb, *args_b, 64, big["scale"])
        got.append(lib.paged_tree_decode(q, c, *args, x["most"], x["scale"], want_lse=True))
    assert lib.kda_get_last_device_error() == 0
    for o, lse in got[1:]:
        same = torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])
        assert same
    check(x, *got[0], expected(x))
