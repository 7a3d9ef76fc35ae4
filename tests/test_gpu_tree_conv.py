"""GPU tests of the KDA pre-step over trees against the plain fp64 definition.

Tolerances (derived, per element): the convolution is four fp32 products and sums, off by up to
4 x 2^-24 of sum |w x|; SiLU has slope at most 1.1 and adds some 2^-20 of itself (ex2 and rcp of the
special-function unit); the norm of q and k scales by at most 1 / |y| and adds 2^-20; the bf16
output is rounded by up to 2^-8 of itself."""
import numpy as np
import pytest
import torch

from oracle import tree
from parity_utils import DEV, f64
from test_gpu_tree_attention import random_tree, signed

pytestmark = pytest.mark.gpu


def case(counts, C, chain=False, seed=0, spare=2):
    gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    B, N = len(counts), sum(counts)
    return dict(x=[torch.randn(N, C, generator=gen).to(torch.bfloat16) for _ in range(3)],
                w=[0.5 * torch.randn(C, 4, generator=gen) for _ in range(3)],
                pool=torch.randn(B + spare, 3, 3, C, generator=gen).to(torch.bfloat16),
                slots=torch.tensor(rng.permutation(B + spare)[:B], dtype=torch.int32),
                cu=torch.tensor([sum(counts[:b]) for b in range(B + 1)], dtype=torch.int32),
                words=[w for n in counts for w in random_tree(n, rng, chain)], counts=counts,
                most=max(counts + [1]))


def device(x):
    return ([t.to(DEV) for t in x["x"]], [t.to(DEV) for t in x["w"]], x["pool"].to(DEV), x["slots"].to(DEV),
            x["cu"].to(DEV), signed(x["words"]).to(DEV))


def check(x, ys):
    for b, n in enumerate(x["counts"]):
        lo, slot = int(x["cu"][b]), int(x["slots"][b])
        for z in range(3 if n else 0):
            y, a, mag = tree.conv(f64(x["x"][z][lo:lo + n]), f64(x["w"][z]), f64(x["pool"][slot, z]),
                                  x["words"][lo:lo + n], z < 2)
            e = 1.1 * 4 * 2.0 ** -24 * mag + 2.0 ** -20 * np.abs(a)
            if z < 2:
                s = (a / (1 + np.exp(-a))).reshape(n, -1, 128)
                norm = np.sqrt((s * s).sum(-1, keepdims=True) + 1e-6)
                h = e.reshape(n, -1, 128)                  # an error of the norm, too
                e = (h / norm + np.abs(s) / norm ** 2 * np.sqrt((h * h).sum(-1, keepdims=True))).reshape(n, -1)
            tol = e + (2.0 ** -20 + 2.0 ** -8) * np.abs(y) + e * 2.0 ** -8
            err = np.abs(f64(ys[z][lo:lo + n]) - y)
            assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("counts", [[1], [2, 0, 3], [64, 1, 9], [17] * 5], ids=str)
@pytest.mark.parametrize("C", [128, 256, 640, 12288])
@pytest.mark.parametrize("chain", [False, True])
def test_every_node(lib, counts, C, chain):
    if C == 12288 and sum(counts) > 20:
        counts = counts[:1] + [3]
    x = case(counts, C, chain, seed=C)
    xs, ws, pool, slots, cu, words = device(x)
    ys = lib.short_conv_tree(*xs, *ws, pool, cu, words, x["most"], slots)
    assert lib.kda_get_last_device_error() == 0
    check(x, ys)
    assert torch.equal(pool.cpu(), x["pool"])


@pytest.mark.parametrize("C", [128, 2176, 12288])
def test_commit(lib, C):
    counts = [1, 5, 3, 30, 2, 4, 0]
    x = case(counts, C, seed=3)
    last = [0, 4, -1, 29, 1, 0, -1]
    xs, _, pool, slots, cu, words = device(x)
    lib.kda_short_conv_tree_commit(*xs, pool, slots, cu, words,
                                   torch.tensor(last, dtype=torch.int32, device=DEV), 30)
    assert lib.kda_get_last_device_error() == 0
    want = x["pool"].clone()
    for b, n in enumerate(counts):
        lo, slot = int(x["cu"][b]), int(x["slots"][b])
        for z in range(3):
            at = tree.path(x["words"][lo:lo + n], last[b])
            want[slot, z] = torch.cat([x["pool"][slot, z], x["x"][z][lo:lo + n][at]])[-3:]
    assert torch.equal(pool.cpu(), want)


def test_a_path_is_the_chain_of_steps(lib):
    x = case([20], 256, seed=6)
    xs, ws, pool, slots, cu, words = device(x)
    ys = lib.short_conv_tree(*xs, *ws, pool, cu, words, 20, slots)
    steps = pool.clone()
    for j in tree.path(x["words"], 19):
        one = lib.short_conv_step(*(t[j:j + 1].contiguous() for t in xs), *ws, steps, slots)
        assert all(torch.equal(a[0], b[j]) for a, b in zip(one, ys))
    lib.kda_short_conv_tree_commit(*xs, pool, slots, cu, words, torch.tensor([19], dtype=torch.int32,
                                                                             device=DEV), 20)
    assert torch.equal(pool, steps)


def test_inactive_refused_and_rows_behind(lib):
    x = case([3, 5, 2], 384, seed=2)
    xs, ws, pool, slots, cu, words = device(x)
    before = pool.clone()

    def call(slots=slots, cu=cu, most=5):
        ys = [torch.full((10, 384), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        lib.kda_short_conv_qkv_tree(*xs, *ws, pool, slots, cu, words, most, *ys)
        return ys, lib.kda_get_last_device_error()
    bad = slots.clone()
    bad[1] = -3
    ys, err = call(slots=bad)
    assert err == 0 and not any(y[3:8].any() for y in ys)
    check(dict(x, counts=[3]), ys)
    bad[1] = pool.shape[0]
    ys, err = call(slots=bad)
    assert err == 1 and not any(y[3:8].any() for y in ys)
    ys, err = call(most=4)
    assert err == 1 and not any(y[3:8].any() for y in ys)
    check(dict(x, counts=[3]), ys)
    ys, err = call(cu=torch.tensor([0, 3, 8, 8], dtype=torch.int32, device=DEV))
    assert err == 0 and all((y[8:] == 7).all() for y in ys)
    check(dict(x, counts=[3, 5]), ys)
    for wrong in ([0, 3, 8, 11], [-1, 3, 8, 10], [0, 3, 2, 10]):
        assert call(cu=torch.tensor(wrong, dtype=torch.int32, device=DEV))[1] == 1
    for last in ([3, -1, -1], [-1, 5, -1]):                  # past the nodes
        lib.kda_short_conv_tree_commit(*xs, pool, slots, cu, words,
                                       torch.tensor(last, dtype=torch.int32, device=DEV), 5)
        assert lib.kda_get_last_device_error() == 1
    assert torch.equal(pool, before)
