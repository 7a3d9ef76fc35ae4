"""Blocks that walk over many requests: more units of work than blocks, empty, inactive and refused
requests among them.  A request's outputs do not depend on which others are in the call, so they are
the bits of a call with that request alone (which the other tests hold against the oracle)."""
import numpy as np
import pytest
import torch

from parity_utils import DEV
from test_gpu_tree_attention import random_tree, signed

pytestmark = pytest.mark.gpu


def batch(counts, most, seed, inactive):
    """Offsets, words and slots; a request of more than `most` nodes is refused."""
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    words = signed([w for n in counts for w in random_tree(min(n, 64), rng) + [1] * max(n - 64, 0)])
    slots = rng.permutation(len(counts)).astype(np.int32)
    slots[rng.random(len(counts)) < inactive] = -1
    return cu, words.to(DEV), slots


def alone(cu, words, slots, b):
    lo, hi = int(cu[b]), int(cu[b + 1])
    return (slice(lo, hi), torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV), words[lo:hi].clone(),
            torch.tensor([slots[b]], dtype=torch.int32, device=DEV))


def compare(lib, counts, most, cu, words, slots, call, rows):
    """call(row slice, cu, words, slots) -> outputs; all of them together and some alone."""
    N = int(cu[-1])
    together = call(slice(0, N), torch.from_numpy(cu).to(DEV), words, torch.from_numpy(slots).to(DEV))
    assert (lib.kda_get_last_device_error() != 0) == any(n > most for n in counts)
    for b in rows:
        at, *rest = alone(cu, words, slots, b)
        if at.start == at.stop:
            continue
        got = [t[at] for t in together]
        if counts[b] > most or slots[b] < 0:
            assert all(not t.any() for t in got)
        else:
            assert all(torch.equal(t, ref) for t, ref in zip(got, call(at, *rest)))
    assert lib.kda_get_last_device_error() == 0


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,most,refused", [(240, 16, False), (240, 11, True), (90, 64, True), (90, 23, False)])
def test_recurrence_walks(lib, B, most, refused, state):
    H = 3                                    # 720 units, or 270 of the form with a block an SM
    rng = np.random.default_rng(B + most)
    counts = [int(n) for n in rng.integers(0, most + 1, B)]
    if refused:
        for b in (0, B // 3, B - 1):
            counts[b] = most + 1
    counts[5:9] = [0] * 4
    cu, words, slots = batch(counts, most, most, 0.1)
    gen = torch.Generator(device=DEV).manual_seed(most)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)
    N = int(cu[-1])
    q, k, v = (normal(N, H, 128).to(torch.bfloat16) for _ in range(3))
    g, beta = -torch.nn.functional.softplus(normal(N, H, 128)), torch.sigmoid(normal(N, H))
    pool = (0.3 * normal(B, H, 128, 128)).to(state)

    def call(at, cu, words, slots):
        return lib.recurrent_tree_decode(*(t[at].clone() for t in (q, k, v, g, beta)), pool, cu, words, most,
                                         state_indices=slots, scale=0.1)
    compare(lib, counts, most, cu, words, slots, call, list(range(0, B, 3)) + [B - 1])


@pytest.mark.parametrize("B,C,most,refused", [(700, 128, 9, True), (30, 12288, 12, True), (60, 2176, 64, False)])
def test_pre_step_walks(lib, B, C, most, refused):
    rng = np.random.default_rng(C)
    counts = [int(n) for n in rng.integers(0, most + 1, B)]
    if refused:
        for b in (1, B // 2, B - 1):
            counts[b] = most + 3
    cu, words, slots = batch(counts, most, C, 0.1)
    gen = torch.Generator(device=DEV).manual_seed(C)
    N = int(cu[-1])
    xs = [torch.randn(N, C, device=DEV, generator=gen).to(torch.bfloat16) for _ in range(3)]
    ws = [torch.randn(C, 4, device=DEV, generator=gen) for _ in range(3)]
    pool = torch.randn(B, 3, 3, C, device=DEV, generator=gen).to(torch.bfloat16)

    def call(at, cu, words, slots):
        return lib.short_conv_tree(*(x[at].clone() for x in xs), *ws, pool, cu, words, most, state_indices=slots)
    compare(lib, counts, most, cu, words, slots, call, range(0, B, 7))
