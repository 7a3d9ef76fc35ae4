"""The recurrence's form for trees of 17 to 32 nodes (left operands as fp32 words, two blocks an SM; the state
in four parts, or whole where it is bf16) against the fp64 recurrence, element by element, and the commits
of its updates.  Tolerances: test_gpu_tree_recurrent.py, which are for up to 64 nodes."""
import numpy as np
import pytest
import torch

from oracle import tree
from parity_utils import DEV, f64
from test_gpu_tree_recurrent import GAMMA, case, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("state,o_dtype", [("fp32", torch.float32), ("fp32", torch.bfloat16),
                                           ("bf16", torch.float32), ("bf16", torch.bfloat16)])
@pytest.mark.parametrize("counts", [[17], [24, 3, 32], [31, 8, 0, 25], [18, 1] * 9], ids=str)
@pytest.mark.parametrize("chain", [False, True])
def test_every_node(lib, counts, chain, state, o_dtype):
    x = case(counts, 3, state, chain, seed=len(counts) + counts[0])
    o, u, _, _ = run(lib, x, o_dtype)
    assert lib.kda_get_last_device_error() == 0
    check(x, o, u)


@pytest.mark.parametrize("state", ["fp32", "bf16"])
@pytest.mark.parametrize("most", [32, 24, 17])
def test_decays_of_every_strength(lib, most, state):
    x = case([most, 9], 2, state, chain=True, seed=most)
    x["g"][..., ::3] = 0
    x["g"][..., 1::7] = -40.0
    x["g"][..., 2::11] = -200.0
    x["g"][3, :, 5] = -float("inf")
    o, u, _, _ = run(lib, x)
    assert lib.kda_get_last_device_error() == 0
    assert torch.isfinite(o).all() and torch.isfinite(u).all()
    check(x, o, u)


@pytest.mark.parametrize("state", ["fp32", "bf16"])
def test_commit(lib, state):
    counts = [20, 32, 27]
    x = case(counts, 2, state, seed=8)
    last = [19, 31, 14]
    _, u, d, words = run(lib, x)
    lib.kda_recurrent_tree_commit(d["k"], d["g"], u, d["pool"], x["slots"].to(DEV), d["cu"], words,
                                  torch.tensor(last, dtype=torch.int32, device=DEV), x["most"])
    assert lib.kda_get_last_device_error() == 0
    for b, n in enumerate(counts):
        lo, slot = int(x["cu"][b]), int(x["slots"][b])
        ref, mag = tree.commit(f64(x["pool"][slot]), f64(x["k"][lo:lo + n]), f64(x["g"][lo:lo + n]),
                               f64(u[lo:lo + n]), x["words"][lo:lo + n], last[b])
        tol = GAMMA * mag + (2.0 ** -8 * np.abs(ref) if state == "bf16" else 0)
        assert (np.abs(f64(d["pool"][slot]) - ref) <= tol).all()
