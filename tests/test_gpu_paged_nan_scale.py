"""Attention over a paged cache with a NaN scale: every output that it enters is NaN, as the
definition has it (GPU)."""
import pytest
import torch

from oracle import paged
from parity_utils import f64
from test_gpu_paged import attention_case, run_decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_nan_scale(lib, cache, D, o_dtype):
    x = attention_case([40, 0, 3000], 2, 3, D, 16, cache, seed=D)
    x["scale"] = float("nan")
    o, lse = run_decode(lib, x, o_dtype)
    assert lib.kda_get_last_device_error() == 0
    held = x["lens"] > 0
    assert bool(torch.isnan(o[held]).all()) and bool(torch.isnan(lse[held]).all())
    assert float(o[~held].abs().max()) == 0.0 and bool(torch.isneginf(lse[~held]).all())


@pytest.mark.parametrize("half", [0, 1])
def test_nan_scale_of_a_head(lib, half):
    """A NaN in the keys' or the values' scale of one key head stays with that head."""
    x = attention_case([40, 0, 3000], 2, 3, 128, 16, "fp8", seed=1)
    good, good_lse = run_decode(lib, x, torch.float32)
    x["scales"][half][1] = float("nan")
    o, lse = run_decode(lib, x, torch.float32)
    held = x["lens"] > 0
    assert bool(torch.isnan(o[held][:, 3:]).all())
    assert torch.equal(o[:, :3], good[:, :3]) and torch.equal(lse[:, :3], good_lse[:, :3])
    assert float(o[~held].abs().max()) == 0.0
    if half == 0:
        assert bool(torch.isnan(lse[held][:, 3:]).all())
    else:
        assert torch.equal(lse, good_lse)
