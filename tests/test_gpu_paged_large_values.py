"""Attention over a bf16 paged cache whose values are near the end of bf16's range: finite
results are finite (GPU).  One value in a channel is large, so that the 32-bit definition, a sum of
weights of at most 1 times values, gives finite numbers; the tolerances are those of the attention
tests."""
import pytest
import torch

from test_gpu_paged import attention_case, check_decode, run_decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("period", [16, 32])
@pytest.mark.parametrize("D,G,L", [(64, 1, 760), (64, 20, 380), (128, 4, 380), (128, 24, 250), (256, 3, 250)])
def test_one_large_value_in_a_channel(lib, D, G, L, period, o_dtype):
    """Scores alternate between 0 and 4.75 (weights 1 and 116) every 16 or 32 keys, in short
    sequences whose units a block keeps whole: a warp often meets keys that outweigh all before
    them.  One of the heavier keys has a value of 2.6e38 in a channel, another one in each."""
    B, page = 20, 64
    x = attention_case([L] * B, 1, G, D, page, seed=D + G)
    x["q"].zero_()
    x["q"][..., 0] = 1.0
    x["scale"] = 1.0
    score = torch.where(torch.arange(L) // period % 2 == 1, 4.75, 0.0)
    heavy = [t for t in range(L) if t // period % 2]
    gen = torch.Generator().manual_seed(0)
    for b in range(B):
        for i in range(-(-L // page)):
            n = min(page, L - i * page)
            x["k"][int(x["table"][b, i]), :n, 0, 0] = score[i * page:i * page + n].to(torch.bfloat16)
        for c in range(D):
            t = heavy[int(torch.randint(len(heavy), (), generator=gen))]
            x["v"][int(x["table"][b, t // page]), t % page, 0, c] = 3.0 * 2.0 ** 126
    o, lse = run_decode(lib, x, o_dtype)
    assert lib.kda_get_last_device_error() == 0
    check_decode(x, o, lse)
