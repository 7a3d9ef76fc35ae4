"""Attention over an 8-bit paged cache where one key holds nearly all the weight and its values
are 0 in half of the channels (GPU): there the outputs are the other keys' alone, whose weights
are down to 2^-28.9 of the largest.  The tolerances are those of the attention tests, relative
to the weighted values of the channel: 2^-8, of which rounding a bf16 output takes 2^-9 and
weights kept to 2^-38 of the largest 2^-9.1; 2^-17 for an fp32 output, of which weights kept to
2^-49 take 2^-20."""
import pytest
import torch

from test_gpu_paged import attention_case, check_decode, run_decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gap", [8.0, 16.0, 18.0, 20.0])        # e^-20 = 2^-28.9
@pytest.mark.parametrize("L,H,G,D", [(3, 1, 2, 128), (40, 2, 4, 128), (700, 2, 16, 64), (30000, 1, 8, 128),
                                     (5000, 1, 24, 128), (3000, 1, 20, 256), (5000, 1, 32, 64)])
def test_small_weights(lib, L, H, G, D, gap, o_dtype):
    page = 64
    x = attention_case([L], H, G, D, page, "fp8", seed=int(gap) + G)
    x["scale"] = 1.0
    x["scales"] = (torch.ones(H), x["scales"][1])
    x["q"].zero_()
    x["q"][..., 0] = 1.0                                        # a key's score is its channel 0
    k = x["k"].float()
    for i in range(-(-L // page)):
        k[int(x["table"][0, i])] = 0.0
    sink = min(L - 1, 5)
    p = int(x["table"][0, 0])
    k[p, sink, :, 0] = gap
    x["k"] = k.to(torch.float8_e4m3fn)
    v = x["v"].float()
    v[p, sink, :, ::2] = 0.0
    x["v"] = v.to(torch.float8_e4m3fn)
    o, lse = run_decode(lib, x, o_dtype)
    assert lib.kda_get_last_device_error() == 0
    check_decode(x, o, lse)
