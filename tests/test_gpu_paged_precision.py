"""The precision of fp32 attention outputs over a paged cache (GPU), as a relative 2-norm of the
error against fp64.

Short lists pin the weights: scores near 0 are exact to some 2^-26, a weight's exponential is off
by 2^-22 of itself at most, its words by 2^-24, the fp32 products and sums of up to eight keys
and the division by some 2^-23 together: 2^-22 + 2^-24 + 2^-23 < 4.2e-7, all at their worst.
(Weights of 16 bits are off by 2^-18 at most and near 1.1e-6 in the mean.)

Long lists pin the sums.  Within a tile a channel takes at most 12 matrix instructions, each of
which may cut off 2^-24 of the sum in it: 12 2^-24 = 7.2e-7 at the worst, half of that in the
mean; adding the tiles in fp32 rounds both ways and stays below 1e-7 for some hundred of them.
With the weights' 2^-22 at their worst: below 1e-6.  (One running sum over the tiles is cut off
some 12 times a tile: above 1e-5 after 200 tiles a warp.)"""
import pytest
import torch

from parity_utils import DEV

pytestmark = pytest.mark.gpu


def far(lib, lens, H, G, D, cache, seed):
    page = 64
    gen = torch.Generator(device=DEV).manual_seed(seed)
    held = [-(-n // page) for n in lens]
    num_pages = sum(held)
    dtype = torch.float8_e4m3fn if cache == "fp8" else torch.bfloat16
    k, v = (torch.empty(num_pages, page, H, D, dtype=dtype, device=DEV) for _ in range(2))
    for i in range(0, num_pages, 1024):
        shape = k[i:i + 1024].shape
        k[i:i + 1024].copy_(torch.randn(shape, device=DEV, generator=gen))
        v[i:i + 1024].copy_(1.0 + 0.5 * torch.rand(shape, device=DEV, generator=gen))
    first = torch.tensor([sum(held[:b]) for b in range(len(lens))], device=DEV)
    col = torch.arange(max(held), device=DEV)
    table = (first[:, None] + col).clamp(max=num_pages - 1).to(torch.int32)
    q = torch.randn(len(lens), H * G, D, device=DEV, generator=gen).to(torch.bfloat16)
    scale = 0.25 * D ** -0.5
    ones = torch.ones(H, device=DEV) if cache == "fp8" else None
    o, lse = lib.paged_decode(q, lib.PagedCache(k, v, ones, ones), table,
                              torch.tensor(lens, dtype=torch.int32, device=DEV), scale,
                              o_dtype=torch.float32, want_lse=True)
    assert lib.kda_get_last_device_error() == 0
    num = den = 0.0
    for b, n in enumerate(lens):
        for h in range(H):
            rows = slice(sum(held[:b]), sum(held[:b]) + held[b])
            kk = k[rows, :, h].float().double().reshape(-1, D)[:n]
            vv = v[rows, :, h].float().double().reshape(-1, D)[:n]
            s = (q[b, h * G:(h + 1) * G].double() @ kk.T) * scale
            ref = torch.softmax(s, -1) @ vv
            num += float(((o[b, h * G:(h + 1) * G].double() - ref) ** 2).sum())
            den += float((ref ** 2).sum())
    return (num / den) ** 0.5


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (128, 16), (256, 2)])
def test_weights_of_fp32_outputs(lib, D, G, cache):
    assert far(lib, [2, 3, 4, 5, 6, 7, 8] * 20, 2, G, D, cache, seed=D) < 4.2e-7


@pytest.mark.parametrize("D,G,cache,L", [(64, 1, "bf16", 500000), (128, 8, "bf16", 250000),
                                         (64, 2, "fp8", 700000)])
def test_sums_of_fp32_outputs(lib, D, G, cache, L):
    """Some 200 tiles and more a warp."""
    assert far(lib, [L, L], 16, G, D, cache, seed=D + 1) < 1e-6
