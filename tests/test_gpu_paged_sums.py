"""bf16 attention outputs of up to 8 heads a key head over long lists are fp32 outputs rounded
once (GPU): the sums of a warp's some 300 tiles lose nothing that a bf16 output shows.

Derivation of the share that may differ.  Values of one sign make the outputs as large as their
weighted values.  A tile takes at most four matrix instructions, each of which cuts off at most
2^-24 of the sum in it, adding the tiles in fp32 and the fp32 output's own error are below 4e-7
each, and the weights' 16 bits round both ways, to nothing over thousands of keys: within 1e-6 in
all.  Two outputs that are 1e-6 apart are rounded apart where a boundary lies between them, and
those are 2^-8 apart at the nearest: in a share of 2.6e-4.  (One running sum over the tiles differs
in a share of 1e-2.)"""
import pytest
import torch

from parity_utils import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,H,G,D,L", [("bf16", 16, 8, 128, 75001), ("fp8", 16, 8, 128, 150000),
                                           ("bf16", 16, 8, 64, 150000)])
def test_bf16_outputs_are_fp32_outputs_rounded(lib, cache, H, G, D, L):
    B, page = 8, 64
    gen = torch.Generator(device=DEV).manual_seed(D)
    held = -(-L // page)
    dtype = torch.float8_e4m3fn if cache == "fp8" else torch.bfloat16
    k, v = (torch.empty(B * held, page, H, D, dtype=dtype, device=DEV) for _ in range(2))
    for b in range(B):
        part = slice(b * held, (b + 1) * held)
        base = 1.0 + torch.rand(H, D, device=DEV, generator=gen)    # outputs all over bf16's steps
        k[part].copy_(torch.randn(k[part].shape, device=DEV, generator=gen))
        v[part].copy_(base + 0.5 * torch.rand(v[part].shape, device=DEV, generator=gen))
    table = torch.arange(B * held, dtype=torch.int32, device=DEV).view(B, held)
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    q = torch.randn(B, H * G, D, device=DEV, generator=gen).to(torch.bfloat16)
    ones = torch.ones(H, device=DEV) if cache == "fp8" else None
    c = lib.PagedCache(k, v, ones, ones)
    o, _ = lib.paged_decode(q, c, table, lens, 0.5 * D ** -0.5)
    wide, _ = lib.paged_decode(q, c, table, lens, 0.5 * D ** -0.5, o_dtype=torch.float32)
    assert lib.kda_get_last_device_error() == 0
    assert float((o != wide.to(torch.bfloat16)).double().mean()) < 2.6e-4
