"""Tree attention over caches in which some values are not finite, in batches where a block has many
units: what sees one gets it, in its channel; all else is as it was, however long the contexts are."""
import numpy as np
import pytest
import torch

from parity_utils import DEV
from test_gpu_tree_attention import check, on_device, tree_case
from test_gpu_tree_attention_units import expected, many_units

pytestmark = pytest.mark.gpu


def spoil(x, v, b, j, head, channel, value):
    """v [pages, page, heads, channels] on the device: key j of request b."""
    page = v.shape[1]
    raw = v.view(torch.uint8) if v.element_size() == 1 else v
    value = torch.tensor([value]).to(v.dtype)
    if v.element_size() == 1:
        value = value.view(torch.uint8)
    raw[int(x["table"][b, j // page]), j % page, head, channel] = value.to(DEV)[0]


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("cache,D,H,G,wide", [("bf16", 128, 8, 8, 4), ("fp8", 128, 8, 8, 4), ("bf16", 64, 6, 12, 3),
                                              ("fp8", 64, 8, 2, 0), ("bf16", 256, 8, 4, 0),
                                              ("fp8", 256, 4, 8, 0)])
def test_values_of_some_requests(lib, cache, D, H, G, wide, value):
    if cache == "fp8" and np.isinf(value):
        value = float("nan")                                   # 8 bits hold no infinity
    x = many_units(D, H, G, wide, cache, 1500, seed=D + G)
    c, args = on_device(lib, x)
    q = x["q"].to(DEV)
    o0, lse0 = lib.paged_tree_decode(q, c, *args, x["most"], x["scale"], want_lse=True)
    ref = expected(x)
    check(x, o0, lse0, ref)
    hit = torch.zeros(o0.shape, dtype=torch.bool)
    touched = torch.zeros(len(hit), dtype=torch.bool, device=DEV)
    rng = np.random.default_rng(D)
    for b in rng.choice(60, 25, replace=False):
        lo, hi = int(x["cu"][b]), int(x["cu"][b + 1])
        L, h, ch = int(x["lens"][b]), int(rng.integers(0, H)), int(rng.integers(0, D))
        if b % 2:                                              # of the context
            spoil(x, c.v_cache, b, int(rng.integers(0, L - (hi - lo))), h, ch, value)
            rows = list(range(lo, hi))
        else:                                                  # of a drafted token
            node = int(rng.integers(0, hi - lo))
            spoil(x, c.v_cache, b, L - (hi - lo) + node, h, ch, value)
            rows = [r for r in range(lo, hi) if x["words"][r] >> node & 1]
        touched[lo:hi] = True
        for r in rows:
            hit[r, h * G:(h + 1) * G, ch] = True
    o, lse = lib.paged_tree_decode(q, c, *args, x["most"], x["scale"], want_lse=True)
    assert lib.kda_get_last_device_error() == 0
    got = o.cpu()[hit].float()
    assert (torch.isnan(got) if np.isnan(value) else got == value).all()
    assert torch.equal(lse, lse0)
    o = torch.where(hit.to(DEV), o0, o)                        # everything else
    check(x, o, lse, ref)
    assert torch.equal(o[~touched], o0[~touched])              # other requests: the same bits


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_a_long_context_among_many(lib, cache):
    """One value of a long context that 64 nodes of 8 heads see (512 rows over 8192 keys), next to 64
    requests: no wait runs out, and the others' outputs are what they were."""
    x = tree_case([(64, 8128)] + [(8, 1000 + 7 * i) for i in range(64)], 8, 8, 128, 64, cache, seed=3)
    c, args = on_device(lib, x)
    q = x["q"].to(DEV)

    def call():
        return lib.paged_tree_decode(q, c, *args, 64, x["scale"], want_lse=True)
    o0, lse0 = call()
    spoil(x, c.v_cache, 0, 4000, 5, 17, float("nan"))
    o, lse = call()
    assert lib.kda_get_last_device_error() == 0
    assert torch.equal(lse, lse0) and torch.equal(o[64:], o0[64:])
    assert torch.isnan(o[:64, 40:48, 17]).all()
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[:64, 40:48, 16:24] = False                            # the eight channels that are computed again
    assert torch.equal(o[keep], o0[keep])
    near = [16, 18, 19, 20, 21, 22, 23]
    err = (o[:64, 40:48, near].float() - o0[:64, 40:48, near].float()).abs()
    assert (err <= 2.0 ** -6 * o0[:64, 40:48].float().abs().amax()).all()
