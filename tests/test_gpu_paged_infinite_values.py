"""Attention over a bf16 paged cache that holds infinite or NaN values (GPU): as in fp32
arithmetic, a channel with an infinite value of a key that has weight is infinite, NaN where
infinities of both signs or a NaN meet, and NaN where the key's weight is 0 (0 times infinity).
The other channels are within the attention tests' tolerances."""
import numpy as np
import pytest
import torch

from test_gpu_paged import attention_case, check_decode, run_decode

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def at(x, b, t):
    page = x["k"].shape[1]
    return int(x["table"][b, t // page]), t % page


def check(x, o, lse, special):
    """special: {(sequence, key head, channel): what it has to be}."""
    ref = dict(x, v=x["v"].clone())
    bad = ~torch.isfinite(x["v"].float())
    ref["v"][bad] = 0.0
    o = o.cpu().clone()
    for (b, h, c), want in special.items():
        got = o[b, h * x["G"]:(h + 1) * x["G"], c].float()
        if want != want:
            assert bool(torch.isnan(got).all()), ((b, h, c), want, got)
        else:
            assert bool((got == want).all()), ((b, h, c), want, got)
        o[b, h * x["G"]:(h + 1) * x["G"], c] = 0.0
    # what is left is compared; a special channel counts as 0 with any weight
    for (b, h, c) in special:
        n, page = int(x["lens"][b]), x["k"].shape[1]
        for i in range(-(-n // page)):
            ref["v"][int(x["table"][b, i]), :min(page, n - i * page), h, c] = 0.0
    check_decode(ref, o, lse)


@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,G,D,page", [(2, 4, 128, 16), (1, 1, 64, 24), (3, 12, 128, 64),
                                        (2, 16, 64, 1), (2, 24, 64, 64), (1, 32, 128, 64),
                                        (1, 20, 256, 7), (4, 1, 64, 64), (2, 8, 256, 128)])
def test_infinite_values(lib, H, G, D, page, o_dtype):
    lens = [50, 1, 700, 0, 17]
    x = attention_case(lens, H, G, D, page, seed=D + G)
    special = {}

    def put(b, h, c, **values):
        for t, v in values.items():
            x["v"][at(x, b, int(t[1:]))][h, c] = v
    put(0, 0, 5, k3=INF)
    special[0, 0, 5] = INF
    put(0, H - 1, D - 1, k49=-INF)
    special[0, H - 1, D - 1] = -INF
    put(1, 0, 0, k0=INF)                      # the only key: its weight is 1
    special[1, 0, 0] = INF
    put(1, 0, 33, k0=NAN)
    special[1, 0, 33] = NAN
    put(2, 0, 17, k3=INF, k690=-INF)          # both signs, far apart
    special[2, 0, 17] = NAN
    put(2, 0, 18, k350=-INF, k351=-INF, k699=-INF)
    special[2, 0, 18] = -INF
    put(2, 0, 40, k350=INF, k20=NAN)
    special[2, 0, 40] = NAN
    put(2, H - 1, 41, k0=INF)
    special[2, H - 1, 41] = INF
    put(4, 0, 63, k16=-INF, k15=-INF)
    special[4, 0, 63] = -INF
    o, lse = run_decode(lib, x, o_dtype)
    assert lib.kda_get_last_device_error() == 0
    check(x, o, lse, special)


@pytest.mark.parametrize("H,G,D", [(2, 4, 128), (8, 1, 64), (1, 24, 64), (1, 20, 256), (1, 96, 128)])
def test_infinite_values_in_long_lists(lib, H, G, D):
    """Units that are cut between warps and blocks, and two heads side by side."""
    lens = [40000, 0, 21003]
    x = attention_case(lens, H, G, D, 64, seed=D + G)
    gen = np.random.default_rng(G)
    special = {}
    for c in range(0, D, 3):
        b, h = int(gen.choice([0, 2])), int(gen.integers(H))
        v = float(gen.choice([INF, -INF]))
        x["v"][at(x, b, int(gen.integers(lens[b])))][h, c] = v
        special[b, h, c] = v
    x["v"][at(x, 0, 7)][0, 1], x["v"][at(x, 0, 39999)][0, 1] = INF, -INF
    special[0, 0, 1] = NAN
    o, lse = run_decode(lib, x, torch.bfloat16)
    assert lib.kda_get_last_device_error() == 0
    check(x, o, lse, special)


@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
def test_infinite_value_without_weight(lib, o_dtype):
    """A key whose score is -infinity, or so low that its weight is 0 in fp32, times infinity."""
    x = attention_case([40], 1, 2, 64, 16, seed=2)
    x["q"][:] = -1.0
    x["scale"] = 1.0
    x["k"][at(x, 0, 7)][0, 5] = INF                     # score -inf
    x["v"][at(x, 0, 7)][0, 9] = INF
    x["k"][at(x, 0, 20)][0, 0] = 3000.0                 # score near -3000
    x["v"][at(x, 0, 20)][0, 10] = -INF
    o, lse = run_decode(lib, x, o_dtype)
    got = o.cpu().float()
    assert bool(torch.isnan(got[..., 9:11]).all())
    rest = torch.isfinite(got).sum()
    assert int(rest) == got.numel() - 4


def test_infinite_value_on_a_bad_page(lib):
    """A page that is left out, and values past a sequence's end, are not met."""
    x = attention_case([40, 20], 1, 4, 64, 16, seed=3)
    x["v"][int(x["table"][0, 0]), 3, 0, 5] = INF
    x["v"][int(x["table"][1, 1]), 4:, 0, 6] = INF        # past the 20 keys
    special = {(0, 0, 5): INF}
    whole = x["table"].clone()
    x["table"][0, 1] = x["k"].shape[0]                   # keys 16..31 are on no page
    o, lse = run_decode(lib, x, torch.float32)
    assert lib.kda_get_last_device_error() == 1
    cut = dict(x, table=whole.clone())
    cut["table"][0, :2] = whole[0, [0, 2]]
    cut["lens"] = torch.tensor([24, 20], dtype=torch.int32)
    check(cut, o, lse, special)
