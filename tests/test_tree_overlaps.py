"""Outputs that overlap an input, another output or the workspace: the calls over trees refuse them."""
import ctypes

import pytest
import torch

import gated_delta_rule_33_gb300 as kda
from test_paged_boundary import _cache, _fake
from test_tree_boundary import INVALID, far

FP8 = dict(dtype=2, k=0x500000000, v=0x600000000, k_scale=0x700000000, v_scale=0x710000000)


@pytest.fixture(scope="module")
def clib():
    kda.build()
    return kda.load()


def address(p):
    return ctypes.cast(p, ctypes.c_void_p).value


def inside(p, at):
    return _fake(address(p) + at)


def test_recurrence(clib):
    N, B, H = 24, 9, 2
    good = dict(q=far(0), k=far(1), v=far(2), g=far(3), beta=far(4), pool=far(5), idx=far(6), cu=far(7), anc=far(8),
                o=far(9), u=far(10))
    last = dict(q=N * H * 256, k=N * H * 256, v=N * H * 256, g=N * H * 512, beta=N * H * 4, pool=11 * H * 65536,
                idx=B * 4, cu=B * 4 + 4, anc=N * 8)

    def call(**kw):
        a = {**good, **kw}
        return clib.kda_recurrent_tree_decode(a["q"], a["k"], a["v"], a["g"], a["beta"], a["pool"], 1, a["idx"], 11,
                                              a["cu"], a["anc"], B, N, 4, H, 128, 128, 1.0, a["o"], 0, a["u"], None)
    for name, size in last.items():
        for out in ("o", "u"):
            assert call(**{out: good[name]}) == INVALID, (name, out)
            assert call(**{out: inside(good[name], (size - 1) // 16 * 16)}) == INVALID, (name, out)
            assert call(**{name: inside(good[out], N * H * 256 - 16)}) == INVALID, (name, out)
    assert call(o=good["u"]) == INVALID and call(o=inside(good["u"], N * H * 512 - 16)) == INVALID


def test_pre_step(clib):
    N, B, C = 24, 9, 256
    good = dict(x=far(0), w=far(1), pool=far(2), idx=far(3), cu=far(4), anc=far(5), q=far(6), k=far(7), v=far(8))
    last = dict(x=N * C * 2, w=C * 16, pool=11 * 9 * C * 2, idx=B * 4, cu=B * 4 + 4, anc=N * 8)

    def call(**kw):
        a = {**good, **kw}
        return clib.kda_short_conv_qkv_tree(a["x"], a["x"], a["x"], a["w"], a["w"], a["w"], a["pool"], a["idx"], 11,
                                            a["cu"], a["anc"], B, N, 4, C, a["q"], a["k"], a["v"], None)
    for name, size in last.items():
        for out in ("q", "k", "v"):
            assert call(**{out: good[name]}) == INVALID, (name, out)
            assert call(**{out: inside(good[name], (size - 1) // 16 * 16)}) == INVALID, (name, out)
            assert call(**{name: inside(good[out], N * C * 2 - 16)}) == INVALID, (name, out)


def test_attention(clib):
    N, B, P, Hq, D = 24, 9, 6, 8, 128
    need = kda.kda_paged_tree_decode_workspace_size(B, 4, Hq, 4, D)
    cache = dict(page_stride=16 * 4 * 128, token_stride=4 * 128, head_stride=128, num_pages=10, page_size=16)
    good = dict(q=far(0), table=far(1), lens=far(2), cu=far(3), anc=far(4), o=far(5), lse=far(6), ws=far(7))
    outs = dict(o=N * Hq * D * 2, lse=N * Hq * 4, ws=need)
    row = 3 * Hq * D                                       # q: rows of a fused projection
    last = dict(q=(N - 1) * row * 2 + Hq * D * 2, table=B * P * 4, lens=B * 4, cu=B * 4 + 4, anc=N * 8)

    def call(c=FP8, **kw):
        a = {**good, **kw}
        return clib.kda_paged_tree_decode(a["q"], row, _cache(**{**cache, **c}), a["table"], P, a["lens"], a["cu"],
                                          a["anc"], B, N, 4, Hq, 1.0, a["o"], a["lse"], a["ws"], need, None)
    for out, size in outs.items():
        for name, n in last.items():
            assert call(**{out: good[name]}) == INVALID, (name, out)
            assert call(**{out: inside(good[name], (n - 1) // 16 * 16)}) == INVALID, (name, out)
            assert call(**{name: inside(good[out], size - 16)}) == INVALID, (name, out)
        for name in ("k", "v", "k_scale", "v_scale"):
            assert call(**{out: _fake(FP8[name])}) == INVALID, (name, out)
        for name in ("k", "v"):                            # the last page's last row
            assert call(**{out: _fake(FP8[name] + 10 * 16 * 4 * 128 - 16)}) == INVALID, (name, out)
        for other, n in outs.items():
            if other != out:
                assert call(**{out: good[other]}) == INVALID
                assert call(**{out: inside(good[other], n - 16)}) == INVALID
    # outputs as long as the way from row to row of q meet one wherever they begin in it
    for at in (-N * Hq * D * 2 + 16, Hq * D * 2, row * 2, (N - 2) * row * 2 + Hq * D * 2):
        assert call(o=inside(good["q"], at)) == INVALID, at


def test_compact(clib):
    cache = dict(k=0x500000000, v=0x600000000)
    for at in (0x500000000, 0x600000000, 0x600000000 + 10 * 16 * 4 * 128 * 2 - 16):
        assert clib.kda_paged_compact(_cache(**cache), far(1), 4, far(2), far(3), far(4), far(5), 9, 24, 4,
                                      _fake(at), None) == INVALID


@pytest.mark.gpu
def test_an_output_between_the_rows_of_q(lib):
    """What lies between rows that are far apart is not an input."""
    H, D = 2, 64
    gen = torch.Generator().manual_seed(0)
    k, v = (torch.randn(4, 16, H, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    wide = torch.randn(2, 6 * H * D, generator=gen).to(torch.bfloat16).cuda()
    q = wide[:, :H * D].view(2, H, D)
    table = torch.tensor([[2, 0]], dtype=torch.int32).cuda()
    lens, cu = (torch.tensor(t, dtype=torch.int32).cuda() for t in ([20], [0, 2]))
    words = kda.ancestor_words([-1, 0], "cuda")
    want, _ = lib.paged_tree_decode(q.clone(), lib.PagedCache(k, v), table, lens, cu, words, 2, 0.1)
    o = wide.view(-1)[2 * H * D:4 * H * D].view(2, H, D)
    ws = torch.empty(lib.kda_paged_tree_decode_workspace_size(1, 2, H, H, D), dtype=torch.uint8, device="cuda")
    lib.kda_paged_tree_decode(q, lib.PagedCache(k, v), table, lens, cu, words, 2, 0.1, o, None, ws)
    assert torch.equal(o, want) and lib.kda_get_last_device_error() == 0
