"""Host-side checks of the paged-cache entry points (no GPU): every refusal by its status code."""
import ctypes

import pytest
import torch

INVALID, SHAPE, DTYPE, MISALIGNED, WORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def clib():
    import gated_delta_rule_33_gb300 as kda
    kda.build()
    return kda.load()


def _fake(addr=0x10000):
    return ctypes.c_void_p(addr)


def _cache(**kw):
    from gated_delta_rule_33_gb300.kda import _CacheStruct
    a = dict(k=0x10000, v=0x20000, k_scale=None, v_scale=None, page_stride=16 * 4 * 128,
             token_stride=4 * 128, head_stride=128, dtype=0, num_pages=10, page_size=16, heads=4,
             head_dim=128)
    a.update(kw)
    return ctypes.byref(_CacheStruct(**a))


def test_plan_argument_checks(clib):
    def call(**kw):
        a = dict(cached=_fake(0x1000), new=_fake(0x2000), free=_fake(0x3000), F=4,
                 table=_fake(0x4000), P=3, B=2, ps=16, pages=10, seq=_fake(0x5000),
                 cu=_fake(0x6000), slots=_fake(0x7000), N=0x100, used=_fake(0x8000))
        a.update(kw)
        return clib.kda_page_plan(a["cached"], a["new"], a["free"], a["F"], a["table"], a["P"],
                                  a["B"], a["ps"], a["pages"], a["seq"], a["cu"], a["slots"],
                                  a["N"], a["used"], None)
    for bad in (dict(B=-1), dict(N=-1), dict(N=1 << 31), dict(F=-1), dict(P=-1), dict(ps=0),
                dict(pages=-1), dict(cached=None), dict(new=None), dict(free=None),
                dict(table=None), dict(seq=None), dict(cu=None), dict(slots=None),
                dict(used=None), dict(seq=_fake(0x1000)), dict(cu=_fake(0x2000)),
                dict(slots=_fake(0x4000)), dict(used=_fake(0x3000)), dict(table=_fake(0x3000)),
                dict(seq=_fake(0x6000))):
        assert call(**bad) == INVALID, bad
    assert call(pages=1 << 28) == SHAPE          # slots past 2^31
    assert call(free=_fake(0x90002)) == MISALIGNED   # 4 bytes are enough: an advanced list
    for name in ("cached", "new", "table", "seq", "cu", "slots", "used"):
        assert call(**{name: _fake(0x90004)}) == MISALIGNED


def test_cache_description_checks(clib):
    P = _fake(0x900000)

    def both(want, **kw):
        c = _cache(**kw)
        assert clib.kda_paged_append(P, P, 512, 512, P, 1, c, None) == want, kw
        assert clib.kda_paged_decode(P, 512, c, P, 4, P, 1, 4, 1.0, P, 0, None, P, 1 << 30,
                                     None) == want, kw
    for bad in (dict(num_pages=0), dict(page_size=0), dict(heads=0), dict(k=None), dict(v=None),
                dict(dtype=2, k_scale=0x30000), dict(k_scale=0x30000, v_scale=0x30000),
                dict(head_stride=64), dict(token_stride=128), dict(page_stride=512),
                dict(head_stride=16 * 128, token_stride=64), dict(page_stride=-8192),
                dict(page_stride=1 << 60)):
        both(INVALID, **bad)
    both(SHAPE, head_dim=96)
    both(SHAPE, num_pages=1 << 27, page_size=16)
    both(DTYPE, dtype=1)
    both(DTYPE, dtype=7)
    both(MISALIGNED, k=0x10008)
    both(MISALIGNED, token_stride=516)
    both(MISALIGNED, dtype=2, token_stride=520, page_stride=16 * 520)  # 520 bytes
    both(MISALIGNED, dtype=2, k_scale=0x30004, v_scale=0x30000)
    assert clib.kda_paged_append(P, P, 512, 512, P, 1, None, None) == INVALID


def test_append_argument_checks(clib):
    P = _fake(0x900000)

    def call(k=P, v=P, ks=512, vs=512, slots=P, N=3, cache=None):
        return clib.kda_paged_append(k, v, ks, vs, slots, N, cache or _cache(), None)
    for bad in (dict(N=-1), dict(N=1 << 31), dict(k=None), dict(v=None), dict(slots=None),
                dict(ks=504), dict(vs=0), dict(ks=1 << 61), dict(cache=_cache(v=0x10000))):
        assert call(**bad) == INVALID, bad
    assert call(ks=516) == MISALIGNED
    assert call(v=_fake(0x900008)) == MISALIGNED
    assert call(slots=_fake(0x900004)) == MISALIGNED
    assert call(N=0, k=None, v=None, slots=None) == 0       # nothing to do, no device touched


def test_decode_argument_checks(clib):
    import gated_delta_rule_33_gb300 as kda
    P = _fake(0x900000)
    need = kda.kda_paged_decode_workspace_size(2, 8, 4, 128)
    assert need > 0
    assert kda.kda_paged_decode_workspace_size(2, 6, 4, 128) == 0
    assert kda.kda_paged_decode_workspace_size(2, 8, 4, 96) == 0
    assert kda.kda_paged_decode_workspace_size(-1, 8, 4, 128) == 0

    def call(**kw):
        a = dict(q=P, qs=1024, cache=_cache(), table=P, P=4, lens=P, B=2, Hq=8, o=P, odt=0,
                 lse=None, ws=P, wsb=need)
        a.update(kw)
        return clib.kda_paged_decode(a["q"], a["qs"], a["cache"], a["table"], a["P"], a["lens"],
                                     a["B"], a["Hq"], 1.0, a["o"], a["odt"], a["lse"], a["ws"],
                                     a["wsb"], None)
    for bad in (dict(B=-1), dict(P=-1), dict(Hq=0), dict(q=None), dict(table=None),
                dict(lens=None), dict(o=None), dict(qs=1016), dict(qs=1 << 61)):
        assert call(**bad) == INVALID, bad
    assert call(Hq=6) == SHAPE
    assert call(Hq=1 << 30) == SHAPE
    assert call(odt=2) == DTYPE                             # 8 bits are cache storage only
    for bad in (dict(q=_fake(0x900008)), dict(qs=1028), dict(table=_fake(0x900004)),
                dict(lens=_fake(0x900004)), dict(o=_fake(0x900008)), dict(lse=_fake(0x900004)),
                dict(ws=_fake(0x900008))):
        assert call(**bad) == MISALIGNED, bad
    assert call(wsb=need - 1) == WORKSPACE
    assert call(ws=None) == WORKSPACE
    assert call(B=0, q=None, lens=None, table=None, o=None) == 0


def test_python_checks():
    import gated_delta_rule_33_gb300 as kda
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    c = kda.PagedCache(k, k.clone())
    assert (c.num_pages, c.page_size, c.heads, c.head_dim) == (4, 16, 2, 64)
    view = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16).permute(0, 2, 1, 3)
    assert kda.PagedCache(view, view.clone(memory_format=torch.preserve_format)).page_size == 16
    with pytest.raises(ValueError):
        kda.PagedCache(k, view)                             # unequal strides
    with pytest.raises(ValueError):
        kda.PagedCache(k, k[:3])
    with pytest.raises(ValueError):
        kda.PagedCache(k[..., ::2], k[..., ::2])
    with pytest.raises(TypeError):
        kda.PagedCache(k.float(), k.float())
    f8 = k.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        kda.PagedCache(f8, f8.clone(), torch.ones(3), torch.ones(3))
    slots = torch.zeros(5, dtype=torch.int32)
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        kda.kda_paged_append(x.float(), x, slots, c)
    with pytest.raises(ValueError):
        kda.kda_paged_append(x[:4], x, slots, c)
    with pytest.raises(ValueError):
        kda.kda_paged_append(x.transpose(1, 2), x, slots, c)
    with pytest.raises(TypeError):
        kda.kda_paged_append(x, x, slots.long(), c)
