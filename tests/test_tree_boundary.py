"""Host-side checks of the entry points over trees and shared pages (no GPU): every refusal by its
status code, and the binding's own checks."""
import ctypes

import pytest
import torch

import gated_delta_rule_33_gb300 as kda
from gated_delta_rule_33_gb300 import tree as binding
from test_paged_boundary import _cache, _fake

INVALID, SHAPE, DTYPE, MISALIGNED, WORKSPACE = 1, 2, 3, 4, 5
ODD = _fake(0x7000008)


@pytest.fixture(scope="module")
def clib():
    kda.build()
    return kda.load()


def far(i):
    """Addresses that lie apart."""
    return _fake(0x10000000 * (i + 1))


def refuses(call, good, table):
    for status, cases in table.items():
        for bad in cases:
            assert set(bad) <= set(good), bad
            assert call(**{**good, **bad}) == status, bad


def sizes(**kw):
    return dict(B=2, N=8, most=4, **kw)


COMMON = {INVALID: [dict(B=-1), dict(B=65536), dict(N=-1), dict(N=1 << 31), dict(cu=None), dict(anc=None)],
          SHAPE: [dict(most=0), dict(most=65)]}


def test_recurrent_tree_decode_checks(clib):
    good = sizes(q=far(0), k=far(1), v=far(2), g=far(3), beta=far(4), pool=far(5), sdt=1, idx=far(6), slots=3,
                 cu=far(7), anc=far(8), H=2, K=128, V=128, o=far(9), odt=0, u=far(10))

    def call(**a):
        return clib.kda_recurrent_tree_decode(
            a["q"], a["k"], a["v"], a["g"], a["beta"], a["pool"], a["sdt"], a["idx"], a["slots"], a["cu"],
            a["anc"], a["B"], a["N"], a["most"], a["H"], a["K"], a["V"], 1.0, a["o"], a["odt"], a["u"], None)
    refuses(call, good, COMMON)
    refuses(call, good, {
        INVALID: [dict(H=0), dict(slots=-1), dict(idx=None, slots=1), dict(pool=None), dict(o=None)]
        + [{n: None} for n in ("q", "k", "v", "g", "beta")]
        + [dict(o=good[n]) for n in ("q", "k", "v", "g", "pool", "u")] + [dict(u=good["pool"]), dict(u=good["k"])],
        SHAPE: [dict(K=64), dict(V=256), dict(B=65535, slots=65535, H=1 << 16)],
        DTYPE: [dict(sdt=2), dict(odt=2), dict(odt=9)],
        MISALIGNED: [{n: ODD} for n in ("q", "k", "v", "g", "beta", "pool", "idx", "cu", "anc", "o", "u")]})
    assert call(**{**good, "B": 0, "cu": None}) == 0


def test_recurrent_tree_commit_checks(clib):
    good = sizes(k=far(1), g=far(3), u=far(4), pool=far(5), sdt=0, idx=far(6), slots=3, cu=far(7), anc=far(8),
                 last=far(9), H=2, K=128, V=128)

    def call(**a):
        return clib.kda_recurrent_tree_commit(a["k"], a["g"], a["u"], a["pool"], a["sdt"], a["idx"], a["slots"],
                                              a["cu"], a["anc"], a["last"], a["B"], a["N"], a["most"], a["H"],
                                              a["K"], a["V"], None)
    refuses(call, good, COMMON)
    refuses(call, good, {
        INVALID: [dict(H=0), dict(slots=-1), dict(idx=None, slots=1), dict(last=None)]
        + [{n: None} for n in ("k", "g", "u", "pool")],
        SHAPE: [dict(K=64), dict(V=256)], DTYPE: [dict(sdt=2)],
        MISALIGNED: [{n: ODD} for n in ("k", "g", "u", "pool", "idx", "cu", "anc", "last")]})
    assert call(**{**good, "B": 0, "cu": None}) == 0


def test_conv_checks(clib):
    good = sizes(x=far(0), w=far(1), pool=far(2), idx=far(3), slots=3, cu=far(4), anc=far(5), C=256, q=far(6),
                 k=far(7), v=far(8))

    def call(**a):
        return clib.kda_short_conv_qkv_tree(a["x"], a["x"], a["x"], a["w"], a["w"], a["w"], a["pool"], a["idx"],
                                            a["slots"], a["cu"], a["anc"], a["B"], a["N"], a["most"], a["C"],
                                            a["q"], a["k"], a["v"], None)
    refuses(call, good, COMMON)
    refuses(call, good, {
        INVALID: [dict(slots=-1), dict(idx=None, slots=1)] + [{n: None} for n in ("x", "w", "pool", "q", "k", "v")]
        + [dict(q=good[n]) for n in ("x", "w", "pool", "k", "v")],
        SHAPE: [dict(C=0), dict(C=200)],
        MISALIGNED: [{n: ODD} for n in ("x", "w", "pool", "idx", "cu", "anc", "q", "k", "v")]})
    good["last"] = far(9)

    def commit(**a):
        return clib.kda_short_conv_tree_commit(a["x"], a["x"], a["x"], a["pool"], a["idx"], a["slots"], a["cu"],
                                               a["anc"], a["last"], a["B"], a["N"], a["most"], a["C"], None)
    refuses(commit, good, COMMON)
    refuses(commit, good, {
        INVALID: [dict(slots=-1), dict(idx=None, slots=1)] + [{n: None} for n in ("x", "pool", "last")],
        SHAPE: [dict(C=0), dict(C=200)],
        MISALIGNED: [{n: ODD} for n in ("x", "pool", "idx", "cu", "anc", "last")]})
    assert call(**{**good, "B": 0, "cu": None}) == 0 and commit(**{**good, "B": 0, "cu": None}) == 0


def test_attention_checks(clib):
    need = kda.kda_paged_tree_decode_workspace_size(2, 4, 8, 4, 128)
    assert need > 0
    for bad in ((-1, 4, 8, 4, 128), (65536, 4, 8, 4, 128), (2, 0, 8, 4, 128), (2, 65, 8, 4, 128),
                (2, 4, 6, 4, 128), (2, 4, 8, 0, 128), (2, 4, 0, 4, 128), (2, 4, 8, 4, 96),
                (65535, 64, 1 << 20, 1, 64)):
        assert kda.kda_paged_tree_decode_workspace_size(*bad) == 0, bad
    good = sizes(q=far(0), qs=1024, cache=_cache(), table=far(1), P=4, lens=far(2), cu=far(3), anc=far(4), Hq=8,
                 o=far(5), lse=far(6), ws=far(7), wsb=need)

    def call(**a):
        return clib.kda_paged_tree_decode(a["q"], a["qs"], a["cache"], a["table"], a["P"], a["lens"], a["cu"],
                                          a["anc"], a["B"], a["N"], a["most"], a["Hq"], 1.0, a["o"], a["lse"],
                                          a["ws"], a["wsb"], None)
    refuses(call, good, COMMON)
    refuses(call, good, {
        INVALID: [dict(P=-1), dict(Hq=0), dict(qs=1016), dict(qs=1 << 61), dict(cache=None),
                  dict(cache=_cache(heads=0)), dict(cache=_cache(k_scale=0x30000))]
        + [{n: None} for n in ("q", "table", "lens", "o")],
        SHAPE: [dict(Hq=6), dict(Hq=1 << 30), dict(cache=_cache(head_dim=96)), dict(Hq=1 << 20, N=1 << 30)],
        DTYPE: [dict(cache=_cache(dtype=1))],
        MISALIGNED: [{n: ODD} for n in ("q", "table", "lens", "cu", "anc", "o", "lse", "ws")] + [dict(qs=1028)],
        WORKSPACE: [dict(wsb=need - 1), dict(ws=None)]})
    assert call(**{**good, "B": 0, "N": 0, "cu": None, "lens": None}) == 0
    assert call(**{**good, "N": 0, "q": None, "o": None, "anc": None}) == 0


def test_compact_and_copy_checks(clib):
    good = sizes(cache=_cache(), table=far(1), P=4, lens=far(2), cu=far(3), anc=far(4), last=far(5), kept=far(6))

    def call(**a):
        return clib.kda_paged_compact(a["cache"], a["table"], a["P"], a["lens"], a["cu"], a["anc"], a["last"],
                                      a["B"], a["N"], a["most"], a["kept"], None)
    refuses(call, good, COMMON)
    refuses(call, good, {
        INVALID: [dict(P=-1), dict(cache=None), dict(cache=_cache(v=0x10000))]
        + [{n: None} for n in ("table", "lens", "last")]
        + [dict(kept=good[n]) for n in ("table", "lens", "cu", "anc", "last")],
        MISALIGNED: [{n: ODD} for n in ("table", "lens", "cu", "anc", "last", "kept")]})
    assert call(**{**good, "B": 0, "cu": None, "lens": None, "last": None}) == 0

    def copy(copies=far(0), n=3, cache=None):
        return clib.kda_paged_copy(copies, n, cache or _cache(), None)
    assert copy(n=-1) == INVALID and copy(copies=None) == INVALID and copy(copies=ODD) == MISALIGNED
    assert copy(cache=_cache(v=0x10000)) == INVALID and copy(cache=_cache(head_dim=32)) == SHAPE
    assert copy(copies=None, n=0) == 0


def test_fork_and_release_checks(clib):
    good = dict(src=far(0), dst=far(1), F=3, lens=far(2), free=far(3), nf=5, table=far(4), P=4, B=6, ps=16,
                pages=100, shares=far(5), copies=far(6), used=far(7))

    def call(**a):
        return clib.kda_page_fork(a["src"], a["dst"], a["F"], a["lens"], a["free"], a["nf"], a["table"], a["P"],
                                  a["B"], a["ps"], a["pages"], a["shares"], a["copies"], a["used"], None)
    refuses(call, good, {
        INVALID: [dict(F=-1), dict(nf=-1), dict(P=-1), dict(B=-1), dict(ps=0), dict(pages=-1)]
        + [{n: None} for n in ("src", "dst", "lens", "free", "table", "shares", "copies", "used")]
        + [dict(lens=good[n]) for n in ("table", "shares", "copies", "used", "src", "dst", "free")]
        + [dict(shares=good["table"]), dict(copies=good["src"]), dict(used=good["free"])],
        SHAPE: [dict(pages=1 << 28)],
        MISALIGNED: [{n: ODD} for n in ("src", "dst", "lens", "table", "shares", "copies", "used")]
        + [dict(free=_fake(0x7000002))]})
    good = dict(lens=far(0), kept=far(1), table=far(2), P=4, B=6, ps=16, pages=100, shares=far(3), freed=far(4),
                most=100, num=far(5))

    def release(**a):
        return clib.kda_page_release(a["lens"], a["kept"], a["table"], a["P"], a["B"], a["ps"], a["pages"],
                                     a["shares"], a["freed"], a["most"], a["num"], None)
    refuses(release, good, {
        INVALID: [dict(P=-1), dict(B=-1), dict(ps=0), dict(pages=-1), dict(most=-1)]
        + [{n: None} for n in ("lens", "kept", "table", "shares", "freed", "num")]
        + [dict(shares=good[n]) for n in ("lens", "kept", "table", "freed", "num")]
        + [dict(freed=good["table"]), dict(num=good["kept"])],
        SHAPE: [dict(pages=1 << 28)],
        MISALIGNED: [{n: ODD} for n in ("lens", "kept", "table", "shares", "num")] + [dict(freed=_fake(0x7000002))]})


def test_ancestor_words():
    assert kda.ancestor_words([-1, 0, 0, 2, -1]).tolist() == [1, 3, 5, 13, 16]
    assert kda.ancestor_words([]).tolist() == []
    chain = kda.ancestor_words([i - 1 for i in range(64)])
    assert chain[62] == 2 ** 63 - 1 and chain[63] == -1
    for bad in ([0], [-1, 1], [-2], [-1] * 65):
        with pytest.raises(ValueError):
            kda.ancestor_words(bad)


class OnGpu(torch.Tensor):
    """A host tensor that says it is on GPU `index`; its memory is never reached."""
    index = 0

    def get_device(self):
        return self.index


def on_gpu(t, index=0):
    out = t.as_subclass(OnGpu)
    out.index = index
    return out


def calls():
    """Every entry point as (function of (cache, tensors), tensors)."""
    i32, f32, b16 = dict(dtype=torch.int32), dict(dtype=torch.float32), dict(dtype=torch.bfloat16)
    N, H, B = 5, 2, 3
    row = torch.zeros(N, H, 128, **b16)
    cu, anc, per = torch.zeros(B + 1, **i32), torch.zeros(N, dtype=torch.int64), torch.zeros(B, **i32)
    pool, conv = torch.zeros(4, H, 128, 128), torch.zeros(4, 3, 3, 256, **b16)
    x, w, table = torch.zeros(N, 256, **b16), torch.zeros(256, 4), torch.zeros(B, 2, **i32)
    q = torch.zeros(N, 4, 64, **b16)
    return {
        "kda_recurrent_tree_decode": (lambda c, t, s: kda.kda_recurrent_tree_decode(*t[:9], 4, 1.0, *t[9:], stream=s),
                                      [row, row, row, row.float(), torch.zeros(N, H, **f32), pool, per, cu, anc, row,
                                       row.float()]),
        "kda_recurrent_tree_commit": (lambda c, t, s: kda.kda_recurrent_tree_commit(*t, 4, stream=s),
                                      [row, row.float(), row.float(), pool, per, cu, anc, per]),
        "kda_short_conv_qkv_tree": (lambda c, t, s: kda.kda_short_conv_qkv_tree(*t[:10], 4, *t[10:], stream=s),
                                    [x, x, x, w, w, w, conv, per, cu, anc, x, x, x]),
        "kda_short_conv_tree_commit": (lambda c, t, s: kda.kda_short_conv_tree_commit(*t, 4, stream=s),
                                       [x, x, x, conv, per, cu, anc, per]),
        "kda_paged_tree_decode": (lambda c, t, s: kda.kda_paged_tree_decode(t[0], c, *t[1:5], 4, 1.0, *t[5:], stream=s),
                                  [q, table, per, cu, anc, q, torch.zeros(N, 4), torch.zeros(1 << 16, dtype=torch.uint8)]),
        "kda_paged_compact": (lambda c, t, s: kda.kda_paged_compact(c, *t[:5], 4, t[5], stream=s),
                              [table, per, cu, anc, per, per]),
        "kda_page_fork": (lambda c, t, s: kda.kda_page_fork(*t[:5], 16, *t[5:], stream=s),
                          [per, per, per, torch.zeros(9, **i32), table, torch.zeros(20, **i32),
                           torch.zeros(3, 3, **i32), torch.zeros(1, **i32)]),
        "kda_paged_copy": (lambda c, t, s: kda.kda_paged_copy(*t, c, stream=s), [torch.zeros(2, 3, **i32)]),
        "kda_page_release": (lambda c, t, s: kda.kda_page_release(*t[:3], 16, *t[3:], stream=s),
                             [per, per, table, torch.zeros(20, **i32), torch.zeros(20, **i32), torch.zeros(1, **i32)]),
    }


@pytest.fixture
def reached(monkeypatch):
    """Stands for the library: notes the calls that pass the binding's checks."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0
    monkeypatch.setattr(kda.kda, "_lib", Lib())
    return seen


@pytest.mark.parametrize("stream", [0, 77])
@pytest.mark.parametrize("name", sorted(calls()))
def test_every_tensor_is_checked(reached, name, stream):
    call, tensors = calls()[name]
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    cache = kda.PagedCache(on_gpu(k), on_gpu(k.clone()))
    call(cache, [on_gpu(t.clone()) for t in tensors], stream)
    assert reached == [name]
    for i, t in enumerate(tensors):
        for wrong in (t.clone(), on_gpu(t.clone(), 1),                        # on the host, on another GPU
                      on_gpu(t.to(torch.float64)),
                      on_gpu(torch.zeros([n + 1 for n in t.shape], dtype=t.dtype))):
            if wrong.shape != t.shape and (
                    t.numel() == 0 or (name, i) in {("kda_paged_tree_decode", 7), ("kda_paged_compact", 3), ("kda_page_fork", 3),
                                                    ("kda_page_fork", 5), ("kda_page_release", 3),
                                                    ("kda_page_release", 4)}):
                continue                                                      # any length will do
            if wrong.dtype is torch.float64 and (name, i) == ("kda_paged_tree_decode", 7):
                continue                                                      # a workspace of any type
            a = [on_gpu(x.clone()) for x in tensors]
            a[i] = wrong
            with pytest.raises((ValueError, TypeError)):
                call(cache, a, stream)
    assert reached == [name]


CONVENIENCES = {"recurrent_tree_decode": 1, "short_conv_tree": 1, "paged_tree_decode": 1, "paged_compact": 1,
                "page_fork": 1, "page_release": 1}


def test_conveniences_allocate_on_the_given_stream(monkeypatch):
    import inspect
    names = [n for n, f in vars(binding).items()
             if inspect.isfunction(f) and f.__module__ == binding.__name__ and not n.startswith(("_", "kda_"))
             and "stream" in inspect.signature(f).parameters]
    assert sorted(names) == sorted(CONVENIENCES)
    on, made = [], []

    class Context:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            on.append(self.stream)

        def __exit__(self, *_):
            on.pop()
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: ("stream", h))
    monkeypatch.setattr(torch.cuda, "stream", Context)
    for maker in ("empty", "empty_like"):
        real = getattr(torch, maker)
        monkeypatch.setattr(torch, maker, lambda *a, _f=real, **kw: made.append(list(on)) or _f(*a, **kw))
    for entry in [n for n in vars(binding) if n.startswith("kda_")]:
        monkeypatch.setattr(binding, entry, (lambda *a: 4096) if entry.endswith("_size") else lambda *a, **kw: None)
    i32 = torch.zeros(3, dtype=torch.int32)
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    x = torch.zeros(5, 2, 64)
    have = dict(q=x, k=x, v=x, g=x, beta=x, state_pool=x, cu_seqlens=i32, ancestors=i32, x_q=x, x_k=x, x_v=x, w_q=x,
                w_k=x, w_v=x, conv_state_pool=x, cache=kda.PagedCache(k, k.clone()), block_table=i32.view(3, 1),
                seq_lens=i32, last=i32, src=i32, dst=i32, free_pages=i32, page_size=16, shares=i32, kept_lens=i32)
    for name in names:
        f = getattr(binding, name)
        for handle in (None, 77):
            made.clear()
            f(**{n: have[n] for n, p in inspect.signature(f).parameters.items()
                 if p.default is inspect.Parameter.empty}, stream=handle)
            want = [] if handle is None else [("stream", handle)]
            assert made and all(m == want for m in made) and not on, name
