"""GPU tests of the calls that move, share and free pages: exact, against the plain definitions."""
import numpy as np
import pytest
import torch

from oracle import paged, tree
from parity_utils import DEV
from test_gpu_paged import as_device
from test_gpu_tree_attention import random_tree, signed

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device=DEV)


def filled(pages, page, H, D, cache, order, seed):
    gen = torch.Generator().manual_seed(seed)
    dtype = torch.float8_e4m3fn if cache == "fp8" else torch.bfloat16
    out = []
    for _ in range(2):
        shape = (pages, H, page, D) if order == "head" else (pages, page, H, D)
        t = torch.randn(shape, generator=gen).to(dtype)
        out.append(t.permute(0, 2, 1, 3) if order == "head" else t)
    return out


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


@pytest.mark.parametrize("cache,order", [("bf16", "token"), ("fp8", "head")])
@pytest.mark.parametrize("H,D,page", [(2, 64, 16), (8, 128, 24), (1, 256, 1), (3, 128, 7)])
def test_compact(lib, H, D, page, cache, order):
    rng = np.random.default_rng(H * D + page)
    shapes = [(1, 0), (64, 3), (0, 9), (17, 100), (5, 2), (64, 0), (30, 31), (8, 50)]
    lens = [n + c for n, c in shapes]
    held = [paged.pages(x, page) for x in lens]
    pages = sum(held) + 2
    perm = rng.permutation(pages)
    table = np.full((len(shapes), max(held)), -1)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    cu = np.concatenate([[0], np.cumsum([n for n, _ in shapes])])
    words = [w for b, (n, _) in enumerate(shapes) for w in random_tree(n, rng, chain=b == 5)]
    last = [0, 63, -1, 16, -1, 63, int(rng.integers(0, 30)), 7]
    k, v = filled(pages, page, H, D, cache, order, 1)
    c = lib.PagedCache(as_device(k), as_device(v))
    kept = lib.paged_compact(c, torch.tensor(table, **I32), torch.tensor(lens, **I32), torch.tensor(cu, **I32),
                             signed(words).to(DEV), torch.tensor(last, **I32), 64)
    assert lib.kda_get_last_device_error() == 0
    for got, t in ((c.k_cache, k), (c.v_cache, v)):
        want, lens_ref = tree.compact(bits(t).view(pages, page, -1).numpy(), table, lens, cu, words, last, page)
        assert kept.tolist() == lens_ref
        for b, (n, _) in enumerate(shapes):                # behind the kept length nothing is defined
            for p in range(lens_ref[b]):
                at = table[b][p // page], p % page
                assert (bits(got).view(pages, page, -1)[at].numpy() == want[at]).all()
        spare = perm[sum(held):]
        assert torch.equal(bits(got).view(pages, page, -1)[spare], bits(t).view(pages, page, -1)[spare])


def test_compact_refusals(lib):
    k, v = filled(8, 16, 2, 64, "bf16", "token", 0)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], **I32)
    lens, cu = torch.tensor([20, 18, 17], **I32), torch.tensor([0, 6, 10, 13], **I32)
    words = signed(tree.words([-1, -1, 0, 1, 1, 4]) + tree.words([-1, 0, 0, 0]) + tree.words([-1, -1, 1])).to(DEV)
    last = torch.tensor([5, 3, 2], **I32)

    def call(table=table, lens=lens, cu=cu, last=last, most=6):
        c = lib.PagedCache(k.to(DEV), v.to(DEV))
        kept = torch.full((3,), -7, **I32)
        lib.kda_paged_compact(c, table, lens, cu, words, last, most, kept)
        return c, kept.tolist(), lib.kda_get_last_device_error()
    c, kept, err = call()
    assert err == 0 and kept == [14 + 3, 14 + 2, 14 + 2]
    good = c.k_cache.cpu()
    for bad in (dict(last=torch.tensor([6, 3, 2], **I32)), dict(most=5), dict(lens=torch.tensor([5, 18, 17], **I32)),
                dict(lens=torch.tensor([33, 18, 17], **I32))):
        c, kept, err = call(**bad)
        assert err == 1 and kept[1:] == [16, 16]
        assert kept[0] == (0 if "lens" in bad else 14)
        assert torch.equal(c.k_cache[:2].cpu(), k[:2]) and torch.equal(c.k_cache[2:].cpu(), good[2:])
    for page in (-1, 8, 2 ** 31 - 1):
        bad = table.clone()
        bad[0, 1] = page                                   # rows 16 .. stay where they are
        c, kept, err = call(table=bad)
        assert err == 1 and torch.equal(c.k_cache[2:].cpu(), good[2:])
    for wrong in ([0, 6, 10, 14], [0, 6, 5, 13], [-2, 6, 10, 13]):
        assert call(cu=torch.tensor(wrong, **I32))[2] == 1


@pytest.mark.parametrize("cache,order", [("bf16", "head"), ("fp8", "token")])
@pytest.mark.parametrize("H,D,page", [(2, 64, 16), (8, 128, 33), (5, 256, 1), (1, 64, 200)])
def test_copy(lib, H, D, page, cache, order):
    k, v = filled(20, page, H, D, cache, order, 2)
    c = lib.PagedCache(as_device(k), as_device(v))
    rng = np.random.default_rng(page)
    entries = [[int(s), int(d), int(rng.integers(1, page + 1))]
               for s, d in zip(rng.integers(0, 10, 8), 10 + rng.permutation(10)[:8])]
    entries += [[-1, -1, 0], [3, 3, page]]
    lib.kda_paged_copy(torch.tensor(entries, **I32), c)
    assert lib.kda_get_last_device_error() == 0
    for got, t in ((c.k_cache, k), (c.v_cache, v)):
        want = bits(t).view(20, page, -1).clone()
        for s, d, n in entries[:8]:
            want[d, :n] = bits(t).view(20, page, -1)[s, :n]
        assert torch.equal(bits(got).view(20, page, -1), want)
    before = bits(c.k_cache)
    for bad in ([20, 1, 1], [1, 20, 1], [-1, 1, 1], [1, -1, 1], [1, 2, page + 1], [1, 2, -1]):
        lib.kda_paged_copy(torch.tensor([bad], **I32), c)
        assert lib.kda_get_last_device_error() == 1
    assert torch.equal(bits(c.k_cache), before)
    lib.kda_paged_copy(torch.zeros(0, 3, **I32), c)


def fork(lib, src, dst, lens, free, table, page, pages, shares):
    seq, t, s = (torch.tensor(np.asarray(x), **I32) for x in (lens, table, shares))
    copies, used = lib.page_fork(torch.tensor(src, **I32), torch.tensor(dst, **I32), seq,
                                 torch.tensor(free, **I32), t, page, s)
    return seq.tolist(), t.cpu().numpy(), s.cpu().numpy(), copies.tolist(), int(used)


def check_fork(lib, *args):
    got = fork(lib, *args)
    want = tree.fork(*args)
    assert lib.kda_get_last_device_error() == int(want[5])
    assert got[0] == want[0] and (got[1] == want[1]).all() and (got[2] == want[2]).all()
    assert got[3] == want[3] and got[4] == want[4]
    return want


def world(B, page, longest, seed, spare=50):
    """Requests with pages of their own; every third row is empty."""
    rng = np.random.default_rng(seed)
    lens = [0 if b % 3 == 0 else int(rng.integers(0, longest + 1)) for b in range(B)]
    held = [paged.pages(n, page) for n in lens]
    pages = sum(held) + spare
    perm = rng.permutation(pages)
    table = np.full((B, paged.pages(longest, page) + 1), -1)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    return rng, lens, table, pages, [int(p) for p in perm[at:]]


@pytest.mark.parametrize("B,page,longest", [(3, 4, 9), (40, 16, 300), (600, 16, 100), (2000, 1, 12), (9, 64, 20000)])
def test_fork_then_release(lib, B, page, longest):
    rng, lens, table, pages, free = world(B, page, longest, B, spare=B)
    dst = [b for b in range(B) if b % 3 == 0]
    src = [int(rng.choice([b for b in range(B) if b % 3])) for _ in dst]
    seq, t, shares, _, used, bad = check_fork(lib, src, dst, lens, free, table, page, pages, np.zeros(pages, int))
    assert not bad and used == sum(1 for s in src if lens[s] % page)
    for _ in range(2):                                     # what remains is released in two steps
        kept = [0 if rng.random() < 0.4 else int(rng.integers(0, n + 1)) for n in seq]
        s = torch.tensor(shares, **I32)
        freed, num = lib.page_release(torch.tensor(seq, **I32), torch.tensor(kept, **I32), torch.tensor(t, **I32),
                                      page, s)
        shares, want, bad = tree.release(seq, kept, t, page, pages, shares)
        assert lib.kda_get_last_device_error() == 0 and not bad
        assert freed[:int(num)].tolist() == want and (s.cpu().numpy() == shares).all()
        seq = kept
    s = torch.tensor(shares, **I32)
    freed, num = lib.page_release(torch.tensor(seq, **I32), torch.zeros(B, **I32), torch.tensor(t, **I32), page, s)
    assert not s.any()                                     # nobody holds a page


def test_fork_refusals(lib):
    _, lens, table, pages, free = world(12, 4, 30, 5)
    lens[1], lens[2], lens[4] = 9, 8, 0
    table[1, :3], table[2, :2] = [0, 1, 2], [3, 4]
    zero = np.zeros(pages, int)

    def refused(src, dst, free=free, lens=lens, table=table):
        want = check_fork(lib, src, dst, lens, free, table, 4, pages, zero)
        assert want[5]
    refused([1, 12, -1, 2], [0, 3, 6, 9])                  # sources out of range
    refused([1, 2, 1], [12, -1, 0])                        # destinations out of range
    refused([1, 2, 1], [0, 0, 3])                          # one destination twice
    refused([1, 0, 2], [0, 3, 6])                          # a destination that is a source
    refused([1, 1, 2, 1], [0, 3, 6, 9], free=free[:2])     # two pages for three
    refused([1], [0], free=[])
    refused([1, 2], [0, 3], lens=[0, -9, 8] + lens[3:])
    refused([1, 2], [0, 3], lens=[0, table.shape[1] * 4 + 1, 8] + lens[3:])
    for page in (-1, pages, 2 ** 31 - 1):
        bad = table.copy()
        bad[1, 0], bad[2, 1] = page, page
        refused([1, 2], [0, 3], table=bad)                 # a full page that is not one
        bad = table.copy()
        bad[1, 2] = page
        refused([1, 2], [0, 3], table=bad)                 # a last page
    check_fork(lib, [], [], lens, free, table, 4, pages, zero)
    check_fork(lib, [4], [0], lens, free, table, 4, pages, zero)   # an empty source


def test_release_refusals(lib):
    table = [[0, 1, 2], [3, 4, 5], [1, 6, 7], [8, -1, 10]]
    for seq, kept in (([12, -1, 4, 4], [0, 0, 0, 0]), ([12, 13, 4, 4], [0, 0, 0, 0]),
                      ([12, 8, 4, 4], [0, 9, 0, 0]), ([12, 8, 4, 4], [0, -1, 0, 0]),
                      ([8, 8, 4, 0], [0, 0, 0, 0]),        # page 1 is given back twice
                      ([4, 0, 4, 12], [0, 0, 0, 0]),       # a page that is not one
                      ([4, 0, 0, 12], [0, 0, 0, 5])):
        shares = np.zeros(10, int)
        s = torch.tensor(shares, **I32)
        freed, num = lib.page_release(torch.tensor(seq, **I32), torch.tensor(kept, **I32),
                                      torch.tensor(table, **I32), 4, s)
        want_s, want, bad = tree.release(seq, kept, table, 4, 10, shares)
        assert lib.kda_get_last_device_error() == int(bad) == 1
        assert freed[:int(num)].tolist() == want and (s.cpu().numpy() == want_s).all()
    # a list that is too short, and what lies behind the freed pages
    s, freed, num = torch.zeros(10, **I32), torch.full((9,), -7, **I32), torch.zeros(1, **I32)
    args = (torch.tensor([12], **I32), torch.tensor([0], **I32), torch.tensor(table[:1], **I32), 4, s)
    lib.kda_page_release(*args, freed[3:], num)
    assert lib.kda_get_last_device_error() == 0
    assert freed.tolist() == [-7, -7, -7, 0, 1, 2, -7, -7, -7] and int(num) == 3
    freed.fill_(-7)
    lib.kda_page_release(*args, freed[5:7], num)
    assert lib.kda_get_last_device_error() == 1
    assert freed.tolist() == [-7] * 5 + [0, 1] + [-7] * 2 and int(num) == 2 and not s.any()
    lib.kda_page_release(*(t[:0] for t in args[:3]), 4, s, freed, num)
    assert int(num) == 0 and lib.kda_get_last_device_error() == 0


def test_release_of_a_pool_past_the_bitmap(lib):
    """More pages than one pass marks."""
    pages = (1 << 20) * 2 + 77
    rng = np.random.default_rng(0)
    own = np.sort(rng.choice(pages, 5000, replace=False))
    table = rng.permutation(own).reshape(50, 100)
    s = torch.zeros(pages, **I32)
    freed, num = torch.full((6000,), -7, **I32), torch.zeros(1, **I32)
    lib.kda_page_release(torch.full((50,), 100, **I32), torch.zeros(50, **I32), torch.tensor(table, **I32), 1,
                         s, freed, num)
    assert lib.kda_get_last_device_error() == 0
    assert int(num) == 5000 and (freed[:5000].cpu().numpy() == own).all() and (freed[5000:] == -7).all()
    assert not s.any()
