"""Requests that go back behind the point where they were forked: the last page that they keep is shared.
Forked into an empty row they go on in a page of their own, and the others' keys stay as they are."""
import pytest
import torch

from parity_utils import DEV
from test_gpu_paged import as_device
from test_gpu_tree_pages import I32, filled

pytestmark = pytest.mark.gpu


def held(cache, table, row, n, page):
    """The first n keys and values of a row."""
    at = table[row, :-(-n // page)].long()
    return [bits(t)[at].flatten(0, 1)[:n].clone() for t in (cache.k_cache, cache.v_cache)]


def bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


@pytest.mark.parametrize("who", ["fork", "source"])
@pytest.mark.parametrize("cache,order,page,length,back", [("bf16", "token", 16, 40, 20), ("fp8", "head", 16, 48, 47),
                                                          ("bf16", "head", 24, 100, 1), ("fp8", "token", 1, 9, 4),
                                                          ("bf16", "token", 7, 30, 14)])
def test_go_back_fork_and_go_on(lib, cache, order, page, length, back, who):
    H, D, pages, width = 2, 64, 60, 40
    c = lib.PagedCache(*(as_device(t) for t in filled(pages, page, H, D, cache, order, 3)),
                       *((torch.ones(H, device=DEV),) * 2 if cache == "fp8" else ()))
    table = torch.full((3, width), -1, **I32)
    order_of = torch.randperm(pages).to(**I32)
    table[0, :-(-length // page)] = order_of[:-(-length // page)]
    free, lens, shares = order_of[-(-length // page):].clone(), torch.tensor([length, 0, 0], **I32), torch.zeros(pages, **I32)

    def fork(src, dst):
        nonlocal free
        copies, used = lib.page_fork(torch.tensor([src], **I32), torch.tensor([dst], **I32), lens, free, table, page, shares)
        lib.kda_paged_copy(copies, c)
        free = free[int(used):]

    def release(kept):
        nonlocal free, lens
        kept = torch.tensor(kept, **I32)
        freed, num = lib.page_release(lens, kept, table, page, shares)
        free, lens = torch.cat([freed[:int(num)], free]), kept
    fork(0, 1)
    mine, other = (1, 0) if who == "fork" else (0, 1)
    kept = lens.tolist()
    kept[mine] = back                                      # one goes back, the other keeps all
    release(kept)
    theirs, ours = held(c, table, other, length, page), held(c, table, mine, back, page)
    fork(mine, 2)                                          # it goes on in row 2
    kept = lens.tolist()
    kept[mine] = 0
    release(kept)
    n = 2 * page + 1
    lens, _, slots, used = lib.page_plan(lens, torch.tensor([0, 0, n], **I32), free, table, page, pages, n)
    free = free[int(used):]
    new = [torch.randn(n, H, D, device=DEV).to(torch.bfloat16) for _ in range(2)]
    lib.kda_paged_append(*new, slots, c)
    assert lib.kda_get_last_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(held(c, table, other, length, page), theirs))
    assert lens[2] == back + n
    got = held(c, table, 2, back + n, page)
    dtype = c.k_cache.dtype
    for t, old, x in zip(got, ours, new):
        assert torch.equal(t[:back], old) and torch.equal(t[back:], bits(x.to(dtype)))
    release([0, 0, 0])                                     # every page comes back once
    assert sorted(free.tolist()) == list(range(pages)) and not shares.any()
    assert lib.kda_get_last_device_error() == 0
