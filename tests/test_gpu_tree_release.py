"""Pages given back by many requests at once (several blocks): refusals among them, pools of a few
pages and of more than one pass marks, lists that are too short, a captured and replayed call."""
import numpy as np
import pytest
import torch

from oracle import tree
from parity_utils import DEV

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device=DEV)


def check(lib, seq, kept, table, page, pages, shares):
    s = torch.tensor(shares, **I32)
    freed, num = lib.page_release(torch.tensor(seq, **I32), torch.tensor(kept, **I32), torch.tensor(table, **I32),
                                  page, s)
    want_s, want, bad = tree.release(seq, kept, table, page, pages, shares)
    assert lib.kda_get_last_device_error() == int(bad)
    assert freed[:int(num)].tolist() == want and (s.cpu().numpy() == want_s).all()
    return bad


@pytest.mark.parametrize("B", [64, 65, 300, 1500])
@pytest.mark.parametrize("pages", [1, 31, 257, 5000])
def test_shared_and_refused(lib, B, pages):
    rng = np.random.default_rng(B + pages)
    width, page = 4, 8
    table = rng.integers(0, pages, (B, width))
    seq = rng.integers(0, width * page + 1, B)
    kept = (seq * rng.random(B)).astype(int)
    held = np.bincount([p for n, row in zip(seq, table) for p in row[:-(-int(n) // page)]], minlength=pages)
    shares = np.maximum(held - 1, 0)
    assert not check(lib, seq.tolist(), kept.tolist(), table, page, pages, shares)
    bad = rng.random(B) < 0.1                  # lengths that do not fit, pages that are none, pages twice
    seq[bad] = rng.choice([-1, width * page + 1, 2 ** 31 - 1], bad.sum())
    table[rng.random((B, width)) < 0.05] = pages
    kept[rng.random(B) < 0.05] = -5
    check(lib, seq.tolist(), kept.tolist(), table, page, pages, np.minimum(shares, 1))


def test_past_the_bitmap_and_short_lists(lib):
    pages = (1 << 20) * 2 + 77
    rng = np.random.default_rng(1)
    own = np.sort(rng.choice(pages, 20000, replace=False))
    own[-1] = pages - 1
    table = torch.tensor(rng.permutation(own).reshape(200, 100), **I32)
    seq, zero = torch.full((200,), 100, **I32), torch.zeros(200, **I32)
    for room in (20000, 12345):
        s, freed, num = torch.zeros(pages, **I32), torch.full((20008,), -7, **I32), torch.zeros(1, **I32)
        lib.kda_page_release(seq, zero, table, 1, s, freed[:room], num)
        assert lib.kda_get_last_device_error() == int(room < 20000)
        assert int(num) == room and (freed[:room].cpu().numpy() == own[:room]).all() and (freed[room:] == -7).all()
        assert not s.any()


def test_captured_and_replayed(lib):
    B, width = 130, 30
    pages = B * width
    table = torch.randperm(pages).view(B, width).to(**I32)
    seq, zero = torch.full((B,), width * 4, **I32), torch.zeros(B, **I32)
    s, freed, num = torch.zeros(pages, **I32), torch.zeros(pages, **I32), torch.zeros(1, **I32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            lib.kda_page_release(seq, zero, table, 4, s, freed, num)
    for _ in range(3):
        freed.fill_(-7)
        num.zero_()
        graph.replay()
        assert int(num) == pages and (freed.cpu() == torch.arange(pages, dtype=torch.int32)).all() and not s.any()
    assert lib.kda_get_last_device_error() == 0
