"""Pins of the paged-cache oracle (CPU): values worked by hand, the 8-bit rounding against
torch's conversion over every bf16 value, attention against a direct softmax and under splits."""
import numpy as np
import torch

from oracle import paged


def test_plan_by_hand():
    # pages of 4; request 0 holds 3 tokens on page 9 and gets 2 (one more page), request 1 is
    # new with 5, request 2 idle with 4, request 3 holds 4 (a full page) and gets 1
    table = np.array([[9, -1], [-1, -1], [7, -1], [6, -1]])
    t, seq, cu, slots, used, bad = paged.plan([3, 0, 4, 4], [2, 5, 0, 1], [2, 0, 5, 1, 3], table, 4,
                                              10, 9)
    assert t.tolist() == [[9, 2], [0, 5], [7, -1], [6, 1]]
    assert seq.tolist() == [5, 5, 4, 5] and cu.tolist() == [0, 2, 7, 7, 8]
    assert slots.tolist() == [39, 8, 0, 1, 2, 3, 20, 4, -1]
    assert used == 4 and not bad


def test_plan_refusals_by_hand():
    # request 1 needs two pages where one is left; request 2 is negative; request 3 fits its row
    table = np.full((4, 2), -1)
    t, seq, cu, slots, used, bad = paged.plan([0, 0, -3, 0], [4, 5, 2, 0], [8, 1], table, 4, 10, 20)
    assert t.tolist() == [[8, -1], [-1, -1], [-1, -1], [-1, -1]]
    assert seq.tolist() == [4, 0, 0, 0] and cu.tolist() == [0, 4, 9, 11, 11]
    assert slots[:4].tolist() == [32, 33, 34, 35] and (slots[4:] == -1).all()
    assert used == 1 and bad


def test_e4m3_matches_torch_on_every_bf16():
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x)]
    ref = x.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(paged.e4m3(x.double().numpy()), ref)


def test_decode_against_softmax_and_splits():
    gen = np.random.default_rng(0)
    B, H, G, D, ps = 3, 2, 3, 8, 4
    k, v = gen.standard_normal((2, 12, ps, H, D))
    q = gen.standard_normal((B, H * G, D))
    table = gen.permutation(12).reshape(3, 4)
    lens = [7, 0, 16]
    o, lse, weight, _ = paged.decode(q, k, v, table, lens, 0.4)
    assert (o[1] == 0).all() and np.isneginf(lse[1]).all()
    for b in (0, 2):
        kk = torch.tensor(k[table[b]].reshape(-1, H, D)[:lens[b]])
        vv = torch.tensor(v[table[b]].reshape(-1, H, D)[:lens[b]])
        s = torch.einsum("hgd,nhd->hgn", torch.tensor(q[b]).view(H, G, D), kk) * 0.4
        ref = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), vv).reshape(H * G, D)
        np.testing.assert_allclose(o[b], ref.numpy(), atol=1e-13)
        np.testing.assert_allclose(lse[b], torch.logsumexp(s, -1).reshape(-1).numpy(), atol=1e-13)
    assert (weight >= np.abs(o) - 1e-13).all()
    # joining the results over two sets of keys by their lse gives the whole
    a = paged.decode(q, k, v, table[:, :2], [4, 0, 8], 0.4)
    c = paged.decode(q, k, v, table[:, 1:2], [3, 0, 0], 0.4), paged.decode(q, k, v, table[:, 2:], [0, 0, 8], 0.4)
    for b, rest in ((0, c[0]), (2, c[1])):
        w = np.exp(np.stack([a[1][b], rest[1][b]]) - lse[b])[..., None]
        np.testing.assert_allclose(w[0] * a[0][b] + w[1] * rest[0][b], o[b], atol=1e-13)
