"""Pins of the tree oracle (CPU): a chain against the serial recurrence, trees against their
paths, the commit against the states, hand-worked forks, releases and compactions."""
import numpy as np
import pytest

import oracle
from oracle import paged, tree


def inputs(n, H=2, seed=0):
    gen = np.random.default_rng(seed)
    q, k, v = gen.standard_normal((3, n, H, 128))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    g = -np.log1p(np.exp(gen.standard_normal((n, H, 128)) - 2))
    return q, k, v, g, gen.uniform(0.1, 1, (n, H)), gen.standard_normal((H, 128, 128))


PARENTS = [-1, 0, 0, 1, 1, 2, 4, -1, 6]


def test_words():
    assert tree.words(PARENTS)[8] == sum(1 << j for j in (0, 1, 4, 6, 8))
    assert tree.ancestors(tree.words(PARENTS)[8], 8) == [6, 4, 1, 0]
    assert tree.path(tree.words(PARENTS), 5) == [0, 2, 5] and tree.path([], -1) == []


def test_recurrence_follows_every_path():
    q, k, v, g, beta, S0 = inputs(len(PARENTS))
    w = tree.words(PARENTS)
    o, u, mag_o, mag_u, states = tree.recurrent(q, k, v, g, beta, S0, w, 0.3)
    for e in range(len(PARENTS)):
        at = tree.path(w, e)
        ref, S = oracle.recurrent(q[at], k[at], v[at], g[at], beta[at], scale=0.3,
                                  initial_state=S0[None])
        np.testing.assert_allclose(o[e], ref[-1], rtol=1e-10, atol=1e-12)
        np.testing.assert_allclose(states[e], S[0], rtol=1e-10, atol=1e-12)
        got, mag = tree.commit(S0, k, g, u, w, e)
        np.testing.assert_allclose(got, S[0], rtol=1e-10, atol=1e-12)
        assert (mag >= np.abs(got) - 1e-12).all()
    assert (mag_o >= np.abs(o) - 1e-12).all() and (mag_u >= np.abs(u) - 1e-12).all()
    assert (tree.commit(S0, k, g, u, w, -1)[0] == S0).all()


@pytest.mark.parametrize("norm", [False, True])
def test_conv_follows_every_path(norm):
    from oracle import shortconv
    gen = np.random.default_rng(1)
    x, wt, carried = gen.standard_normal((9, 256)), gen.standard_normal((256, 4)), gen.standard_normal((3, 256))
    w = tree.words(PARENTS)
    y, _, _ = tree.conv(x, wt, carried, w, norm)
    for e in range(9):
        at = tree.path(w, e)
        ref, state = shortconv.short_conv(x[at], wt, np.array([0, len(at)]), carried[None],
                                          norm_dim=128 if norm else None)
        np.testing.assert_allclose(y[e], ref[-1], rtol=1e-9, atol=1e-12)
        np.testing.assert_allclose(tree.conv_commit(x, carried, w, e), state[0])


def test_attention_follows_every_path():
    gen = np.random.default_rng(2)
    H, G, D, ps = 2, 2, 8, 4
    k, v = gen.standard_normal((2, 9, ps, H, D))
    q = gen.standard_normal((9, H * G, D))
    table = gen.permutation(9)[None, :5]
    w = tree.words(PARENTS)
    o, lse, _, _ = tree.attend(q, k, v, table, [14], [0, 9], w, 0.4)
    flat_k, flat_v = (x[table[0]].reshape(1, -1, H, D)[0] for x in (k, v))
    for e in range(9):
        at = list(range(5)) + [5 + j for j in tree.path(w, e)]
        ref = paged.decode(q[e:e + 1], flat_k[at][None], flat_v[at][None], [[0]], [len(at)], 0.4)
        np.testing.assert_allclose(o[e], ref[0][0], atol=1e-13)
        np.testing.assert_allclose(lse[e], ref[1][0], atol=1e-13)
    o, lse, _, _ = tree.attend(q[:2], k, v, table, [2], [0, 2], [0, 3], 0.4)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all() and np.isfinite(lse[1]).all()


def test_compact_by_hand():
    # pages of 4, context 2, nodes at positions 2 .. 6; the path 0, 2, 4 moves to 2, 3, 4
    cache = np.arange(12.0).reshape(3, 4)
    table = [[2, 0]]
    out, kept = tree.compact(cache, table, [7], [0, 5], tree.words([-1, 0, 0, 1, 2]), [4], 4)
    assert kept == [5]
    assert out[2].tolist() == [8, 9, 10, 0] and out[0].tolist() == [2, 1, 2, 3]
    out, kept = tree.compact(cache, table, [7], [0, 5], tree.words([-1, 0, 0, 1, 2]), [-1], 4)
    assert kept == [2] and (out == cache).all()


def test_fork_and_release_by_hand():
    # pages of 4: request 0 holds 9 tokens on pages 5, 3, 7; it is forked to rows 1 and 3
    table = [[5, 3, 7], [-1, -1, -1], [6, -1, -1], [-1, -1, -1]]
    shares = np.zeros(10, int)
    seq, t, shares, copies, used, bad = tree.fork([0, 0, 2], [1, 3, 0], [9, 0, 4, 0], [2, 8, 1], table, 4,
                                                  10, shares)
    assert bad and used == 2                              # the third fork's destination is a source
    assert seq == [9, 9, 4, 9]
    assert t.tolist() == [[5, 3, 7], [5, 3, 2], [6, -1, -1], [5, 3, 8]]
    assert copies == [[7, 2, 1], [7, 8, 1], [-1, -1, 0]]
    assert shares.tolist() == [0, 0, 0, 2, 0, 2, 0, 0, 0, 0]
    s1, freed, bad = tree.release([9, 9, 4, 9], [0, 8, 4, 2], t, 4, 10, shares)
    assert not bad and freed == [2, 7, 8]
    assert s1.tolist() == [0, 0, 0, 0, 0, 1, 0, 0, 0, 0]
    # the last two holders of page 5 end together: free once
    s2, freed, bad = tree.release([0, 8, 4, 2], [0, 0, 4, 0], t, 4, 10, s1)
    assert not bad and freed == [3, 5] and (s2 == 0).all()
    _, freed, bad = tree.release([4, 4], [0, 0], [[1], [1]], 4, 10, np.zeros(10, int))
    assert bad and freed == [1]
