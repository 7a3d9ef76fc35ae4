"""Plain fp64 / integer definitions of the operators over trees of drafted tokens and over shared
pages (numpy, loops over requests, nodes, heads and pages)."""
import numpy as np

from . import paged


def words(parents):
    """A word for each node: its ancestors and itself."""
    w = []
    for i, p in enumerate(parents):
        w.append((w[p] if p >= 0 else 0) | 1 << i)
    return w


def ancestors(word, i):
    """The nodes above node i, nearest first."""
    return [j for j in range(i - 1, -1, -1) if word >> j & 1]


def path(words_, e):
    """The accepted path's nodes, first to last."""
    return [] if e < 0 else ancestors(words_[e], e)[::-1] + [e]


def recurrent(q, k, v, g, beta, S0, words_, scale):
    """One request: q, k, v, g [n, H, 128], beta [n, H], S0 [H, 128, 128].  Each node's state is
    its nearest ancestor's after one step.  Returns (o, u, mag_o, mag_u, states): the magnitudes are
    what fp32 rounding errors of sums and products are relative to, carried through the updates
    that later nodes read."""
    n, H, D = q.shape
    o, u = np.zeros((n, H, D)), np.zeros((n, H, D))
    mag_o, mag_u = np.zeros((n, H, D)), np.zeros((n, H, D))
    states = []
    for i in range(n):
        up = ancestors(words_[i], i)
        S = np.exp(g[i])[:, :, None] * (states[up[0]] if up else S0)
        u[i] = beta[i][:, None] * (v[i] - np.einsum("hkv,hk->hv", S, k[i]))
        S = S + k[i][:, :, None] * u[i][:, None, :]
        o[i] = np.einsum("hkv,hk->hv", S, scale * q[i])
        states.append(S)
        # |S_0| behind the decays, and every ancestor's product with its update and that one's error
        e = np.exp(g[i])
        prod = []
        for j in up:
            prod.append((j, e.copy()))
            e = e * np.exp(g[j])
        first = np.abs(S0) * e[:, :, None]
        for x, out in ((k[i], mag_u[i]), (scale * q[i], mag_o[i])):
            out += np.einsum("hkv,hk->hv", first, np.abs(x))
            for j, ej in prod:
                w = (ej * np.abs(k[j]) * np.abs(x)).sum(-1)
                out += w[:, None] * (np.abs(u[j]) + mag_u[j])
        mag_u[i] = np.abs(beta[i])[:, None] * (np.abs(v[i]) + mag_u[i])
        w = (np.abs(k[i]) * np.abs(scale * q[i])).sum(-1)
        mag_o[i] += w[:, None] * (np.abs(u[i]) + mag_u[i])
    return o, u, mag_o, mag_u, states


def commit(S0, k, g, u, words_, e):
    """The state after the path of node e from the nodes' updates u, and its magnitude."""
    S, mag = np.array(S0, np.float64), np.abs(S0)
    for j in path(words_, e):
        S = np.exp(g[j])[:, :, None] * S + k[j][:, :, None] * u[j][:, None, :]
        mag = np.exp(g[j])[:, :, None] * mag + np.abs(k[j][:, :, None] * u[j][:, None, :])
    return S, mag


def conv(x, w, carried, words_, norm):
    """One request's stream: x [n, C], w [C, 4], carried [3, C] (oldest first).  Returns
    (y, a, mag): a the convolution, mag sum |w x|."""
    y, a, mag = (np.zeros(x.shape) for _ in range(3))
    for i in range(len(x)):
        rows = np.concatenate([carried, x[ancestors(words_[i], i)[::-1]], x[i:i + 1]])[-4:]
        a[i], mag[i] = (rows * w.T).sum(0), np.abs(rows * w.T).sum(0)
    y = a / (1 + np.exp(-a))
    if norm:
        h = y.reshape(len(x), x.shape[1] // 128, 128)
        y = (h / np.sqrt((h * h).sum(-1, keepdims=True) + 1e-6)).reshape(x.shape)
    return y, a, mag


def conv_commit(x, carried, words_, e):
    return np.concatenate([carried, x[path(words_, e)]])[-3:]


def attend(q, k_cache, v_cache, table, seq_lens, cu, words_, scale, k_scale=None, v_scale=None):
    """fp64 attention of q [N, Hq, D]; words_ one for each row.  Returns (o, lse, weight, spread)
    as paged.decode does, each node over the keys that it sees."""
    N, Hq, D = q.shape
    page_size, H = k_cache.shape[1:3]
    G = Hq // H
    o, weight = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    lse, spread = np.full((N, Hq), -np.inf), np.zeros((N, Hq))
    for b in range(len(seq_lens)):
        n, L = int(cu[b + 1] - cu[b]), int(seq_lens[b])
        pg = np.asarray(table[b][:paged.pages(L, page_size)], np.int64)
        kk = k_cache[pg].reshape(-1, H, D)[:L].astype(np.float64)
        vv = v_cache[pg].reshape(-1, H, D)[:L].astype(np.float64)
        if k_scale is not None:
            kk = kk * np.asarray(k_scale, np.float64)[:, None]
            vv = vv * np.asarray(v_scale, np.float64)[:, None]
        for i in range(n):
            r = int(cu[b]) + i
            seen = list(range(L - n)) + [L - n + j for j in range(n) if words_[r] >> j & 1]
            if not seen:
                continue
            for h in range(Hq):
                k, v = kk[seen, h // G], vv[seen, h // G]
                s = (k @ q[r, h].astype(np.float64)) * scale
                m = s.max()
                p = np.exp(s - m)
                lse[r, h] = m + np.log(p.sum())
                p /= p.sum()
                o[r, h], weight[r, h] = p @ v, p @ np.abs(v)
                spread[r, h] = abs(scale) * (np.abs(k) @ np.abs(q[r, h].astype(np.float64))).max()
    return o, lse, weight, spread


def compact(cache, table, seq_lens, cu, words_, last, page_size):
    """Returns (cache, kept_lens); cache [num_pages, page_size, ...]."""
    out, kept = np.array(cache), []
    for b in range(len(seq_lens)):
        n = int(cu[b + 1] - cu[b])
        C = int(seq_lens[b]) - n
        nodes = path(words_[int(cu[b]):int(cu[b + 1])], int(last[b]))
        for r, j in enumerate(nodes):
            to, frm = C + r, C + j
            out[table[b][to // page_size], to % page_size] = \
                cache[table[b][frm // page_size], frm % page_size]
        kept.append(C + len(nodes))
    return out, kept


def fork(src, dst, seq_lens, free, table, page_size, num_pages, shares):
    """Returns (seq_lens, table, shares, copies, pages_used, any refused or bad page)."""
    seq, table, shares = list(seq_lens), np.array(table), np.array(shares)
    B, width = table.shape
    copies, off, bad = [], 0, False
    for f, (s, d) in enumerate(zip(src, dst)):
        n = seq_lens[s] if 0 <= s < B else -1
        known = 0 <= n <= width * page_size
        takes = known and n % page_size != 0
        served = known and 0 <= d < B and d not in src and d not in dst[:f] \
            and (not takes or off < len(free))
        entry = [-1, -1, 0]
        if served:
            full = n // page_size
            for i in range(full):
                p = table[d, i] = table[s, i]
                if 0 <= p < num_pages:
                    shares[p] += 1
                else:
                    bad = True
            if takes:
                a, c = int(table[s, full]), int(free[off])
                table[d, full] = c
                if 0 <= a < num_pages and 0 <= c < num_pages:
                    entry = [a, c, n % page_size]
                else:
                    bad = True
            seq[d] = n
        else:
            bad = True
        copies.append(entry)
        off += takes
    return seq, table, shares, copies, min(off, len(free)), bad


def release(seq_lens, kept_lens, table, page_size, num_pages, shares):
    """Returns (shares, freed, any refused or bad page)."""
    shares, freed, bad = np.array(shares), set(), False
    width = len(table[0]) if len(table) else 0
    for b, (n, m) in enumerate(zip(seq_lens, kept_lens)):
        if not 0 <= m <= n <= width * page_size:
            bad = True
            continue
        for i in range(paged.pages(m, page_size), paged.pages(n, page_size)):
            p = int(table[b][i])
            if not 0 <= p < num_pages or p in freed:
                bad = True
            elif shares[p] > 0:
                shares[p] -= 1
            else:
                freed.add(p)
    return shares, sorted(freed), bad
