"""Plain fp64 / integer definitions of the paged key-value cache operators
(numpy, loops over requests, tokens and heads): the page plan, the cache append
with its rounding to 8 bits, and one-token softmax attention over the cache."""
import numpy as np


def pages(n, page_size):
    return -(-n // page_size)


def plan(cached, new, free, table, page_size, num_pages, N):
    """Returns (table, seq_lens, cu_seqlens, slot_map, pages_used, any refused or bad page)."""
    table = np.array(table)
    B, width = table.shape
    seq, cu = np.zeros(B, np.int64), np.zeros(B + 1, np.int64)
    slots = np.full(N, -1, np.int64)
    row = off = used = 0
    bad = False
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        fits = c >= 0 and n >= 0 and c + n <= min(width * page_size, 2 ** 31 - 1)
        n_rows = max(n, 0)
        held = pages(max(c, 0), page_size)
        need = pages(c + n, page_size) - held if fits else 0
        served = fits and (need == 0 or off + need <= len(free)) and (n == 0 or row + n <= N)
        if served:
            for i in range(need):
                table[b, held + i] = free[off + i]
            if need:
                used = off + need
            for j in range(n):
                page = int(table[b, (c + j) // page_size])
                if 0 <= page < num_pages:
                    slots[row + j] = page * page_size + (c + j) % page_size
                else:
                    bad = True
            seq[b] = c + n
        else:
            bad = True
            seq[b] = c if 0 <= c <= width * page_size else 0
        row += n_rows
        off += need
        cu[b + 1] = min(row, N)
    return table, seq, cu, slots, used, bad


def e4m3(x):
    """x rounded to the nearest 8-bit float of 4 exponent and 3 mantissa bits (ties to even,
    magnitudes limited to 448, subnormal steps of 2^-9), as fp64 values."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)                                 # |x| in [2^(e-1), 2^e)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def append(k_cache, k, slots, scale=None):
    """k_cache fp64 [num_pages, page_size, H, D] with the tokens k [N, H, D] written; an 8-bit
    cache (scale [H]) holds e4m3(fp32 quotient)."""
    out = np.array(k_cache, np.float64, order="C")
    flat = out.reshape(-1, *out.shape[2:])
    for n, s in enumerate(slots):
        if 0 <= s < len(flat):
            x = np.asarray(k[n], np.float64)
            if scale is not None:
                q = x.astype(np.float32) / np.asarray(scale, np.float32)[:, None]
                x = e4m3(q)
            flat[s] = x
    return out


def decode(q, k_cache, v_cache, table, seq_lens, scale, k_scale=None, v_scale=None):
    """fp64 attention of q [B, Hq, D] over the cached keys.  Returns (o, lse, weight, spread):
    weight [B, Hq, D] = sum_j p_j |v_j| and spread [B, Hq] = max_j scale sum_d |q_d k_jd|, the
    magnitudes that rounding errors of the weights and of the scores are relative to."""
    B, Hq, D = q.shape
    page_size, H = k_cache.shape[1:3]
    G = Hq // H
    o, weight = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, spread = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    for b in range(B):
        n = int(seq_lens[b])
        if n == 0:
            continue
        pg = np.asarray(table[b][:pages(n, page_size)], np.int64)
        kk = k_cache[pg].reshape(-1, H, D)[:n].astype(np.float64)
        vv = v_cache[pg].reshape(-1, H, D)[:n].astype(np.float64)
        if k_scale is not None:
            kk = kk * np.asarray(k_scale, np.float64)[:, None]
            vv = vv * np.asarray(v_scale, np.float64)[:, None]
        for h in range(Hq):
            k, v = kk[:, h // G], vv[:, h // G]
            s = (k @ q[b, h].astype(np.float64)) * scale
            m = s.max()
            p = np.exp(s - m)
            lse[b, h] = m + np.log(p.sum())
            p /= p.sum()
            o[b, h], weight[b, h] = p @ v, p @ np.abs(v)
            spread[b, h] = abs(scale) * (np.abs(k) @ np.abs(q[b, h].astype(np.float64))).max()
    return o, lse, weight, spread
