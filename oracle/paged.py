"""Float64 oracle of the paged-cache operators: append with rotary positions, page selection, decode attention.

Caches are [n_pages, Hkv, page, d] arrays, tables [B, pages]; every function walks sequences, heads and
positions one at a time, as the definitions read.
"""
import numpy as np


def rope(x, cos, sin, interleaved):
    """x [H, d] at one position; cos, sin [R/2]."""
    y = x.copy()
    for i in range(len(cos)):
        u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + len(cos))
        y[:, u] = x[:, u] * cos[i] - x[:, w] * sin[i]
        y[:, w] = x[:, w] * cos[i] + x[:, u] * sin[i]
    return y


def append(k, v, table, token_seq, token_pos, k_cache, v_cache, k_bounds=None, q=None, table_rope=None,
           interleaved=False):
    """Writes into the given (float64) caches and bounds; returns the rotated queries (None without q). The bounds are
    of the unrounded keys this oracle wrote."""
    page = k_cache.shape[2]
    q_out = None if q is None else q.copy()
    last = {}
    for i in range(len(token_seq)):
        b, p = int(token_seq[i]), int(token_pos[i])
        if b < 0:
            continue
        key = k[i]
        if table_rope is not None:
            half = table_rope.shape[1] // 2
            key = rope(key, table_rope[p, :half], table_rope[p, half:], interleaved)
            if q is not None:
                q_out[i] = rope(q[i], table_rope[p, :half], table_rope[p, half:], interleaved)
        at = int(table[b, p // page])
        k_cache[at, :, p % page] = key
        v_cache[at, :, p % page] = v[i]
        last[at] = max(last.get(at, 0), p % page)
    if k_bounds is not None:
        for at, off in last.items():
            k_bounds[at, :, 0] = k_cache[at, :, :off + 1].min(1)
            k_bounds[at, :, 1] = k_cache[at, :, :off + 1].max(1)
    return q_out


def keys_of(cache, table_row, g, length, pages=None):
    """[n, d]: the cached rows of one sequence at kv head g, or of the listed pages of it."""
    page = cache.shape[2]
    rows = []
    for p in range(length):
        if pages is not None and p // page not in pages:
            continue
        rows.append(cache[int(table_row[p // page]), g, p % page])
    return np.array(rows).reshape(-1, cache.shape[3])


def decode(q, k_cache, v_cache, table, lens, scale, pages=None):
    """(o [B, Hq, d], lse [B, Hq], spread [B, Hq, d], reach [B, Hq]): the attention, and for error bounds
    sum_j p_j |v_j| and the largest scale * sum_i |q_i k_ji|."""
    B, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    o, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf)
    spread, reach = np.zeros((B, Hq, d)), np.zeros((B, Hq))
    for b in range(B):
        for g in range(Hkv):
            chosen = None if pages is None else set(int(x) for x in pages[b, g] if x >= 0)
            k = keys_of(k_cache, table[b], g, int(lens[b]), chosen)
            v = keys_of(v_cache, table[b], g, int(lens[b]), chosen)
            if not len(k):
                continue
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                s = scale * (k @ q[b, h])
                top = s.max()
                w = np.exp(s - top)
                lse[b, h] = top + np.log(w.sum())
                w /= w.sum()
                o[b, h], spread[b, h] = w @ v, w @ np.abs(v)
                reach[b, h] = scale * (np.abs(k) @ np.abs(q[b, h])).max()
    return o, lse, spread, reach


def scores(q, k_bounds, table_row, g, count):
    """[count]: each page's bound on the sum of the group's scores (unscaled), as sums of maxima."""
    G = q.shape[0] // k_bounds.shape[1]
    out = np.zeros(count)
    for p in range(count):
        lo, hi = k_bounds[int(table_row[p]), g]
        for h in range(g * G, (g + 1) * G):
            out[p] += np.maximum(q[h] * lo, q[h] * hi).sum()
    return out


def select(q, k_bounds, table, lens, page, n_select, keep_first, keep_last):
    B, Hkv = q.shape[0], k_bounds.shape[1]
    out = np.full((B, Hkv, n_select), -1, dtype=np.int64)
    for b in range(B):
        count = -(-int(lens[b]) // page)
        for g in range(Hkv):
            s = scores(q[b], k_bounds, table[b], g, count)
            kept = [p < keep_first or p >= count - keep_last for p in range(count)]
            order = sorted(range(count), key=lambda p: (not kept[p], 0.0 if kept[p] else -s[p], p))
            taken = sorted(order[:n_select])
            out[b, g, :len(taken)] = taken
    return out
