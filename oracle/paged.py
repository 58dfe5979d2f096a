"""Plain fp64 definitions of rotary positions and of the paged key/value cache's operators.

Test infrastructure only (see the package docstring).  Everything is written
per sequence, per head and per token over gathered keys; nothing is shared with
the CUDA path.  Layouts: packed q [T, H, D], k and v [T, H_kv, D] with offsets
cu [B + 1]; pages [num_pages, H_kv, page, D]; weights [num_pages, H_kv, page];
table [B, max_pages]; kv_len [B] with the new tokens counted.
"""

from __future__ import annotations

import math

import numpy as np


def rope(x, positions, freq, interleaved=False, mscale=1.0, inverse=False):
    """Rows x [..., N, D] turned by positions [N] (angles positions * freq), the values behind
    2 * len(freq) unchanged; inverse: the transposed map."""
    x = np.asarray(x, dtype=np.float64)
    half = len(freq)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freq, dtype=np.float64)
    c, s = mscale * np.cos(ang), mscale * np.sin(ang) * (-1.0 if inverse else 1.0)
    y = x.copy()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    a, b = x[..., first], x[..., second]
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


def slots(table_row, length, page):
    """(page, offset) of the keys 0..length-1 of a sequence."""
    j = np.arange(length)
    return np.asarray(table_row)[j // page], j % page


def append(q, k, v, k_cache, v_cache, weights, cu, kv_len, table, positions=None, freq=None, interleaved=False,
           mscale=1.0):
    """The turned q, and copies of the cache with the new tokens in their slots (weights there 0)."""
    page = k_cache.shape[2]
    kc, vc = np.array(k_cache, dtype=np.float64), np.array(v_cache, dtype=np.float64)
    wc = None if weights is None else np.array(weights, dtype=np.float64)
    qo = None if q is None else np.array(q, dtype=np.float64)
    for b in range(len(kv_len)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            t = cu[b] + i
            slot = kv_len[b] - n + i
            pos = slot if positions is None else positions[t]
            turn = (lambda x: x) if freq is None else \
                (lambda x: rope(x[:, None, :], [pos], freq, interleaved, mscale)[:, 0])
            if qo is not None:
                qo[t] = turn(np.asarray(q[t], dtype=np.float64))
            if slot < 0:
                continue
            p, o = table[b][slot // page], slot % page
            kc[p, :, o] = turn(np.asarray(k[t], dtype=np.float64))
            vc[p, :, o] = v[t]
            if wc is not None:
                wc[p, :, o] = 0.0
    return qo, kc, vc, wc


def attention_paged(q, k_cache, v_cache, cu, kv_len, table, scale):
    """(o [T, H, D], lse [T, H]); rows outside every sequence NaN, rows that see no key 0 and -inf."""
    T, H, D = q.shape
    Hkv, page = k_cache.shape[1:3]
    o = np.full((T, H, D), np.nan)
    lse = np.full((T, H), np.nan)
    for b in range(len(kv_len)):
        n, L = cu[b + 1] - cu[b], int(kv_len[b])
        p, f = slots(table[b], L, page)
        for h in range(H):
            k = np.asarray(k_cache[p, h // (H // Hkv), f], dtype=np.float64)
            v = np.asarray(v_cache[p, h // (H // Hkv), f], dtype=np.float64)
            for i in range(n):
                t, seen = cu[b] + i, max(0, L - n + i + 1)
                if seen == 0:
                    o[t, h], lse[t, h] = 0.0, -math.inf
                    continue
                z = scale * (k[:seen] @ np.asarray(q[t, h], dtype=np.float64))
                m = z.max()
                e = np.exp(z - m)
                o[t, h] = e @ v[:seen] / e.sum()
                lse[t, h] = m + math.log(e.sum())
    return o, lse


def paged_weights(q, lse, k_cache, weights, cu, kv_len, table, scale):
    """weights plus what every key's probabilities sum to over the rows of its group that see it."""
    H = q.shape[1]
    Hkv, page = k_cache.shape[1:3]
    w = np.array(weights, dtype=np.float64)
    for b in range(len(kv_len)):
        n, L = cu[b + 1] - cu[b], int(kv_len[b])
        p, f = slots(table[b], L, page)
        for h in range(H):
            g = h // (H // Hkv)
            k = np.asarray(k_cache[p, g, f], dtype=np.float64)
            for i in range(n):
                t, seen = cu[b] + i, max(0, L - n + i + 1)
                z = scale * (k[:seen] @ np.asarray(q[t, h], dtype=np.float64))
                w[p[:seen], g, f[:seen]] += np.exp(z - float(lse[t, h]))
    return w


def evict(k_cache, v_cache, weights, table, kv_len, dst_table, n_keep, n_recent):
    """(k, v, weights, kept [B, H_kv, n_keep], kv_len) after the eviction; nothing else changes."""
    Hkv, page = k_cache.shape[1:3]
    kc, vc, wc = k_cache.copy(), v_cache.copy(), weights.copy()
    kept = np.full((len(kv_len), Hkv, n_keep), -1, dtype=np.int32)
    new_len = np.minimum(kv_len, n_keep).astype(np.int32)
    for b in range(len(kv_len)):
        L = int(kv_len[b])
        p, f = slots(table[b], L, page)
        for h in range(Hkv):
            if L <= n_keep:
                at = list(range(L))
            else:
                w = [float(x) for x in weights[p[:L - n_recent], h, f[:L - n_recent]]]
                order = sorted(range(L - n_recent), key=lambda j: (math.inf if math.isnan(w[j]) else -w[j], j))
                at = sorted(order[:n_keep - n_recent]) + list(range(L - n_recent, L))
            kept[b, h, :len(at)] = at
            dp, df = slots(dst_table[b], len(at), page)
            for old, new in ((k_cache, kc), (v_cache, vc), (weights, wc)):
                new[dp, h, df] = old[p[at], h, f[at]]
    return kc, vc, wc, kept, new_len
