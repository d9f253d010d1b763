"""The attention-side operators from their definitions, in 64 bits and one row at a time.

Inputs are float64 arrays (the exact values of the 16-bit tensors); nothing is rounded here.
"""
from __future__ import annotations

import numpy as np

__all__ = ["norm_rope", "kv_append", "paged_attention"]


def norm_rope(x, weight, eps, positions, cos_sin, interleaved):
    """x [t, h, d] -> (y, a): the normed and rotated rows, and for each value the sum of the
    magnitudes of its rotation's terms (what its fp32 rounding errors are relative to)."""
    t, h, d = x.shape
    y, mag = np.array(x, dtype=np.float64), np.zeros(x.shape)
    rot = 0 if cos_sin is None else cos_sin.shape[1]
    for i in range(t):
        for j in range(h):
            row = y[i, j]
            if weight is not None:
                row = row / np.sqrt(np.mean(row * row) + eps) * weight
            out, m = row.copy(), np.abs(row)
            if rot:
                p = int(positions[i])
                if 0 <= p < cos_sin.shape[0]:
                    for f in range(rot // 2):
                        a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + rot // 2)
                        c, s = cos_sin[p, f], cos_sin[p, rot // 2 + f]
                        out[a], out[b] = row[a] * c - row[b] * s, row[b] * c + row[a] * s
                        m[a], m[b] = abs(row[a] * c) + abs(row[b] * s), abs(row[b] * c) + abs(row[a] * s)
                else:
                    out, m = np.zeros(d), np.zeros(d)
            y[i, j], mag[i, j] = out, m
    return y, mag


def kv_append(cache, rows, slots):
    """The cache [n_pages, page_size, hk, d] with rows [t, hk, d] at their slots."""
    out = np.array(cache)
    n_pages, page = out.shape[:2]
    for r, s in zip(rows, slots):
        if 0 <= s < n_pages * page:
            out[s // page, s % page] = r
    return out


def paged_attention(q, k_cache, v_cache, block_table, cu_q, kv_lens, scale, window=0, sinks=None):
    """-> (out, a, info): out [t, hq, d]; a [t, hq, d] the weighted sums of |v|; info [t, hq, 4] the
    largest sum |q_i k_i| * scale and |score| of a visible key, the count of visible keys, and
    the sum of e^(score - max) (0 keys: zeros)."""
    t, hq, d = q.shape
    n_pages, page, hk, _ = k_cache.shape
    out, mag, info = np.zeros(q.shape), np.zeros(q.shape), np.zeros((t, hq, 4))
    for s in range(len(kv_lens)):
        n = int(cu_q[s + 1]) - int(cu_q[s])
        kv = int(kv_lens[s])
        pages = np.array([block_table[s][j // page] for j in range(kv)], dtype=np.int64)
        place = np.arange(kv) % page
        held = (pages >= 0) & (pages < n_pages)
        for i in range(n):
            p = kv - n + i
            j = np.arange(kv)
            see = held & (j <= p)
            if window:
                see &= j > p - window
            if not see.any():
                continue
            for h in range(hq):
                k = k_cache[pages[see], place[see], h // (hq // hk)]
                v = v_cache[pages[see], place[see], h // (hq // hk)]
                row = q[cu_q[s] + i, h]
                x = (k @ row) * scale
                m = x.max() if sinks is None or np.isinf(sinks[h]) else max(x.max(), sinks[h])
                e = np.exp(x - m)
                z = e.sum() + (0.0 if sinks is None else np.exp(sinks[h] - m))  # infinite sinks: 0 or infinity
                out[cu_q[s] + i, h] = (e @ v) / z
                mag[cu_q[s] + i, h] = (e @ np.abs(v)) / z
                info[cu_q[s] + i, h] = ((np.abs(k) @ np.abs(row)).max() * scale, np.abs(x).max(), see.sum(),
                                        np.exp(x - x.max()).sum())
    return out, mag, info
