"""The operators around a cache in 4 bits and around routed experts, from their definitions, one row at a
time in 64 bits (fp32 where the definition says so)."""
from __future__ import annotations

import numpy as np

from . import attention_oracle as A
from . import qlinear_oracle as O

__all__ = ["stored_rows", "quantize_rows", "row_values", "kv_extend", "select_experts", "combine_experts"]


def stored_rows(x, weight, eps, positions, cos_sin, interleaved, dtype):
    """Rows of k [t, h, d] (float64 of 16-bit values) as they are quantized: normed and rotated in 64 bits, then
    rounded to fp32 and from there to dtype ("bf16" or "f16") -> float32."""
    y, _ = A.norm_rope(x, weight, eps, positions, cos_sin, interleaved)
    return O.bits_to_f64(dtype, O.to_bits(dtype, y.astype(np.float32))).astype(np.float32)


def quantize_rows(rows, group):
    """fp32 rows [.., d] -> (codes uint32 [.., d/8], groups float16 [.., d/group, 2])."""
    shape, d = rows.shape[:-1], rows.shape[-1]
    v = np.ascontiguousarray(rows, dtype=np.float32).reshape(-1, d)
    odd = ~(np.abs(v).reshape(-1, d // group, group) <= 32768).all(axis=-1)
    clean = np.where(np.repeat(odd, group, axis=1), np.float32(0), v)
    words, s, b = O.affine_quantize(clean, 4, group, "f16")
    s, b = s.view(np.float16).copy(), b.view(np.float16).copy()
    s[odd], b[odd] = 0, np.nan
    return words.reshape(*shape, d // 8), np.stack([s, b], axis=-1).reshape(*shape, d // group, 2)


def row_values(codes, groups):
    """Values (float64) of codes [.., d/8] and groups [.., g, 2]."""
    d = codes.shape[-1] * 8
    c = np.stack([(codes.astype(np.uint32) >> np.uint32(4 * i)) & np.uint32(15) for i in range(8)], axis=-1)
    c = c.reshape(*codes.shape[:-1], d).astype(np.float64)
    per = d // groups.shape[-2]
    return c * np.repeat(groups[..., 0].astype(np.float64), per, axis=-1) + np.repeat(groups[..., 1].astype(np.float64), per, axis=-1)


def kv_extend(counts, lens, table, page, rows, free=None):
    """-> (cu_q, positions, slots, lens, table, free list, info); free is the list of free pages and the
    capacity of its array, or None."""
    counts, lens = [int(c) for c in counts], [int(x) for x in lens]
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    fits = all(0 <= x <= width * page and (c < 0 or x + c <= width * page) for c, x in zip(counts, lens))
    pages = lambda n: -(-n // page)  # noqa: E731
    stack, cap = (list(free[0]), free[1]) if free is not None else ([], 0)
    why = int(sum(max(c, 0) for c, x in zip(counts, lens) if 0 <= x <= width * page and (c < 0 or x + c <= width * page)) > rows)
    why += 0 if fits else 4
    if free is not None:
        ok = [0 <= x <= width * page and (c < 0 or x + c <= width * page) for c, x in zip(counts, lens)]
        back = sum(pages(x) for c, x, o in zip(counts, lens, ok) if c < 0 and o)
        need = sum(pages(x + c) - pages(x) for c, x, o in zip(counts, lens, ok) if c > 0 and o)
        why += 2 * (need > len(stack) + back) + 8 * (len(stack) + back > cap)
    pos, slots, cu, taken = [], [], [0], 0
    if why:
        cu += [0] * len(counts)
    else:
        if free is not None:
            for s, c in enumerate(counts):
                if c < 0:
                    stack += table[s][:pages(lens[s])]
        for s, c in enumerate(counts):
            if c < 0:
                lens[s] = 0
        for s, c in enumerate(counts):
            for p in range(lens[s], lens[s] + max(c, 0)):
                if p % page == 0 and free is not None:
                    table[s][p // page] = stack.pop()
                    taken += 1
                pos.append(p)
                slots.append(table[s][p // page] * page + p % page)
            lens[s] += max(c, 0)
            cu.append(len(pos))
    info = [len(pos), taken, why, len(stack)]
    fill = rows - len(pos)
    return cu, pos + [0] * fill, slots + [-1] * fill, lens, table, stack, info


def select_experts(logits, k, sigmoid=False, bias=None, n_groups=1, top_groups=1, group_top=1, renormalize=True,
                   scale=1.0):
    """Router logits [t, e] (float64) -> (ids, weights float64)."""
    t, e = logits.shape
    m = e // n_groups
    ids, weights = np.zeros((t, k), dtype=np.int64), np.zeros((t, k))
    with np.errstate(all="ignore"):
        for i in range(t):
            x = np.where(np.isnan(logits[i]), -np.inf, logits[i])
            if sigmoid:
                p = 1 / (1 + np.exp(-x))
            elif x.max() == -np.inf:
                p = np.zeros(e)
            else:
                p = np.where(x == x.max(), 1.0, np.exp(x - x.max()))
                p = p / p.sum()
            c = p if bias is None else p + bias
            c = np.where(np.isnan(c), -np.inf, c)
            stay = range(n_groups)
            if n_groups > 1:
                score = [sum(sorted(c[g * m:(g + 1) * m])[-group_top:]) for g in range(n_groups)]
                stay = sorted(range(n_groups), key=lambda g: (-score[g], g))[:top_groups]
            left = [j for g in stay for j in range(g * m, (g + 1) * m)]
            ids[i] = sorted(left, key=lambda j: (-c[j], j))[:k]
            w = p[ids[i]]
            if renormalize:
                w = w / w.sum() if w.sum() > 0 else np.zeros(k)
            weights[i] = w * scale
    return ids, weights


def combine_experts(y, weights, ids=None, e=0, residual=None):
    """y [t * k, n], weights [t, k] (float64) -> (out [t, n], the sums of the terms' magnitudes)."""
    t, k = weights.shape
    out, mag = np.zeros((t, y.shape[1])), np.zeros((t, y.shape[1]))
    for i in range(t):
        if residual is not None:
            out[i], mag[i] = residual[i], np.abs(residual[i])
        for j in range(k):
            if ids is None or 0 <= ids[i, j] < e:
                out[i] += weights[i, j] * y[i * k + j]
                mag[i] += np.abs(weights[i, j] * y[i * k + j])
    return out, mag
