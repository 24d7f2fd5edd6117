"""fp64 restatement of the rotation, the append, the key bounds, the selection of pages and the attention over them.

Plain numpy from the definitions in include/pagedattn.h; shares nothing with
the library.  What the definitions round to fp32 is rounded here at the same
places, so that codes and lists can be compared bit for bit.
"""
from __future__ import annotations

import math

import numpy as np

F = np.float32


def rope(x, positions, inv_freq, axes=None, interleaved=False, scale=1.0, inverse=False):
    """x [n, heads, D] rotated; positions [num_axes, n]; and |a| + |b| of each value's pair (0 where none is)."""
    x, w = np.array(x, np.float64), np.asarray(inv_freq, np.float64)
    pairs = len(w)
    axes = np.zeros(pairs, int) if axes is None else np.asarray(axes)
    angle = np.asarray(positions, np.float64)[axes].T * w * (-1 if inverse else 1)  # [n, pairs]
    c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale
    i = np.arange(pairs)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    a, b = x[..., first], x[..., second]
    out, size = x.copy(), np.zeros_like(x)
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = (np.abs(a) + np.abs(b)) * abs(scale)
    return out, size


def bounds(keys):
    """Codes int8 [2, D] and the fp32 scale of a page's keys [rows, D] (values of 16 bits)."""
    keys = np.asarray(keys, F)
    if not np.isfinite(keys).all():
        return np.stack([np.full(keys.shape[1], 127), np.full(keys.shape[1], -127)]).astype(np.int8), F(np.inf)
    top, low = keys.max(0), keys.min(0)
    a = F(max(np.abs(top).max(), np.abs(low).max()))
    if a < F(2.0 ** -100):
        return np.zeros((2, keys.shape[1]), np.int8), F(0)
    f = F(127) * (F(1) / a)
    return np.stack([np.minimum(F(127), np.ceil(top * f)), np.maximum(F(-127), np.floor(low * f))]).astype(np.int8), a * (F(1) / F(127))


def query_codes(q):
    """Codes (whole numbers) [2 * D] of a group's queries [G, D]: the positive parts' sum, then the negative parts'."""
    q = np.asarray(q, np.float64)
    D = q.shape[1]
    if not np.isfinite(q).all() or not q.any():
        return np.zeros(2 * D, np.int64)
    x = np.rint(q * 2.0 ** (15 - math.frexp(np.abs(q).max())[1]))
    parts = np.concatenate([np.maximum(x, 0).sum(0), np.minimum(x, 0).sum(0)])
    most = np.abs(parts).max()
    if most == 0:
        return np.zeros(2 * D, np.int64)
    return np.rint(parts.astype(F) * (F(127) * (F(1) / F(most)))).astype(np.int64)


def scores(codes, bounds_codes, scales):
    """fp32 scores of pages with codes [n, 2, D] and scales [n]."""
    sums = bounds_codes.reshape(len(scales), len(codes)).astype(np.int64) @ codes
    with np.errstate(invalid="ignore"):
        z = sums.astype(F) * scales
    return np.where(np.isnan(z), F(np.inf), z)


def select(score, num_blocks, first, last):
    """The selected blocks of a query that has len(score) of them: ascending, -1 behind."""
    n = len(score)
    if n <= num_blocks:
        chosen = np.arange(n)
    else:
        i = np.arange(n)
        always = (i < first) | (i >= n - last)
        order = np.lexsort((i, -score.astype(np.float64), ~always))
        chosen = np.sort(order[:num_blocks])
    return np.concatenate([chosen, np.full(num_blocks - len(chosen), -1)]).astype(np.int32)


def rows_of(data, pages, half, h, hnd):
    """Keys (or values) [pages * page_size, D] of one head in the order of the pages."""
    x = data[pages, half, h] if hnd else data[pages, half, :, h]
    return x.reshape(-1, x.shape[-1])


def queries(qo_indptr, page_indptr, last, page_size):
    """(request, first entry of its pages, their number, position) of each query token."""
    out = []
    for b in range(len(last)):
        n = int(page_indptr[b + 1] - page_indptr[b])
        kv = (n - 1) * page_size + int(last[b]) if n else 0
        qo = int(qo_indptr[b + 1] - qo_indptr[b])
        out += [(b, int(page_indptr[b]), n, kv - qo + i) for i in range(qo)]
    return out


def attention(q, data, lists, qo_indptr, page_indptr, pages, last, page_size, hnd):
    """(out, lse, spread) as oracle.kv4.attention gives them, of q [T, Hq, D] over the listed blocks."""
    T, Hq, D = q.shape
    q, Hkv = np.asarray(q, np.float64), lists.shape[1]
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    av, sv, sabs, seen = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq), int)
    for i, (_, start, n, pos) in enumerate(queries(qo_indptr, page_indptr, last, page_size)):
        for h in range(Hkv):
            listed = [int(e) for e in lists[i, h]]
            end = next((j for j, e in enumerate(listed) if e < 0), len(listed))
            if any(e >= 0 for e in listed[end:]) or any(a >= b for a, b in zip(listed[:end], listed[1:end])):
                continue  # out of order: as an empty list
            mine = [e for e in listed[:end] if e < n and e * page_size <= pos]
            if not mine:
                continue
            ids = np.asarray(pages)[start + np.array(mine)]
            at = (np.array(mine)[:, None] * page_size + np.arange(page_size)).reshape(-1)
            k, v = (rows_of(data, ids, half, h, hnd)[at <= pos].astype(np.float64) for half in (0, 1))
            for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                z = k @ q[i, j] / np.sqrt(D)
                top = z.max()
                p = np.exp(z - top)
                total = p.sum()
                out[i, j], lse[i, j] = p @ v / total, top + np.log(total)
                av[i, j], sv[i, j] = p @ np.abs(v) / total, np.abs(v).sum(0)
                sabs[i, j], seen[i, j] = (np.abs(k) @ np.abs(q[i, j])).max() / np.sqrt(D), len(k)
    return out, lse, {"av": av, "v": sv, "s": sabs, "n": seen}
