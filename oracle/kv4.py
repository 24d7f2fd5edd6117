"""fp64 restatement of the device-built tables, the 4-bit cache and the attention over it.

Plain numpy from the definitions in include/pagedattn.h; shares nothing with
the library.  Caches are uint8 arrays as the library lays them out.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3: sign, 4 exponent bits of bias 7, 3 of mantissa; 0x7F is NaN, no infinities
E4M3 = np.array([(b % 8) / 8 * 2.0 ** -6 if b < 8 else (1 + b % 8 / 8) * 2.0 ** (b // 8 - 7) for b in range(127)])
GROUP = 16


def nearest(a, grid):
    """Index of the grid value nearest to a >= 0, halfway to the even index, beyond the last to the last."""
    i = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo, hi = a - grid[i - 1], grid[i] - a
    return np.where((hi < lo) | ((hi == lo) & (i % 2 == 0)), i, i - 1)


def quantise(x, g):
    """x [..., D] (float64 of values in 16 bits) -> codes [..., D/2], scales [..., D/16] (bytes), values [..., D].

    The scale and the unit scale * g are rounded to fp32 as documented (one
    correctly rounded operation each); with g a power of two they are exact.
    """
    x = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    amax = np.abs(x).max(-1)
    nan = np.isnan(x).any(-1)
    g6 = np.float64(np.float32(6) * np.float32(g))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        s = np.minimum(np.float32(amax / g6).astype(np.float64), 448.0)
        sb = np.where(nan, 0x7F, nearest(np.where(nan, 0.0, s), E4M3)).astype(np.uint8)
        scale = np.where(nan, 0.0, E4M3[np.where(nan, 0, sb)])
        unit = np.float32(scale * np.float64(np.float32(g))).astype(np.float64)[..., None]
        y = np.where(unit > 0, x / np.where(unit > 0, unit, 1.0), 0.0)
        y = np.float32(y).astype(np.float64)
    mag = nearest(np.minimum(np.abs(y), 1e30), E2M1)
    code = (mag + 8 * np.signbit(y)).astype(np.uint8)
    code = np.where((unit > 0) & np.ones_like(mag, bool), code, 0).astype(np.uint8)
    flat = code.reshape(*code.shape[:-2], code.shape[-2] * GROUP)
    codes = (flat[..., 0::2] | (flat[..., 1::2] << 4)).astype(np.uint8)
    return codes, sb, values(codes, sb) * np.float64(np.float32(g))


def values(codes, scales):
    """What codes and scale bytes stand for, without the cache's own scales."""
    table = np.concatenate([E2M1, -E2M1])
    x = np.stack([table[codes & 15], table[codes >> 4]], -1).reshape(*codes.shape[:-1], codes.shape[-1] * 2 // GROUP, GROUP)
    s = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])[scales]
    return (x * s[..., None]).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def rows(cache, page, half, slot, hnd):
    """Rows [..., heads, bytes] of the given pages and slots."""
    return cache[page, half, :, slot] if hnd else cache[page, half, slot]


def tables(qo_lens, kv_lens, block_table, free_pages, free_count, page_size):
    """The documented outputs of build_tables for a batch that fits, as a dict; block_table is changed."""
    B = len(qo_lens)
    qo, kv = np.asarray(qo_lens, np.int64), np.asarray(kv_lens, np.int64)
    old, new = -(-kv // page_size), -(-(kv + qo) // page_size)
    top = int(free_count)
    indices, slots, positions = [], [], []
    for b in range(B):
        for i in range(int(old[b]), int(new[b])):
            top -= 1
            block_table[b, i] = free_pages[top]
        indices += list(block_table[b, : int(new[b])])
        for pos in range(int(kv[b]), int(kv[b] + qo[b])):
            positions.append(pos)
            slots.append(int(block_table[b, pos // page_size]) * page_size + pos % page_size)
    cum = lambda n: np.concatenate([[0], np.cumsum(n)])  # noqa: E731
    return {"qo_indptr": cum(qo), "kv_page_indptr": cum(new), "new_page_indptr": cum(new - old),
            "kv_page_indices": np.array(indices, np.int64), "slot_mapping": np.array(slots, np.int64),
            "positions": np.array(positions, np.int64), "kv_lens": kv + qo,
            "kv_last_page_len": np.where(new > 0, kv + qo - (new - 1) * page_size, 0), "free_count": top}


def attention(q, codes, scales, k_scale, v_scale, qo_indptr, page_indptr, pages, last, page_size, hnd, causal):
    """(out, lse, spread) in float64 for q [T, Hq, D]; rows without keys: 0, -inf.

    spread holds what an error bound needs of each row: "av" [T, Hq, D] =
    sum p |v|, "v" = sum |v| over the visible keys, "s" [T, Hq] = the largest
    scale * sum_d |q_d k_d|, "n" [T, Hq] = the keys seen.
    """
    T, Hq, D = q.shape
    q = np.asarray(q, np.float64)
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    av, sv, sabs, seen = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq), int)
    for b in range(len(last)):
        r0, r1 = int(qo_indptr[b]), int(qo_indptr[b + 1])
        ids = np.asarray(pages[int(page_indptr[b]): int(page_indptr[b + 1])], np.int64)
        n = (len(ids) - 1) * page_size + int(last[b]) if len(ids) else 0
        if r1 == r0 or n == 0:
            continue
        t = np.arange(n)
        k, v = (values(rows(codes, ids[t // page_size], h, t % page_size, hnd),
                       rows(scales, ids[t // page_size], h, t % page_size, hnd)) * s
                for h, s in ((0, k_scale), (1, v_scale)))  # [n, Hkv, D]
        G = Hq // k.shape[1]
        for i in range(r0, r1):
            m = n - (r1 - r0) + (i - r0) + 1 if causal else n
            if m <= 0:
                continue
            for h in range(Hq):
                kk, vv = k[:m, h // G], v[:m, h // G]
                z = kk @ q[i, h] / np.sqrt(D)
                top = z.max()
                p = np.exp(z - top)
                total = p.sum()
                out[i, h] = p @ vv / total
                lse[i, h] = top + np.log(total)
                av[i, h], sv[i, h] = p @ np.abs(vv) / total, np.abs(vv).sum(0)
                sabs[i, h], seen[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() / np.sqrt(D), m
    return out, lse, {"av": av, "v": sv, "s": sabs, "n": seen}
