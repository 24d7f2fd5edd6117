"""Pins for the fp64 oracle of the tables, the 4-bit format and the attention over it.

Each check compares ``oracle.kv4`` with something other than itself: torch's
own e4m3 type, values written out by hand, a simulation token by token, or
torch's scaled_dot_product_attention.  ``test_planted_mistakes`` then swaps in
a plausible mistake at a time and requires a pin to fail.
"""
import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import kv4


def pin_formats():
    bytes_ = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(kv4.E4M3, bytes_[:127])
    # code c: sign c >> 3, exponent (c >> 1) & 3 of bias 1, mantissa c & 1
    for c in range(8):
        e, m = c >> 1, c & 1
        assert kv4.E2M1[c] == (m / 2 if e == 0 else (1 + m / 2) * 2 ** (e - 1))
    one = np.zeros((1, 8), np.uint8)
    one[0, 0], one[0, 1], one[0, 7] = 0x71, 0x0F, 0xA0  # elements 0, 1 = 0.5, 6; 2, 3 = -6, 0; 14, 15 = 0, -1
    got = kv4.values(one, np.array([[0x38]], np.uint8))[0]  # scale 1
    assert got[[0, 1, 2, 3, 14, 15]].tolist() == [0.5, 6.0, -6.0, 0.0, 0.0, -1.0] and not got[4:14].any()
    assert kv4.values(one, np.array([[0x38 + 8]], np.uint8))[0, 1] == 12.0
    assert np.isnan(kv4.values(one, np.array([[0x7F]], np.uint8))).all()


def pin_scales():
    """The scale is torch's rounding of amax / 6 to e4m3, the codes are the nearest by search over all 16."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((500, 32)) * 2.0 ** rng.integers(-12, 12, (500, 1))).half()
    for g in (1.0, 0.5, 8.0):
        codes, sb, val = kv4.quantise(x.double().numpy(), g)
        blocks = x.float().unflatten(-1, (2, 16))
        s = (blocks.abs().amax(-1) / np.float32(6 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        np.testing.assert_array_equal(sb, s.view(torch.uint8).numpy())
        unit = s.double().numpy()[..., None] * g
        grid = np.concatenate([kv4.E2M1, -kv4.E2M1]) * unit[..., None]
        best = np.abs(blocks.double().numpy()[..., None] - grid).min(-1)
        err = np.abs(blocks.double().numpy() - val.reshape(500, 2, 16))
        np.testing.assert_array_equal(err[(unit > 0)[..., 0]], best[(unit > 0)[..., 0]])
        assert (codes.reshape(500, 2, 8)[(unit == 0)[..., 0]] == 0).all()


def pin_ties_and_specials():
    x = np.zeros((1, 16))
    x[0] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0.26, 0.24, 5.01, -0.0, 0.0]
    codes, sb, _ = kv4.quantise(x, 1.0)
    assert sb[0, 0] == 0x38
    low, high = codes[0] & 15, codes[0] >> 4
    flat = np.stack([low, high], -1).ravel().tolist()
    assert flat == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 14, 1, 0, 7, 8, 0]
    # amax / 6 halfway between 1 and 1.125 goes to 1 (even mantissa), between 1.125 and 1.25 to 1.25
    for amax, byte in ((6 * 1.0625, 0x38), (6 * 1.1875, 0x3A), (1e9, 0x7E), (6 * 2.0 ** -10, 0), (6 * 2.0 ** -9.9, 1)):
        x[:] = 0
        x[0, 3] = -amax
        assert kv4.quantise(x, 1.0)[1][0, 0] == byte, amax
    x[0, 3] = np.inf
    x[0, 4] = 1.0
    codes, sb, val = kv4.quantise(x, 1.0)
    assert sb[0, 0] == 0x7E and val[0, 3] == 6 * 448.0 and val[0, 4] == 0
    x[0, 5] = np.nan
    codes, sb, val = kv4.quantise(x, 1.0)
    assert sb[0, 0] == 0x7F and np.isnan(val).all()


def pin_tables():
    """Token after token, request after request: a token that finds its request's pages full takes one."""
    rng = np.random.default_rng(3)
    for page in (1, 4, 16):
        qo, kv = rng.integers(0, 30, 9), rng.integers(0, 60, 9)
        kv[2] = qo[2] = 0
        held = [list(rng.integers(100, 200, -(-k // page))) for k in kv]
        table = np.full((9, 100), -1, np.int64)
        for b, h in enumerate(held):
            table[b, : len(h)] = h
        free = np.arange(900, 900 + 400)
        got = kv4.tables(qo, kv, table, free, len(free), page)
        stack, slots, positions, fresh = list(free), [], [], []
        for b in range(9):
            before = len(held[b])
            for pos in range(kv[b], kv[b] + qo[b]):
                if pos == len(held[b]) * page:
                    held[b].append(stack.pop())
                slots.append(held[b][pos // page] * page + pos % page)
                positions.append(pos)
            fresh.append(len(held[b]) - before)
        assert got["slot_mapping"].tolist() == slots and got["positions"].tolist() == positions
        assert got["kv_page_indices"].tolist() == [p for h in held for p in h] and got["free_count"] == len(stack)
        for name, n in (("qo_indptr", qo), ("kv_page_indptr", [len(h) for h in held]), ("new_page_indptr", fresh)):
            assert got[name].tolist() == [sum(n[:i]) for i in range(10)]
        assert got["kv_lens"].tolist() == [k + q for k, q in zip(kv, qo)]
        assert got["kv_last_page_len"].tolist() == [((k + q - 1) % page + 1) if k + q else 0 for k, q in zip(kv, qo)]
        assert [list(table[b, : len(h)]) for b, h in enumerate(held)] == held


def pin_attention():
    """torch's attention over the values gathered one key at a time."""
    rng = np.random.default_rng(5)
    page, Hq, Hkv, D = 4, 6, 2, 32
    qo, kv = [1, 5, 0, 3, 2], [9, 5, 8, 20, 0]
    pages = [-(-n // page) for n in kv]
    ids = rng.permutation(sum(pages) + 2)
    indptr = lambda n: np.concatenate([[0], np.cumsum(n)])  # noqa: E731
    q = rng.standard_normal((sum(qo), Hq, D))
    for hnd in (False, True):
        mid = (Hkv, page) if hnd else (page, Hkv)
        codes = rng.integers(0, 256, (len(ids), 2, *mid, D // 2), dtype=np.uint8)
        scales = rng.integers(0x20, 0x40, (len(ids), 2, *mid, D // 16), dtype=np.uint8)
        last = [(n - 1) % page + 1 if n else 0 for n in kv]
        for causal in (True, False):
            out, lse, spread = kv4.attention(q, codes, scales, 0.5, 2.0, indptr(qo), indptr(pages), ids, last, page, hnd, causal)
            for b in range(5):
                r0, n, m = indptr(qo)[b], kv[b], qo[b]
                if n == 0:
                    assert (out[r0: r0 + m] == 0).all() and np.isneginf(lse[r0: r0 + m]).all()
                    continue
                x = np.zeros((2, n, Hkv, D))
                for t in range(n):
                    at = ids[indptr(pages)[b] + t // page]
                    for h in range(Hkv):
                        for half in range(2):
                            place = (at, half, h, t % page) if hnd else (at, half, t % page, h)
                            x[half, t, h] = kv4.values(codes[place], scales[place])
                k, v = (torch.from_numpy(y * s).repeat_interleave(Hq // Hkv, 1).transpose(0, 1) for y, s in zip(x, (0.5, 2.0)))
                Q = torch.from_numpy(q[r0: r0 + m]).transpose(0, 1)
                mask = torch.ones(m, n, dtype=torch.bool)
                if causal:
                    mask = torch.arange(n)[None] <= n - m + torch.arange(m)[:, None]
                want = F.scaled_dot_product_attention(Q, k, v, attn_mask=mask).transpose(0, 1).numpy()
                z = (Q @ k.transpose(1, 2) / math.sqrt(D)).masked_fill(~mask, -math.inf)
                np.testing.assert_allclose(out[r0: r0 + m], want, rtol=1e-12, atol=1e-12)
                np.testing.assert_allclose(lse[r0: r0 + m], torch.logsumexp(z, -1).t().numpy(), rtol=1e-12, atol=1e-12)
                p = torch.softmax(z, -1)
                np.testing.assert_allclose(spread["av"][r0: r0 + m], (p @ v.abs()).transpose(0, 1).numpy(), rtol=1e-12, atol=0)
                seen = mask.double().expand(Hq, m, n)
                np.testing.assert_allclose(spread["v"][r0: r0 + m], (seen @ v.abs()).transpose(0, 1).numpy(), rtol=1e-12, atol=0)
                s = (Q.abs() @ k.abs().transpose(1, 2) / math.sqrt(D)).masked_fill(~mask, 0.0).amax(-1).t().numpy()
                np.testing.assert_allclose(spread["s"][r0: r0 + m], s, rtol=1e-12, atol=0)
                assert (spread["n"][r0: r0 + m] == mask.sum(-1).numpy()[:, None]).all()


def pin_rows_before_their_keys():
    """Causal with more queries than keys: the first rows see nothing."""
    out, lse, _ = kv4.attention(np.ones((3, 1, 16)), np.full((1, 2, 4, 1, 8), 0x22, np.uint8), np.full((1, 2, 4, 1, 1), 0x38, np.uint8),
                                1.0, 1.0, [0, 3], [0, 1], [0], [2], 4, False, True)
    assert np.isneginf(lse[0, 0]) and not out[0].any()
    assert lse[1, 0] == 4.0 and lse[2, 0] == pytest.approx(4 + math.log(2), abs=1e-14) and (out[1:] == 1).all()


PINS = [pin_formats, pin_scales, pin_ties_and_specials, pin_tables, pin_attention, pin_rows_before_their_keys]


@pytest.mark.parametrize("pin", PINS, ids=lambda f: f.__name__)
def test_pins(pin):
    pin()


def half_up(a, grid):
    i = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    return np.where(grid[i] - a <= a - grid[i - 1], i, i - 1)


def swapped_nibbles(codes, scales, real=kv4.values):
    return real(((codes << 4) | (codes >> 4)).astype(np.uint8), scales)


def always_nhd(cache, page, half, slot, hnd):
    return cache[page, half, slot]


MISTAKES = {"ties away from even": ("nearest", half_up), "high nibble first": ("values", swapped_nibbles),
            "layout ignored": ("rows", always_nhd),
            "bias 6": ("E4M3", kv4.E4M3 * 2), "no 3 among the codes": ("E2M1", np.array([0, 0.5, 1, 1.5, 2, 2.5, 4, 6.0]))}


@pytest.mark.parametrize("name", MISTAKES)
def test_planted_mistakes(name, monkeypatch):
    monkeypatch.setattr(kv4, *MISTAKES[name])
    caught = 0
    for pin in PINS:
        try:
            pin()
        except (AssertionError, IndexError, ValueError):
            caught += 1
    assert caught, name
