"""CPU oracle of the attention operations (clover_kv_write, clover_kv_read,
clover_kv_attention, clover_prompt_attention): plain fp64 definitions, loops
over sequences, rows and heads.

TEST INFRASTRUCTURE, like clover_oracle.py: it shares no code with the
library or its binding."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """The value of every e4m3 byte."""
    out = np.zeros(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v = np.nan if (b & 127) == 127 else (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        out[b] = -v if b & 128 else v
    return out


E4M3 = e4m3_values()


def _nearest(values, x):
    """Index of the value (ascending) nearest to x >= 0, ties to the even index."""
    i = int(np.searchsorted(values, x))
    if i == 0:
        return 0
    if i == len(values):
        return i - 1
    lo, hi = x - values[i - 1], values[i] - x
    return i - 1 if lo < hi or (lo == hi and (i - 1) % 2 == 0) else i


def quantize_row(x, exp):
    """x [dim] -> (codes uint8 [dim / 2], scales uint8 [dim / 16])."""
    codes, scales = np.zeros(len(x), dtype=np.uint8), np.zeros(len(x) // 16, dtype=np.uint8)
    for b in range(len(x) // 16):
        with np.errstate(over="ignore", invalid="ignore"):
            y = np.float32(x[16 * b:16 * b + 16]) * np.float32(2.0 ** -exp)
        if not np.isfinite(y).all():
            scales[b] = 127
            continue
        y = y.astype(np.float64)
        sb = _nearest(E4M3[:127], np.abs(y).max() / 6.0)
        scales[b] = sb
        if sb:
            for i in range(16):
                codes[16 * b + i] = _nearest(E2M1, abs(y[i]) / E4M3[sb]) + (8 if np.signbit(y[i]) else 0)
    return codes[0::2] | codes[1::2] << 4, scales


def decode_row(codes, scales, exp):
    n = np.stack([codes & 15, codes >> 4], -1).reshape(-1)
    v = E2M1[n & 7] * np.where(n > 7, -1.0, 1.0)
    return v * np.repeat(E4M3[scales], 16) * 2.0 ** exp


def _place(pages, table_row, p):
    """(page, sixteen, row) of position p, or None."""
    page_tokens = 16 * pages.shape[2]
    page = table_row[p // page_tokens]
    if page < 0 or page >= pages.shape[0]:
        return None
    return page, p % page_tokens // 16, p % 16


def _parts(six, r, dim, value):
    """Views of row r's codes and scales in a sixteen."""
    base = 9 * dim if value else 0
    return (six[base + r * (dim // 2):base + (r + 1) * (dim // 2)],
            six[base + 8 * dim + r * (dim // 16):base + 8 * dim + (r + 1) * (dim // 16)])


def rows_of(offsets, n_rows):
    """(sequence, row, index of the row in the sequence, rows of the sequence) of every row."""
    off = np.clip(offsets, 0, n_rows)
    return [(s, r, r - off[s], off[s + 1] - off[s]) for s in range(len(off) - 1) for r in range(off[s], off[s + 1])]


def write(pages, k, v, offsets, lens, table, k_exp=0, v_exp=0):
    """The pages (uint8 [n][heads][sixteens][18 dim]) after the call."""
    pages = pages.copy()
    dim, cap = pages.shape[3] // 18, table.shape[1] * 16 * pages.shape[2]
    for s, r, i, n in rows_of(offsets, len(k)):
        p = min(max(int(lens[s]), 0), cap) - n + i
        at = None if p < 0 else _place(pages, table[s], p)
        if at is None:
            continue
        for h in range(pages.shape[1]):
            for x, value, exp in ((k, False, k_exp), (v, True, v_exp)):
                c, sc = _parts(pages[at[0], h, at[1]], at[2], dim, value)
                c[:], sc[:] = quantize_row(x[r, h], exp)
    return pages


def positions(pages, table_row, length, k_exp=0, v_exp=0):
    """Keys and values [length][heads][dim] of one sequence in fp64, and which positions have a page."""
    heads, dim = pages.shape[1], pages.shape[3] // 18
    out, there = np.zeros((2, length, heads, dim)), np.zeros(length, dtype=bool)
    for p in range(length):
        at = _place(pages, table_row, p)
        if at is None:
            continue
        there[p] = True
        for h in range(heads):
            for value, exp in ((0, k_exp), (1, v_exp)):
                out[value, p, h] = decode_row(*_parts(pages[at[0], h, at[1]], at[2], dim, value), exp)
    return out[0], out[1], there


def limit(p, length, block):
    return length if block == 0 else (0 if p < 0 else min(length, (p // block + 1) * block))


def attend(q, k, v, there, block, scale):
    """q [n][Hq][D], the last n positions of k, v [L][H][D] (fp64) -> out, lse, and what errors are measured by: per result
    the sum of p |v|, the largest sum of |q k| scale of a visible position, and the sum of |v|."""
    n, Hq, D = q.shape
    L, H, _ = k.shape
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    mag, size, total = np.zeros((n, Hq, D)), np.zeros((n, Hq)), np.zeros((n, Hq, D))
    for i in range(n):
        lim = limit(L - n + i, L, block)
        see = np.nonzero(there[:lim])[0]
        if len(see) == 0:
            continue
        for h in range(Hq):
            kk, vv = k[see, h // (Hq // H)], v[see, h // (Hq // H)]
            with np.errstate(invalid="ignore", over="ignore"):
                z = scale * (kk @ q[i, h])
                m = z.max()
                if m == -np.inf:
                    continue
                e = np.exp(z - m)
                out[i, h] = (e / e.sum()) @ vv
                mag[i, h] = (e / e.sum()) @ np.abs(vv)
                lse[i, h] = m + np.log(e.sum())
                size[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
                total[i, h] = np.abs(vv).sum(0)
    return out, lse, mag, size, total


def kv_attention(q, pages, offsets, lens, table, block, scale, k_exp=0, v_exp=0):
    """Results of every row (rows of no sequence: NaN), as `attend` gives them."""
    n, Hq, D = q.shape
    res = [np.full((n, Hq, D), np.nan), np.full((n, Hq), np.nan), np.zeros((n, Hq, D)), np.zeros((n, Hq)),
           np.zeros((n, Hq, D))]
    off = np.clip(offsets, 0, n)
    cap = table.shape[1] * 16 * pages.shape[2]
    for s in range(len(off) - 1):
        k, v, there = positions(pages, table[s], min(max(int(lens[s]), 0), cap), k_exp, v_exp)
        r = slice(off[s], off[s + 1])
        for x, y in zip(res, attend(q[r], k, v, there, block, scale)):
            x[r] = y
    return res


def prompt_attention(q, k, v, offsets, k_offsets, block, scale):
    n, Hq, D = q.shape
    res = [np.full((n, Hq, D), np.nan), np.full((n, Hq), np.nan), np.zeros((n, Hq, D)), np.zeros((n, Hq)),
           np.zeros((n, Hq, D))]
    off, koff = np.clip(offsets, 0, n), np.clip(k_offsets, 0, len(k))
    for s in range(len(off) - 1):
        r, c = slice(off[s], off[s + 1]), slice(koff[s], koff[s + 1])
        for x, y in zip(res, attend(q[r], k[c], v[c], np.ones(koff[s + 1] - koff[s], dtype=bool), block, scale)):
            x[r] = y
    return res
