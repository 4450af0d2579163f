"""CPU oracle of the routed-expert operations (clover_route,
clover_quantize_fp4, clover_fp4_product, clover_moe_combine): plain fp64
definitions, loops over tokens and rows.

TEST INFRASTRUCTURE, like clover_oracle.py: it shares no code with the
library or its binding."""
from __future__ import annotations

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def route_token(z, top_k, score="softmax", bias=None, n_groups=1, top_groups=1, group_rank=1, renormalise=True,
                scale=1.0):
    """One token's logits z [E] -> (experts in descending key order, weights), at most top_k of them."""
    z = np.minimum(np.asarray(z, dtype=np.float64), FLT_MAX)
    E = z.shape[0]
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    live = [e for e in range(E) if z[e] > -np.inf and b[e] > -np.inf]
    if not live:
        return [], np.zeros(0)
    s = np.zeros(E)
    with np.errstate(over="ignore"):
        if score == "softmax":
            m = max(z[e] for e in range(E) if z[e] > -np.inf)
            tot = sum(np.exp(z[e] - m) for e in range(E) if z[e] > -np.inf)
            for e in live:
                s[e] = np.exp(z[e] - m) / tot
        else:
            for e in live:
                s[e] = 1.0 / (1.0 + np.exp(-z[e]))
    key = {e: (z[e] if bias is None else s[e] + b[e]) for e in live}
    if n_groups > 1:
        size = E // n_groups
        ranks = []
        for g in range(n_groups):
            mem = [e for e in live if e // size == g]
            if not mem:
                ranks.append(-np.inf)
            elif group_rank == 1:
                ranks.append(max(key[e] for e in mem))
            else:
                ranks.append(sum(sorted((s[e] + b[e] for e in mem), reverse=True)[:2]))
        keep = sorted(range(n_groups), key=lambda g: (-ranks[g], g))[:top_groups]
        live = [e for e in live if e // size in keep]
    sel = sorted(live, key=lambda e: (-key[e], e))[:top_k]
    if not sel:
        return [], np.zeros(0)
    if renormalise:  # in logarithms, so that scores below the smallest double still have a ratio
        ls = np.array([z[e] if score == "softmax" else -np.logaddexp(0.0, -z[e]) for e in sel])
        w = np.exp(ls - ls.max())
        w = w / w.sum()
    else:
        w = s[sel]
    return sel, w * scale


def route(z, top_k, **kw):
    """[M][E] logits -> dict idx, w, offsets, rows (valid part), pos."""
    z = np.asarray(z)
    M, E = z.shape
    idx = np.full((M, top_k), -1, dtype=np.int32)
    w = np.zeros((M, top_k))
    for t in range(M):
        sel, wt = route_token(z[t], top_k, **kw)
        idx[t, :len(sel)] = sel
        w[t, :len(sel)] = wt
    rows, offsets = [], [0]
    pos = np.full((M, top_k), -1, dtype=np.int32)
    for e in range(E):
        for t, k in zip(*np.nonzero(idx == e)):
            pos[t, k] = len(rows)
            rows.append(t * top_k + k)
        offsets.append(len(rows))
    return {"idx": idx, "w": w, "offsets": np.array(offsets, dtype=np.int32), "rows": np.array(rows, dtype=np.int32),
            "pos": pos}


# ------------------------------------------------------------ 4-bit formats


def e4m3_value(byte):
    b = int(byte)
    if b & 0x7F == 0x7F:
        return np.nan
    e, m = (b >> 3) & 15, b & 7
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if b & 0x80 else v


E4M3 = np.array([e4m3_value(b) for b in range(127)])  # ascending, 0 .. 448


def nearest(table, v):
    """Index of the entry of an ascending table nearest to v >= 0; a tie goes to the even index."""
    i = int(np.searchsorted(table, v))
    if i == 0:
        return 0
    if i == len(table):
        return len(table) - 1
    lo, hi = v - table[i - 1], table[i] - v
    if lo == hi:
        return i if i % 2 == 0 else i - 1
    return i - 1 if lo < hi else i


def quantize_block(x, fmt, scale_exp=0):
    """One block (fp32 values as fp64) -> (code nibbles, scale byte)."""
    with np.errstate(invalid="ignore", under="ignore"):
        y = (np.asarray(x, dtype=np.float32) * np.float32(2.0 ** -scale_exp)).astype(np.float64)
    if not np.all(np.isfinite(y)):
        return np.zeros(len(y), dtype=np.uint8), 0x7F if fmt == "nv" else 0xFF
    amax = np.abs(y).max()
    if fmt == "nv":
        sb = nearest(E4M3, min(amax / 6.0, 448.0))
        s = E4M3[sb]
    else:
        e = -127 if amax == 0 else max(int(np.frexp(amax)[1]) - 3, -127)
        sb, s = e + 127, 2.0 ** e
    codes = np.zeros(len(y), dtype=np.uint8)
    if s > 0:
        for i, v in enumerate(y):
            codes[i] = nearest(E2M1, abs(v) / s) + (8 if np.signbit(v) else 0)
    return codes, sb


def quantize(x, fmt, scale_exp=0):
    """[rows][cols] -> (codes [rows][cols] one nibble each, scale bytes [rows][blocks])."""
    block = 16 if fmt == "nv" else 32
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    codes = np.zeros((rows, cols), dtype=np.uint8)
    sb = np.zeros((rows, cols // block), dtype=np.uint8)
    for r in range(rows):
        for b in range(cols // block):
            codes[r, b * block:(b + 1) * block], sb[r, b] = quantize_block(x[r, b * block:(b + 1) * block], fmt,
                                                                           scale_exp)
    return codes, sb


def scale_values(sb, fmt):
    if fmt == "nv":
        return np.vectorize(e4m3_value, otypes=[np.float64])(sb)
    return np.where(sb == 255, np.nan, 2.0 ** (sb.astype(np.float64) - 127))


def dequantize(codes, sb, fmt, scale_exp=0):
    block = 16 if fmt == "nv" else 32
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(scale_values(sb, fmt), block, axis=1) * 2.0 ** scale_exp


def pack_codes(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def scale_tiles(n_tiles, blocks):
    return np.zeros((n_tiles, -(-blocks // 4), 512), dtype=np.uint8)


def scale_place(row, block):
    """(row tile, column tile, byte) of a scale in its tiles."""
    r = row % 128
    return row // 128, block // 4, (r % 32) * 16 + (r // 32) * 4 + block % 4


def grouped_scale_row(i, offsets):
    """The row of the scale tiles that grouped row i takes: group g starts at tile offsets[g] / 128 + g."""
    g = max(g for g in range(len(offsets) - 1) if offsets[g] <= i < offsets[g + 1])
    return (offsets[g] // 128 + g) * 128 + (i - offsets[g])


def product(a, b, offsets, alpha=None, swiglu=False):
    """a [rows][K], b [groups][N][K] (values) -> y rows of their group's product (gate rows of b first)."""
    out = []
    for g in range(len(offsets) - 1):
        y = np.asarray(a)[offsets[g]:offsets[g + 1]] @ np.asarray(b)[g].T
        if alpha is not None:
            y = y * alpha[g]
        if swiglu:
            h = y.shape[1] // 2
            y = y[:, :h] / (1.0 + np.exp(-y[:, :h])) * y[:, h:]
        out.append(y)
    return np.concatenate(out)


def combine(y, pos, w, x=None, shared=None):
    y, pos, w = np.asarray(y, dtype=np.float64), np.asarray(pos), np.asarray(w, dtype=np.float64)
    M, K = pos.shape
    out = np.zeros((M, y.shape[1])) if x is None else np.asarray(x, dtype=np.float64).copy()
    for t in range(M):
        for k in range(K):
            if 0 <= pos[t, k] < y.shape[0]:
                out[t] += w[t, k] * y[pos[t, k]]
    return out if shared is None else out + np.asarray(shared, dtype=np.float64)
