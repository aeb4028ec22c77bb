"""Plain 64-bit implementations (numpy) of the cache and sampling operators, for the tests.

Written from the definitions in include/pspec.h; they share no code with the kernels."""
import math

import numpy as np
import torch

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # eps / 2: one rounding


def f64(t):
    return t.detach().double().cpu().numpy()


def e4m3_grid():
    """The finite non-negative e4m3 values by code 0 .. 126."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out, np.float64)


GRID = e4m3_grid()


def nearest_code(x, grid):
    """Index of the grid value nearest to x >= 0, ties to the even index, the largest above it."""
    hi = np.clip(np.searchsorted(grid, x), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - x, x - grid[lo]
    take = (up < down) | ((up == down) & (hi % 2 == 0)) | (x >= grid[-1])
    return np.where(take, hi, lo)


def quantise(x, g):
    """(codes [..., D], scale codes [..., D/16]) of x [..., H, D], head scales g [H]."""
    y = np.where(np.isnan(x), 0.0, x)
    b = y.reshape(*y.shape[:-1], -1, 16)
    gg = g[:, None]
    s_code = nearest_code(np.abs(b).max(-1) / gg / 6, GRID)
    s = GRID[s_code]
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(s[..., None] > 0, np.abs(b) / gg[..., None] / s[..., None], 0.0)
    code = nearest_code(np.where(np.isnan(z), 0.0, z), LEVELS)
    sign = np.signbit(b) & ~np.isnan(x.reshape(b.shape))
    return (code + 8 * sign).reshape(x.shape).astype(np.uint8), s_code.astype(np.uint8)


def values(code, s_code, g):
    """What codes [..., H, D] with scale codes [..., H, D/16] and head scales g [H] stand for."""
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(GRID[s_code], 16, axis=-1) * g[:, None]


def rotate(x, pos, inv_freq, interleaved):
    """x [T, H, D] with its first 2 len(inv_freq) elements turned by pos * inv_freq."""
    h = len(inv_freq)
    ang = pos.astype(np.float64)[:, None] * inv_freq.astype(np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    out = x.copy()
    ia, ib = (np.arange(0, 2 * h, 2), np.arange(1, 2 * h, 2)) if interleaved else (np.arange(h), np.arange(h, 2 * h))
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    return out


def unpack(pages):
    """Codes [..., D] of bytes [..., D/2]."""
    return np.stack((pages & 15, pages >> 4), -1).reshape(*pages.shape[:-1], -1)


def pack(code):
    return (code[..., ::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def cache_values(cache, which):
    """[num_blocks, heads, block_size, D] values of a 4-bit cache."""
    pages = getattr(cache, which).cpu().numpy()
    sc = getattr(cache, which + "_block_scales").view(torch.uint8).cpu().numpy()
    g = getattr(cache, which + "_scale")
    g = np.ones(pages.shape[1]) if g is None else f64(g)
    sc = np.where(sc <= 126, sc, 0)                            # NaN and negative scales count as 0
    return values(unpack(pages).swapaxes(1, 2), sc.swapaxes(1, 2), g).swapaxes(1, 2)


def attend(q, kv, vv, table, qsl, pos, lens, scale, block_size, row_kind=None):
    """(out, lse, seen, a, vmax): the definition row by row; seen: rows of a sequence that are
    computed; a: max over keys of sum |q_d k_d| * |scale| (for error bounds); vmax: largest
    value magnitude a row may average per element."""
    T, Hq, D = q.shape
    Hkv = kv.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    seen, a, vmax = np.zeros(T, bool), np.zeros((T, Hq)), np.zeros((T, Hq, D))
    nb = kv.shape[0]
    for i in range(len(lens)):
        lo, hi = int(qsl[i]), int(qsl[i + 1])
        if lo < 0 or hi < lo or hi > T:
            continue
        n = max(0, min(int(lens[i]), table.shape[1] * block_size))
        j = np.arange(n)
        blk = table[i, j // block_size] if n else np.zeros(0, np.int64)
        ok = (blk >= 0) & (blk < nb)
        kk = kv[np.where(ok, blk, 0), :, j % block_size]        # [n, Hkv, D]
        vvv = vv[np.where(ok, blk, 0), :, j % block_size]
        for t in range(lo, hi):
            if row_kind is not None and row_kind[t] >= 3:
                continue
            seen[t] = True
            vis = ok & (j <= pos[t])
            if not vis.any():
                continue
            for h in range(Hq):
                k1, v1 = kk[vis, h // G], vvv[vis, h // G]
                x = k1 @ q[t, h] * scale
                m = x.max()
                p = np.exp(x - m)
                z = p.sum()
                out[t, h] = p @ v1 / z
                lse[t, h] = m + math.log(z)
                a[t, h] = (np.abs(k1) @ np.abs(q[t, h])).max() * abs(scale)
                vmax[t, h] = np.abs(v1).max(0)
    return out, lse, seen, a, vmax


def attend_bounds(dtype, D, ref, a, vmax):
    """Elementwise error bound of the kernel's output against the exact one.

    A score is a sum of D exact products in fp32 (tensor core: at most D roundings of partial
    sums, each at most 2^-23 relative: truncation allowed) and three fp32 factors: off by at
    most (D + 4) 2^-23 a in the exponent's units, with the exponential (2^-22) and the fp32
    argument (2^-24 of |x - m| <= 2a, in base-2 units 1.45 times that) the weight is off by
    d = (D + 8) 2^-23 a + 2^-21 relative; a weighted mean moves by at most 2 d vmax.  Rounding
    the weights to fp16 (bf16 rows): 2^-11 vmax more, and 2^-24 / 2^7 of the largest weight per
    key below its subnormals, far less.  fp32 rows: two terms of 11 bits of queries and weights
    each (2^-22 of a, 2^-22 vmax).  Sums over keys in fp32: 2^-20 vmax covers 2^3 roundings of
    each of the levels' partial sums.  Last, one rounding to the dtype."""
    d = (D + 8) * 2.0 ** -23 * a + 2.0 ** -21 + 2.0 ** -20
    if dtype == torch.bfloat16:
        d2 = 2.0 ** -11
    else:
        d2 = 2.0 ** -22
        d = d + 2.0 ** -21 * a
    return HALF_STEP[dtype] * np.abs(ref) * 1.01 + (2 * d[..., None] + d2) * vmax + 1e-30, d


def filtered(logits, u, temperature, top_k, top_p, min_p):
    """(token, probability, margin) of one row: margin is how far u lies from the drawn token's
    borders in the running mass (relative), infinite where nothing is drawn."""
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    V = len(x)
    M = x.max()
    if M == -np.inf:
        return 0, 0.0, np.inf
    if temperature == 0:
        return int(np.argmax(x)), 1.0, np.inf
    with np.errstate(invalid="ignore"):
        w = np.where(x == M, 1.0, np.exp((x - M) / temperature))
    order = np.lexsort((np.arange(V), -x))
    n = V
    if top_k > 0:
        n = min(n, top_k)
    if top_p < 1:
        c = np.cumsum(w[order[:n]])
        before = np.concatenate(([0.0], c[:-1]))
        n = max(1, int((before < top_p * c[-1]).sum()))
    if min_p > 0:
        n = max(1, int((w[order[:n]] >= min_p).sum()))
    keep = np.sort(order[:n])
    c = np.cumsum(w[keep])
    z = c[-1]
    over = np.nonzero(c > u * z)[0]
    i = int(over[0]) if len(over) else int(np.nonzero(w[keep] > 0)[0][-1])
    lo = c[i] - w[keep[i]]
    margin = min(abs(u * z - lo) if i else np.inf, abs(c[i] - u * z)) / z
    return int(keep[i]), w[keep[i]] / z, margin
