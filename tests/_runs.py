"""Plain forms, in 64 bits and on the host, of the operators on runs of several
tokens: a cache's tokens as values, the rotation, and attention of ragged runs.
They read the oracle's cache (or a device cache brought to the host) by the layout's
definition."""

import numpy as np

HALF_STEP = 2.0 ** -11  # the most one rounding to fp16 moves a value, relative to it


def tokens_of(r, which, b):
    """Sequence b's tokens in order (sink, packed, residual), float64 [H][n][d], of
    oracle cache r; which: "k" or "v"."""
    B, H, d, bits, cap, Nr, S, hyb = r.shape
    ns = int(r.sink_len[b]) if S else 0
    npk, nres, head = int(r.packed_len[b]), int(r.res_len[b]), int(r.res_head[b])
    codes = getattr(r, which + "_codes")[b, :, :npk].astype(np.int64)
    e = np.arange(d)
    wide = np.concatenate([codes, np.zeros_like(codes[..., :1])], -1)
    pair = wide[..., e * bits // 8] | wide[..., e * bits // 8 + 1] << 8
    code = (pair >> (e * bits % 8)) & ((1 << bits) - 1)
    p = np.ascontiguousarray(getattr(r, which + "_params")[b, :, :npk]).view(np.float16)
    p = p.reshape(H, npk, d // 32, 2).astype(np.float64).repeat(32, 2)
    x = [p[..., 1] + code * p[..., 0]]
    if S:
        x.insert(0, getattr(r, which + "_sink")[b, :, :ns].view(np.float16).astype(np.float64))
    if Nr:
        ring = (head + np.arange(nres)) % Nr
        x.append(getattr(r, which + "_res")[b][:, ring].view(np.float16).astype(np.float64))
    return np.concatenate(x, 1)


def attend(k, v, q, seen):
    """softmax(q k^T / sqrt(d)) v of rows q [T][Hq][d], row i over its first seen[i]
    tokens (zeros where there is none), and for each value the most that the kernel's
    roundings may move it: keys, values and weights are rounded to fp16 once, which
    moves a score by at most E = HALF_STEP * max_j sum |q k_j| / sqrt(d), a weight by
    (e^(2E) - 1) + HALF_STEP relative and a value by HALF_STEP; the output's own rounding
    is a third HALF_STEP; sums are in fp32
    (n * 2^-23 relative, the order left open) and the exponential within 2^-20."""
    H, n, d = k.shape
    T, Hq, _ = q.shape
    gq = Hq // H
    out = np.zeros((T, Hq, d))
    bound = np.zeros((T, Hq, d))
    for h in range(Hq):
        kk, vv = k[h // gq], v[h // gq]
        s = q[:, h] @ kk.T / np.sqrt(d)
        mag = np.abs(q[:, h]) @ np.abs(kk).T / np.sqrt(d)
        mask = np.arange(n)[None] < np.asarray(seen)[:, None]
        s = np.where(mask, s, -np.inf)
        mx = s.max(1, keepdims=True, initial=-np.inf)
        p = np.where(mask, np.exp(s - np.where(np.isfinite(mx), mx, 0.0)), 0.0)
        tot = p.sum(1, keepdims=True)
        p = p / np.where(tot > 0, tot, 1.0)
        out[:, h] = p @ vv
        E = (HALF_STEP + d * 2.0 ** -23) * np.where(mask, mag, 0.0).max(1, initial=0.0)
        rel = np.expm1(2 * E) + 3 * HALF_STEP + (n + 64) * 2.0 ** -23 + 2.0 ** -19
        bound[:, h] = rel[:, None] * (p @ np.abs(vv)) + 1e-7
    return out, bound


def rotate(x, table, pos, rotary, interleaved):
    """R1 on fp16 x [n][heads][d] at rows pos of table (fp32 [rows][rotary/2][2])."""
    if not rotary:
        return x
    y = x.copy()
    cs = table[np.clip(pos, 0, len(table) - 1)][:, None]
    c, s = cs[..., 0], cs[..., 1]
    half = rotary // 2
    a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, half), slice(half, rotary))
    xa, xb = x[..., a].astype(np.float32), x[..., b].astype(np.float32)
    y[..., a] = (xa * c - xb * s).astype(np.float16)
    y[..., b] = (xb * c + xa * s).astype(np.float16)
    return y
