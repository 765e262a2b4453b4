"""The 8-bit serving operators, as their plain definitions (oracle; test only).

Row quantization to INT8, the product of two such operands, position rotation, the paged
key/value cache and attention over it. Binary64 throughout; where the definition fixes a
binary32 operation (fl32) the binary64 result is rounded, which equals the binary32
operation (53 >= 2 * 24 + 2 bits).
"""
from __future__ import annotations

import numpy as np


def f32(x):
    return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def row_quant(X, c=None):
    """(codes int64, scales float64) of each row (last axis): d = max(fl32(a/127), 2^-126),
    q = RNE(fl32(x~ fl32(1/d))); an all-zero row has codes and scale 0."""
    x = np.asarray(X, dtype=np.float64)
    if c is not None:
        x = f32(x * np.asarray(c, dtype=np.float64))
    a = np.max(np.abs(x), axis=-1, keepdims=True)
    d = np.maximum(f32(a / 127.0), 2.0 ** -126)
    q = np.clip(np.rint(f32(x * f32(1.0 / d))), -127, 127)
    q = np.where(a == 0, 0.0, q)
    return q.astype(np.int64), np.where(a == 0, 0.0, d)[..., 0]


def w8a8_gemm(xq, xs, wq, ws):
    """fl32(fl32(sum) * fl32(xs ws)), the sum in 64-bit integers."""
    acc = np.asarray(xq, dtype=np.int64) @ np.asarray(wq, dtype=np.int64).T
    s = f32(np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)[None, :])
    return f32(f32(acc) * s)


def rotate(x, cos, sin, positions, interleaved=False):
    """x [T, heads, D]: the first 2 * cos.shape[1] channels turned by cos, sin [rows, dim/2]."""
    y = np.array(x, dtype=np.float64)
    h = cos.shape[1]
    ct = np.asarray(cos, np.float64)[positions][:, None]
    st = np.asarray(sin, np.float64)[positions][:, None]
    if interleaved:
        ia, ib = np.arange(0, 2 * h, 2), np.arange(1, 2 * h, 2)
    else:
        ia, ib = np.arange(h), np.arange(h, 2 * h)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = f32(f32(a * ct) - f32(b * st))
    y[..., ib] = f32(f32(b * ct) + f32(a * st))
    return y


def attention(q, k, v, causal, scale):
    """One sequence: q [n, H, D], k, v [m, G, D] -> o [n, H, D], and sum_j w_j |v_j| / sum_j w_j
    and max_j scale * sum_d |q_d k_d| per (token, head), the scales of its rounding errors."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, H, D = q.shape
    m, G, _ = k.shape
    o, mag, dot = np.zeros((n, H, D)), np.zeros((n, H, D)), np.zeros((n, H))
    for h in range(H):
        g = h // (H // G)
        s = scale * (q[:, h] @ k[:, g].T)
        sa = abs(scale) * (np.abs(q[:, h]) @ np.abs(k[:, g]).T)
        for i in range(n):
            seen = min(m, max(0, m - n + i + 1)) if causal else m
            if seen == 0:
                continue
            w = np.exp(s[i, :seen] - s[i, :seen].max())
            w /= w.sum()
            o[i, h] = w @ v[:seen, g]
            mag[i, h] = w @ np.abs(v[:seen, g])
            dot[i, h] = sa[i, :seen].max()
    return o, mag, dot
