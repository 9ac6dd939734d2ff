"""Host definitions, in 64 bits, of rotary positions, the paged key-value cache and the attention of a
step's rows over it (TEST INFRASTRUCTURE ONLY). Plain numpy, request by request and token by token."""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot_dim, theta=10000.0, scaling=None, factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """(radians per position of each pair, amplitude)"""
    f = np.array([theta ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "by_parts":
        w = (original_len * f / (2.0 * math.pi) - beta_slow) / (beta_fast - beta_slow)
        w = np.minimum(np.maximum(w, 0.0), 1.0)
        return f * (w + (1.0 - w) / factor), (0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0)
    return f, 1.0


def rope(x, pos, f, interleaved=False, amplitude=1.0, inverse=False):
    """x [rows, heads, dim] float64, pos [rows] integers, f radians per position: the rotated rows."""
    x = np.array(x, dtype=np.float64)
    rot = 2 * len(f)
    angle = np.asarray(pos, dtype=np.float64)[:, None] * f[None, :]
    c, s = amplitude * np.cos(angle)[:, None, :], amplitude * np.sin(angle)[:, None, :]
    if inverse:
        s = -s
    if interleaved:
        one, two = np.arange(0, rot, 2), np.arange(1, rot, 2)
    else:
        one, two = np.arange(rot // 2), np.arange(rot // 2, rot)
    out = x.copy()
    a, b = x[:, :, one], x[:, :, two]
    out[:, :, one] = a * c - b * s
    out[:, :, two] = b * c + a * s
    return out


def e4m3_value(code):
    """The number an e4m3 code stands for (S EEEE MMM, bias 7, no infinity, S1111111 is NaN)."""
    s, e, m = code >> 7, (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if s else v


E4M3 = np.array([e4m3_value(c) for c in range(256)])
_POSITIVE = E4M3[:127]                                   # 0 .. 448, ascending


def e4m3_code(x):
    """Codes of x (float64, |x| <= 448 where finite), to nearest, ties to the even code; not finite -> NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = (_POSITIVE[hi] - a < a - _POSITIVE[lo]) | ((_POSITIVE[hi] - a == a - _POSITIVE[lo]) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.int64)
    code = np.where(np.isfinite(x), code, 127)
    sign = np.where(np.signbit(x) & np.isfinite(x), 128, 0)
    return (code + sign).astype(np.uint8)


def e4m3_exponent(x):
    """Exponent of the head x (last axis): smallest e >= -126 with max |finite x| <= 448 * 2^e, 0 for zeros."""
    x = np.asarray(x, dtype=np.float64)
    top = np.max(np.where(np.isfinite(x), np.abs(x), 0.0), axis=-1)
    e = np.full(top.shape, -126, dtype=np.int64)
    for k in range(-125, 128):
        e = np.where(top > 448.0 * 2.0 ** (k - 1), k, e)
    return np.where(top == 0, 0, e)


def owners(cu, B):
    """(request, index within it) of every row, in order."""
    return [(b, j) for b in range(B) for j in range(int(cu[b + 1]) - int(cu[b]) + 1)]


def attention(q, k, v, cached, scale, window=0):
    """One request: q [n, heads, dim] at tokens cached .. cached + n - 1, k and v [tokens, kv_heads, dim], all
    float64. Returns (out, lse, spread): spread = sum p |v|, by which rounded weights may move out."""
    n, H, D = q.shape
    G = H // k.shape[1]
    out, spread, lse = np.zeros((n, H, D)), np.zeros((n, H, D)), np.full((n, H), -np.inf)
    for j in range(n):
        first = max(0, cached + j - window + 1) if window else 0
        K, V = k[first: cached + j + 1], v[first: cached + j + 1]
        for h in range(H):
            with np.errstate(invalid="ignore"):
                z = scale * (K[:, h // G] @ q[j, h])
                m = z.max()
                if m == -np.inf:
                    continue
                p = np.exp(z - m)
                total = p.sum()
                keep = p > 0
                out[j, h] = p[keep] @ V[keep, h // G] / total
                spread[j, h] = p[keep] @ np.abs(V[keep, h // G]) / total
                lse[j, h] = m + np.log(total)
    return out, lse, spread
