"""The 8-bit frame cache and what a layer does around it, in float64, from the definitions.

Row format ("Head Forcing", §2: per-head caches; the format itself is this library's): blocks
of 32 elements, e4m3 codes times the smallest power of two 2^e, e in [-124, 119], with
max |x| <= 448 * 2^e.  Codes are returned as the values that they stand for (code values, not
bytes), rounded to nearest even by arithmetic on the spacing of e4m3 numbers.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32
E_MIN, E_MAX = -124, 119
E4M3_MAX = 448.0


def norm_rope(x, weight=None, eps=None, positions=None, inv_freq=None, axis_pairs=(), scale=1.0, layout="interleaved"):
    """x [B, heads, L, d], positions [B, L, axes]: (result, magnitude), the magnitude of element i
    of a pair being |a| + |b| of its two (normed) elements times the scale: what rounding errors
    of the rotation are relative to."""
    y = np.asarray(x, np.float64)
    if eps is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    out, mag = y.copy(), np.abs(y)
    half = sum(axis_pairs)
    p = 0
    for axis, n in enumerate(axis_pairs):
        for _ in range(n):
            i, j = (p, p + half) if layout == "half" else (2 * p, 2 * p + 1)
            angle = (np.asarray(positions, np.float64)[:, None, :, axis] * float(inv_freq[p]))
            c, s = np.cos(angle), np.sin(angle)
            out[..., i] = scale * (y[..., i] * c - y[..., j] * s)
            out[..., j] = scale * (y[..., j] * c + y[..., i] * s)
            mag[..., i] = mag[..., j] = abs(scale) * (np.abs(y[..., i]) + np.abs(y[..., j]))
            p += 1
    return out, mag


def e4m3_round(y):
    """Nearest e4m3 value (ties to even, saturated): numbers of 4 significant bits, spaced at
    least 2^-9 apart."""
    y = np.clip(np.asarray(y, np.float64), -E4M3_MAX, E4M3_MAX)
    _, ex = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(ex - 4, -9))
    return np.rint(y / step) * step  # np.rint: ties to even


def block_exponent(top):
    """Smallest e in [E_MIN, E_MAX] with top <= 448 * 2^e."""
    e = np.full(np.shape(top), E_MIN, np.int64)
    for x in range(E_MIN, E_MAX):
        e = np.where(np.asarray(top) > math.ldexp(E4M3_MAX, x), x + 1, e)
    return e


def quantise(x):
    """(code values [..., d], exponents [..., d / 32])."""
    x = np.asarray(x, np.float64)
    blk = x.reshape(x.shape[:-1] + (-1, BLOCK))
    e = block_exponent(np.abs(blk).max(-1))
    return e4m3_round(np.ldexp(blk, -e[..., None])).reshape(x.shape), e


def dequantise(codes, e):
    blk = np.asarray(codes, np.float64).reshape(codes.shape[:-1] + (-1, BLOCK))
    return np.ldexp(blk, np.asarray(e)[..., None]).reshape(codes.shape)


def place(table, heads, page_len, b, h, j):
    """(page, head of the page, row) of logical token j of (b, h); table [B][H_kv or 1][N]."""
    row = table[b][h if len(table[b]) > 1 else 0]
    return int(row[j // page_len]), (h if heads > 1 else 0), j % page_len


def attention(q, k, v, scale, causal=False):
    """One head: q [L, d] over k, v [n, d].  Causal: query i sees j <= n - L + i.  Rows that see
    nothing give O = 0 and LSE = -inf.  Returns (O, LSE, sum_j p_j |v_j|)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    L, n = q.shape[0], k.shape[0]
    o, lse, mag = np.zeros((L, v.shape[1])), np.full(L, -np.inf), np.zeros((L, v.shape[1]))
    s = scale * (q @ k.T)
    for i in range(L):
        m = n - L + i + 1 if causal else n
        if m <= 0:
            continue
        x = s[i, :m]
        top = x.max()
        p = np.exp(x - top)
        total = p.sum()
        o[i] = p @ v[:m] / total
        mag[i] = p @ np.abs(v[:m]) / total
        lse[i] = top + math.log(total)
    return o, lse, mag
