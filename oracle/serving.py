"""Rotary positions, cache quantisation and one-token attention in float64, from their definitions."""
import math

import numpy as np

SCALE_MIN = 2.0 ** -126
E4M3_MAX = 448.0


def rotary_frequencies(rot_dim, base=10000.0, kind="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """Angles a position of the rot_dim / 2 pairs."""
    i = np.arange(rot_dim // 2, dtype=np.float64)
    if kind == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    f = base ** (-2.0 * i / rot_dim)
    if kind == "linear":
        f = f / factor
    if kind == "by_parts":
        turns = original_len * f / (2.0 * math.pi)
        keep = np.clip((turns - low) / (high - low), 0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f


def rotary(x, positions, frequencies, interleaved=False, factor=1.0, inverse=False):
    """x (B, H, S, D) with its pairs turned by positions (B, S) times the frequencies."""
    x = np.asarray(x, dtype=np.float64)
    n = len(frequencies)
    a = np.asarray(positions, dtype=np.float64)[:, None, :, None] * np.asarray(frequencies, dtype=np.float64)
    c, s = factor * np.cos(a), factor * np.sin(-a if inverse else a)
    y = x.copy()
    one = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    two = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def _half_even(y):
    return np.rint(y)          # numpy rounds halves to even


def quantise_s8(rows):
    """(codes, scales) of rows (..., D): scale = max(fp32(amax / 127), 2^-126)."""
    x = np.asarray(rows, dtype=np.float64)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    scale = np.maximum(np.float64(np.float32(np.abs(x).max(-1) / 127.0)), SCALE_MIN)
    return _half_even(x / scale[..., None]), np.where(bad, np.nan, scale)


def round_e4m3(y):
    """Nearest e4m3 values (3 mantissa bits, smallest normal 2^-6), ties to even, |y| <= 448."""
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    e = np.where(np.exp2(e + 1) <= np.abs(y), e + 1, np.where(np.exp2(e) > np.maximum(np.abs(y), 2.0 ** -6), e - 1, e))
    step = np.exp2(e - 3)
    return _half_even(y / step) * step


def quantise_e4m3(rows):
    """(code values, scales): scale = the smallest power of two >= 2^-126 with amax / scale <= 448."""
    x = np.asarray(rows, dtype=np.float64)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    amax = np.abs(x).max(-1)
    m, e = np.frexp(amax)                      # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 2^9
    scale = np.maximum(np.where(amax > 0, np.exp2(np.where(m <= 0.875, e - 9, e - 8).astype(np.float64)), 0.0), SCALE_MIN)
    return round_e4m3(x / scale[..., None]), np.where(bad, np.nan, scale)


def decode(q, keys, values, length, window=0, softcap=None, slopes=None, scale=None, vscale=None):
    """q (HQ, D) over keys and values (H, n, D): (out (HQ, D), lse (HQ,), sum p |v| (HQ, D),
    largest sum |q k| scale, max(p s) sum |v| / s (HQ, D) with s the values' row scales (H, n) or 1)
    with the query at position length - 1."""
    q, K, V = (np.asarray(t, dtype=np.float64) for t in (q, keys, values))
    HQ, D = q.shape
    H = K.shape[0]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    lo = max(0, length - window) if window else 0
    out, lse, weight, reach, fine = np.zeros((HQ, D)), np.full(HQ, -np.inf), np.zeros((HQ, D)), 0.0, np.zeros((HQ, D))
    if length - lo <= 0:
        return out, lse, weight, reach, fine
    pos = np.arange(lo, length)
    for h in range(HQ):
        k, v = K[h // (HQ // H), lo:length], V[h // (HQ // H), lo:length]
        x = scale * (k @ q[h])
        reach = max(reach, float((scale * (np.abs(k) @ np.abs(q[h]))).max()))
        if softcap is not None:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            x = x + slopes[h] * (pos - (length - 1))
        top = x.max()
        p = np.exp(x - top)
        lse[h] = top + math.log(p.sum())
        p = p / p.sum()
        out[h], weight[h] = p @ v, p @ np.abs(v)
        s = np.ones(len(p)) if vscale is None else np.asarray(vscale, dtype=np.float64)[h // (HQ // H), lo:length]
        fine[h] = (p * s).max() * (np.abs(v) / s[:, None]).sum(0)
    return out, lse, weight, reach, fine
