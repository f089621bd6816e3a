"""CPU oracle of the attention entry points, in plain numpy.

Angles, scores, softmax and sums are fp64. What include/moe.h fixes to fp32
(the rotation's products and sums, and the quantisation) is done in fp32 here
too, so that stored codes can be compared exactly. Shares no code with the
CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

F32 = np.float32
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
GROUP = 16


def e4m3_values() -> np.ndarray:
    """The 256 values of an e4m3 byte (1 sign, 4 exponent, 3 mantissa bits,
    bias 7; 0x7f and 0xff are NaN)."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = math.nan if (b & 0x7f) == 0x7f else v * (-1 if b & 0x80 else 1)
    return out


E4M3 = e4m3_values()


def nearest_even(x, steps):
    """Index of the nearest of ascending `steps`; ties to the even index;
    saturating."""
    mids = (steps[1:] + steps[:-1]) / 2
    lo, hi = np.searchsorted(mids, x, side="left"), np.searchsorted(mids, x, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def frequencies(R, base, kind="none", factor=1.0, original=0.0, slow=0.0, fast=0.0, gain=0.0):
    """(radians per position of the R/2 pairs, factor on cosines and sines)."""
    slow = slow or 1.0
    fast = fast or (32.0 if kind == "yarn" else 4.0)
    if kind == "ntk":
        base = base * factor ** (R / (R - 2))
    f = np.array([base ** (-2.0 * i / R) for i in range(R // 2)])
    if kind == "linear":
        f = f / factor
    elif kind == "parts":
        turns = original * f / (2 * math.pi)
        keep = np.clip((turns - slow) / (fast - slow), 0, 1)
        f = f * keep + f / factor * (1 - keep)
    elif kind == "yarn":
        lo, hi = (R * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
                  for turns in (fast, slow))
        lo, hi = math.floor(lo), math.ceil(hi)
        if hi < 0:          # the whole ramp lies before the first pair
            lo, hi = -1, 0
        elif lo > R - 1:    # or behind the last
            hi = lo + 1
        else:
            lo, hi = max(lo, 0), min(hi, R - 1)
            hi = hi + 0.001 if hi == lo else hi
        ramp = np.clip((np.arange(R // 2) - lo) / (hi - lo), 0, 1)
        f = f * (1 - ramp) + f / factor * ramp
        gain = gain or 0.1 * math.log(factor) + 1.0
    return f, gain or 1.0


def rope_table(positions, R, base, **kw):
    """[n, R] fp64 rows: cosines of the pairs, then sines."""
    f, gain = frequencies(R, base, **kw)
    a = np.asarray(positions, dtype=np.float64)[:, None] * f
    return gain * np.concatenate([np.cos(a), np.sin(a)], axis=1)


def rotate(x, positions, table, R, interleaved, inverse=False, dtype=F32):
    """x [T, heads, D] with its first R channels turned, products and sums
    rounded one by one in `dtype`."""
    x = np.array(x, dtype=dtype)
    if R == 0:
        return x
    rows = np.asarray(table, dtype=dtype)[positions][:, None]
    c, s = rows[..., :R // 2], rows[..., R // 2:]
    s = -s if inverse else s
    ia = np.arange(R // 2) * 2 if interleaved else np.arange(R // 2)
    ib = ia + 1 if interleaved else ia + R // 2
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = (a * c).astype(dtype) - (b * s).astype(dtype)
    x[..., ib] = (b * c).astype(dtype) + (a * s).astype(dtype)
    return x


def quantise(x, scale=1.0):
    """Signed code values (multiples of a level) and scale bytes of fp32 rows
    [..., D]."""
    y = np.asarray(x, dtype=F32) * (F32(1) / F32(scale))
    y = np.where(np.isnan(y), F32(0), y).astype(F32)
    g = y.reshape(*y.shape[:-1], y.shape[-1] // GROUP, GROUP)
    with np.errstate(over="ignore"):
        want = np.abs(g).max(-1) * F32(1.0 / 6.0)
    s8 = nearest_even(np.minimum(want.astype(np.float64), 448), E4M3[:127])
    s = E4M3[s8].astype(F32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, np.abs(g) / s, F32(0)).astype(F32)
    mag = nearest_even(q.astype(np.float64), LEVELS)
    return (LEVELS[mag] * np.where(g < 0, -1.0, 1.0)).reshape(y.shape), s8.astype(np.uint8)


def stored_values(codes, scales, scale=1.0):
    """fp64 values of code values [..., D] and scale bytes [..., D/16]."""
    return codes * np.repeat(E4M3[scales], GROUP, axis=-1) * float(F32(scale))


def pack_cache(k, v, page_size):
    """The cache bytes of k and v, each (codes [pages, page_size, heads, D],
    scale bytes [..., D/16]): [pages, heads, block bytes]."""
    parts = []
    for codes, scales in (k, v):
        n = codes.shape[0]
        nib = nearest_even(np.abs(codes), LEVELS).astype(np.uint8) | \
            (np.signbit(codes).astype(np.uint8) << 3)
        b = nib[..., 0::2] | (nib[..., 1::2] << 4)
        for a in (b, scales):
            parts.append(np.moveaxis(a, 2, 1).reshape(n, codes.shape[2], -1))
    return np.concatenate(parts, axis=-1)


def unpack_cache(cache, page_size, D):
    """Inverse of pack_cache: ((k codes, k scales), (v codes, v scales))."""
    n, heads, _ = cache.shape
    out, at = [], 0
    for _ in range(2):
        b = cache[..., at:at + page_size * D // 2].reshape(n, heads, page_size, D // 2)
        at += page_size * D // 2
        s = cache[..., at:at + page_size * D // 16].reshape(n, heads, page_size, D // 16)
        at += page_size * D // 16
        nib = np.stack([b & 15, b >> 4], axis=-1).reshape(n, heads, page_size, D)
        codes = LEVELS[nib & 7] * np.where(nib & 8, -1.0, 1.0)
        out.append((np.moveaxis(codes, 1, 2), np.moveaxis(s, 1, 2)))
    return out


def attention(q, k, v, n, scale, window=0):
    """One request: q [m, heads, D], k and v [>= n, kv heads, D] fp64 values;
    the queries are the last m of its n tokens. Returns (out, lse,
    sum of p |v|, largest sum of |q k| * scale of a seen key)."""
    m, heads, D = q.shape
    g = heads // k.shape[1]
    out, lse = np.zeros((m, heads, D)), np.full((m, heads), -np.inf)
    size, reach = np.zeros((m, heads, D)), np.zeros((m, heads))
    for i in range(m):
        p = n - m + i
        first = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        for h in range(heads):
            ks, vs = k[first:p + 1, h // g], v[first:p + 1, h // g]
            x = ks @ q[i, h] * scale
            top = x.max()
            e = np.exp(x - top)
            w = e / e.sum()
            lse[i, h] = top + np.log(e.sum())
            out[i, h], size[i, h] = w @ vs, w @ np.abs(vs)
            reach[i, h] = (np.abs(ks) @ np.abs(q[i, h])).max() * scale
    return out, lse, size, reach
