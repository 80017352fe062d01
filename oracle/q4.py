"""Definitions of the paged cache in 4 bits.

TEST INFRASTRUCTURE ONLY, as the rest of this package: plain numpy and integers,
sharing no code with the library.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .scored import _f64, _int

GROUP = 64


def bf16_below(x):
    """The largest bf16 numbers not above fp32 numbers x, as float64."""
    b = np.asarray(x, dtype=np.float32).view(np.int32)
    low = b & 0xffff
    return np.where((b < 0) & (low != 0), b - low + 0x10000, b - low).astype(np.int32).view(np.float32).astype(np.float64)


def _scale(span):
    """The smallest bf16 numbers not below span / 15 and 2^-100 (span >= 0)."""
    with np.errstate(over="ignore"):
        near = np.asarray(span / 15).astype(np.float32).view(np.int32) >> 16
    found = np.full(np.shape(span), np.inf)
    for step in (1, 0, -1):  # from above: the last that is large enough
        c = (np.maximum(near + step, 0) << 16).astype(np.int32).view(np.float32).astype(np.float64)
        found = np.where(15 * c >= span, c, found)
    return np.maximum(found, 2.0 ** -100)


def quantise(x):
    """Rows [..., D] of finite bf16 or fp32 numbers -> codes [..., D] (0 .. 15), scales and offsets [..., D / 64].

    In float64, whose differences and borders are exact while the numbers of a group lie within 2^28 of each other
    (quantise_one has no such limit).
    """
    v = _f64(x)
    v = v.reshape(*v.shape[:-1], -1, GROUP)
    z = bf16_below(v.min(-1))
    s = _scale(v.max(-1) - z)
    d = v - z[..., None]
    c = sum((d >= (n - 0.5) * s[..., None]).astype(np.int64) for n in range(1, 16))
    return c.reshape(*c.shape[:-2], -1), s, z


def quantise_one(values):
    """One group by rational numbers: (codes, scale, offset)."""
    x = [Fraction(float(v)) for v in values]
    z = Fraction(float(bf16_below(np.float32(float(min(x))))))
    span = max(x) - z
    s = Fraction(float(_scale(np.float64(float(span)))))
    # (the float64 quotient may be off next to a bf16 number: settled by rational ones)
    up = lambda f, n: Fraction(float(np.int32((np.float32(float(f)).view(np.int32) >> 16) + n << 16).view(np.float32)))
    while 15 * s < span:
        s = up(s, 1)
    while s > Fraction(1, 2 ** 100) and 15 * up(s, -1) >= span:
        s = up(s, -1)
    return [sum(v - z >= (n - Fraction(1, 2)) * s for n in range(1, 16)) for v in x], float(s), float(z)


def pack(codes):
    """Codes [..., D] -> bytes [..., D / 2]."""
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(data):
    b = _int(data)
    return np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1)


def values(data, scales):
    """What bytes [..., D / 2] and scales [..., D / 64, 2] stand for, exactly as float64 holds it."""
    sz = np.repeat(_f64(scales), GROUP, axis=-2)
    return sz[..., 1] + sz[..., 0] * unpack(data)


def as_rows(cache):
    """[pages, heads, page, x] -> [pages, page, heads, x], as the other cache lies."""
    return np.swapaxes(cache, 1, 2)


def append(new, data, scales, table, seq_lens, new_lens=None):
    """(bytes, scales) after the new tokens [B, T, Hkv, D]; scales as float64."""
    data, scales = _int(data).astype(np.uint8).copy(), _f64(scales).copy()
    codes, s, z = quantise(new)
    B, T = codes.shape[:2]
    page = data.shape[2]
    for b in range(B):
        for t in range(T if new_lens is None else max(0, min(T, int(new_lens[b])))):
            pos = int(seq_lens[b]) + t
            p, r = int(table[b][pos // page]), pos % page
            data[p, :, r] = pack(codes[b, t])
            scales[p, :, r] = np.stack((s[b, t], z[b, t]), -1)
    return data, scales
