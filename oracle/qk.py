"""Float64 definitions of the head norm with rotary positions.

TEST INFRASTRUCTURE ONLY, as the rest of this package: plain numpy, sharing no
code with the library.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .scored import _f64, _int


# 2^200 / 2 pi
_PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
_TURN = int(Fraction(1 << 200) / (2 * _PI))


def angles(positions, freqs, axes=None):
    """positions [B, S, axes] -> radians [B, S, pairs] without their whole turns, by integers of any length."""
    p, f = _int(positions), _f64(freqs)
    axes = [0] * len(f) if axes is None else list(axes)
    t = np.empty((*p.shape[:2], len(f)))
    for i, x in enumerate(f):
        m, of = float(x).as_integer_ratio()
        step, whole = m * _TURN, of << 200  # of a position, and of a turn
        for n in np.unique(p[:, :, axes[i]]):
            t[:, :, i][p[:, :, axes[i]] == n] = 2 * np.pi * float(Fraction(int(n) * step % whole, whole))
    return t


def rotate(x, t, interleaved):
    """x [B, S, H, D], its first pairs turned by t [B, S, pairs]."""
    n, y = t.shape[2], x.copy()
    u, v = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    c, s = np.cos(t)[:, :, None], np.sin(t)[:, :, None]
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., u] * s + x[..., v] * c
    return y


def forward(x, t, interleaved, eps=None, weight=None):
    x = _f64(x)
    if eps is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if weight is None else _f64(weight))
    return rotate(x, t, interleaved)


def backward(x, grad, t, interleaved, eps=None, weight=None):
    """(dx, dweight) of L = sum(forward * grad); dweight None without a norm."""
    g = rotate(_f64(grad), -t, interleaved)
    if eps is None:
        return g, None
    x = _f64(x)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    unit, gw = x * r, g * (1.0 if weight is None else _f64(weight))
    return r * (gw - unit * (gw * unit).mean(-1, keepdims=True)), (g * unit).sum((0, 1, 2))
