"""Pins of the float64 oracle of the head norm with rotary positions: closed
forms, plain angles where 64 bits hold them, torch's autograd and differences."""
import numpy as np
import pytest
import torch

from oracle import qk


def data(B=2, S=5, H=3, D=64, seed=0):
    g = np.random.default_rng(seed)
    return g.standard_normal((B, S, H, D)), g.standard_normal((B, S, H, D)), g.standard_normal(D)


def test_angles():
    g = np.random.default_rng(1)
    pos = g.integers(-5000, 5000, (2, 7, 3))
    f = 10000.0 ** -(np.arange(8) / 8)
    axes = [0, 0, 1, 1, 1, 2, 2, 0]
    t = qk.angles(pos, f, axes)
    plain = pos[:, :, axes] * f
    assert np.abs(np.exp(1j * t) - np.exp(1j * plain)).max() < 1e-11
    # far out: additive in the position, where the sum is exact
    a, b = qk.angles(np.full((1, 1, 1), 2 ** 30), f), qk.angles(np.full((1, 1, 1), -2 ** 30 + 3), f)
    assert np.abs(np.exp(1j * (a + b)) - np.exp(3j * f)).max() < 1e-14
    assert np.all(qk.angles(np.zeros((1, 1, 1)), f) == 0)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(inter):
    x, y, _ = data()
    f = 0.5 ** np.arange(16)
    p = np.arange(10).reshape(2, 5, 1)
    dot = lambda shift: (qk.rotate(x, qk.angles(p + shift, f), inter) * qk.rotate(y, qk.angles(3 * p + shift, f), inter)).sum(-1)
    assert np.abs(dot(0) - dot(12345)).max() < 1e-10
    r = qk.rotate(x, qk.angles(p, f), inter)
    assert np.allclose((r * r).sum(-1), (x * x).sum(-1), rtol=1e-13)
    assert np.array_equal(r[..., 32:], x[..., 32:])
    back = qk.rotate(r, -qk.angles(p, f), inter)
    assert np.abs(back - x).max() < 1e-14
    # position 0 turns nothing; a quarter turn of one pair
    one = np.zeros((1, 1, 1, 64))
    one[..., 0] = 1.0
    q = qk.rotate(one, np.full((1, 1, 4), np.pi / 2), inter)
    assert abs(q[0, 0, 0, 1 if inter else 4] - 1) < 1e-15 and abs(q[0, 0, 0, 0]) < 1e-15


def test_norm_closed_forms():
    x = np.full((1, 1, 1, 64), 3.0)
    t = np.zeros((1, 1, 4))
    assert np.allclose(qk.forward(x, t, True, eps=0.0), 1.0)
    assert np.allclose(qk.forward(x, t, True, eps=7.0), 0.75)          # 3 / sqrt(9 + 7)
    w = np.arange(64.0)
    assert np.allclose(qk.forward(x, t, False, eps=0.0, weight=w)[0, 0, 0], w)
    # without eps the gradient is at right angles to x
    x, g, w = data()
    dx, _ = qk.backward(x, g, np.zeros((2, 5, 4)), False, eps=0.0, weight=w)
    assert np.abs((dx * x).sum(-1)).max() < 1e-12


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("eps,weighted", [(None, False), (1e-6, True), (0.3, False)])
def test_backward_by_autograd_and_differences(inter, eps, weighted):
    x, g, w = data(seed=3)
    w = w if weighted else None
    t = qk.angles(np.arange(10).reshape(2, 5, 1) * 7, 0.7 ** np.arange(20))
    dx, dw = qk.backward(x, g, t, inter, eps, w)
    f = lambda x, w: (qk.forward(x, t, inter, eps, w) * g).sum()
    r = np.random.default_rng(5)
    for _ in range(5):
        d, h = r.standard_normal(x.shape), 1e-5
        assert abs((f(x + h * d, w) - f(x - h * d, w)) / (2 * h) - (dx * d).sum()) < 1e-7
        if eps is not None:
            d = r.standard_normal(64)
            w0 = np.ones(64) if w is None else w
            assert abs((f(x, w0 + h * d) - f(x, w0 - h * d)) / (2 * h) - (dw * d).sum()) < 1e-7
    # torch's own gradient of the same formulas, written out for it
    xt = torch.tensor(x, requires_grad=True)
    y = xt
    if eps is not None:
        y = xt / (xt.square().mean(-1, keepdim=True) + eps).sqrt() * (1.0 if w is None else torch.tensor(w))
    n = t.shape[2]
    z = torch.exp(1j * torch.tensor(t))[:, :, None]
    pair = torch.complex(y[..., 0:2 * n:2], y[..., 1:2 * n:2]) if inter else torch.complex(y[..., :n], y[..., n:2 * n])
    pair = pair * z
    gr = torch.tensor(g)
    gu, gv = (gr[..., 0:2 * n:2], gr[..., 1:2 * n:2]) if inter else (gr[..., :n], gr[..., n:2 * n])
    ((pair.real * gu).sum() + (pair.imag * gv).sum() + (y[..., 2 * n:] * gr[..., 2 * n:]).sum()).backward()
    assert np.abs(xt.grad.numpy() - dx).max() < 1e-12


def test_planted_mistakes_are_found():
    x, g, w = data(seed=4)
    t = qk.angles(np.arange(10).reshape(2, 5, 1), 0.7 ** np.arange(20))
    d = np.random.default_rng(6).standard_normal(x.shape)
    f = lambda x: (qk.forward(x, t, True, 1e-6, w) * g).sum()
    slope = (f(x + 1e-5 * d) - f(x - 1e-5 * d)) / 2e-5
    right, _ = qk.backward(x, g, t, True, 1e-6, w)
    assert abs((right * d).sum() - slope) < 1e-7
    for wrong in (qk.backward(x, g, -t, True, 1e-6, w), qk.backward(x, g, t, False, 1e-6, w),
                  qk.backward(x, g, t, True, 0.1, w), qk.backward(x, g, t, True, 1e-6, None),
                  qk.backward(x, g, t, True, None, w)):
        assert abs((wrong[0] * d).sum() - slope) > 1e-3
