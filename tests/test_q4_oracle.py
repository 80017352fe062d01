"""Pins of the oracle of the cache in 4 bits: rational numbers, closed forms, and
what the definition promises of every value."""
import numpy as np
import pytest
import torch

from oracle import q4


def bf16(x):
    return torch.tensor(np.asarray(x), dtype=torch.float32).to(torch.bfloat16).double().numpy()


def groups(n=40, seed=0):
    g = np.random.default_rng(seed)
    rows = [bf16(g.standard_normal(64) * 10.0 ** g.integers(-6, 6)) for _ in range(n)]
    rows += [np.float64(np.float32(g.standard_normal(64) + g.integers(-50, 50))) for _ in range(n)]
    rows += [g.integers(-8, 9, 64) * 0.5 for _ in range(n)]                   # many ties
    rows += [np.zeros(64), np.full(64, -3.5), np.r_[np.zeros(63), 15.0], np.r_[np.ones(63), 1 + 2.0 ** -7]]
    return rows


def test_rational_numbers_agree():
    for x in groups():
        c, s, z = q4.quantise(x)
        rc, rs, rz = q4.quantise_one(x)
        assert c.tolist() == rc and float(s[0]) == rs and float(z[0]) == rz


def test_what_the_definition_promises():
    for x in groups(seed=1):
        c, s, z = q4.quantise(x)
        assert z[0] <= x.min() and bf16(z[0]) == z[0] and bf16(s[0]) == s[0]
        assert x.min() - z[0] <= abs(x.min()) * 2.0 ** -7
        assert 15 * s[0] >= x.max() - z[0] and (s[0] == 2.0 ** -100 or 15 * s[0] * (1 - 2.0 ** -7) <= x.max() - z[0])
        assert np.abs(x - (z[0] + s[0] * c)).max() <= s[0] / 2        # half a step
        assert c.min() >= 0 and c.max() <= 15


def test_closed_forms():
    x = np.arange(64) % 16
    c, s, z = q4.quantise(x)
    assert s[0] == 1 and z[0] == 0 and np.array_equal(c, x)
    c, s, z = q4.quantise(np.r_[np.zeros(31), 0.5, 1.5, np.full(31, 15.0)])   # ties go up
    assert c[31] == 1 and c[32] == 2
    c, s, z = q4.quantise(np.full(64, 7.25))
    assert z[0] == 7.25 and s[0] == 2.0 ** -100 and not c.any()
    assert q4.bf16_below(np.float32(-1 - 2.0 ** -20)) == -1 - 2.0 ** -7 and q4.bf16_below(np.float32(1 + 2.0 ** -20)) == 1


def test_bytes_and_values():
    g = np.random.default_rng(2)
    c = g.integers(0, 16, (3, 2, 128))
    data = q4.pack(c)
    assert data.shape == (3, 2, 64) and data.dtype == np.uint8 and np.array_equal(q4.unpack(data), c)
    assert data[0, 0, 5] == c[0, 0, 10] + 16 * c[0, 0, 11]
    sz = g.standard_normal((3, 2, 2, 2))
    v = q4.values(data, sz)
    assert v[2, 1, 70] == sz[2, 1, 1, 1] + sz[2, 1, 1, 0] * c[2, 1, 70]


@pytest.mark.parametrize("new", [None, [2, 0]])
def test_append(new):
    g = np.random.default_rng(3)
    data, sz = g.integers(0, 256, (6, 2, 16, 32)), g.standard_normal((6, 2, 16, 1, 2))
    table = np.array([[4, 1], [0, 5]])
    x = bf16(g.standard_normal((2, 3, 2, 64)))
    d, s = q4.append(x, data, sz, table, [15, 7], new)
    c, sc, z = q4.quantise(x)
    assert np.array_equal(d[4, 1, 15], q4.pack(c[0, 0, 1])) and np.array_equal(d[1, :, 0], q4.pack(c[0, 1]))
    assert s[1, 0, 0, 0, 0] == sc[0, 1, 0, 0] and s[1, 0, 0, 0, 1] == z[0, 1, 0, 0]
    same = (d == data).all(-1)
    assert same[2].all() and same[3].all() and same[5].all() and (same[0].all() or new is None)
