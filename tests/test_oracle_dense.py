"""The dense operators' definitions (oracle/dense.py): gradients against
differences, codes against exact quotients (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import dense as OD


def test_silu_mul_values():
    g, u = np.array([0.0, 1.0, -1.0, 40.0, -800.0]), np.array([3.0, 2.0, 2.0, 0.5, 7.0])
    s1 = 1.0 / (1.0 + np.exp(-1.0))
    np.testing.assert_allclose(OD.silu_mul(g, u), [0.0, 2.0 * s1, -2.0 * (1.0 - s1), 20.0, 0.0], rtol=1e-15, atol=1e-300)


def test_block_gradients_against_differences():
    rng = np.random.default_rng(5)
    T, H, I = 4, 6, 5
    x, dout, base = rng.standard_normal((3, T, H))
    w1, w2 = rng.standard_normal((2 * I, H)), rng.standard_normal((H, I))
    dx, dw1, dw2 = OD.ffn_backward(dout, x, w1, w2, base)

    def goal(**kw):
        a = dict(x=x, w1=w1, w2=w2)
        a.update(kw)
        return float((OD.ffn(a["x"], a["w1"], a["w2"])[0] * dout).sum())

    step = 1e-5
    for name, at, grad in (("x", x, dx - base), ("w1", w1, dw1), ("w2", w2, dw2)):
        for i in np.ndindex(at.shape):
            up, down = at.copy(), at.copy()
            up[i] += step
            down[i] -= step
            diff = (goal(**{name: up}) - goal(**{name: down})) / (2 * step)
            # the difference's own error: step^2 of third derivatives, 2^-52 / step of the goal
            assert abs(diff - grad[i]) <= 1e-7 * (1 + abs(grad[i])), (name, i)


@pytest.mark.parametrize("amax", [1.0, 127.0, 448.0, 1e-30, 3e38, 1.1754944e-38, 1e-45])
def test_int8_codes_are_the_nearest(amax):
    rng = np.random.default_rng(11)
    row = (rng.uniform(-1, 1, 64) * amax).astype(np.float32)
    row[0] = amax
    scale = OD.int8_scale(amax)
    # values at and one float either side of the halves
    halves = ((np.arange(-6, 6) + 0.5) * np.float64(scale)).astype(np.float32)
    row = np.concatenate([row, halves, np.nextafter(halves, np.float32(np.inf)), np.nextafter(halves, np.float32(-np.inf))])
    row = row[np.abs(row) <= np.float32(amax)]
    codes, scales = OD.int8_quantize(row[None])
    assert scales[0] == scale
    for v, c in zip(row, codes[0]):
        exact = Fraction(float(v)) / Fraction(float(scale))
        assert abs(exact - int(c)) <= Fraction(1, 2) and OD.int8_code(v, scale) == c


def test_int8_rows_of_special_values():
    x = np.array([[0, 0], [np.inf, 1], [np.nan, 2], [-127, 63.5]], np.float32)
    codes, scales = OD.int8_quantize(x)
    assert codes.tolist() == [[0, 0], [0, 0], [0, 0], [-127, 64]]
    assert scales[0] == 1 and np.isnan(scales[1]) and np.isnan(scales[2]) and scales[3] == 1
