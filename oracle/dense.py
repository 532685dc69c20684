"""The dense operators beside the layer, on the CPU in float64.

TEST INFRASTRUCTURE ONLY, like the rest of this package: written from the
definitions (include/moe.h states them), sharing no code with the GPU path.
tests/test_oracle_dense.py pins the gradients to differences of the forward
function and the 8-bit codes to the exact quotients.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, e) / (1.0 + e)


def silu_mul(g, u):
    return g * sigmoid(g) * u


def silu_mul_backward(g, u, dh):
    """Gradients of gate and up from that of silu(g) * u."""
    s = sigmoid(g)
    return dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s


def ffn(x, w1, w2, base=0.0):
    """out, and g, u, h of every token."""
    half = w1.shape[0] // 2
    g, u = x @ w1[:half].T, x @ w1[half:].T
    h = silu_mul(g, u)
    return base + h @ w2.T, g, u, h


def ffn_backward(dout, x, w1, w2, dx_base=0.0):
    """dx, dw1, dw2."""
    _, g, u, h = ffn(x, w1, w2)
    dg, du = silu_mul_backward(g, u, dout @ w2)
    d = np.concatenate([dg, du], axis=1)
    return dx_base + d @ w1, d.T @ x, dout.T @ h


def int8_scale(amax):
    """Scale of a row with this largest magnitude (float32)."""
    amax = np.float32(amax)
    if not np.isfinite(amax):
        return np.float32(np.nan)
    if amax == 0:
        return np.float32(1.0)
    return np.maximum(amax * (np.float32(1.0) / np.float32(127.0)), np.float32(2.0 ** -126))


def int8_code(v, scale):
    """The integer nearest to v / scale, ties to even, in exact arithmetic."""
    return round(Fraction(float(v)) / Fraction(float(scale)))


def int8_quantize(x):
    """codes int8, scales float32 of the rows of x.  A double's quotient of two
    float32 numbers lies on the same side of every half as the exact one (it is
    off by 2^-53 of itself, and differs from a half by 2^-34 of it at least or
    not at all)."""
    x = np.asarray(x, np.float32)
    codes = np.zeros(x.shape, np.int8)
    scales = np.empty(x.shape[0], np.float32)
    for i, row in enumerate(x):
        top = np.abs(row).max() if np.isfinite(row).all() else np.inf
        scales[i] = int8_scale(top)
        if np.isfinite(top):
            codes[i] = np.rint(row.astype(np.float64) / np.float64(scales[i])).astype(np.int8)
    return codes, scales


def int8_matmul(codes, scales, w, w_scales, base=0.0):
    sums = codes.astype(np.float64) @ w.astype(np.float64).T  # exact: below 2^53
    return base + sums * scales.astype(np.float64)[:, None] * w_scales.astype(np.float64)
