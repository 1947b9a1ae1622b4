"""Plain forms of the 8-bit integer layers, written from the definitions in numpy: 64 bits, and
float32 where the definition rounds to it."""

from __future__ import annotations

import numpy as np

from tests import _q8

LEAST = np.float32(2.0 ** -100)
STEP = 2.0 ** -24  # half a step of float32


def codes(z: np.ndarray):
    """(codes, a) of the rows of z, float32: whole rows of zeros where z is not finite."""
    assert z.dtype == np.float32
    finite = np.isfinite(z).all(axis=1)
    z = np.where(finite[:, None], z, np.float32(0))
    a = np.maximum(np.abs(z).max(axis=1), LEAST)
    inv = np.float32(127) / a
    return np.rint(z * inv[:, None]).astype(np.int8), a, finite


def store(x: np.ndarray):
    """(codes, scales) of x, float32 (bf16 values widened)."""
    q, a, finite = codes(x)
    return q, np.where(finite, a / np.float32(127), np.float32(np.nan)).astype(np.float32)


def norm(x: np.ndarray, r, w: np.ndarray, eps: float):
    """(codes, scales in 64 bits, s in float32): codes from the operations in float32, the scales
    from the formula."""
    with np.errstate(over="ignore", invalid="ignore"):
        s = x if r is None else x + r
        q, _, finite = codes(s * w)
        s64 = x.astype(np.float64) + (0.0 if r is None else r.astype(np.float64))
        y = s64 * w / np.sqrt((s64 * s64).mean(axis=1, keepdims=True) + eps)
        return q, np.where(finite, np.abs(y).max(axis=1) / 127, np.nan), s


def norm_bound(cols: int) -> float:
    """Relative error of a scale of norm: the squares are added in a thread's order (at most 32 of
    them, or an eighth of a 4096th of the row beyond 16384 columns), over 32 lanes in 5 steps and
    over 16 warps, s itself and eps with one rounding each, half of all that through the root; then
    the rounded mean, root, quotient, z (s, and s w), a / 127 and the product."""
    each = 32 if cols <= 16384 else 8 * -(-cols // 4096)
    return ((each + 5 + 16 + 2 + 1 + 1) / 2 + 7) * STEP


def value_bound(y: np.ndarray) -> np.ndarray:
    """How far a product's float32 value may be from y: the sum, and two products, rounded (one
    more covers their second order); below the normal numbers steps of 2^-149."""
    return 3.01 * STEP * np.abs(y) + 3 * 2.0 ** -149


def gated_bound(g: np.ndarray, u: np.ndarray, act: str) -> np.ndarray:
    """The same for act(g) u: act's own error, its slope times g's, u's, and a rounding."""
    a, d = _q8.act(g, act)
    # the slope changes by less than 1.2 a unit of g, which is below 2^-22 |g| away
    da = _q8.act_bound(g, act)[0] + (np.abs(d) + 2.0 ** -20) * value_bound(g)
    return da * np.abs(u) * (1 + 4 * STEP) + np.abs(a) * value_bound(u) + \
        2 * STEP * np.abs(a * u) + 2.0 ** -126


def rounded(bound: np.ndarray, y: np.ndarray, dtype: str) -> np.ndarray:
    """The bound after rounding to the output's type: half a step of bf16 is 2^-8."""
    return bound if dtype == "float32" else bound + 2.0 ** -8 * (np.abs(y) + bound) + 2.0 ** -134
