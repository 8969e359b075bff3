"""Activations of the product's epilogue, their slopes, and the epilogue's gradient.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).  float64, from the
definitions: relu, the tanh form of gelu, silu.
"""

import numpy as np

NONE, RELU, GELU, SILU = 0, 1, 2, 3
_C = np.sqrt(2.0 / np.pi)
_A = 0.044715


def act(z, kind):
    """act(z) of a float64 array."""
    z = np.asarray(z, dtype=np.float64)
    if kind == RELU:
        return np.where(z < 0, 0.0, z)
    if kind == GELU:
        # 1 + tanh(v) = 2 / (1 + e^-2v), without the cancellation at v << 0
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-2.0 * _C * (z + _A * z ** 3)))
    if kind == SILU:
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-z))
    return z


def slope(z, kind):
    """d act / dz."""
    z = np.asarray(z, dtype=np.float64)
    if kind == RELU:
        return np.where(z <= 0, 0.0, 1.0)
    with np.errstate(over="ignore"):
        if kind == GELU:
            # (1 + tanh(w/2)) / 2 = p and (1 - tanh^2) / 4 = p q, again without cancellation
            w = 2.0 * _C * (z + _A * z ** 3)
            p, q = 1.0 / (1.0 + np.exp(-w)), 1.0 / (1.0 + np.exp(w))
            return p + z * p * q * 2.0 * _C * (1 + 3 * _A * z * z)
        if kind == SILU:
            p, q = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
            return p + z * p * q
    return np.ones_like(z)


def value_error(z, kind):
    """Allowed |float32 act(z) - act(z)| for a float32 z, U = 2^-24.

    e^-|w| by the fast exponential: 2 + 1.2 |w| ulp, one ulp at most 2 U; w
    itself (gelu) rounds four times, 4 U |w| in the exponent; 1 + t and the
    final products once each, the fast division 2 ulp.  Where e^-w leaves
    float32's range, the value, below 2^-119, may be 0.
    """
    z = np.asarray(z, dtype=np.float64)
    return np.abs(act(z, kind)) * _relative(z, kind) + 2.0 ** -119


def slope_error(z, kind):
    """Allowed |float32 slope - slope|: p and q have the error above, their product twice
    it, and the terms are added, not their rounded sum's size."""
    z = np.asarray(z, dtype=np.float64)
    if kind in (NONE, RELU):
        return np.zeros_like(z)
    w = 2 * _C * (z + _A * z ** 3) if kind == GELU else z
    dw = 2 * _C * (1 + 3 * _A * z * z) if kind == GELU else np.ones_like(z)
    with np.errstate(over="ignore"):
        p, q = 1.0 / (1.0 + np.exp(-w)), 1.0 / (1.0 + np.exp(w))
    return _relative(z, kind) * (p + 2 * np.abs(z * p * q * dw)) + 2.0 ** -126


def _relative(z, kind):
    U = 2.0 ** -24
    if kind in (NONE, RELU):
        return np.zeros_like(z)
    w = np.abs(2 * _C * (z + _A * z ** 3) if kind == GELU else z)
    return U * (2 * (2 + 1.2 * w) + 4 * w + 2 * 2 + 6)


def backward(dy, z, kind, u=None):
    """(dz, du) of y = act(z) [* u]; du is None without u."""
    dy = np.asarray(dy, dtype=np.float64)
    d = dy if u is None else dy * np.asarray(u, dtype=np.float64)
    s = slope(z, kind)
    if kind == RELU:
        d = np.where(s == 0, 0.0, d)  # nothing passes where the slope is 0
    return d * s, None if u is None else dy * act(z, kind)
