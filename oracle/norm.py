"""Root-mean-square norm with the residual's addition, its FP8 output and its gradient.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

float64 throughout, except the two roundings that the definition contains:
the stream ``h = round(x + residual)`` is kept in the input's type and the
norm reads that rounded value; codes are rounded to the format's values.
The gradient takes the codes' cast as the identity.
"""

import numpy as np

from . import fp8_formats as F

FMAX = {F.E4M3: 448.0, F.E5M2: 57344.0}


def rmsnorm(h, gamma, eps):
    """(y, rstd) of float64 rows h: y = h * rstd * gamma, rstd = (mean h^2 + eps)^-1/2."""
    h = np.asarray(h, dtype=np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * np.asarray(gamma, dtype=np.float64), rstd


def rmsnorm_backward(dy, h, rstd, gamma, dres=None):
    """(dx, dgamma), from the stream h and the rstd that the forward stored."""
    dy, h, rstd, gamma = (np.asarray(v, dtype=np.float64) for v in (dy, h, rstd, gamma))
    n = h * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - n * np.mean(g * n, axis=1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, dtype=np.float64)
    return dx, np.sum(dy * n, axis=0)


def row_scales(y, fmt):
    """Current scale of every row: FP8_MAX / max |y|, 1 where that is not a positive finite number."""
    a = np.max(np.abs(y), axis=1) if y.shape[1] else np.zeros(y.shape[0])
    with np.errstate(divide="ignore", invalid="ignore"):
        s = FMAX[fmt] / a
    return np.where((a > 0) & np.isfinite(a) & np.isfinite(s), s, 1.0)
