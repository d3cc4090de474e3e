"""CPU oracle for the root-mean-square norm (forward and backward).

TEST INFRASTRUCTURE.  Only the tests and the package smoke check may import
or run this module.  It shares no code with the CUDA path and never takes an
input or an expected value from it.  Plain numpy, float64.

    rstd = 1 / sqrt(mean(s^2) + eps),   y = s rstd w
    ds = rstd (w dy - s rstd^2 mean(s w dy)) + carry,   dw = sum over rows of dy s rstd
"""

from __future__ import annotations

import numpy as np


def rmsnorm_forward(s, weight, eps) -> dict:
    """s [rows, d] (already x + residual), weight [d]."""
    s, w = np.asarray(s, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    rstd = 1.0 / np.sqrt((s * s).mean(-1) + eps)
    with np.errstate(invalid="ignore"):
        y = s * rstd[:, None] * w
    return {"y": y, "rstd": rstd}


def rmsnorm_group_scale(y, group) -> np.ndarray:
    """The e4m3 scale of each group of columns: its largest |y| / 448, 1 for zeros."""
    rows, d = y.shape
    top = np.abs(y).reshape(rows, d // group, group).max(-1)
    return np.where(top > 0, top / 448.0, 1.0)


def rmsnorm_backward(s, weight, eps, grad_y, carry=None) -> dict:
    s, w, dy = (np.asarray(a, dtype=np.float64) for a in (s, weight, grad_y))
    rstd = (1.0 / np.sqrt((s * s).mean(-1) + eps))[:, None]
    ds = rstd * (w * dy - s * rstd ** 2 * (s * w * dy).mean(-1, keepdims=True))
    if carry is not None:
        ds = ds + np.asarray(carry, dtype=np.float64)
    return {"grad_x": ds, "grad_weight": (dy * s * rstd).sum(0)}
