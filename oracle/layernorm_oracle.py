"""CPU oracle for the layer norm (forward and backward).

TEST INFRASTRUCTURE.  Only the tests and the package smoke check may import
or run this module.  It shares no code with the CUDA path and never takes an
input or an expected value from it.  Plain numpy, float64.

    n = (s - mean(s)) rstd,  rstd = 1 / sqrt(mean((s - mean(s))^2) + eps),   y = n w + b
    ds = rstd (w dy - mean(w dy) - n mean(w dy n)) + carry,   dw = sum over rows of dy n,   db = sum of dy
"""

from __future__ import annotations

import numpy as np


def layernorm_forward(s, weight, bias, eps) -> dict:
    """s [rows, d] (already x + residual), weight [d], bias [d] or None."""
    s, w = np.asarray(s, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    mean = s.mean(-1)
    with np.errstate(invalid="ignore"):
        c = s - mean[:, None]
        rstd = 1.0 / np.sqrt((c * c).mean(-1) + eps)
        n = c * rstd[:, None]
        y = n * w + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
    return {"y": y, "n": n, "mean": mean, "rstd": rstd}


def layernorm_backward(s, weight, eps, grad_y, carry=None) -> dict:
    ref = layernorm_forward(s, weight, None, eps)
    n, rstd = ref["n"], ref["rstd"][:, None]
    w, dy = np.asarray(weight, dtype=np.float64), np.asarray(grad_y, dtype=np.float64)
    dn = w * dy
    ds = rstd * (dn - dn.mean(-1, keepdims=True) - n * (dn * n).mean(-1, keepdims=True))
    if carry is not None:
        ds = ds + np.asarray(carry, dtype=np.float64)
    return {"grad_x": ds, "grad_weight": (dy * n).sum(0), "grad_bias": dy.sum(0)}
