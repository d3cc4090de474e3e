"""CPU oracle for the selective scan and its short convolution (forward and backward).

TEST INFRASTRUCTURE.  Only the tests and the package smoke check may import
or run this module.  It shares no code with the CUDA path and never takes an
input or an expected value from it.  Plain numpy, float64, one token at a time.

The convolution, per channel with weights w [W], over the rows of its sequence:

    pre_t = b + sum_j w_j x_{t-W+1+j},   y = pre sigmoid(pre) or pre

The scan, per channel with a state h [N] and B, C of the channel's group:

    dt = log(1 + exp(delta + bias)),   h_t = exp(dt A) h_{t-1} + dt x B
    y  = (C . h_t + D x) z sigmoid(z)

Given the gradients dy of y and dh of h_t (final state's, then carried back), with
g = dy z sigmoid(z):

    dh += g C                 dC = g h_t              dD = g x
    ddt = dh . (A exp(dt A) h_{t-1} + x B)            dA = dt dh exp(dt A) h_{t-1}
    dx = dt dh . B + D g      dB = dt x dh            ddelta = ddt sigmoid(delta + bias)
    dh_{t-1} = exp(dt A) dh

Rows of all sequences lie one after another; offsets has the first row of each
and the number of rows.
"""

from __future__ import annotations

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def conv_forward(x, weight, bias, offsets, initial_state=None, silu=True) -> dict:
    """x [rows, channels], weight [channels, W], states [sequences, W - 1, channels]."""
    x, weight, bias, init = map(_f64, (x, weight, bias, initial_state))
    d, W = weight.shape
    n = len(offsets) - 1
    pre, final = np.zeros_like(x), np.zeros((n, W - 1, d))
    for i in range(n):
        a, b = offsets[i], offsets[i + 1]
        seen = np.concatenate([np.zeros((W - 1, d)) if init is None else init[i], x[a:b]])
        for t in range(b - a):
            pre[a + t] = (weight.T * seen[t:t + W]).sum(0) + (0 if bias is None else bias)
        final[i] = seen[b - a:]
    return {"pre": pre, "y": pre * sigmoid(pre) if silu else pre, "final_state": final}


def conv_backward(x, weight, bias, offsets, grad_y, initial_state=None, grad_final_state=None, silu=True) -> dict:
    """Gradients of <y, grad_y> + <final_state, grad_final_state>."""
    pre = conv_forward(x, weight, bias, offsets, initial_state, silu)["pre"]
    x, weight, init, gy, gfinal = map(_f64, (x, weight, initial_state, grad_y, grad_final_state))
    d, W = weight.shape
    s = sigmoid(pre)
    p = gy * s * (1 + pre * (1 - s)) if silu else gy
    gx, gw = np.zeros_like(x), np.zeros_like(weight)
    ginit = np.zeros((len(offsets) - 1, W - 1, d))
    for i in range(len(offsets) - 1):
        a, b = offsets[i], offsets[i + 1]
        seen = np.concatenate([np.zeros((W - 1, d)) if init is None else init[i], x[a:b]])
        into = np.zeros_like(seen)
        for t in range(b - a):
            into[t:t + W] += weight.T * p[a + t]
            gw += (seen[t:t + W] * p[a + t]).T
        if gfinal is not None:
            into[b - a:] += gfinal[i]
        ginit[i], gx[a:b] = into[:W - 1], into[W - 1:]
    return {"grad_x": gx, "grad_weight": gw, "grad_bias": p.sum(0), "grad_initial_state": ginit}


def ssm_forward(x, delta, A, B, C, offsets, D=None, z=None, bias=None, initial_state=None, keep=False) -> dict:
    """x, delta, z [rows, channels], A [channels, N], B, C [rows, groups, N]; states [sequences, channels, N]."""
    x, delta, A, B, C, D, z, bias = map(_f64, (x, delta, A, B, C, D, z, bias))
    rows, d = x.shape
    N = A.shape[1]
    group = np.arange(d) // (d // B.shape[1])
    dt = np.logaddexp(0.0, delta + (0 if bias is None else bias))
    n = len(offsets) - 1
    inner, final = np.zeros_like(x), np.zeros((n, d, N))
    before = np.zeros((rows, d, N)) if keep else None
    for i in range(n):
        h = np.zeros((d, N)) if initial_state is None else np.array(initial_state[i], dtype=np.float64)
        for t in range(offsets[i], offsets[i + 1]):
            if keep:
                before[t] = h
            h = np.exp(dt[t][:, None] * A) * h + (dt[t] * x[t])[:, None] * B[t][group]
            inner[t] = (h * C[t][group]).sum(1)
        final[i] = h
    if D is not None:
        inner = inner + D * x
    return {"y": inner if z is None else inner * z * sigmoid(z), "inner": inner, "final_state": final, "before": before}


def ssm_backward(x, delta, A, B, C, offsets, grad_y, D=None, z=None, bias=None, initial_state=None,
                 grad_final_state=None) -> dict:
    """Gradients of <y, grad_y> + <final_state, grad_final_state>."""
    ref = ssm_forward(x, delta, A, B, C, offsets, D, z, bias, initial_state, keep=True)
    before, inner = ref["before"], ref["inner"]
    x, delta, A, B, C, D, z, bias, gy = map(_f64, (x, delta, A, B, C, D, z, bias, grad_y))
    rows, d = x.shape
    N, groups = A.shape[1], B.shape[1]
    group = np.arange(d) // (d // groups)
    pre = delta + (0 if bias is None else bias)
    dt, out = np.logaddexp(0.0, pre), {}
    if z is None:
        g = gy
    else:
        s = sigmoid(z)
        g = gy * z * s
        out["grad_z"] = gy * inner * s * (1 + z * (1 - s))
    gx = g * D if D is not None else np.zeros_like(x)
    gdt, gA = np.zeros_like(x), np.zeros_like(A)
    gB, gC = np.zeros_like(B), np.zeros_like(C)
    ginit = np.zeros((len(offsets) - 1, d, N))
    for i in range(len(offsets) - 1):
        dh = np.zeros((d, N)) if grad_final_state is None else np.array(grad_final_state[i], dtype=np.float64)
        for t in range(offsets[i + 1] - 1, offsets[i] - 1, -1):
            a, b = np.exp(dt[t][:, None] * A), B[t][group]
            h = a * before[t] + (dt[t] * x[t])[:, None] * b
            np.add.at(gC[t], group, g[t][:, None] * h)
            dh = dh + g[t][:, None] * C[t][group]
            np.add.at(gB[t], group, (dt[t] * x[t])[:, None] * dh)
            gdt[t] = (dh * (A * a * before[t] + x[t][:, None] * b)).sum(1)
            gx[t] += dt[t] * (dh * b).sum(1)
            gA += dt[t][:, None] * dh * a * before[t]
            dh = a * dh
        ginit[i] = dh
    gdelta = gdt * sigmoid(pre)
    out.update(grad_x=gx, grad_delta=gdelta, grad_A=gA, grad_B=gB, grad_C=gC, grad_D=(g * x).sum(0),
               grad_delta_bias=gdelta.sum(0), grad_initial_state=ginit)
    return out
