"""CPU oracle for the gated delta rule (forward and backward through time).

TEST INFRASTRUCTURE.  Only the tests and the package smoke check may import
or run this module.  It shares no code with the CUDA path and never takes an
input or an expected value from it.  Plain numpy, float64, one token at a time.

Per sequence and value head, with a state S [d_k, d_v], and per token

    S'  = exp(g) S_{t-1}
    u   = beta (v - S'^T k)
    S_t = S' + k u^T
    o   = scale S_t^T q

q and k of value head h are those of head h // (v_heads / k_heads).  Given the
gradients dO of o and dS of S_t (final state's, then carried back):

    dS  += scale q dO^T       dq = scale S_t dO
    du   = dS^T k             dk = dS u
    dv   = beta du            dbeta = du . (v - S'^T k)
    dS'  = dS - beta k du^T   dk -= beta S' du
    dg   = exp(g) <dS', S_{t-1}>
    dS_{t-1} = exp(g) dS'

Rows of all sequences lie one after another; offsets has the first row of each
and the number of rows.
"""

from __future__ import annotations

import numpy as np


def _f64(*arrays):
    return [np.asarray(a, dtype=np.float64) for a in arrays]


def gdr_forward(q, k, v, g, beta, scale, offsets, initial_state=None, keep=False) -> dict:
    """q, k [rows, hk, dk], v [rows, hv, dv], g, beta [rows, hv];
    o [rows, hv, dv], final_state [sequences, hv, dk, dv]."""
    q, k, v, g, beta = _f64(q, k, v, g, beta)
    rows, hv, dv = v.shape
    hk, dk = q.shape[1:]
    head = np.arange(hv) // (hv // hk)
    n = len(offsets) - 1
    o = np.zeros((rows, hv, dv))
    final = np.zeros((n, hv, dk, dv))
    kept = np.zeros((rows + 1, hv, dk, dv)) if keep else None     # S_{t-1} of each row
    for i in range(n):
        S = np.zeros((hv, dk, dv)) if initial_state is None else np.array(initial_state[i], dtype=np.float64)
        for t in range(offsets[i], offsets[i + 1]):
            if keep:
                kept[t] = S
            S = np.exp(g[t])[:, None, None] * S
            kt, qt = k[t, head], q[t, head]
            u = beta[t][:, None] * (v[t] - np.einsum("hk,hkv->hv", kt, S))
            S = S + kt[:, :, None] * u[:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", qt, S)
        final[i] = S
    out = {"o": o, "final_state": final}
    if keep:
        out["before"] = kept
    return out


def gdr_backward(q, k, v, g, beta, scale, offsets, grad_o, initial_state=None, grad_final_state=None) -> dict:
    """Gradients of <o, grad_o> + <final_state, grad_final_state>."""
    before = gdr_forward(q, k, v, g, beta, scale, offsets, initial_state, keep=True)["before"]
    q, k, v, g, beta, grad_o = _f64(q, k, v, g, beta, grad_o)
    rows, hv, dv = v.shape
    hk, dk = q.shape[1:]
    head = np.arange(hv) // (hv // hk)
    n = len(offsets) - 1
    gq, gk = np.zeros((rows, hv, dk)), np.zeros((rows, hv, dk))
    gv, gg, gb = np.zeros_like(v), np.zeros_like(g), np.zeros_like(beta)
    ginit = np.zeros((n, hv, dk, dv))
    for i in range(n):
        dS = np.zeros((hv, dk, dv)) if grad_final_state is None else np.array(grad_final_state[i], dtype=np.float64)
        for t in range(offsets[i + 1] - 1, offsets[i] - 1, -1):
            kt, qt, bt = k[t, head], q[t, head], beta[t][:, None]
            a = np.exp(g[t])[:, None, None]
            S1 = a * before[t]
            e = v[t] - np.einsum("hk,hkv->hv", kt, S1)
            S = S1 + kt[:, :, None] * (bt * e)[:, None, :]
            gq[t] = scale * np.einsum("hkv,hv->hk", S, grad_o[t])
            dS = dS + scale * qt[:, :, None] * grad_o[t][:, None, :]
            du = np.einsum("hkv,hk->hv", dS, kt)
            gk[t] = np.einsum("hkv,hv->hk", dS, bt * e) - np.einsum("hkv,hv->hk", S1, bt * du)
            gv[t] = bt * du
            gb[t] = (du * e).sum(-1)
            dS1 = dS - kt[:, :, None] * (bt * du)[:, None, :]
            gg[t] = a[:, 0, 0] * (dS1 * before[t]).sum((1, 2))
            dS = a * dS1
        ginit[i] = dS
    per = hv // hk
    return {"grad_q": gq.reshape(rows, hk, per, dk).sum(2), "grad_k": gk.reshape(rows, hk, per, dk).sum(2),
            "grad_v": gv, "grad_g": gg, "grad_beta": gb, "grad_initial_state": ginit}
