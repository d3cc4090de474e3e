"""The 64-bit oracles of the gated delta rule and the residual norm, held to
their definitions: closed forms, and central differences of the forward."""

import numpy as np
import pytest

from oracle.gdr_oracle import gdr_backward, gdr_forward
from oracle.rmsnorm_oracle import rmsnorm_backward, rmsnorm_forward, rmsnorm_group_scale


def _inputs(rng, rows, hk, hv, dk, dv):
    q, k = rng.standard_normal((2, rows, hk, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return [q, k, rng.standard_normal((rows, hv, dv)), -rng.uniform(0, 1, (rows, hv)), rng.uniform(0, 1, (rows, hv))]


def test_no_decay_and_full_strength_replaces_what_a_key_holds():
    """beta = 1, g = 0 and unit keys: reading a key just written gives its value,
    an orthogonal key's stays."""
    k = np.zeros((3, 1, 4))
    k[0, 0, 0] = k[1, 0, 1] = k[2, 0, 0] = 1
    v = np.arange(6.0).reshape(3, 1, 2) + 1
    r = gdr_forward(k, k, v, np.zeros((3, 1)), np.ones((3, 1)), 1.0, [0, 3])
    np.testing.assert_array_equal(r["o"], v)
    np.testing.assert_array_equal(r["final_state"][0, 0, :2], [v[2, 0], v[1, 0]])


def test_a_reset_forgets_everything_before_it():
    rng = np.random.default_rng(1)
    x = _inputs(rng, 9, 1, 2, 4, 3)
    x[3][5] = -np.inf
    whole = gdr_forward(*x, 0.5, [0, 9], rng.standard_normal((1, 2, 4, 3)))
    after = gdr_forward(*(a[5:] for a in x), 0.5, [0, 4])
    np.testing.assert_array_equal(whole["o"][5:], after["o"])
    np.testing.assert_array_equal(whole["final_state"], after["final_state"])


def test_sequences_are_independent_and_empty_ones_keep_their_state():
    rng = np.random.default_rng(2)
    x = _inputs(rng, 7, 1, 1, 4, 2)
    s0 = rng.standard_normal((3, 1, 4, 2))
    r = gdr_forward(*x, 1.0, [0, 3, 3, 7], s0)
    np.testing.assert_array_equal(r["final_state"][1], s0[1])
    np.testing.assert_array_equal(r["o"][3:], gdr_forward(*(a[3:] for a in x), 1.0, [0, 4], s0[2:])["o"])


def test_rule_gradients_match_differences():
    rng = np.random.default_rng(3)
    off = [0, 5, 5, 6, 13]
    x = _inputs(rng, 13, 2, 4, 4, 3)
    s0 = rng.standard_normal((4, 4, 4, 3))
    w, wf = rng.standard_normal((13, 4, 3)), rng.standard_normal((4, 4, 4, 3))

    def loss(x, s0):
        r = gdr_forward(*x, 0.7, off, s0)
        return (r["o"] * w).sum() + (r["final_state"] * wf).sum()

    got = gdr_backward(*x, 0.7, off, w, s0, wf)
    names = ("grad_q", "grad_k", "grad_v", "grad_g", "grad_beta", "grad_initial_state")
    eps = 1e-6
    for i, name in enumerate(names):
        a = (x + [s0])[i]
        flat = a.reshape(-1)
        for j in rng.choice(flat.size, min(flat.size, 12), replace=False):
            old = flat[j]
            flat[j] = old + eps
            up = loss(x, s0)
            flat[j] = old - eps
            down = loss(x, s0)
            flat[j] = old
            assert got[name].reshape(-1)[j] == pytest.approx((up - down) / (2 * eps), rel=1e-6, abs=1e-7), (name, j)


def test_norm_gradients_match_differences():
    rng = np.random.default_rng(4)
    s, w, dy, carry = rng.standard_normal((3, 5)), rng.standard_normal(5), rng.standard_normal((3, 5)), rng.standard_normal((3, 5))
    got = rmsnorm_backward(s, w, 1e-3, dy, carry)
    eps = 1e-6
    for a, name in ((s, "grad_x"), (w, "grad_weight")):
        flat = a.reshape(-1)
        for j in range(flat.size):
            old, f = flat[j], []
            for d in (eps, -eps):
                flat[j] = old + d
                f.append((rmsnorm_forward(s, w, 1e-3)["y"] * dy).sum() + (s * carry).sum())
            flat[j] = old
            assert got[name].reshape(-1)[j] == pytest.approx((f[0] - f[1]) / (2 * eps), rel=1e-6, abs=1e-7)


def test_norm_of_equal_values_and_group_scales():
    r = rmsnorm_forward(np.full((2, 8), -3.0), np.full(8, 2.0), 0.0)
    np.testing.assert_allclose(r["y"], -2.0)
    np.testing.assert_allclose(r["rstd"], 1 / 3)
    y = np.array([[0.0, 0.0, -448.0, 1.0]])
    np.testing.assert_array_equal(rmsnorm_group_scale(y, 2), [[1.0, 1.0]])
