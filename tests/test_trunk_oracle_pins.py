"""The oracles of the scan, its convolution and the layer norm: closed forms, and every gradient against central
differences in 64 bits (step 1e-6: truncation 1e-12 and rounding 1e-10 of the value, 1e-7 relative is ample)."""

import numpy as np
import pytest

from oracle.layernorm_oracle import layernorm_backward, layernorm_forward
from oracle.ssm_oracle import conv_backward, conv_forward, ssm_backward, ssm_forward

OFF = [0, 3, 3, 4, 9]


def check(loss, inputs, grads):
    """loss(**inputs) against central differences in every element of every input that has a gradient."""
    for name, g in grads.items():
        a = inputs[name]
        num = np.zeros(a.shape)
        for at in np.ndindex(a.shape):
            keep = a[at]
            a[at] = keep + 1e-6
            up = loss(**inputs)
            a[at] = keep - 1e-6
            num[at] = (up - loss(**inputs)) / 2e-6
            a[at] = keep
        np.testing.assert_allclose(g, num, rtol=1e-6, atol=1e-8, err_msg=name)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_gradients(W, silu):
    rng = np.random.default_rng(W)
    n, d = len(OFF) - 1, 3
    inp = dict(x=rng.standard_normal((9, d)), weight=rng.standard_normal((d, W)), bias=rng.standard_normal(d),
               initial_state=rng.standard_normal((n, W - 1, d)))
    gy, gf = rng.standard_normal((9, d)), rng.standard_normal((n, W - 1, d))

    def loss(x, weight, bias, initial_state):
        r = conv_forward(x, weight, bias, OFF, initial_state, silu)
        return (r["y"] * gy).sum() + (r["final_state"] * gf).sum()

    g = conv_backward(inp["x"], inp["weight"], inp["bias"], OFF, gy, inp["initial_state"], gf, silu)
    check(loss, inp, {k[5:]: v for k, v in g.items()})


def test_conv_of_an_impulse_is_the_weights_reversed():
    w = np.array([[1.0, 2.0, 3.0, 4.0]])
    x = np.zeros((6, 1))
    x[0] = 1
    r = conv_forward(x, w, None, [0, 6], silu=False)
    assert r["y"][:, 0].tolist() == [4, 3, 2, 1, 0, 0]
    assert conv_forward(x[:1], w, None, [0, 1], np.array([[[7.0], [8.0], [9.0]]]), False)["final_state"][0, :, 0].tolist() == [8, 9, 1]
    assert conv_forward(x[:0], w, None, [0, 0], np.array([[[7.0], [8.0], [9.0]]]), False)["final_state"][0, :, 0].tolist() == [7, 8, 9]


@pytest.mark.parametrize("gate", [True, False])
def test_scan_gradients(gate):
    rng = np.random.default_rng(int(gate))
    n, d, N, groups = len(OFF) - 1, 4, 3, 2
    inp = dict(x=rng.standard_normal((9, d)), delta=rng.standard_normal((9, d)), A=-rng.uniform(0.1, 2, (d, N)),
               B=rng.standard_normal((9, groups, N)), C=rng.standard_normal((9, groups, N)), D=rng.standard_normal(d),
               z=rng.standard_normal((9, d)), bias=rng.standard_normal(d), initial_state=rng.standard_normal((n, d, N)))
    if not gate:
        inp["z"] = None
    gy, gf = rng.standard_normal((9, d)), rng.standard_normal((n, d, N))

    def loss(**kw):
        r = ssm_forward(offsets=OFF, **kw)
        return (r["y"] * gy).sum() + (r["final_state"] * gf).sum()

    g = ssm_backward(offsets=OFF, grad_y=gy, grad_final_state=gf, **inp)
    g["grad_bias"] = g.pop("grad_delta_bias")
    assert ("grad_z" in g) == gate
    check(loss, inp, {k[5:]: v for k, v in g.items()})


def test_scan_with_constant_steps_is_a_sum_of_powers():
    """One state, dt = ln 2 (delta = 0), A = -1: a decay of 1/2 a token."""
    x = np.array([[1.0], [0.0], [0.0]])
    one = np.ones((3, 1, 1))
    r = ssm_forward(x, np.zeros((3, 1)), [[-1.0]], one, one, [0, 3])
    np.testing.assert_allclose(r["y"][:, 0], np.log(2) * np.array([1, 0.5, 0.25]), rtol=1e-15)
    np.testing.assert_allclose(ssm_forward(x, np.zeros((3, 1)), [[-1.0]], one, one, [0, 3], D=[2.0])["y"][0, 0], np.log(2) + 2)
    # a bias so low that dt vanishes keeps the state, whatever the inputs
    r = ssm_forward(x, np.zeros((3, 1)), [[-1.0]], one, one, [0, 3], bias=[-800.0], initial_state=[[[5.0]]])
    assert r["final_state"].item() == 5.0


def test_layernorm_gradients():
    rng = np.random.default_rng(3)
    inp = dict(s=rng.standard_normal((4, 5)) + 3, weight=rng.standard_normal(5), bias=rng.standard_normal(5))
    gy, carry = rng.standard_normal((4, 5)), rng.standard_normal((4, 5))

    def loss(s, weight, bias):
        return (layernorm_forward(s, weight, bias, 1e-3)["y"] * gy).sum() + (carry * s).sum()

    g = layernorm_backward(inp["s"], inp["weight"], 1e-3, gy, carry)
    check(loss, inp, {"s": g["grad_x"], "weight": g["grad_weight"], "bias": g["grad_bias"]})


def test_layernorm_against_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(4)
    s, w, b = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal(7)
    want = torch.nn.functional.layer_norm(torch.from_numpy(s), (7,), torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    np.testing.assert_allclose(layernorm_forward(s, w, b, 1e-5)["y"], want.numpy(), rtol=1e-12, atol=1e-14)
