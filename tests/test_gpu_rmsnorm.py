"""The residual RMS norm on the GPU against the 64-bit oracle.

Tolerances.  The stream s = x + residual is one fp32 addition and one rounding
to the stored type, which torch does bit for bit on the CPU; the oracle goes
on from it.  rstd: a sum of at most 32768 squares in fp32, added pairwise over lanes
and warps but up to 256 in a row within a thread: 256 x 2^-24 / 2 = 8e-6 at worst,
2e-6 expected; 4e-6.  y = s rstd w: that and two roundings: 5e-6 relative in fp32;
in bf16 half a unit on top, 2^-8 at most.  y8: half a unit of e4m3, 2^-4
relative or, below 2^-6, 2^-10 of a scale, on a y that is off by 5e-6.  grad_x is a
difference of two terms: 1e-5 of them in fp32, 2^-8 of itself on top in
bf16.  grad_weight: fp32 sums over rows: 1e-5 of the sum of absolute values.
"""

import os
import subprocess
import sys

import numpy as np
import pytest

import recurrent_cell_gb300 as cfc
from oracle.rmsnorm_oracle import rmsnorm_backward, rmsnorm_forward, rmsnorm_group_scale

from gpu_common import require_gpu, torch_mod

pytestmark = pytest.mark.gpu

FP32, BF16 = cfc.MATH_FP32, cfc.MATH_BF16
MODES = pytest.mark.parametrize("math", [FP32, BF16], ids=["fp32", "bf16"])
EPS = 1e-6
# one element, less than a vector, odd, around the steps from lanes to warps to wider rows
WIDTHS = [1, 3, 7, 8, 64, 100, 128, 250, 256, 257, 512, 520, 1001, 1024, 2048, 2560, 4099, 5000, 8192, 16384, 16385, 32768]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def half_unit(math):
    return 0.0 if math == FP32 else 2.0 ** -8


def inputs(rows, d, math, seed=0, size=1.0):
    torch = torch_mod()
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if math == FP32 else torch.bfloat16
    x = [(size * torch.randn(rows, d, generator=gen)).to(dt) for _ in range(4)]
    w = 1 + 0.3 * torch.randn(d, generator=gen)
    return x, w, dt


def stream_of(x, residual):
    return (x.float() + residual.float()).to(x.dtype)


def nans(*shape, dtype):
    torch = torch_mod()
    if dtype is torch.uint8:
        return torch.full(shape, 255, dtype=dtype, device="cuda")
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def check_y(y, ref, math, what):
    got = y.double().cpu().numpy()
    bad = np.abs(got - ref["y"]) > (half_unit(math) + 5e-6) * np.abs(ref["y"])
    assert not bad.any(), f"{what}: {bad.sum()} values"


def check_y8(y8, scale, ref, group, what):
    y = ref["y"]
    c = scale.double().cpu().numpy()
    np.testing.assert_allclose(c, rmsnorm_group_scale(y, group), rtol=5e-6, err_msg=what)
    wide = np.repeat(c, group, axis=1)
    got = y8.view(torch_mod().float8_e4m3fn).float().double().cpu().numpy() * wide
    assert (np.abs(got - y) <= (2.0 ** -4 + 1e-5) * np.abs(y) + 2.0 ** -10 * (1 + 1e-5) * wide).all(), what


@MODES
@pytest.mark.parametrize("d", WIDTHS)
def test_forward_and_backward(d, math):
    torch = torch_mod()
    for rows in (1, 2, 33, 700 if d <= 2560 else 5):
        (x, r, dy, carry), w, dt = inputs(rows, d, math, seed=d + rows)
        s = stream_of(x, r)
        ref = rmsnorm_forward(s.double(), w, EPS)
        y, out, rstd = nans(rows, d, dtype=dt), nans(rows, d, dtype=dt), nans(rows, dtype=torch.float32)
        xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
        cfc.cfc_rmsnorm_forward(xd, wd, y=y, residual=rd, residual_out=out, rstd=rstd, eps=EPS, math=math)
        what = f"{rows} x {d}"
        assert torch.equal(out.cpu(), s), what
        np.testing.assert_allclose(rstd.cpu().double(), ref["rstd"], rtol=4e-6, err_msg=what)
        check_y(y, ref, math, what)
        plain = nans(rows, d, dtype=dt)
        cfc.cfc_rmsnorm_forward(out, wd, y=plain, eps=EPS, math=math)          # without the residual
        assert torch.equal(plain, y), what

        ws = torch.full((cfc.cfc_rmsnorm_workspace_bytes(rows, d),), 255, dtype=torch.uint8, device="cuda")
        for c in (carry, None):
            gx, gw = nans(rows, d, dtype=dt), nans(d, dtype=torch.float32)
            cfc.cfc_rmsnorm_backward(out, wd, rstd, dy.cuda(), gx, gw, ws, grad_residual_out=None if c is None else c.cuda(),
                                     math=math)
            want = rmsnorm_backward(s.double(), w, EPS, dy.double(), None if c is None else c.double())
            terms = rmsnorm_terms(s.double().numpy(), w.double().numpy(), dy.double().numpy())
            got = gx.double().cpu().numpy()
            assert (np.abs(got - want["grad_x"]) <= half_unit(math) * np.abs(want["grad_x"]) + 1e-5 * (
                terms + (0 if c is None else np.abs(c.double().numpy())))).all(), what
            sums = np.abs(dy.double().numpy() * s.double().numpy() * ref["rstd"][:, None]).sum(0)
            assert (np.abs(gw.double().cpu().numpy() - want["grad_weight"]) <= 1e-5 * sums).all(), what


def rmsnorm_terms(s, w, dy):
    rstd = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + EPS)
    return rstd * (np.abs(w * dy) + np.abs(s) * rstd ** 2 * np.abs(s * w * dy).mean(-1, keepdims=True))


@MODES
@pytest.mark.parametrize("d,group", [(64, 64), (64, 16), (64, 1), (96, 3), (128, 128), (256, 64), (1024, 128), (1001, 7),
                                     (1001, 1001), (4096, 4096), (4096, 64), (8192, 128), (8192, 8192), (32768, 32768),
                                     (2560, 2560), (5000, 1000)])
def test_eight_bits(d, group, math):
    torch = torch_mod()
    for rows in (1, 37):
        (x, r, _, _), w, dt = inputs(rows, d, math, seed=d + group)
        ref = rmsnorm_forward(stream_of(x, r).double(), w, EPS)
        y8, scale = nans(rows, d, dtype=torch.uint8), nans(rows, d // group, dtype=torch.float32)
        y, out = nans(rows, d, dtype=dt), nans(rows, d, dtype=dt)
        args = dict(residual=r.cuda(), y8=y8, y8_scale=scale, eps=EPS, math=math)
        cfc.cfc_rmsnorm_forward(x.cuda(), w.cuda(), y=y, residual_out=out, **args)
        check_y8(y8, scale, ref, group, f"{rows} x {d} / {group}")
        check_y(y, ref, math, f"{rows} x {d}")
        first, scale1 = y8.clone(), scale.clone()
        y8.fill_(0)
        cfc.cfc_rmsnorm_forward(x.cuda(), w.cuda(), **args)                    # the 8-bit output alone
        assert torch.equal(y8, first) and torch.equal(scale, scale1)


@MODES
def test_rows_of_zeros_and_of_extremes(math):
    """Zeros: y = 0, scale 1.  Rows at the ends of the type's range whose squares fp32 holds."""
    torch = torch_mod()
    (x, r, _, _), w, dt = inputs(6, 256, math, seed=3)
    x[0] = r[0] = 0
    x[1], r[1] = x[1] * 1e17, 0
    x[2], r[2] = x[2] * 1e-15, 0
    r[3] = -x[3]
    x[4] = r[4] = 0
    x[4, 100] = 5.0
    ref = rmsnorm_forward(stream_of(x, r).double(), w, EPS)
    y, y8, scale = nans(6, 256, dtype=dt), nans(6, 256, dtype=torch.uint8), nans(6, 2, dtype=torch.float32)
    cfc.cfc_rmsnorm_forward(x.cuda(), w.cuda(), y=y, residual=r.cuda(), y8=y8, y8_scale=scale, eps=EPS, math=math)
    check_y(y, ref, math, "extremes")
    check_y8(y8, scale, ref, 128, "extremes")
    assert (scale[[0, 3]] == 1).all() and (scale[4].cpu().numpy()[1] == 1)


@MODES
@pytest.mark.parametrize("d", [64, 257, 4096])
def test_nan_and_infinity_stay_in_their_rows(d, math):
    torch = torch_mod()
    (x, _, dy, _), w, dt = inputs(40, d, math, seed=4)
    outs = []
    for bad in (None, float("nan"), float("inf")):
        if bad is not None:
            x[7, d // 2] = bad
        y, rstd, y8, scale = nans(40, d, dtype=dt), nans(40, dtype=torch.float32), nans(40, d, dtype=torch.uint8), nans(40, 1, dtype=torch.float32)
        cfc.cfc_rmsnorm_forward(x.cuda(), w.cuda(), y=y, rstd=rstd, y8=y8, y8_scale=scale, eps=EPS, math=math)
        gx, gw = nans(40, d, dtype=dt), nans(d, dtype=torch.float32)
        ws = torch.empty(cfc.cfc_rmsnorm_workspace_bytes(40, d), dtype=torch.uint8, device="cuda")
        cfc.cfc_rmsnorm_backward(x.cuda(), w.cuda(), rstd, dy.cuda(), gx, gw, ws, math=math)
        outs.append([a.cpu().view(torch.uint8).reshape(40, -1) for a in (y, rstd, y8, scale, gx)])
        if bad is not None:
            assert torch.isnan(y[7, d // 2])
            if bad != bad:
                assert torch.isnan(y[7]).all() and torch.isnan(rstd[7])
    rest = [i for i in range(40) if i != 7]
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a[rest], b[rest])


@MODES
@pytest.mark.parametrize("d", [96, 257, 5000])
def test_outputs_over_inputs(d, math):
    torch = torch_mod()
    (x, r, dy, carry), w, dt = inputs(50, d, math, seed=5)
    ref = nans(50, d, dtype=dt), nans(50, d, dtype=dt)
    cfc.cfc_rmsnorm_forward(x.cuda(), w.cuda(), y=ref[0], residual=r.cuda(), residual_out=ref[1], math=math)
    for over in ("x", "residual"):
        xd, rd, y = x.cuda(), r.cuda(), nans(50, d, dtype=dt)
        out = xd if over == "x" else rd
        cfc.cfc_rmsnorm_forward(xd, w.cuda(), y=y, residual=rd, residual_out=out, math=math)
        assert torch.equal(y, ref[0]) and torch.equal(out, ref[1])
    rstd = torch.rand(50, device="cuda") + 0.5
    ws = torch.empty(cfc.cfc_rmsnorm_workspace_bytes(50, d), dtype=torch.uint8, device="cuda")
    gw = nans(2, d, dtype=torch.float32) if d % 4 == 0 else [nans(d, dtype=torch.float32) for _ in range(2)]
    gx = nans(50, d, dtype=dt)
    cfc.cfc_rmsnorm_backward(ref[1], w.cuda(), rstd, dy.cuda(), gx, gw[0], ws, grad_residual_out=carry.cuda(), math=math)
    for over in ("dy", "carry"):
        a, b = dy.cuda(), carry.cuda()
        cfc.cfc_rmsnorm_backward(ref[1], w.cuda(), rstd, a, a if over == "dy" else b, gw[1], ws, grad_residual_out=b, math=math)
        assert torch.equal(a if over == "dy" else b, gx) and torch.equal(gw[0], gw[1])


@MODES
def test_gradients_match_differences(math):
    """Against central differences of the 64-bit forward; grad_x in bf16 is off by a rounding,
    2^-9 of its norm, and both by 1e-5 of the terms."""
    torch = torch_mod()
    (s, dy, _, _), w, dt = inputs(9, 200, math, seed=6)
    y, rstd = nans(9, 200, dtype=dt), nans(9, dtype=torch.float32)
    cfc.cfc_rmsnorm_forward(s.cuda(), w.cuda(), y=y, rstd=rstd, eps=EPS, math=math)
    gx, gw = nans(9, 200, dtype=dt), nans(200, dtype=torch.float32)
    ws = torch.empty(cfc.cfc_rmsnorm_workspace_bytes(9, 200), dtype=torch.uint8, device="cuda")
    cfc.cfc_rmsnorm_backward(s.cuda(), w.cuda(), rstd, dy.cuda(), gx, gw, ws, math=math)
    S, W, D = s.double().numpy(), w.double().numpy(), dy.double().numpy()
    loss = lambda a, b: (rmsnorm_forward(a, b, EPS)["y"] * D).sum()  # noqa: E731
    rng = np.random.default_rng(0)
    for _ in range(4):
        a, b = rng.standard_normal(S.shape), rng.standard_normal(W.shape)
        fd = (loss(S + 1e-5 * a, W) - loss(S - 1e-5 * a, W)) / 2e-5
        g = gx.double().cpu().numpy()
        assert abs((g * a).sum() - fd) <= (half_unit(math) / 2 + 2e-5) * np.linalg.norm(g) * np.linalg.norm(a) + 1e-6
        fd = (loss(S, W + 1e-5 * b) - loss(S, W - 1e-5 * b)) / 2e-5
        g = gw.double().cpu().numpy()
        assert abs((g * b).sum() - fd) <= 2e-5 * np.linalg.norm(g) * np.linalg.norm(b) + 1e-6


def test_no_rows():
    torch = torch_mod()
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    cfc.cfc_rmsnorm_forward(e, w, y=e, math=FP32)
    gw = nans(64, dtype=torch.float32)
    ws = torch.empty(max(cfc.cfc_rmsnorm_workspace_bytes(0, 64), 16), dtype=torch.uint8, device="cuda")
    cfc.cfc_rmsnorm_backward(e, w, torch.empty(0, device="cuda"), e, e, gw, ws, math=FP32)
    assert (gw == 0).all()


@MODES
def test_same_bits_on_another_stream_and_in_a_graph(math):
    torch = torch_mod()
    (x, r, dy, carry), w, dt = inputs(999, 1024, math, seed=7)
    dev = [a.cuda() for a in (x, r, dy, carry, w)]
    ws = torch.empty(cfc.cfc_rmsnorm_workspace_bytes(999, 1024), dtype=torch.uint8, device="cuda")

    def make():
        return [nans(999, 1024, dtype=dt), nans(999, 1024, dtype=dt), nans(999, dtype=torch.float32),
                nans(999, 1024, dtype=dt), nans(1024, dtype=torch.float32)]

    def run(o, stream=None):
        cfc.cfc_rmsnorm_forward(dev[0], dev[4], y=o[0], residual=dev[1], residual_out=o[1], rstd=o[2], math=math, stream=stream)
        cfc.cfc_rmsnorm_backward(o[1], dev[4], o[2], dev[2], o[3], o[4], ws, grad_residual_out=dev[3], math=math, stream=stream)

    a, b, c = make(), make(), make()
    run(a)
    torch.cuda.synchronize()
    run(b, torch.cuda.Stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c)
    graph.replay()
    torch.cuda.synchronize()
    for u, v, z in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, z)


def test_more_rows_than_32_bit_offsets():
    """Rows past 2^31 elements, read in place of their copies at the front."""
    torch = torch_mod()
    rows, d = 2 ** 31 // 4096 + 10, 4096
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    x[-10:] = torch.randn(10, d, device="cuda")
    x[:10] = x[-10:]
    w = torch.rand(d, device="cuda")
    y = torch.empty_like(x)
    cfc.cfc_rmsnorm_forward(x, w, y=y)
    assert torch.equal(y[-10:], y[:10])
    check_y(y[-10:], rmsnorm_forward(x[-10:].double().cpu(), w.cpu(), EPS), BF16, "far rows")


def test_binding_refuses_what_does_not_fit():
    torch = torch_mod()
    x, w = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    y, f8 = torch.empty_like(x), torch.empty(4, 64, dtype=torch.uint8, device="cuda")
    for err, args, kw in [
        (TypeError, (x.float(), w), {"y": y}),
        (TypeError, (x, w.bfloat16()), {"y": y}),
        (TypeError, (x, w), {"y8": f8.int()}),
        (ValueError, (x, w[:32]), {"y": y}),
        (ValueError, (x, w), {"y": y[:2]}),
        (ValueError, (x, w), {"y8": f8}),
        (ValueError, (x, w), {"y8": f8, "y8_scale": torch.empty(4, 5, device="cuda")}),
        (cfc.CfcError, (x, w), {}),
    ]:
        with pytest.raises(err):
            cfc.cfc_rmsnorm_forward(*args, **kw)
    with pytest.raises(cfc.CfcError):
        cfc.cfc_rmsnorm_backward(x, w, torch.ones(4, device="cuda"), y, y, torch.empty(64, device="cuda"),
                                 torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_widths_at_the_default_limit_of_shared_memory_in_a_fresh_process():
    """Rows that the element-wise backward takes, whose sums just fill 48 KB beside its own few words: in a
    process that has asked for no more yet."""
    code = ("import test_gpu_rmsnorm as t\n"
            "for d in (12256, 12257, 12264, 12280, 12288, 12289):\n"
            "    for math in (t.FP32, t.BF16):\n"
            "        t.test_forward_and_backward(d, math)\n")
    here = os.path.dirname(os.path.abspath(__file__))
    path = os.pathsep.join([here, os.path.dirname(here)])
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(here), env={**os.environ, "PYTHONPATH": path},
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
