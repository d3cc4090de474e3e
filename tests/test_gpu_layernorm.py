"""The residual layer norm on the GPU against the 64-bit oracle.

Tolerances.  The stream s = x + residual is one fp32 addition and one rounding to the stored type, which torch does bit
for bit on the CPU; the oracle goes on from it.  Sums are of at most 32768 terms in fp32, added pairwise over lanes and
warps but up to 64 in a row within a thread: 64 x 2^-24 / 2 = 2e-6 of the sum of absolute values, less in practice.
mean: 4e-6 of the mean of |s|; what it is off by moves n by as much times rstd.  rstd: 4e-6 relative, and what the
mean's error adds, second order.  y: 6e-6 of |w| (|n| + mean|s| rstd) + |b|, in bf16 half a step, 2^-8, on top.  grad_x is a
difference of three terms: 2e-5 of them, in bf16 2^-8 of itself on top.  grad_weight and grad_bias: fp32 sums over
rows: 1e-5 of the sum of absolute values."""

import numpy as np
import pytest

import recurrent_cell_gb300 as cfc
from oracle.layernorm_oracle import layernorm_backward, layernorm_forward

from gpu_common import require_gpu, torch_mod

pytestmark = pytest.mark.gpu

FP32, BF16 = cfc.MATH_FP32, cfc.MATH_BF16
MODES = pytest.mark.parametrize("math", [FP32, BF16], ids=["fp32", "bf16"])
EPS = 1e-5
# one element, less than a vector, odd, around the steps from lanes to warps, to wider rows and past the registers
WIDTHS = [1, 3, 7, 8, 64, 100, 128, 250, 256, 257, 512, 520, 1001, 1024, 2048, 2560, 4099, 5000, 8192, 8200, 16384, 16385, 32768]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def inputs(rows, d, math, seed=0, shift=0.0, size=1.0):
    torch = torch_mod()
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if math == FP32 else torch.bfloat16
    t = [(shift * (i == 0) + size * torch.randn(rows, d, generator=gen)).to(dt) for i in range(4)]
    return t, 1 + 0.3 * torch.randn(d, generator=gen), 0.3 * torch.randn(d, generator=gen), dt


def nans(*shape, dtype):
    return torch_mod().full(shape, float("nan"), dtype=dtype, device="cuda")


def run(rows, d, math, seed, residual=True, bias=True, carry=True, shift=0.0, size=1.0):
    torch = torch_mod()
    (x, r, dy, c), w, b, dt = inputs(rows, d, math, seed, shift, size)
    s = (x.float() + r.float()).to(dt) if residual else x
    f32, what = torch.float32, f"{rows} x {d}"
    half = 0.0 if math == FP32 else 2.0 ** -8
    y, out, mean, rstd = nans(rows, d, dtype=dt), nans(rows, d, dtype=dt), nans(rows, dtype=f32), nans(rows, dtype=f32)
    wd, bd = w.cuda(), b.cuda() if bias else None
    cfc.cfc_layernorm_forward(x.cuda(), wd, y, bias=bd, residual=r.cuda() if residual else None, residual_out=out, mean=mean,
                              rstd=rstd, eps=EPS, math=math)
    assert torch.equal(out.cpu(), s), what
    sd = s.double().numpy()
    ref = layernorm_forward(sd, w, b if bias else None, EPS)
    size_of = np.abs(sd).mean(-1)
    assert (np.abs(mean.double().cpu().numpy() - ref["mean"]) <= 4e-6 * size_of).all(), what
    moved = 4e-6 * size_of * ref["rstd"]                          # what the mean's error moves n by
    np.testing.assert_allclose(rstd.cpu().double(), ref["rstd"], rtol=float((4e-6 + moved ** 2).max()), err_msg=what)
    wn, bn = np.abs(w.double().numpy()), np.abs(b.double().numpy()) if bias else 0.0
    terms = wn * (np.abs(ref["n"]) + (size_of * ref["rstd"])[:, None]) + bn
    assert (np.abs(y.double().cpu().numpy() - ref["y"]) <= half * np.abs(ref["y"]) + 6e-6 * terms).all(), what

    ws = torch.full((cfc.cfc_layernorm_workspace_bytes(rows, d),), 255, dtype=torch.uint8, device="cuda")
    gx, gw, gb = nans(rows, d, dtype=dt), nans(d, dtype=f32), nans(d, dtype=f32)
    cfc.cfc_layernorm_backward(out, wd, mean, rstd, dy.cuda(), gx, gw, ws, grad_bias=gb if bias else None,
                               grad_residual_out=c.cuda() if carry else None, math=math)
    dyn = dy.double().numpy()
    want = layernorm_backward(sd, w, EPS, dyn, c.double().numpy() if carry else None)
    dn, n = np.abs(w.double().numpy() * dyn), np.abs(ref["n"]) + (size_of * ref["rstd"])[:, None]
    terms = ref["rstd"][:, None] * (dn + dn.mean(-1, keepdims=True) + n * (dn * n).mean(-1, keepdims=True))
    terms = terms + (np.abs(c.double().numpy()) if carry else 0)
    got = gx.double().cpu().numpy()
    assert (np.abs(got - want["grad_x"]) <= half * np.abs(want["grad_x"]) + 2e-5 * terms).all(), what
    assert (np.abs(gw.double().cpu().numpy() - want["grad_weight"]) <= 1e-5 * (np.abs(dyn) * n).sum(0)).all(), what
    if bias:
        assert (np.abs(gb.double().cpu().numpy() - want["grad_bias"]) <= 1e-5 * np.abs(dyn).sum(0)).all(), what


@MODES
@pytest.mark.parametrize("d", WIDTHS)
def test_forward_and_backward(d, math):
    for rows in (1, 2, 33, 700 if d <= 2560 else 5):
        run(rows, d, math, seed=d + rows)


@MODES
@pytest.mark.parametrize("d", [64, 1001, 2560, 20000])
def test_optional_inputs(d, math):
    for i, (residual, bias, carry) in enumerate([(False, True, True), (True, False, True), (True, True, False), (False, False, False)]):
        run(20, d, math, i, residual, bias, carry)


@pytest.mark.parametrize("d", [8, 257, 512, 2560, 16385])
def test_rows_far_from_zero_keep_their_digits(d):
    """fp32 rows around 1000 with a deviation of 1: the variance is not a difference of squares (whose error
    would be 1e6 x 6e-8 = 0.06 of it)."""
    run(40, d, FP32, 1, residual=False, shift=1000.0)


def test_more_rows_than_blocks():
    run(70000, 64, BF16, 1)
    run(9000, 1000, FP32, 2)


@MODES
def test_a_constant_row_and_no_rows(math):
    torch = torch_mod()
    dt = torch.float32 if math == FP32 else torch.bfloat16
    x, w, b = torch.full((3, 96), 5.0, dtype=dt, device="cuda"), torch.ones(96, device="cuda"), torch.arange(96.0, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(3, device="cuda")
    cfc.cfc_layernorm_forward(x, w, y, bias=b, rstd=rstd, eps=EPS, math=math)
    assert torch.equal(y, b.to(dt).expand(3, 96)) and torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5))
    gw, gb = nans(96, dtype=torch.float32), nans(96, dtype=torch.float32)
    ws = torch.empty(cfc.cfc_layernorm_workspace_bytes(0, 96), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 96, dtype=dt, device="cuda")
    cfc.cfc_layernorm_forward(none, w, none.clone(), math=math)
    cfc.cfc_layernorm_backward(none, w, rstd[:0], rstd[:0], none, none.clone(), gw, ws, grad_bias=gb, math=math)
    assert not gw.any() and not gb.any()


@MODES
@pytest.mark.parametrize("d", [100, 512, 2560, 20000])
def test_in_place_streams_and_gradients(d, math):
    torch = torch_mod()
    (x, r, dy, c), w, b, dt = inputs(50, d, math, 7)
    x, r, dy, c, w, b = (t.cuda() for t in (x, r, dy, c, w, b))
    f32 = torch.float32
    y, s, mean, rstd = nans(50, d, dtype=dt), nans(50, d, dtype=dt), nans(50, dtype=f32), nans(50, dtype=f32)
    call = lambda x, r, s, y: cfc.cfc_layernorm_forward(x, w, y, bias=b, residual=r, residual_out=s, mean=mean, rstd=rstd, math=math)  # noqa: E731
    call(x, r, s, y)
    for which in (0, 1):
        xx, rr, y2 = x.clone(), r.clone(), nans(50, d, dtype=dt)
        call(xx, rr, (xx, rr)[which], y2)
        assert torch.equal(y2, y) and torch.equal((xx, rr)[which], s)
    ws = torch.empty(cfc.cfc_layernorm_workspace_bytes(50, d), dtype=torch.uint8, device="cuda")
    back = lambda dy, c, gx, gw, gb: cfc.cfc_layernorm_backward(s, w, mean, rstd, dy, gx, gw, ws, grad_bias=gb, grad_residual_out=c, math=math)  # noqa: E731
    gx, gw, gb = nans(50, d, dtype=dt), nans(d, dtype=f32), nans(d, dtype=f32)
    back(dy, c, gx, gw, gb)
    for which in (0, 1):
        t = [dy.clone(), c.clone()]
        gw2, gb2 = nans(d, dtype=f32), nans(d, dtype=f32)
        back(*t, t[which], gw2, gb2)
        assert torch.equal(t[which], gx) and torch.equal(gw, gw2) and torch.equal(gb, gb2)


@MODES
@pytest.mark.parametrize("d", [7, 64, 2560])
def test_a_bad_row_stays_its_own(d, math):
    torch = torch_mod()
    (x, _, _, _), w, b, dt = inputs(64, d, math, 3)
    x, w = x.cuda(), w.cuda()
    y0 = nans(64, d, dtype=dt)
    cfc.cfc_layernorm_forward(x, w, y0, math=math)
    for bad in (float("nan"), float("inf")):
        x[5, d // 2] = bad
        y = nans(64, d, dtype=dt)
        cfc.cfc_layernorm_forward(x, w, y, math=math)
        keep = [i for i in range(64) if i != 5]
        assert torch.equal(y[keep], y0[keep]) and y[5].isnan().any()


@MODES
def test_the_same_bits_every_time_and_in_a_graph(math):
    torch = torch_mod()
    (x, r, dy, c), w, b, dt = inputs(3000, 1000, math, 5)
    x, r, dy, c, w, b = (t.cuda() for t in (x, r, dy, c, w, b))

    def run_all():
        f32 = torch.float32
        y, s, mean, rstd = (torch.empty_like(x), torch.empty_like(x), torch.empty(3000, device="cuda"), torch.empty(3000, device="cuda"))
        cfc.cfc_layernorm_forward(x, w, y, bias=b, residual=r, residual_out=s, mean=mean, rstd=rstd, math=math)
        gx, gw, gb = torch.empty_like(x), torch.empty(1000, dtype=f32, device="cuda"), torch.empty(1000, dtype=f32, device="cuda")
        ws = torch.empty(cfc.cfc_layernorm_workspace_bytes(3000, 1000), dtype=torch.uint8, device="cuda")
        cfc.cfc_layernorm_backward(s, w, mean, rstd, dy, gx, gw, ws, grad_bias=gb, grad_residual_out=c, math=math)
        return y, s, mean, rstd, gx, gw, gb

    first = run_all()
    for a, b2 in zip(first, run_all()):
        assert torch.equal(a, b2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run_all()
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    for a, b2 in zip(kept, run_all()):
        assert torch.equal(a, b2)


def test_refusals_of_the_binding():
    torch = torch_mod()
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(16, device="cuda")
    for bad in (dict(weight=w[:8]), dict(bias=w[:8]), dict(y=x[:3]), dict(x=x[:, ::2]), dict(mean=w), dict(residual=x.t())):
        with pytest.raises(ValueError):
            cfc.cfc_layernorm_forward(**{**dict(x=x, weight=w, y=torch.empty_like(x)), **bad})
    with pytest.raises(TypeError):
        cfc.cfc_layernorm_forward(x.float(), w, torch.empty_like(x))
