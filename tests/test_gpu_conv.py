"""The short causal convolution on the GPU against the 64-bit oracle.

Tolerances.  pre is a sum of up to nine fp32 terms: 9 x 6e-8 = 5e-7 of the sum of their absolute values, which the
gate passes on with a slope of at most 1.1; the sigmoid itself is good to 1e-6: 2e-6 of the terms' sum, for which
|w| |x| of the tensors' largest values stands, as 3e-6 of max|y| + max|pre|.  grad_x is a sum of up to eight such
values: 1e-5 of the largest.  grad_weight and grad_bias are sums over rows: 1e-5 of the largest term times the square
root of the number of rows.  In bf16 half a step of the value itself on top, 2^-8.  States are copies: exact."""

import numpy as np
import pytest

import recurrent_cell_gb300 as cfc
from oracle.ssm_oracle import conv_backward, conv_forward

from gpu_common import require_gpu, torch_mod

pytestmark = pytest.mark.gpu

FP32, BF16 = cfc.MATH_FP32, cfc.MATH_BF16
MODES = pytest.mark.parametrize("math", [FP32, BF16], ids=["fp32", "bf16"])


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


class Conv:
    def __init__(self, lens, d, W, math, seed=0, uniform=False, bias=True, init=True, silu=True, wide=True):
        torch = torch_mod()
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.dt = torch.float32 if math == FP32 else torch.bfloat16
        self.rows, self.n, self.d, self.W, self.math, self.silu = sum(lens), len(lens), d, W, math, silu
        self.off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        lead = (self.n, lens[0]) if uniform else (self.rows,)
        self.x = rand(*lead, d + (24 if wide else 0)).to(self.dt).cuda()[..., 8 if wide else 0:][..., :d]
        self.w, self.b = rand(d, W).cuda(), rand(d).cuda() if bias else None
        self.init = rand(self.n, W - 1, d).to(self.dt).cuda() if init else None
        self.gy, self.gfinal = rand(*lead, d).to(self.dt).cuda(), rand(self.n, W - 1, d).to(self.dt).cuda()
        self.so = None if uniform else torch.from_numpy(self.off).cuda()

    def nan(self, *shape, dtype=None):
        return torch_mod().full(shape, float("nan"), dtype=dtype or self.dt, device="cuda")

    def forward(self):
        y, final = self.nan(*self.x.shape), self.nan(self.n, self.W - 1, self.d)
        cfc.cfc_conv_forward(self.x, self.w, y, bias=self.b, seq_offsets=self.so, initial_state=self.init, final_state=final,
                             silu=self.silu, math=self.math)
        return y, final

    def backward(self, gfinal=True, optional=True):
        torch = torch_mod()
        f32 = torch.float32
        out = dict(grad_x=self.nan(*self.x.shape), grad_weight=self.nan(self.d, self.W, dtype=f32))
        more = dict(grad_bias=self.nan(self.d, dtype=f32), grad_initial_state=self.nan(self.n, self.W - 1, self.d)) if optional else {}
        ws = torch.full((cfc.cfc_conv_workspace_bytes(self.rows, self.d, self.W, self.math),), 255, dtype=torch.uint8, device="cuda")
        cfc.cfc_conv_backward(self.x, self.w, self.gy, *out.values(), ws, bias=self.b, seq_offsets=self.so,
                              initial_state=self.init, grad_final_state=self.gfinal if gfinal else None, silu=self.silu,
                              math=self.math, **more)
        return {**out, **more}

    def host(self):
        f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        return dict(x=f(self.x).reshape(self.rows, -1), weight=f(self.w), bias=f(self.b), offsets=self.off,
                    initial_state=f(self.init), silu=self.silu)


def close(got, want, tol, what, half):
    if want.size == 0:
        return
    got = got.double().cpu().numpy().reshape(want.shape)
    excess = np.abs(got - want) - tol - (2.0 ** -8 * np.abs(want) if half else 0)
    assert np.isfinite(got).all() and (excess <= 0).all(), f"{what}: {excess.max():.1e} beyond"


def check(c, gfinal=True):
    torch = torch_mod()
    half = c.math == BF16
    y, final = c.forward()
    h = c.host()
    ref = conv_forward(**h)
    top = np.abs(ref["pre"]).max(initial=0)
    close(y, ref["y"], 6e-6 * top, "y", half)
    np.testing.assert_array_equal(final.double().cpu().numpy(), ref["final_state"])
    gy = c.gy.double().cpu().numpy().reshape(c.rows, -1)
    want = conv_backward(**h, grad_y=gy, grad_final_state=c.gfinal.double().cpu().numpy() if gfinal else None)
    got = c.backward(gfinal)
    most = 1.1 * np.abs(gy).max(initial=1) * np.abs(h["weight"]).max()
    for k in ("grad_x", "grad_initial_state"):
        close(got[k], want[k], 1e-5 * most, k, half)
    x_top = max(np.abs(h["x"]).max(initial=1), 1 if c.init is None else float(c.init.abs().max()))
    for k, scale in (("grad_weight", x_top), ("grad_bias", 1)):
        close(got[k], want[k], 1e-5 * 1.1 * np.abs(gy).max(initial=1) * scale * np.sqrt(max(c.rows, 1)), k, False)
    for k, v in c.backward(gfinal, optional=False).items():
        assert torch.equal(v, got[k]), k


LENS = [[1], [3], [64], [65], [200], [0, 1, 2, 3, 4, 5, 0], [63, 1, 64, 65, 0, 130], [2, 1] * 30]


@MODES
@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v))[:20])
def test_packed_sequences(lens, math):
    check(Conv(lens, 40, 4, math, seed=len(lens)))


@MODES
@pytest.mark.parametrize("W", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("silu", [True, False])
def test_widths(W, silu, math):
    check(Conv([100, 3, 0, 1, 77], 24, W, math, seed=W, silu=silu))


@MODES
@pytest.mark.parametrize("n,t", [(1, 1), (3, 2), (2, 131), (50, 7)])
def test_uniform_sequences(n, t, math):
    check(Conv([t] * n, 32, 4, math, seed=t, uniform=True), gfinal=t != 7)


@MODES
@pytest.mark.parametrize("d", [8, 16, 136, 1000])
@pytest.mark.parametrize("flags", ["", "bias", "init"])
def test_channels_and_optional_inputs(d, flags, math):
    check(Conv([70, 30], d, 4, math, seed=d, bias="bias" in flags, init="init" in flags, wide=d != 16))


@MODES
def test_rows_of_nothing(math):
    torch = torch_mod()
    c = Conv([0, 0], 16, 4, math)
    _, final = c.forward()
    assert torch.equal(final, c.init)
    got = c.backward()
    assert torch.equal(got["grad_initial_state"], c.gfinal) and not got["grad_weight"].any() and not got["grad_bias"].any()


@MODES
@pytest.mark.parametrize("W", [2, 4, 8])
@pytest.mark.parametrize("t", [1, 3, 12])
def test_step_is_the_convolution_continued(W, t, math):
    torch = torch_mod()
    c = Conv([t] * 5, 48, W, math, seed=W + t, uniform=True)
    ref = conv_forward(**c.host())
    pool = torch.full((9, W - 1, 48), 7.0, dtype=c.dt, device="cuda")
    slots = torch.tensor([4, 0, 8, 2, 5], dtype=torch.int32, device="cuda")
    pool[slots.long()] = c.init
    y = c.nan(*c.x.shape)
    cfc.cfc_conv_step(c.x, c.w, pool, y, bias=c.b, slots=slots, math=math)
    close(y, ref["y"], 6e-6 * np.abs(ref["pre"]).max(), "y", math == BF16)
    np.testing.assert_array_equal(pool[slots.long()].double().cpu().numpy(), ref["final_state"])
    assert (pool[[1, 3, 6, 7]] == 7).all()
    bad = torch.tensor([4, -1, 9, 2 ** 30, 5], dtype=torch.int32, device="cuda")
    before = pool.clone()
    cfc.cfc_conv_step(c.x, c.w, pool, y, bias=c.b, slots=bad, math=math)
    assert not y[1:4].any() and torch.equal(pool[[0, 1, 2, 3, 6, 7, 8]], before[[0, 1, 2, 3, 6, 7, 8]])


@MODES
def test_a_nan_reaches_the_rows_that_see_it_only(math):
    torch = torch_mod()
    c = Conv([90, 100], 40, 4, math, seed=3)
    y0, _ = c.forward()
    for row in (88, 130):
        for bad in (float("nan"), float("inf")):
            keep = c.x[row, 7].clone()
            c.x[row, 7] = bad
            y, _ = c.forward()
            same = torch.ones_like(y, dtype=torch.bool)
            same[row:min(row + 4, 90 if row < 90 else 190), 7] = False
            assert torch.equal(y[same], y0[same])
            c.x[row, 7] = keep


@MODES
def test_large_arguments(math):
    """The gate far from zero: nothing but the value or zero, and its slope one or zero."""
    torch = torch_mod()
    c = Conv([8], 8, 2, math, bias=False, init=False, wide=False)
    c.w.zero_()
    c.w[:, 1] = 1
    c.x[:] = torch.tensor([-3e38, -1e4, -200, -100, 100, 200, 1e4, 3e38], device="cuda").to(c.dt)[:, None]
    y, _ = c.forward()
    assert (y[:4].float().abs() <= 1e-37).all() and torch.equal(y[4:], c.x[4:])
    c.gy.fill_(1)
    g = c.backward(gfinal=False)["grad_x"].float()
    assert (g[:4].abs() <= 1e-30).all() and (g[4:] == 1).all()


@MODES
def test_the_same_bits_every_time_in_a_graph_and_on_another_stream(math):
    torch = torch_mod()
    c = Conv([300, 0, 70, 1], 72, 4, math, seed=5)
    run = lambda: [*c.forward(), *c.backward().values()]  # noqa: E731
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run()
    side.synchronize()
    for a, b, o in zip(first, run(), other):
        assert torch.equal(a, b) and torch.equal(a, o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    c.x.copy_(c.x * 0.5)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(kept, run()):
        assert torch.equal(a, b)


@MODES
def test_offsets_outside_the_rows(math):
    torch = torch_mod()
    c = Conv([50, 60, 40], 24, 4, math, seed=8)
    y0, _ = c.forward()
    for off in ([0, 50, 110, 2 ** 31 - 1], [-5, 50, 110, 200], [0, 50, 40, 150], [-2 ** 31, 50, 110, 120]):
        c.so.copy_(torch.tensor(off, dtype=torch.int32))
        guard = torch.full((c.rows + 64, c.d), 3.0, dtype=c.dt, device="cuda")
        y = guard[32:32 + c.rows]
        cfc.cfc_conv_forward(c.x, c.w, y, bias=c.b, seq_offsets=c.so, initial_state=c.init,
                             final_state=c.nan(c.n, c.W - 1, c.d), math=math)
        c.backward()
        assert torch.equal(y[:40], y0[:40]), off
        assert (guard[:32] == 3).all() and (guard[32 + c.rows:] == 3).all()


@MODES
@pytest.mark.parametrize("lens", [[100, 0, 37], [3], [], [0]])
def test_a_padded_batch(lens, math):
    """Rows behind the last sequence are neither read nor written, and add nothing to the sums over rows."""
    torch = torch_mod()
    c, exact = Conv([*lens, 200], 40, 4, math, seed=12), Conv([*lens, 0], 40, 4, math, seed=12)
    used = sum(lens)
    for name in ("x", "gy"):
        setattr(exact, name, getattr(c, name)[:used].clone())
        getattr(c, name)[used:] = float("nan")
    for name in ("w", "b", "init", "gfinal"):
        setattr(exact, name, getattr(c, name))
    c.so = exact.so.clone()
    (y, f), (y1, f1) = c.forward(), exact.forward()
    assert torch.equal(y[:used], y1) and y[used:].isnan().all() and torch.equal(f, f1)
    got, want = c.backward(), exact.backward()
    assert torch.equal(got["grad_x"][:used], want["grad_x"]) and got["grad_x"][used:].isnan().all()
    assert torch.equal(got["grad_initial_state"], want["grad_initial_state"])
    for k in ("grad_weight", "grad_bias"):          # tiles of another length: sums in another order
        assert float((got[k] - want[k]).abs().max()) <= 1e-5 * max(float(want[k].abs().max()), 1e-30) * max(used, 1) ** 0.5


def test_offsets_past_32_bits():
    torch = torch_mod()
    n, t, d = 2100, 16, 65536
    g = torch.Generator("cuda").manual_seed(0)
    x = torch.randn(n, t, d, generator=g, device="cuda", dtype=torch.bfloat16)
    w, b = torch.randn(d, 4, generator=g, device="cuda"), torch.randn(d, generator=g, device="cuda")
    y = torch.full_like(x, float("nan"))
    cfc.cfc_conv_forward(x, w, y, bias=b, math=BF16)
    ref = conv_forward(x[-1].double().cpu().numpy()[:, -64:], w[-64:].double().cpu().numpy(), b[-64:].double().cpu().numpy(), [0, t])
    close(y[-1][:, -64:], ref["y"], 6e-6 * np.abs(ref["pre"]).max(), "y", True)
    assert not torch.isnan(y[::300]).any()


def test_refusals_of_the_binding():
    torch = torch_mod()
    c = Conv([4, 4], 16, 4, BF16, uniform=True, wide=False)
    y = torch.empty_like(c.x)
    for bad in (dict(weight=c.w[:8]), dict(bias=c.w), dict(x=c.x[0]), dict(initial_state=c.init[:, :2]), dict(y=y[:, :3]),
                dict(x=c.x.transpose(0, 1)[:, :, :], y=y.transpose(0, 1))):
        with pytest.raises(ValueError):
            cfc.cfc_conv_forward(**{**dict(x=c.x, weight=c.w, y=y), **bad})
    with pytest.raises(cfc.CfcError, match="overlap"):
        cfc.cfc_conv_forward(c.x, c.w, c.x)
    with pytest.raises(cfc.CfcError, match="overlap"):
        cfc.cfc_conv_forward(c.x, c.w, y, initial_state=c.init, final_state=c.init)
    with pytest.raises(ValueError, match="slots"):
        cfc.cfc_conv_step(c.x, c.w, c.init[:, :2], y)


@MODES
def test_an_output_between_the_rows_of_an_input(math):
    """Overlap is seen row by row: y may lie in what the rows of a wider tensor leave of it, and not a vector further."""
    torch = torch_mod()
    c = Conv([3], 16, 4, math, seed=21, uniform=True, wide=False)
    want, _ = c.forward()
    buffer = torch.full((3, 128), float("nan"), dtype=c.dt, device="cuda")
    x = buffer[None, :, :16]
    x.copy_(c.x)
    y = buffer[1, 16:16 + 48].view(1, 3, 16)
    call = lambda y: cfc.cfc_conv_forward(x, c.w, y, bias=c.b, initial_state=c.init, math=math)  # noqa: E731
    call(y)
    assert torch.equal(y, want) and torch.equal(x, c.x)
    with pytest.raises(cfc.CfcError, match="overlap"):
        call(buffer[1, 8:56].view(1, 3, 16))
    with pytest.raises(cfc.CfcError, match="overlap"):
        call(buffer.view(-1)[128 + 88:][:48].view(1, 3, 16))       # runs into the third row
