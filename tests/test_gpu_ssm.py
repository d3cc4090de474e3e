"""The selective scan on the GPU against the 64-bit oracle.

Tolerances.  A token adds to a state the error of one exponential (1.4e-7 at most, 6e-8 in root mean square), of the
product dt A under it and of three roundings (6e-8 each): 3e-7.  The tests' decays remember some 15 tokens, so a state
and what is read from it are good to 15 x 3e-7 = 5e-6 of the tensor's largest value at worst.  A gradient goes through
the states forward and its own recurrence back: 1e-5.  Sums over rows (grad_A, grad_D, grad_delta_bias) add the same
relative errors of terms of both signs: 1e-5 of the sum of absolute values, for which their largest value times the
square root of the number of rows stands.  In bf16 what leaves in that type is off by half a step of itself more, 2^-8."""

import numpy as np
import pytest

import recurrent_cell_gb300 as cfc
from oracle.ssm_oracle import ssm_backward, ssm_forward

from gpu_common import require_gpu, torch_mod

pytestmark = pytest.mark.gpu

FP32, BF16 = cfc.MATH_FP32, cfc.MATH_BF16
MODES = pytest.mark.parametrize("math", [FP32, BF16], ids=["fp32", "bf16"])


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def offsets_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


class Scan:
    """Inputs of one call on the device, and as the oracle gets them."""

    def __init__(self, lens, d, groups, N, math, seed=0, uniform=False, D=True, z=True, bias=True, init=True, wide=True):
        torch = torch_mod()
        g = torch.Generator().manual_seed(seed)
        self.lens, self.d, self.groups, self.N, self.math, self.uniform = list(lens), d, groups, N, math, uniform
        self.dt = torch.float32 if math == FP32 else torch.bfloat16
        rows, n = sum(lens), len(lens)
        self.rows, self.n, self.off = rows, n, offsets_of(lens)
        lead = (n, lens[0]) if uniform else (rows,)
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        wide_rows = (lambda w, x: torch.cat([rand(*lead, w).to(self.dt), x, rand(*lead, 8).to(self.dt)], -1).cuda()[..., w:w + x.shape[-1]]
                     ) if wide else (lambda w, x: x.cuda())
        self.x = wide_rows(8, rand(*lead, d).to(self.dt))
        self.delta = wide_rows(16, rand(*lead, d).to(self.dt))
        self.z = wide_rows(8, rand(*lead, d).to(self.dt)) if z else None
        self.B, self.C = (wide_rows(8, rand(*lead, groups * N).to(self.dt)).unflatten(-1, (groups, N)) for _ in range(2))
        self.A = -(0.1 + torch.rand(d, N, generator=g)).cuda()
        self.D = rand(d).cuda() if D else None
        self.bias = (0.3 * rand(d)).cuda() if bias else None
        self.init = rand(n, d, N).cuda() if init else None
        self.gy = rand(*lead, d).to(self.dt).cuda()
        self.gfinal = rand(n, d, N).cuda()
        self.so = None if uniform else torch.from_numpy(self.off).cuda()

    def workspace(self, save):
        torch = torch_mod()
        size = cfc.cfc_ssm_workspace_bytes(self.rows, self.n, self.d, self.groups, self.N, self.math, save)
        return torch.full((size,), 255, dtype=torch.uint8, device="cuda")       # NaN in every float

    def nan(self, t, dtype=None):
        return None if t is None else torch_mod().full(t.shape, float("nan"), dtype=dtype or t.dtype, device="cuda")

    def forward(self, ws=None, save=False, **kw):
        y, final = self.nan(self.x), self.nan(self.gfinal)
        ws = self.workspace(save) if ws is None else ws
        cfc.cfc_ssm_forward(self.x, self.delta, self.A, self.B, self.C, y, ws, D=self.D, z=self.z, delta_bias=self.bias,
                            seq_offsets=self.so, initial_state=self.init, final_state=final, save=save, math=self.math, **kw)
        return y, final

    def backward(self, ws, gfinal=True, optional=True):
        out = dict(grad_x=self.nan(self.x), grad_delta=self.nan(self.delta), grad_A=self.nan(self.A), grad_B=self.nan(self.B),
                   grad_C=self.nan(self.C))
        more = dict(grad_z=self.nan(self.z))
        if optional:
            vec = torch_mod().empty(self.d, device="cuda")
            more.update(grad_D=self.nan(vec), grad_delta_bias=self.nan(vec), grad_initial_state=self.nan(self.gfinal))
        cfc.cfc_ssm_backward(self.x, self.delta, self.A, self.B, self.C, self.gy, *out.values(), ws, D=self.D, z=self.z,
                             delta_bias=self.bias, seq_offsets=self.so, initial_state=self.init,
                             grad_final_state=self.gfinal if gfinal else None, math=self.math, **more)
        out.update({k: v for k, v in more.items() if v is not None})
        return out

    def host(self):
        f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        rows = lambda t: None if t is None else f(t).reshape(self.rows, -1)  # noqa: E731
        bc = lambda t: f(t).reshape(self.rows, self.groups, self.N)  # noqa: E731
        return dict(x=rows(self.x), delta=rows(self.delta), A=f(self.A), B=bc(self.B), C=bc(self.C), D=f(self.D), z=rows(self.z),
                    bias=f(self.bias), initial_state=f(self.init), offsets=self.off)


def close(got, want, tol, what, half=False, scale=None):
    if want.size == 0:
        return
    got = got.double().cpu().numpy().reshape(want.shape)
    top = np.abs(want).max() if scale is None else scale
    excess = np.abs(got - want) - tol * top - (2.0 ** -8 * np.abs(want) if half else 0)
    assert np.isfinite(got).all() and (excess <= 0).all(), f"{what}: {excess.max() / top:.1e} of the largest value beyond"


def check(s, gfinal=True):
    half = s.math == BF16
    ws = s.workspace(True)
    y, final = s.forward(ws, save=True)
    h = s.host()
    ref = ssm_forward(**h)
    close(y, ref["y"], 5e-6, "y", half)
    close(final, ref["final_state"], 5e-6, "final state")
    y2, _ = s.forward()                                       # without saving: the same values
    assert torch_mod().equal(y, y2)
    got = s.backward(ws, gfinal)
    want = ssm_backward(**h, grad_y=s.gy.double().cpu().numpy().reshape(s.rows, -1),
                        grad_final_state=s.gfinal.double().cpu().numpy() if gfinal else None)
    for k, v in got.items():
        over_rows = k in ("grad_A", "grad_D", "grad_delta_bias")
        scale = np.abs(want[k]).max() * np.sqrt(max(s.rows, 1)) if over_rows else None
        close(v, want[k], 1e-5, k, half and k in ("grad_x", "grad_delta", "grad_z", "grad_B", "grad_C"), scale)


LENS = [[1], [16], [17], [300], [0, 300, 1, 16, 0, 15, 70, 33, 0, 8], [0, 1, 2, 15, 16, 17, 33, 0], [0, 70, 200, 1, 0, 5, 64, 130], [5, 3] * 20]


@MODES
@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v))[:20])
def test_packed_sequences(lens, math):
    check(Scan(lens, 40, 1, 16, math, seed=len(lens)))


@MODES
@pytest.mark.parametrize("n,t", [(1, 1), (3, 1), (3, 40), (2, 131), (50, 7)])
def test_uniform_sequences(n, t, math):
    check(Scan([t] * n, 32, 1, 16, math, seed=t, uniform=True))


@MODES
@pytest.mark.parametrize("n,t,d", [(1, 700, 32), (2, 500, 64), (9, 263, 8), (9, 264, 8), (3, 401, 40)])
def test_long_uniform_sequences(n, t, d, math):
    """Few of them and long: cut into segments; short ones stay whole."""
    check(Scan([t] * n, d, 1, 16, math, seed=t + n, uniform=True))


@MODES
@pytest.mark.parametrize("N", [1, 3, 4, 8, 12, 16, 24, 32, 40, 64])
@pytest.mark.parametrize("d,groups", [(8, 1), (48, 2)])
def test_states_and_groups(N, d, groups, math):
    check(Scan([37, 0, 90], d, groups, N, math, seed=N))


@MODES
@pytest.mark.parametrize("N", [3, 8, 16, 24, 32, 64])
@pytest.mark.parametrize("d,groups", [(8, 1), (48, 2)])
def test_states_and_groups_of_long_sequences(N, d, groups, math):
    """More rows than one warp takes: sequences that a segment's end cuts, once and more often."""
    check(Scan([150, 0, 1, 237], d, groups, N, math, seed=N))


def test_channels_enough_for_whole_packed_rows():
    """Tiles of channels for every warp of the GPU: packed rows in one segment, and a workspace of their size."""
    d, N = 40000, 2
    small, big = (cfc.cfc_ssm_workspace_bytes(r, 3, d, 1, N, BF16, save=True) for r in (320, 640))
    assert big < 2.1 * small
    check(Scan([100, 0, 220], d, 1, N, BF16, seed=3))


@pytest.mark.parametrize("d,groups", [(8, 1), (24, 3), (136, 1), (128, 1), (160, 2), (1000, 1)])
def test_channels(d, groups):
    check(Scan([20, 70], d, groups, 16, BF16, seed=d))


@MODES
@pytest.mark.parametrize("flags", ["", "D", "z", "bias", "init", "D z", "z bias init"])
def test_optional_inputs(flags, math):
    s = Scan([33, 100], 24, 1, 8, math, seed=len(flags), wide=False,
             **{k: k in flags.split() for k in ("D", "z", "bias", "init")})
    check(s, gfinal="init" in flags)
    ws = s.workspace(True)
    s.forward(ws, save=True)
    want = s.backward(ws)
    for k, v in s.backward(ws, optional=False).items():       # optional gradients left out: the others keep their bits
        assert torch_mod().equal(v, want[k]), k


@MODES
def test_rows_of_nothing(math):
    torch = torch_mod()
    s = Scan([0, 0, 0], 16, 1, 16, math)
    ws = s.workspace(True)
    _, final = s.forward(ws, save=True)
    assert torch.equal(final, s.init)
    got = s.backward(ws)
    assert torch.equal(got["grad_initial_state"], s.gfinal)
    assert not got["grad_A"].any() and not got["grad_D"].any() and not got["grad_delta_bias"].any()
    u = Scan([0, 0], 16, 1, 16, math, uniform=True, init=False)
    _, final = u.forward()
    assert not final.any()


@MODES
@pytest.mark.parametrize("N", [5, 8, 16, 32, 64])
@pytest.mark.parametrize("d,groups", [(8, 1), (72, 1), (96, 4)])
def test_step_is_the_scan_continued(N, d, groups, math):
    torch = torch_mod()
    s = Scan([3] * 5, d, groups, N, math, seed=N + d, uniform=True)
    h = s.host()
    ref = ssm_forward(**h)
    pool = torch.full((9, d, N), 7.0, device="cuda")
    slots = torch.tensor([4, 0, 8, 2, 5], dtype=torch.int32, device="cuda")
    pool[slots.long()] = s.init
    y = s.nan(s.x)
    cfc.cfc_ssm_step(s.x, s.delta, s.A, s.B, s.C, pool, y, D=s.D, z=s.z, delta_bias=s.bias, slots=slots, math=math)
    close(y, ref["y"], 5e-6, "y", math == BF16)
    close(pool[slots.long()], ref["final_state"], 5e-6, "state")
    rest = [i for i in range(9) if i not in slots.tolist()]
    assert (pool[rest] == 7).all()
    # one token at a time, slots in order, the same states to a rounding
    own = s.init.clone()
    for t in range(3):
        part = [v[:, t:t + 1] for v in (s.x, s.delta, s.B, s.C, s.z)]
        one = s.nan(part[0])
        cfc.cfc_ssm_step(part[0], part[1], s.A, part[2], part[3], own, one, D=s.D, z=part[4], delta_bias=s.bias, math=math)
        assert torch.equal(one[:, 0], y[:, t])
    assert torch.equal(own, pool[slots.long()])


@MODES
@pytest.mark.parametrize("N,tokens,none", [(16, 1, ()), (16, 2, (0, 3, 4)), (16, 1, (6,)), (8, 3, (2,)), (12, 1, (1,))])
def test_channels_for_every_warp_and_sequences_one_after_another(N, tokens, none, math):
    """More tiles of channels than half of the GPU's warps: each takes all sequences, with and without states."""
    torch = torch_mod()
    n, d = 7, 65536 + 24
    s = Scan([tokens] * n, d, 1, N, math, seed=N + tokens, uniform=True)
    ref = ssm_forward(**s.host())
    pool = torch.full((n + 2, d, N), 7.0, device="cuda")
    slots = torch.tensor([8, 1, 0, 6, 3, 5, 2], dtype=torch.int32)
    good = np.setdiff1d(np.arange(n), none)
    pool[slots.long()[good]] = s.init[good]
    before, at = pool.clone(), slots.long()[good]
    slots[list(none)] = -1
    y = s.nan(s.x)
    cfc.cfc_ssm_step(s.x, s.delta, s.A, s.B, s.C, pool, y, D=s.D, z=s.z, delta_bias=s.bias, slots=slots.cuda(), math=math)
    assert not y[list(none)].any()
    close(y[good], ref["y"].reshape(n, tokens, d)[good], 5e-6, "y", math == BF16)
    close(pool[at], ref["final_state"][good], 5e-6, "state")
    rest = np.setdiff1d(np.arange(n + 2), at.numpy())
    assert torch.equal(pool[rest], before[rest])


def test_many_sequences_a_warp_and_slots_outside_the_pool():
    torch = torch_mod()
    n, d, N = 700, 64, 16
    s = Scan([1] * n, d, 1, N, BF16, seed=9, uniform=True)
    ref = ssm_forward(**s.host())
    pool = s.init.clone()
    slots = torch.arange(n, dtype=torch.int32)
    bad = [0, 3, 400, 699]
    slots[bad] = torch.tensor([-1, n, 2 ** 30, -2 ** 31], dtype=torch.int32)
    y = s.nan(s.x)
    cfc.cfc_ssm_step(s.x, s.delta, s.A, s.B, s.C, pool, y, D=s.D, z=s.z, delta_bias=s.bias, slots=slots.cuda(), math=BF16)
    good = np.setdiff1d(np.arange(n), bad)
    assert not y[bad].any()
    close(y[good], ref["y"][good], 5e-6, "y", True)
    close(pool[good], ref["final_state"][good], 5e-6, "state")
    assert torch.equal(pool[bad], s.init[bad])


@MODES
def test_a_nan_reaches_its_channel_and_its_sequences_later_tokens_only(math):
    torch = torch_mod()
    s = Scan([90, 100, 30], 40, 1, 16, math, seed=3)
    y0, f0 = s.forward()
    for name, at in (("x", (130, 7)), ("delta", (130, 7)), ("z", (130, 7))):
        t = getattr(s, name)
        for bad in (float("nan"), float("inf")):
            keep = t[at].clone()
            t[at] = bad
            y, f = s.forward()
            same = torch.ones_like(y, dtype=torch.bool)
            same[130:190 if name != "z" else 131, 7] = False
            assert torch.equal(y[same], y0[same]), (name, bad)
            if bad != bad and name != "z":
                assert y[130:190, 7].isnan().all() and f[1, 7].isnan().all()
            keepf = torch.ones_like(f, dtype=torch.bool)
            if name != "z":
                keepf[1, 7] = False
            assert torch.equal(f[keepf], f0[keepf]), (name, bad)
            t[at] = keep
    s.B[130, 0, 2] = float("nan")
    y, _ = s.forward()
    assert torch.equal(y[:130], y0[:130]) and torch.equal(y[190:], y0[190:]) and y[130:190].isnan().all()


@MODES
def test_a_step_of_no_length_leaves_the_state(math):
    """delta of the lowest value, or minus infinity: dt = 0, a factor of exactly one and no input."""
    torch = torch_mod()
    s = Scan([80], 16, 1, 16, math, seed=4)
    for low in (float("-inf"), float(torch.finfo(s.dt).min)):
        s.delta[20:70] = low
        ref = ssm_forward(**{**s.host(), "delta": np.maximum(s.host()["delta"], -1e30)})
        y, f = s.forward()
        close(f, ref["final_state"], 5e-6, "state")
        close(y, ref["y"], 5e-6, "y", math == BF16)
        pool = s.init.clone()
        part = [v[None, 20:21] for v in (s.x, s.delta, s.B, s.C)]
        cfc.cfc_ssm_step(part[0], part[1], s.A, part[2], part[3], pool, s.nan(part[0]), math=math)
        assert torch.equal(pool, s.init)


@MODES
def test_the_same_bits_every_time_in_a_graph_and_on_another_stream(math):
    torch = torch_mod()
    s = Scan([300, 0, 70, 1], 72, 1, 16, math, seed=5)
    ws = s.workspace(True)

    def run():
        y, f = s.forward(ws, save=True)
        return [y, f, *s.backward(ws).values()]

    first = run()
    for a, b in zip(first, run()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run()
    side.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    s.x.copy_(s.x * 0.5)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(kept, run()):
        assert torch.equal(a, b)


def test_two_calls_at_once():
    """Two streams, each with its own workspace: nothing is shared."""
    torch = torch_mod()
    a, b = (Scan([400, 300], 256, 1, 16, BF16, seed=i) for i in (6, 7))
    want = []
    for s in (a, b):
        ws = s.workspace(True)
        want.append([*s.forward(ws, save=True), *s.backward(ws).values()])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (s, st) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(st):
                ws = s.workspace(True)
                got[i] = [*s.forward(ws, save=True), *s.backward(ws).values()]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for u, v in zip(w, g):
                assert torch.equal(u, v)


@MODES
def test_rows_behind_the_last_sequence_and_offsets_outside_the_rows(math):
    """Offsets that leave rows behind the last sequence, exceed the rows or fall: nothing outside the tensors is touched,
    and the sequences before them keep their values."""
    torch = torch_mod()
    s = Scan([50, 60, 40], 24, 1, 16, math, seed=8)
    y0, _ = s.forward()
    for off in ([0, 50, 110, 2 ** 31 - 1], [-5, 50, 110, 200], [0, 50, 40, 150], [-2 ** 31, 50, 110, 120]):
        s.so.copy_(torch.tensor(off, dtype=torch.int32))
        ws = s.workspace(True)
        guard = torch.full((s.rows + 64, s.d), 3.0, dtype=s.dt, device="cuda")
        y = guard[32:32 + s.rows]
        final = s.nan(s.gfinal)
        cfc.cfc_ssm_forward(s.x, s.delta, s.A, s.B, s.C, y, ws, D=s.D, z=s.z, delta_bias=s.bias, seq_offsets=s.so,
                            initial_state=s.init, final_state=final, save=True, math=math)
        s.backward(ws)
        assert torch.equal(y[:40], y0[:40]), off
        assert (guard[:32] == 3).all() and (guard[32 + s.rows:] == 3).all()


@MODES
@pytest.mark.parametrize("lens", [[100, 0, 37], [3], [], [0]])
def test_a_padded_batch(lens, math):
    """Rows behind the last sequence are neither read nor written, and add nothing to the sums over rows."""
    torch = torch_mod()
    pad = 200
    s = Scan([*lens, pad], 40, 1, 16, math, seed=12)
    n = len(lens) + 1
    ends = np.concatenate([offsets_of(lens), [sum(lens)]]).astype(np.int32)      # the last sequence is empty
    exact = Scan([*lens, 0], 40, 1, 16, math, seed=12)
    used = sum(lens)
    for name in ("x", "delta", "z", "B", "C", "gy"):
        t = getattr(s, name)
        setattr(exact, name, t[:used].clone())
        t[used:] = float("nan")
    for name in ("A", "D", "bias", "init", "gfinal"):
        setattr(exact, name, getattr(s, name))
    s.so = torch.from_numpy(ends).cuda()
    assert exact.so.tolist() == ends.tolist() and len(ends) == n + 1
    results = []
    for c in (s, exact):
        ws = c.workspace(True)
        y, f = c.forward(ws, save=True)
        results.append(dict(y=y, f=f, **c.backward(ws)))
    for k, v in results[0].items():
        if k in ("y", "grad_x", "grad_delta", "grad_z", "grad_B", "grad_C"):
            assert v[used:].isnan().all(), k
            v = v[:used]
        want = results[1][k]
        top = float(want.abs().max()) if want.numel() else 0.0
        assert torch.isfinite(v).all() and float((v - want).abs().max() if v.numel() else 0) <= (2e-5 if math == FP32 else 2 ** -7) * top, k


def test_offsets_past_32_bits():
    """More than 2^31 values in x: the last rows against the oracle."""
    torch = torch_mod()
    n, t, d, N = 2100, 16, 65536, 1
    g = torch.Generator("cuda").manual_seed(0)
    x = torch.randn(n, t, d, generator=g, device="cuda", dtype=torch.bfloat16)
    delta = torch.randn(n, t, d, generator=g, device="cuda", dtype=torch.bfloat16)
    assert x.numel() > 2 ** 31
    B, C = (torch.randn(n, t, 1, N, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    A = -torch.rand(d, N, generator=g, device="cuda") - 0.1
    y = torch.full_like(x, float("nan"))
    ws = torch.empty(cfc.cfc_ssm_workspace_bytes(n * t, n, d, 1, N, BF16), dtype=torch.uint8, device="cuda")
    cfc.cfc_ssm_forward(x, delta, A, B, C, y, ws, math=BF16)
    part = lambda v: v[-1].double().cpu().numpy()[:, -64:]  # noqa: E731
    bc = lambda v: v[-1].double().cpu().numpy()  # noqa: E731
    ref = ssm_forward(part(x), part(delta), A[-64:].double().cpu().numpy(), bc(B), bc(C), [0, t])
    close(y[-1][:, -64:], ref["y"], 5e-6, "y", True)
    assert not torch.isnan(y[::300]).any()


def test_refusals_of_the_binding():
    torch = torch_mod()
    s = Scan([4, 4], 16, 1, 16, BF16, uniform=True, wide=False)
    ws, y = s.workspace(False), torch.empty_like(s.x)
    call = lambda **kw: cfc.cfc_ssm_forward(**{**dict(x=s.x, delta=s.delta, A=s.A, B=s.B, C=s.C, y=y, workspace=ws), **kw})  # noqa: E731
    call()
    for bad, what in ((dict(delta=s.delta[:, :3]), "delta"), (dict(A=s.A[:8]), "A must"), (dict(C=s.C.transpose(0, 1)), "evenly"),
                      (dict(x=s.x[..., ::2]), "B must|dense|shape"), (dict(D=s.A), "D must"), (dict(z=s.z[..., :8]), "z must"),
                      (dict(seq_offsets=torch.zeros(3, dtype=torch.int32, device="cuda")), "seq_offsets|x must")):
        with pytest.raises(ValueError):
            call(**bad)
            pytest.fail(what)
    with pytest.raises(TypeError):
        call(x=s.x.float())
    with pytest.raises(cfc.CfcError, match="workspace"):
        call(workspace=ws[:8])
    with pytest.raises(cfc.CfcError, match="overlap"):
        call(y=s.delta)
    with pytest.raises(ValueError, match="slots"):
        cfc.cfc_ssm_step(s.x, s.delta, s.A, s.B, s.C, s.init[:, :8], y)
