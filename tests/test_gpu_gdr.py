"""The gated delta rule on the GPU against the 64-bit oracle: whole sequences
forward and backward, and token by token, in both precision modes.

Tolerances, each normwise per tensor (2-norm) with an elementwise guard of ten
times the same figure of max|ref|:

FP32.  Each operand of a product is two TF32 values, 22 bits, and sums are
fp32: about 2^-21 relative a product.  An output is some eight products and
sums from the inputs, and what the state carries is damped by the decays:
8 x 2^-21 = 4e-6; 1e-5 allows for the inverse's condition.  grad_g is a
difference of sums of that accuracy that are a few times larger: 5e-5.

BF16.  A rounding to bf16 is 2^-8 at most and 0.42 of that, 1.6e-3, in the root
mean square.  o is rounded once and depends on four operands that are (S, R, U,
P T): sqrt(5) x 1.6e-3 = 3.6e-3, allowed 6e-3.  The gradients have about nine in
both directions: 4.9e-3, allowed 1e-2; grad_g and grad_beta, differences of sums:
2e-2.  A final state that is asked for keeps 17 bits on its way, 2^-17 = 8e-6 an
operand: 3e-5.  grad_initial_state comes of the bf16 chain back: as the gradients.

The step is fp32 throughout: state 3e-6; o the same in FP32, and in BF16 one rounding:
2e-3.
"""

import numpy as np
import pytest

import recurrent_cell_gb300 as cfc
from oracle.gdr_oracle import gdr_backward, gdr_forward

from gpu_common import require_gpu, torch_mod

pytestmark = pytest.mark.gpu

FP32, BF16 = cfc.MATH_FP32, cfc.MATH_BF16
MODES = pytest.mark.parametrize("math", [FP32, BF16], ids=["fp32", "bf16"])
GRADS = ("grad_q", "grad_k", "grad_v", "grad_g", "grad_beta")


def tolerance(name, math):
    if math == FP32:
        return 5e-5 if name == "grad_g" else 1e-5
    return {"o": 6e-3, "final_state": 3e-5, "grad_g": 2e-2, "grad_beta": 2e-2}.get(name, 1e-2)


def close(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, what
    if not ref.size:
        return
    assert np.isfinite(got).all(), what
    off, norm = np.linalg.norm(got - ref), np.linalg.norm(ref)
    assert off <= tol * norm, f"{what}: {off / norm if norm else off:.2e} of the norm, {tol:.0e} allowed"
    assert np.abs(got - ref).max() <= 10 * tol * np.abs(ref).max(), what


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    assert cfc.cfc_device_error(clear=True) == 0


class Case:
    """Inputs of one packed batch, rounded to the mode's type, on both sides."""

    def __init__(self, lens, hk, hv, dk, dv, math, seed=0, init=False, decay=0.3):
        torch = torch_mod()
        self.math, self.dtype = math, torch.float32 if math == FP32 else torch.bfloat16
        self.hk, self.hv, self.dk, self.dv = hk, hv, dk, dv
        self.off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.n, self.rows = len(lens), int(self.off[-1])
        rng = np.random.default_rng(seed)
        unit = lambda a: a / np.linalg.norm(a, axis=-1, keepdims=True)  # noqa: E731
        self.rng, self.scale = rng, dk ** -0.5
        self.q = self.rounded(unit(rng.standard_normal((self.rows, hk, dk))))
        self.k = self.rounded(unit(rng.standard_normal((self.rows, hk, dk))))
        self.v = self.rounded(rng.standard_normal((self.rows, hv, dv)))
        self.g = torch.from_numpy(-decay * rng.uniform(0, 1, (self.rows, hv))).float()
        self.beta = torch.from_numpy(rng.uniform(0, 1, (self.rows, hv))).float()
        self.init = torch.from_numpy(rng.standard_normal((self.n, hv, dk, dv))).float() if init else None
        self.go = self.rounded(rng.standard_normal((self.rows, hv, dv)))

    def rounded(self, a):
        return torch_mod().from_numpy(np.ascontiguousarray(a)).to(self.dtype)

    def inputs(self):
        return [self.q, self.k, self.v, self.g, self.beta]

    def host(self):
        return [a.double().numpy() for a in self.inputs()]

    def oracle(self):
        return gdr_forward(*self.host(), self.scale, self.off, None if self.init is None else self.init.numpy())

    def oracle_back(self, gfinal=None):
        return gdr_backward(*self.host(), self.scale, self.off, self.go.double().numpy(),
                            None if self.init is None else self.init.numpy(), gfinal)

    def workspace(self, save, fill=255):
        torch = torch_mod()
        size = cfc.cfc_gdr_workspace_bytes(self.rows, self.n, self.hk, self.hv, self.dk, self.dv, self.math, save)
        assert size > 0
        return torch.full((size,), fill, dtype=torch.uint8, device="cuda")     # NaN wherever nothing is written

    def forward(self, final=True, save=False, packed=True, stream=None):
        torch = torch_mod()
        self.dev = [a.cuda() for a in self.inputs()]
        self.ws = self.workspace(save)
        o = torch.full_like(self.dev[2], float("nan"))
        init = None if self.init is None else self.init.cuda()
        fin = torch.full((self.n, self.hv, self.dk, self.dv), float("nan"), device="cuda") if final else None
        self.offsets = torch.from_numpy(self.off).cuda() if packed else None
        args = self.dev + [o]
        if not packed:
            args = [a.unflatten(0, (self.n, self.rows // self.n)) for a in args]
        torch.cuda.synchronize()            # the call may run on another stream
        cfc.cfc_gdr_forward(*args, self.ws, seq_offsets=self.offsets, initial_state=init, final_state=fin, save=save,
                            math=self.math, stream=stream)
        torch.cuda.synchronize()
        return {"o": o.cpu().double().numpy(), "final_state": fin.cpu().double().numpy() if final else None}

    def backward(self, gfinal=None, packed=True):
        torch = torch_mod()
        like = lambda a: torch.full(a.shape, float("nan"), dtype=self.dtype, device="cuda")  # noqa: E731
        out = {n: like(a) for n, a in zip(GRADS, self.dev)}
        ginit = torch.full((self.n, self.hv, self.dk, self.dv), float("nan"), device="cuda")
        args = self.dev + [self.go.cuda()] + list(out.values())
        if not packed:
            args = [a.unflatten(0, (self.n, self.rows // self.n)) for a in args]
        gf = None if gfinal is None else torch.from_numpy(gfinal).float().cuda()
        cfc.cfc_gdr_backward(*args, self.ws, seq_offsets=self.offsets, grad_final_state=gf, grad_initial_state=ginit,
                             math=self.math)
        torch.cuda.synchronize()
        r = {n: a.cpu().double().numpy() for n, a in out.items()}
        r["grad_initial_state"] = ginit.cpu().double().numpy()
        return r

    def check(self, got, ref, names, what=""):
        for n in names:
            close(got[n], ref[n], tolerance(n, self.math), f"{what}{n}")


SHAPES = [(1, 1, 8, 8), (2, 2, 64, 64), (2, 6, 40, 72), (1, 2, 128, 256), (3, 3, 72, 136), (1, 4, 128, 128)]
LENGTHS = [[1], [63], [64], [65], [0, 1, 64, 0, 130, 2], [200, 5]]


@MODES
@pytest.mark.parametrize("init", [False, True], ids=["zero", "carried"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, init, math):
    for lens in LENGTHS:
        c = Case(lens, *shape, math, seed=len(lens), init=init)
        ref = c.oracle()
        c.check(c.forward(), ref, ("o", "final_state"), f"{lens} ")
        c.check(c.forward(final=False), ref, ("o",), f"{lens} without a final state: ")


@MODES
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, math):
    for lens in LENGTHS:
        c = Case(lens, *shape, math, seed=7 + len(lens))
        ref = c.oracle_back()
        c.check(c.forward(final=False, save=True), c.oracle(), ("o",), f"{lens} ")
        c.check(c.backward(), ref, GRADS + ("grad_initial_state",), f"{lens} ")
        c.check(c.forward(final=True, save=True), c.oracle(), ("o", "final_state"), f"{lens} ")
        c.check(c.backward(), ref, GRADS + ("grad_initial_state",), f"{lens} after a final state ")


@MODES
def test_gradients_of_carried_and_leaving_states(math):
    """Both states take part, and the forward that saves also gives the final one."""
    for lens in ([70, 0, 1, 128],):
        c = Case(lens, 2, 4, 64, 96, math, seed=3, init=True)
        gf = np.float32(c.rng.standard_normal((c.n, c.hv, c.dk, c.dv)))
        c.check(c.forward(final=True, save=True), c.oracle(), ("o", "final_state"))
        ref = c.oracle_back(gf)
        got = c.backward(gf)
        c.check(got, ref, GRADS + ("grad_initial_state",))
        np.testing.assert_allclose(got["grad_initial_state"][1], gf[1], rtol=1e-6)     # an empty sequence hands it on


@MODES
def test_many_heads_take_the_wide_tiles(math):
    """Enough sequences and heads to fill the GPU: the other side of every choice of tile."""
    c = Case([66] * 10 + [0, 129], 8, 16, 64, 128, math, seed=5)
    ref = c.oracle()
    c.check(c.forward(), ref, ("o", "final_state"))
    c.check(c.forward(final=False, save=True), ref, ("o",))
    c.check(c.backward(), c.oracle_back(), GRADS + ("grad_initial_state",))


def test_widest_heads_fill_the_gpu_in_bf16():
    c = Case([65] * 8, 16, 16, 128, 128, BF16, seed=6)
    c.check(c.forward(), c.oracle(), ("o", "final_state"))
    c.check(c.forward(final=False, save=True), c.oracle(), ("o",))
    c.check(c.backward(), c.oracle_back(), GRADS)


@MODES
def test_uniform_sequences_equal_packed_ones(math):
    c = Case([77] * 3, 2, 2, 64, 64, math, seed=8, init=True)
    a, ga = c.forward(save=True), c.backward()
    b, gb = c.forward(save=True, packed=False), c.backward(packed=False)
    for x, y in ((a, b), (ga, gb)):
        for n in x:
            assert np.isfinite(x[n]).all(), n
            np.testing.assert_array_equal(x[n], y[n], err_msg=n)


@MODES
def test_decays_from_none_to_total(math):
    """g = 0, tiny, large, -inf (a reset, in the middle of a chunk, at its ends, alone) and
    beta = 0 and 1."""
    c = Case([150, 64, 1], 1, 2, 64, 64, math, seed=9, init=True)
    g = c.g
    g[5:40] = 0
    g[40:60] = -1e-6
    g[60, 0] = g[64, 0] = g[100, 1] = g[127, 0] = g[128, 0] = g[150, 1] = g[213, 0] = g[214, 0] = -np.inf
    g[61, 0], g[70, 1], g[110, 0] = -500.0, -3e38, -90.0
    c.beta[20:30] = 0
    c.beta[30:50] = 1
    ref = c.oracle()
    c.check(c.forward(), ref, ("o", "final_state"))
    c.check(c.forward(final=False, save=True), ref, ("o",))
    got, ref = c.backward(), c.oracle_back()
    c.check(got, ref, GRADS + ("grad_initial_state",))
    assert (got["grad_g"][np.isneginf(g.numpy())] == 0).all()


@MODES
def test_strong_decays_leave_single_tokens(math):
    """Sums of g down to -64 x 80: exp(G) underflows inside a chunk, ratios do not."""
    c = Case([130], 1, 1, 32, 32, math, seed=10, decay=160.0)
    c.check(c.forward(), c.oracle(), ("o", "final_state"))
    c.forward(final=False, save=True)
    got, ref = c.backward(), c.oracle_back()
    c.check(got, ref, ("grad_q", "grad_k", "grad_v", "grad_beta"))
    # grad_g is small here against the terms that it is a difference of
    x = c.host()
    terms = np.abs(x[0] * ref["grad_q"]).sum(-1) + np.abs(x[1] * ref["grad_k"]).sum(-1)
    assert np.abs(got["grad_g"] - ref["grad_g"]).max() <= tolerance("grad_g", math) * terms.max()


@MODES
def test_repeated_and_opposite_keys(math):
    """The inverse of a chunk is far from the identity when keys repeat: beta |k|^2 = 1 and up to 2.
    The state is then a sum of 64 updates up to twice its size that nearly cancel:
    its error is 2 sqrt(64) = 16 roundings of an update, ten times the usual allowance."""
    for beta, tag in ((1.0, "replace"), (1.9, "reflect")):
        c = Case([100], 1, 1, 64, 32, math, seed=11, decay=0.0 if beta == 1 else 0.2)
        key = np.zeros(64)
        key[3], key[40] = 0.5, np.sqrt(0.75)
        c.k = c.rounded(np.where(np.arange(100)[:, None, None] % 3 == 2, -key, key))
        c.beta[:] = beta
        got, ref = c.forward(), c.oracle()
        for n in ("o", "final_state"):
            close(got[n], ref[n], 10 * tolerance(n, math), f"{tag} {n}")


@MODES
def test_gradient_of_first_tokens_decay_is_exactly_zero(math):
    c = Case([1] * 5 + [70], 1, 2, 64, 64, math, seed=12)
    c.forward(final=False, save=True)
    got = c.backward()
    first = c.off[:-1]
    assert (got["grad_g"][first] == 0).all()
    c.check(got, c.oracle_back(), GRADS)


def test_gradients_match_differences():
    """The FP32 gradients against central differences of the 64-bit forward along
    random directions.  Each is off by 1e-5 (grad_g 5e-5) of |grad| |direction| at
    most, and the differences by the rounding of a loss of order 100: 1e-13 / 1e-5."""
    c = Case([66, 3], 1, 2, 32, 24, FP32, seed=13, init=True)
    gf = np.float32(c.rng.standard_normal((c.n, c.hv, c.dk, c.dv)))
    c.forward(save=True)
    got = c.backward(gf)
    x, go, init = c.host(), c.go.double().numpy(), c.init.double().numpy()

    def loss(x, init):
        r = gdr_forward(*x, c.scale, c.off, init)
        return (r["o"] * go).sum() + (r["final_state"] * gf).sum()

    for i, n in enumerate(GRADS + ("grad_initial_state",)):
        a = (x + [init])[i]
        for _ in range(3):
            d = c.rng.standard_normal(a.shape)
            up, down = ([*x[:i], a + s * d, *x[i + 1:]] if i < 5 else x for s in (1e-5, -1e-5))
            fd = (loss(up, init + 1e-5 * d if i == 5 else init) - loss(down, init - 1e-5 * d if i == 5 else init)) / 2e-5
            allowed = tolerance(n, FP32) * np.linalg.norm(got[n]) * np.linalg.norm(d) + 1e-6
            assert abs((got[n] * d).sum() - fd) <= allowed, (n, fd)


@MODES
def test_one_sequences_nan_reaches_no_other(math):
    lens = [70, 65, 3, 64]
    c = Case(lens, 2, 2, 64, 64, math, seed=14, init=True)
    clean, gclean = c.forward(save=True), c.backward()
    for bad in (float("nan"), float("inf")):
        c.q[75, 0, 3] = c.k[75, 1, 5] = c.v[80, 0, 1] = c.go[90, 0, 0] = bad
        c.g[76, 0] = c.beta[77, 1] = float("nan")
        c.init[1, 0, 0, 0] = bad
        got = {**c.forward(save=True), **c.backward()}
        lo, hi = c.off[1], c.off[2]
        for n, a in {**clean, **gclean}.items():
            if n in ("final_state", "grad_initial_state"):
                np.testing.assert_array_equal(got[n][[0, 2, 3]], a[[0, 2, 3]], err_msg=n)
            else:
                np.testing.assert_array_equal(got[n][:lo], a[:lo], err_msg=n)
                np.testing.assert_array_equal(got[n][hi:], a[hi:], err_msg=n)
        assert np.isnan(got["o"][lo:hi]).any()


@MODES
def test_inputs_may_be_parts_of_one_projection(math):
    torch = torch_mod()
    hk, hv, dk, dv, rows = 2, 4, 64, 40, 133
    c = Case([rows], hk, hv, dk, dv, math, seed=15)
    dense, gdense = c.forward(save=True), c.backward()
    wide = torch.full((rows, 2 * hk * dk + hv * dv + 24), float("nan"), dtype=c.dtype, device="cuda")
    parts, at = [], 8
    for a in (c.q, c.k, c.v):
        w = a.shape[1] * a.shape[2]
        wide[:, at:at + w] = a.cuda().reshape(rows, w)
        parts.append(wide[:, at:at + w].unflatten(1, a.shape[1:]))
        at += w
    assert not parts[0].is_contiguous()
    o = torch.empty_like(c.dev[2])
    ws = c.workspace(True)
    fin = torch.empty(1, hv, dk, dv, device="cuda")         # asked for as above: the same operands' width
    cfc.cfc_gdr_forward(*parts, *c.dev[3:], o, ws, seq_offsets=c.offsets, final_state=fin, save=True, math=math)
    grads = [torch.empty(a.shape, dtype=c.dtype, device="cuda") for a in c.dev]
    cfc.cfc_gdr_backward(*parts, *c.dev[3:], c.go.cuda(), *grads, ws, seq_offsets=c.offsets, math=math)
    close(o.cpu().double(), c.oracle()["o"], tolerance("o", math), "o")
    for n, a in zip(GRADS, grads):
        np.testing.assert_array_equal(a.cpu().double().numpy(), gdense[n], err_msg=n)
    # [sequences, tokens, ...] views of it too
    o4 = torch.empty(1, rows, hv, dv, dtype=c.dtype, device="cuda")
    cfc.cfc_gdr_forward(*[p[None] for p in parts], *[a[None] for a in c.dev[3:]], o4, c.workspace(False), math=math)
    close(o4[0].cpu().double(), dense["o"], tolerance("o", math), "o")


@MODES
def test_initial_and_final_state_may_be_one_buffer(math):
    torch = torch_mod()
    c = Case([100, 0, 30], 1, 2, 64, 64, math, seed=16, init=True)
    apart = c.forward()
    both = c.init.cuda()
    o = torch.empty_like(c.dev[2])
    cfc.cfc_gdr_forward(*c.dev, o, c.workspace(False), seq_offsets=c.offsets, initial_state=both, final_state=both, math=math)
    np.testing.assert_array_equal(both.cpu().double().numpy(), apart["final_state"])
    np.testing.assert_array_equal(apart["final_state"][1], c.init[1].numpy())


@MODES
def test_a_sequence_in_two_parts_equals_the_whole(math):
    """The state handed from one call to the next, cut inside a chunk."""
    torch = torch_mod()
    c = Case([150], 2, 2, 64, 64, math, seed=17)
    whole = c.oracle()
    state = torch.zeros(1, 2, 64, 64, device="cuda")
    got = []
    for lo, hi in ((0, 70), (70, 71), (71, 150)):
        p = [a[lo:hi].cuda()[None] for a in c.inputs()]
        o = torch.empty_like(p[2])
        ws = torch.empty(cfc.cfc_gdr_workspace_bytes(hi - lo, 1, 2, 2, 64, 64, math), dtype=torch.uint8, device="cuda")
        cfc.cfc_gdr_forward(*p, o, ws, initial_state=state, final_state=state, math=math)
        got.append(o[0].cpu())
    close(torch.cat(got).double(), whole["o"], tolerance("o", math), "o")
    close(state.cpu().double(), whole["final_state"], tolerance("final_state", math), "state")


@MODES
def test_rows_zero(math):
    torch = torch_mod()
    c = Case([0, 0], 1, 1, 32, 32, math, seed=18, init=True)
    got = c.forward(save=True)
    np.testing.assert_array_equal(got["final_state"], c.init.numpy())
    gf = np.float32(c.rng.standard_normal((2, 1, 32, 32)))
    np.testing.assert_array_equal(c.backward(gf)["grad_initial_state"], gf)


@MODES
def test_offsets_outside_the_rows_are_held_to_them(math):
    """Wrong offsets touch nothing outside: sequences end at the last row, and one that would
    begin after its end is empty."""
    torch = torch_mod()
    c = Case([40, 60], 1, 1, 32, 32, math, seed=19)
    c.forward()
    guard = torch.full((3, 100, 1, 32), 7.0, dtype=c.dtype, device="cuda")
    off = torch.tensor([-50, 40, 100000], dtype=torch.int32, device="cuda")
    cfc.cfc_gdr_forward(*c.dev, guard[1], c.workspace(False), seq_offsets=off, math=math)
    close(guard[1].cpu().double(), c.oracle()["o"], tolerance("o", math), "o")
    off = torch.tensor([2 ** 31 - 1, -2 ** 31, 50], dtype=torch.int32, device="cuda")
    cfc.cfc_gdr_forward(*c.dev, guard[1], c.workspace(False), seq_offsets=off, math=math)
    torch.cuda.synchronize()
    assert (guard[0] == 7).all() and (guard[2] == 7).all()


@MODES
def test_same_bits_every_time_and_on_another_stream(math):
    torch = torch_mod()
    c = Case([200, 33, 64], 2, 6, 64, 72, math, seed=20)
    a, ga = c.forward(save=True), c.backward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b, gb = c.forward(save=True, stream=side), c.backward()
    for x, y in ((a, b), (ga, gb)):
        for n in x:
            assert np.isfinite(x[n]).all(), n
            np.testing.assert_array_equal(x[n], y[n], err_msg=n)


@MODES
def test_captured_calls_replay_on_new_inputs(math):
    torch = torch_mod()
    c = Case([90, 70], 1, 2, 64, 64, math, seed=21)
    c.forward(final=False, save=True)
    o = torch.empty_like(c.dev[2])
    go = c.go.cuda()
    grads = [torch.empty(a.shape, dtype=c.dtype, device="cuda") for a in c.dev]

    def step():
        cfc.cfc_gdr_forward(*c.dev, o, c.ws, seq_offsets=c.offsets, save=True, math=math)
        cfc.cfc_gdr_backward(*c.dev, go, *grads, c.ws, seq_offsets=c.offsets, math=math)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    d = Case([90, 70], 1, 2, 64, 64, math, seed=22)
    ref = d.forward(final=False, save=True)
    gref = d.backward()
    for x, y in zip(c.dev, d.dev):
        x.copy_(y)
    go.copy_(d.go.cuda())
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(o.cpu().double().numpy(), ref["o"])
    for n, a in zip(GRADS, grads):
        np.testing.assert_array_equal(a.cpu().double().numpy(), gref[n], err_msg=n)


def test_more_sequences_than_are_ordered():
    """Packed batches beyond the longest-first order's limit, most of them empty or short."""
    rng = np.random.default_rng(23)
    lens = np.where(rng.uniform(size=2100) < 0.9, rng.integers(0, 3, 2100), 0)
    lens[2000] = 100
    c = Case(lens.tolist(), 1, 1, 16, 16, BF16, seed=23)
    c.check(c.forward(), c.oracle(), ("o", "final_state"))
    c.forward(final=False, save=True)
    c.check(c.backward(), c.oracle_back(), GRADS)


# ------------------------------------------------------------------- the step
def step_tolerance(name, math):
    return 2e-3 if name == "o" and math == BF16 else 3e-6


def run_step(c, tokens, state, slots=None):
    torch = torch_mod()
    dev = [a.cuda().unflatten(0, (c.n, tokens)) for a in c.inputs()]
    o = torch.full_like(dev[2], float("nan"))
    cfc.cfc_gdr_step(*dev, state, o, slots=slots, math=c.math)
    torch.cuda.synchronize()
    return o.flatten(0, 1).cpu().double().numpy()


@MODES
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("tokens", [1, 2, 5])
def test_step(tokens, shape, math):
    c = Case([tokens] * 3, *shape, math, seed=30 + tokens, init=True)
    state = c.init.cuda()
    o = run_step(c, tokens, state)
    ref = c.oracle()
    close(o, ref["o"], step_tolerance("o", math), "o")
    close(state.cpu().double(), ref["final_state"], step_tolerance("state", math), "state")


@MODES
def test_step_of_many_heads(math):
    c = Case([1] * 80, 8, 16, 128, 128, math, seed=36, init=True)
    state = c.init.cuda()
    o = run_step(c, 1, state)
    ref = c.oracle()
    close(o, ref["o"], step_tolerance("o", math), "o")
    close(state.cpu().double(), ref["final_state"], step_tolerance("state", math), "state")


@MODES
def test_step_by_step_equals_the_whole_sequence(math):
    c = Case([70, 70], 1, 3, 64, 64, math, seed=37)
    torch = torch_mod()
    state = torch.zeros(2, 3, 64, 64, device="cuda")
    whole = c.forward()
    dev = [a.unflatten(0, (2, 70)) for a in c.dev]
    o = torch.empty_like(dev[2])
    for t in range(70):
        one = torch.empty_like(dev[2][:, :1])
        cfc.cfc_gdr_step(*[a[:, t:t + 1].contiguous() for a in dev], state, one, math=math)
        o[:, t:t + 1] = one
    close(o.flatten(0, 1).cpu().double(), whole["o"], 2 * tolerance("o", math), "o")
    close(state.cpu().double(), whole["final_state"], 2 * tolerance("final_state", math), "state")


@MODES
def test_step_slots(math):
    """Sequences in any slot; one without a slot gives zeros and keeps nothing, and no
    other slot changes."""
    torch = torch_mod()
    c = Case([2] * 5, 1, 2, 64, 32, math, seed=38, init=True)
    pool = torch.randn(9, 2, 64, 32, device="cuda")
    slots = torch.tensor([7, -1, 0, 9, 3], dtype=torch.int32, device="cuda")
    for i, s in ((0, 7), (2, 0), (4, 3)):
        pool[s] = c.init[i].cuda()
    before = pool.clone()
    o = run_step(c, 2, pool, slots)
    ref = c.oracle()
    rows = [0, 1, 4, 5, 8, 9]
    close(o[rows], ref["o"][rows], step_tolerance("o", math), "o")
    for i, s in ((0, 7), (2, 0), (4, 3)):
        close(pool[s].cpu().double(), ref["final_state"][i], step_tolerance("state", math), "state")
    assert (o[2:4] == 0).all() and (o[6:8] == 0).all()
    rest = [1, 2, 4, 5, 6, 8]
    assert torch.equal(pool[rest], before[rest])


@MODES
def test_step_resets_and_zero_sizes(math):
    torch = torch_mod()
    c = Case([3, 3], 1, 1, 64, 64, math, seed=39, init=True)
    c.g[1, 0] = c.g[3, 0] = -np.inf
    state = c.init.cuda()
    o = run_step(c, 3, state)
    ref = c.oracle()
    close(o, ref["o"], step_tolerance("o", math), "o")
    close(state.cpu().double(), ref["final_state"], step_tolerance("state", math), "state")
    e = lambda *s, t=c.dtype: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    before = state.clone()
    for n, t in ((0, 1), (2, 0)):
        cfc.cfc_gdr_step(e(n, t, 1, 64), e(n, t, 1, 64), e(n, t, 1, 64), e(n, t, 1, t=torch.float32),
                         e(n, t, 1, t=torch.float32), state, e(n, t, 1, 64), math=math)
    torch.cuda.synchronize()
    assert torch.equal(state, before)


def test_step_state_beyond_32_bit_offsets():
    """A pool of more than 2^31 elements; the slot at its far end."""
    torch = torch_mod()
    per = 64 * 128 * 128
    slots = 2 ** 31 // per + 3
    c = Case([1, 1], 64, 64, 128, 128, BF16, seed=40, init=True)
    pool = torch.empty(slots, 64, 128, 128, device="cuda")
    pool[slots - 1], pool[0] = c.init[0].cuda(), c.init[1].cuda()
    o = run_step(c, 1, pool, torch.tensor([slots - 1, 0], dtype=torch.int32, device="cuda"))
    ref = c.oracle()
    close(o, ref["o"], step_tolerance("o", BF16), "o")
    close(pool[slots - 1].cpu().double(), ref["final_state"][0], step_tolerance("state", BF16), "state")


def test_rows_far_apart_pass_32_bit_offsets():
    """Row strides that carry later rows past 2^31 elements."""
    torch = torch_mod()
    rows, hk, dk = 70, 1, 64
    c = Case([rows], hk, 1, dk, 64, BF16, seed=41)
    ref = c.oracle()
    c.forward()
    ld = (2 ** 31 // rows + 64) // 64 * 64 + 64
    far = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    views = []
    for i, a in enumerate(c.dev[:3]):
        v = torch.as_strided(far, (rows, 1, 64), (ld, 64, 1), 64 * i)
        v.copy_(a)
        views.append(v)
    o = torch.empty_like(c.dev[2])
    cfc.cfc_gdr_forward(*views, *c.dev[3:], o, c.workspace(False), seq_offsets=c.offsets, math=BF16)
    close(o.cpu().double(), ref["o"], tolerance("o", BF16), "o")


def test_binding_refuses_what_does_not_fit():
    torch = torch_mod()
    c = Case([10], 1, 2, 32, 32, BF16, seed=42)
    c.forward()
    q, k, v, g, beta = c.dev
    o, ws, off = torch.empty_like(v), c.ws, c.offsets
    bad = [
        (TypeError, (q.float(), k, v, g, beta, o, ws), {}),
        (TypeError, (q, k, v, g.bfloat16(), beta, o, ws), {}),
        (TypeError, (q.cpu(), k, v, g, beta, o, ws), {}),
        (ValueError, (q[:5], k, v, g, beta, o, ws), {}),
        (ValueError, (q, k, v, g[:, :1], beta, o, ws), {}),
        (ValueError, (q, k, v.transpose(1, 2).contiguous().transpose(1, 2), g, beta, o, ws), {}),
        (ValueError, (q, k[:, :, :24], v, g, beta, o, ws), {}),
        (ValueError, (q, k, v, g, beta, o, ws), {"final_state": torch.empty(1, 2, 32, 16, device="cuda")}),
        (cfc.CfcError, (q, k, v, g, beta, o, ws[:64]), {}),
        (cfc.CfcError, (q, k, v, g, beta, o, ws), {"math": cfc.MATH_TF32}),
    ]
    for err, args, kw in bad:
        with pytest.raises((err, TypeError, ValueError) if err is cfc.CfcError else err):
            cfc.cfc_gdr_forward(*args, seq_offsets=off, **kw)
    with pytest.raises(ValueError):
        cfc.cfc_gdr_forward(*c.dev, o, ws)                                  # rows without offsets
    with pytest.raises(ValueError):
        cfc.cfc_gdr_step(*[a[None] for a in c.dev], torch.empty(1, 2, 16, 32, device="cuda"), o[None])


@pytest.mark.parametrize("shape", [(3, 3, 72, 136), (2, 6, 64, 96), (1, 2, 128, 256), (2, 2, 64, 64)], ids=str)
def test_bits_depend_neither_on_the_run_nor_on_what_the_workspace_held(shape):
    """Blocks with one, two, three and four tiles of value columns, whole and partial chunks."""
    torch = torch_mod()
    c = Case([64, 200, 5], *shape, BF16, seed=43)
    c.forward(final=False, save=True)
    go = c.go.cuda()
    first = None
    for run in range(40):
        ws = c.workspace(True, fill=(255, 0, 63, 1)[run % 4])
        o = torch.empty_like(c.dev[2])
        grads = [torch.empty(a.shape, dtype=c.dtype, device="cuda") for a in c.dev]
        cfc.cfc_gdr_forward(*c.dev, o, ws, seq_offsets=c.offsets, save=True, math=BF16)
        cfc.cfc_gdr_backward(*c.dev, go, *grads, ws, seq_offsets=c.offsets, math=BF16)
        if first is None:
            first = [o] + grads
            c.check({"o": o.cpu().double()}, c.oracle(), ("o",))
        for a, b in zip(first, [o] + grads):
            assert torch.equal(a, b), run


@pytest.mark.parametrize("dv", [96, 128])
def test_one_long_sequence_among_many_heads(dv):
    """Far longer than an even share: it takes tiles of half the width, beside others of the whole."""
    c = Case([3, 700, 0, 64, 10], 12, 24, 32, dv, BF16, seed=44, init=True)
    ref = c.oracle()
    c.check(c.forward(), ref, ("o", "final_state"))
    for final in (False, True):
        c.check(c.forward(final=final, save=True), ref, ("o", "final_state") if final else ("o",))
        c.check(c.backward(), c.oracle_back(), GRADS + ("grad_initial_state",), f"final state {final}: ")


@pytest.mark.parametrize("beta,decay", [(1.0, 0.0), (1.9, 0.0), (1.9, 0.2), (2.0, 0.0)])
def test_repeated_and_opposite_keys_in_training(beta, decay):
    """One chunk from the zero state, no final state asked for.  T's entries reach 2 and its rows
    nearly cancel, so T has to be exact before it is rounded, and P T formed from
    more than bf16's bits: then o has the roundings of P T, R and its own, and grad_v, grad_k no more than
    elsewhere.  dq and dbeta go by S^T k, a sum of 64 updates that nearly cancel: ten times the allowance, as
    above.  dg is a difference of the terms in the last line, and is 0 where each token replaces the one before."""
    c = Case([64, 40, 64, 17], 1, 2, 64, 32, BF16, seed=45, decay=decay)
    key = np.zeros(64)
    key[3], key[40] = 0.5, np.sqrt(0.75)
    c.k = c.rounded(np.where(np.arange(c.rows)[:, None, None] % 3 == 2, -key, key))
    c.beta[:] = beta
    got, ref = c.forward(final=False, save=True), c.oracle()
    close(got["o"], ref["o"], tolerance("o", BF16), "o")
    got, ref = c.backward(), c.oracle_back()
    for n in ("grad_v", "grad_k"):
        close(got[n], ref[n], tolerance(n, BF16), n)
    for n in ("grad_q", "grad_beta"):
        close(got[n], ref[n], 10 * tolerance(n, BF16), n)
    x = c.host()
    terms = np.abs(x[0] * ref["grad_q"]).sum(-1) + np.abs(x[1] * ref["grad_k"]).sum(-1)
    assert np.abs(got["grad_g"] - ref["grad_g"]).max() <= 10 * tolerance("grad_g", BF16) * terms.max()


@MODES
@pytest.mark.parametrize("kind", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("many", [False, True], ids=["few heads", "many heads"])
def test_a_bad_token_reaches_no_earlier_one(many, kind, math):
    """A NaN or an infinity at one token reaches what the recurrence hands it to, and nothing else: not the
    tokens before it in its chunk, not other heads, nor other columns where it is in v.  Everything
    that stays finite has the same bits as without it."""
    lens, shape = ([66] * 9 + [150], (8, 16, 64, 128)) if many else ([70, 150], (2, 4, 64, 96))
    c = Case(lens, *shape, math, seed=46, init=True)
    first = c.off[-2]                               # of the last sequence
    for final in (True, False):
        clean = c.forward(final=final, save=not final)
        for at, bad in ((37, float("nan")), (64 + 21, float("inf")), (149, float("nan"))):
            if kind == "g" and bad == float("inf"):
                bad = float("nan")                  # the log-decay is at most 0
            t = {"q": c.q, "k": c.k, "v": c.v, "g": c.g, "beta": c.beta}[kind]
            i = (first + at, 1, 13)[:t.dim()]
            was = t[i].clone()
            t[i] = bad
            got = c.forward(final=final, save=not final)
            with np.errstate(invalid="ignore", over="ignore"):
                ref = c.oracle()
            t[i] = was
            for n in ("o", "final_state") if final else ("o",):
                fine = np.isfinite(ref[n])
                np.testing.assert_array_equal(np.isfinite(got[n]), fine, err_msg=f"{n} {at} {bad}")
                np.testing.assert_array_equal(got[n][fine], clean[n][fine], err_msg=f"{n} {at} {bad}")
            assert not np.isfinite(ref["o"][i[0]]).all()


@MODES
def test_an_overflow_inside_a_chunk_is_not_hidden(math):
    """Finite keys whose product passes fp32's range: what follows is not finite, what came before is right."""
    c = Case([60], 1, 1, 64, 32, math, seed=47)
    c.g[:] = 0
    c.beta[:] = 0.5
    clean = c.forward()
    c.k[40] = c.k[30] = c.k[30] * 1e25
    got = c.forward()
    np.testing.assert_array_equal(got["o"][:30], clean["o"][:30])
    assert not np.isfinite(got["o"][40:]).any() and not np.isfinite(got["final_state"]).any()
