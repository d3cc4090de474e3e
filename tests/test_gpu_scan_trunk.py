"""The trunk of scan blocks in front of the cell, as it is used: its gradients against the same block in 64-bit torch,
packed sequences and states handed on, decoding against whole sequences, training with clipped gradients.

FP32 tolerance 2e-4 normwise, as for the trunk of rules: the library's operators are good to 1e-5 each (their own
tests) and torch's fp32 products to 1e-6; four of the former lie on a path.  Decoding sums in another order: 1e-4 of
the largest value, in bf16 a few steps of a value."""

import numpy as np
import pytest

from gpu_common import require_gpu, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def exact_block(block, delta, stream):
    """ScanBlock.forward in plain torch, token by token, in the parameters' type (float64)."""
    torch = torch_mod()
    inner, states, rank, width = block.sizes
    s = delta if stream is None else delta + stream
    y = torch.nn.functional.layer_norm(s, s.shape[-1:], block.norm, block.norm_bias, 1e-5)
    x, z = (y @ block.w_in).chunk(2, -1)
    n, T = x.shape[:2]
    seen = torch.cat([torch.zeros(n, width - 1, inner, dtype=x.dtype), x], 1)
    x = torch.nn.functional.silu(sum(seen[:, j:j + T] * block.conv[:, j] for j in range(width)) + block.conv_bias)
    r, B, C = (x @ block.w_x).split([rank, states, states], -1)
    dt = torch.nn.functional.softplus(r @ block.w_dt + block.dt_bias)
    A, h, out = -torch.exp(block.A_log), torch.zeros(n, inner, states, dtype=x.dtype), []
    for t in range(T):
        h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * x[:, t])[..., None] * B[:, t, None]
        out.append((h * C[:, t, None]).sum(-1) + block.D * x[:, t])
    return (torch.stack(out, 1) * torch.nn.functional.silu(z)) @ block.w_out, s


def near(a, b, tol, what):
    a, b = a.detach().cpu().double().numpy(), b.detach().double().numpy()
    assert np.linalg.norm(a - b) <= tol * np.linalg.norm(b), f"{what}: {np.linalg.norm(a - b) / np.linalg.norm(b):.1e}"


def test_two_blocks_match_plain_torch_in_64_bits():
    torch = torch_mod()
    from recurrent_cell_gb300.memory import ScanBlock
    torch.manual_seed(0)
    blocks = [ScanBlock(48, dtype=torch.float32) for _ in range(2)]
    exact = [ScanBlock(48, dtype=torch.float64, device="cpu") for _ in range(2)]
    for b, e in zip(blocks, exact):
        b.norm.data.copy_(1 + 0.2 * torch.randn(48))
        b.norm_bias.data.copy_(0.2 * torch.randn(48))
        b.conv_bias.data.copy_(0.2 * torch.randn(96))
        for p, q in zip(b.parameters(), e.parameters()):
            q.data = p.data.double().cpu()
    x, w = torch.randn(3, 70, 48), torch.randn(3, 70, 48)
    xg = x.cuda().requires_grad_()
    xe = x.double().requires_grad_()
    d, s, _ = blocks[0](xg, None)
    d, s, _ = blocks[1](d, s)
    ((d + s) * w.cuda()).sum().backward()
    de, se = exact_block(exact[0], xe, None)
    de, se = exact_block(exact[1], de, se)
    ((de + se) * w.double()).sum().backward()
    near(d, de, 2e-4, "out")
    near(xg.grad, xe.grad, 2e-4, "grad of x")
    for i, (b, e) in enumerate(zip(blocks, exact)):
        for (name, p), q in zip(b.named_parameters(), e.parameters()):
            near(p.grad, q.grad, 2e-4, f"block {i} {name}")


def test_packed_sequences_and_states_handed_on():
    torch = torch_mod()
    from recurrent_cell_gb300.memory import ScanBlock
    torch.manual_seed(1)
    block = ScanBlock(64, dtype=torch.float32)
    x = torch.randn(100, 64, device="cuda")
    off = torch.tensor([0, 70, 70, 100], dtype=torch.int32, device="cuda")
    packed, _, state = block(x, None, off, want_state=True)
    a, _, sa = block(x[None, :70], None, want_state=True)
    near(packed[:70], a[0].cpu(), 1e-5, "first")
    near(packed[70:], block(x[None, 70:], None)[0][0].cpu(), 1e-5, "last")
    assert not state[0][1].any() and not state[1][1].any()
    h, _, s1 = block(x[None, :33], None, want_state=True)
    t, _, s2 = block(x[None, 33:70], None, state=s1, want_state=True)
    near(torch.cat([h, t], 1), a.cpu(), 1e-5, "in two parts")
    for i in range(2):
        near(state[i][0], sa[i][0].cpu(), 1e-5, "state")
        near(s2[i], sa[i].cpu(), 1e-5, "state in two parts")
    # gradients flow through the states that are handed on
    xa, xb = x[None, :33].clone().requires_grad_(), x[None, :70].clone().requires_grad_()
    _, _, s1 = block(xa, None, want_state=True)
    block(x[None, 33:70], None, state=s1)[0].square().sum().backward()
    block(xb, None)[0][:, 33:].square().sum().backward()
    near(xa.grad, xb.grad[:, :33].cpu(), 1e-4, "gradient through the states")


@pytest.mark.parametrize("dtype,tol", [("float32", 1e-4), ("bfloat16", 0.1)])
def test_decoding_equals_whole_sequences(dtype, tol):
    torch = torch_mod()
    from recurrent_cell_gb300.memory import MemoryCell
    torch.manual_seed(2)
    dt = getattr(torch, dtype)
    model = MemoryCell(64, 32, dtype=dt, kind="scan")
    x = torch.randn(5, 40, 64, device="cuda").to(dt)
    whole = model(x).detach()
    state = model.empty_state(5)
    for t in range(40):
        h, state = model.step(x[:, t], state)
        assert float((h - whole[:, t]).abs().max()) <= tol * float(whole.abs().max()), t


def test_slots_of_a_server():
    """Sequences come and go in the slots of one pool; each gets what it would alone."""
    torch = torch_mod()
    from recurrent_cell_gb300.memory import ScanBlock
    torch.manual_seed(3)
    block = ScanBlock(32, dtype=torch.float32)
    x = torch.randn(4, 6, 32, device="cuda")
    whole = block(x, None)[0].detach()
    pool = block.empty_state(7)
    live = [(0, 5), (1, 2), (2, 6), (3, 0)]
    for t in range(6):
        order = live[t % 4:] + live[:t % 4]
        slots = torch.tensor([s for _, s in order], dtype=torch.int32, device="cuda")
        out, _ = block.step(x[[i for i, _ in order], t][:, None], None, pool, slots)
        for k, (i, _) in enumerate(order):
            near(out[k, 0], whole[i, t].cpu(), 1e-4, f"token {t} of {i}")


def test_training_with_clipped_gradients_runs():
    torch = torch_mod()
    from recurrent_cell_gb300.memory import train_recall
    model, losses = train_recall(steps=20, kind="scan", clip=0.5)
    assert np.isfinite(losses).all()
    norm = torch.sqrt(sum(p.grad.double().square().sum() for p in model.parameters()))
    assert 0 < float(norm) <= 0.5 * (1 + 1e-5)
    _, rule = train_recall(steps=5, clip=0.5)
    assert np.isfinite(rule).all()


def test_clipping_against_torch():
    torch = torch_mod()
    from recurrent_cell_gb300.memory import MemoryCell, clip_gradients
    torch.manual_seed(4)
    model = MemoryCell(32, 16, dtype=torch.float32, kind="scan")
    model(torch.randn(3, 9, 32, device="cuda")).square().sum().backward()
    want = [p.grad.double().clone().requires_grad_() for p in model.parameters()]
    for w in want:
        w.grad = w.detach().clone()
    total = torch.nn.utils.clip_grad_norm_(want, 0.1)
    norm = clip_gradients(model.parameters(), 0.1)
    assert abs(float(norm) - float(total)) <= 2e-6 * float(total)
    for p, w in zip(model.parameters(), want):
        near(p.grad, w.grad.cpu(), 1e-5, "clipped")
    assert float(clip_gradients([], 1.0)) == 0


def test_second_derivatives_are_refused():
    torch = torch_mod()
    from recurrent_cell_gb300.memory import causal_conv, layer_norm, selective_scan
    torch.manual_seed(5)
    leaf = lambda *s: torch.randn(*s, device="cuda").requires_grad_()  # noqa: E731
    x, rows = leaf(2, 5, 16), leaf(6, 32)
    w, A, B = torch.randn(16, 4, device="cuda"), -torch.rand(16, 8, device="cuda"), torch.randn(2, 5, 1, 8, device="cuda")
    for at, out in ((rows, layer_norm(2 * rows, torch.ones(32, device="cuda"))[0]), (x, causal_conv(x.square(), w)[0]),
                    (x, selective_scan(x.square(), x, A, B, B)[0])):
        (grad,) = torch.autograd.grad(out.square().sum(), at, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            grad.square().sum().backward()


@pytest.fixture
def stale():
    """Memory that is allocated and not written holds NaN, as memory may that something else has used."""
    torch = torch_mod()
    torch.use_deterministic_algorithms(True, warn_only=True)
    try:
        assert torch.empty(4, device="cuda").isnan().all()
        yield
    finally:
        torch.use_deterministic_algorithms(False)


@pytest.mark.filterwarnings("ignore:.*deterministic")
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_a_padded_batch_is_the_batch_without_its_padding(stale, dtype):
    """Rows behind the last sequence, whatever the allocator left: outputs of zeros there, and nothing in any gradient.

    A block is good to 2e-4 of 64 bits in FP32 (above), so two runs differ by 4e-4 at most; in bf16 the same values
    are rounded alike but for sums in another order: a step of a value, 2^-7, through the four roundings of a path."""
    torch = torch_mod()
    from recurrent_cell_gb300.memory import ScanBlock
    torch.manual_seed(6)
    dt, tol = getattr(torch, dtype), 4e-4 if dtype == "float32" else 4 * 2.0 ** -7
    blocks = [ScanBlock(48, dtype=dt) for _ in range(2)]
    x = torch.randn(100, 48, device="cuda").to(dt)
    w = torch.randn(70, 48, device="cuda")
    off = torch.tensor([0, 33, 33, 70], dtype=torch.int32, device="cuda")
    got = []
    for rows in (70, 100):
        leaf = x[:rows].clone().requires_grad_()
        delta, stream, last = blocks[0](leaf, None, off, want_state=True)
        delta, stream, _ = blocks[1](delta, stream, off)
        assert not delta[70:].any()
        ((delta + stream)[:70].float() * w).sum().backward()
        got.append({"out": delta[:70], "window": last[0], "state": last[1], "x": leaf.grad[:70],
                    **{f"{i}.{n}": p.grad for i, b in enumerate(blocks) for n, p in b.named_parameters()}})
        assert not leaf.grad[70:].any()
        for b in blocks:
            b.zero_grad(set_to_none=True)
    for name, want in got[0].items():
        near(got[1][name], want.cpu(), tol, name)


@pytest.mark.filterwarnings("ignore:.*deterministic")
def test_padding_of_the_operators_is_zero(stale):
    torch = torch_mod()
    from recurrent_cell_gb300.memory import causal_conv, selective_scan
    torch.manual_seed(7)
    off = torch.tensor([0, 5, 30], dtype=torch.int32, device="cuda")
    leaf = lambda *s: torch.randn(*s, device="cuda").requires_grad_()  # noqa: E731
    x, delta, z, B, C = leaf(41, 16), leaf(41, 16), leaf(41, 16), leaf(41, 1, 8), leaf(41, 1, 8)
    weight, A = leaf(16, 4), -torch.rand(16, 8, device="cuda")
    y, _ = causal_conv(x, weight, seq_offsets=off)
    o, _ = selective_scan(y, delta, A, B, C, z=z, seq_offsets=off)
    assert not y[30:].any() and not o[30:].any() and y[:30].all() and o[:30].all()
    o.sum().backward()
    for t in (x, delta, z, B, C):
        assert t.grad.isfinite().all() and not t.grad[30:].any() and t.grad[:30].any()
    assert weight.grad.isfinite().all()


@pytest.mark.parametrize("kind", ["scan", "rule"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_a_prompt_without_gradients_takes_less_memory_and_gives_the_same_bits(kind, dtype):
    torch = torch_mod()
    from recurrent_cell_gb300.memory import MemoryBlock, ScanBlock
    torch.manual_seed(8)
    dt = getattr(torch, dtype)
    block = ScanBlock(64, dtype=dt) if kind == "scan" else MemoryBlock(64, 2, 2, 32, 32, dt)
    x = torch.randn(2, 300, 64, device="cuda").to(dt)

    def run():
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        out, stream, state = block(x, None, want_state=True)
        return out, stream, state if kind == "scan" else (state,), torch.cuda.max_memory_allocated() - before

    out, stream, state, most = run()
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            o, s, last, some = run()
            assert torch.equal(o, out) and torch.equal(s, stream) and some < most
            assert all(torch.equal(a, b) for a, b in zip(last, state))
    out = block(x, None)[0]
    with torch.no_grad():
        assert torch.equal(block(x, None)[0], out)                 # nor without a final state
