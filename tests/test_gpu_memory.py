"""The memory trunk in front of the cell: its gradients against the same model in
64-bit torch, decoding against whole sequences, and that it learns to recall.

FP32 tolerance 2e-4 normwise: the library's operators are good to 1e-5 to 5e-5
each (their own tests) and torch's fp32 products to 1e-6; four of the former lie
on a path through two blocks, the norm and the cell.  Decoding sums in
another order: 1e-4 of the largest value."""

import numpy as np
import pytest

from gpu_common import require_gpu, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def exact_block(block, delta, stream):
    """MemoryBlock.forward in plain torch, token by token, in the parameters' type (float64)."""
    torch = torch_mod()
    s = delta if stream is None else delta + stream
    y = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-6) * block.norm
    hk, hv, dk, dv = block.sizes
    p = y @ block.w_in
    at = [0, hk * dk, 2 * hk * dk, 2 * hk * dk + hv * dv, 2 * hk * dk + hv * dv + hv, 2 * hk * dk + hv * dv + 2 * hv]
    q, k, v, a, b = (p[..., i:j] for i, j in zip(at, at[1:]))
    rep = hv // hk
    q, k = (torch.nn.functional.normalize(t.unflatten(-1, (hk, dk)), dim=-1).repeat_interleave(rep, -2) for t in (q, k))
    v = v.unflatten(-1, (hv, dv))
    g, beta = -torch.nn.functional.softplus(a + block.bias), torch.sigmoid(b)
    S, out = torch.zeros(delta.shape[0], hv, dk, dv, dtype=delta.dtype), []
    for t in range(delta.shape[1]):
        S = torch.exp(g[:, t])[..., None, None] * S
        u = beta[:, t][..., None] * (v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S))
        S = S + k[:, t][..., None] * u[..., None, :]
        out.append(dk ** -0.5 * torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    return torch.stack(out, 1).flatten(-2) @ block.w_out, s


def near(a, b, tol, what):
    a, b = a.detach().cpu().double().numpy(), b.detach().double().numpy()
    assert np.linalg.norm(a - b) <= tol * np.linalg.norm(b), f"{what}: {np.linalg.norm(a - b) / np.linalg.norm(b):.1e}"


def test_two_blocks_match_plain_torch_in_64_bits():
    torch = torch_mod()
    from recurrent_cell_gb300.memory import MemoryBlock
    torch.manual_seed(0)
    blocks = [MemoryBlock(48, 1, 2, 32, 24, torch.float32) for _ in range(2)]
    exact = [MemoryBlock(48, 1, 2, 32, 24, torch.float64, "cpu") for _ in range(2)]
    for b, e in zip(blocks, exact):
        b.bias.data.copy_(torch.tensor([-1.0, 0.5]))
        b.norm.data.copy_(1 + 0.2 * torch.randn(48))
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
    from recurrent_cell_gb300.memory import MemoryBlock
    torch.manual_seed(1)
    block = MemoryBlock(64, 2, 2, 32, 32, torch.float32)
    x = torch.randn(100, 64, device="cuda")
    off = torch.tensor([0, 70, 70, 100], dtype=torch.int32, device="cuda")
    packed, _, state = block(x, None, off, want_state=True)
    a, _, sa = block(x[None, :70], None, want_state=True)
    near(packed[:70], a[0].cpu(), 1e-6, "first")
    near(packed[70:], block(x[None, 70:], None)[0][0].cpu(), 1e-6, "last")
    near(state[0], sa[0].cpu(), 1e-6, "state")
    h, _, s1 = block(x[None, :33], None, want_state=True)
    t, _, s2 = block(x[None, 33:70], None, state=s1, want_state=True)
    near(torch.cat([h, t], 1), a.cpu(), 1e-5, "in two parts")
    near(s2, sa.cpu(), 1e-5, "state in two parts")


@pytest.mark.parametrize("dtype,tol", [("float32", 1e-4), ("bfloat16", 0.1)])
def test_decoding_equals_whole_sequences(dtype, tol):
    """bf16: the streams are rounded alike but the rule's outputs not: a few bf16 steps of a value."""
    torch = torch_mod()
    from recurrent_cell_gb300.memory import MemoryCell
    torch.manual_seed(2)
    dt = getattr(torch, dtype)
    model = MemoryCell(64, 32, dtype=dt)
    x = torch.randn(5, 40, 64, device="cuda").to(dt)
    whole = model(x).detach()
    state = model.empty_state(5)
    for t in range(40):
        h, state = model.step(x[:, t], state)
        assert float((h - whole[:, t]).abs().max()) <= tol * float(whole.abs().max()), t


def test_it_learns_to_recall():
    """Guessing the sign of each value is a loss of 0.25; less than half of that needs the memory."""
    from recurrent_cell_gb300.memory import train_recall
    _, losses = train_recall(steps=300)
    assert np.isfinite(losses).all()
    assert np.mean(losses[-20:]) < 0.125, losses[::20]


def test_second_derivatives_are_refused():
    """The gradients are kernels' results, not differentiable themselves: asking for their gradient is an
    error, also where other operations lie on the path and would give a part of it."""
    torch = torch_mod()
    from recurrent_cell_gb300.memory import MemoryBlock, MemoryCell, gated_delta_rule, residual_norm
    torch.manual_seed(3)
    leaf = lambda *s: torch.randn(*s, device="cuda").requires_grad_()  # noqa: E731
    block, cell = MemoryBlock(32, 1, 2, 16, 16, torch.float32), MemoryCell(32, 16, dtype=torch.float32)
    x, rows, q = leaf(2, 5, 32), leaf(6, 32), leaf(1, 5, 1, 16)
    g, beta = -torch.rand(1, 5, 1, device="cuda"), torch.rand(1, 5, 1, device="cuda")
    for name, at, out in (("norm", rows, residual_norm(2 * rows, block.norm.detach())[0]),
                          ("rule", q, gated_delta_rule(q.square(), q, q, g, beta)[0]),
                          ("block", x, block(x, None)[0]), ("cell", x, cell(x))):
        (grad,) = torch.autograd.grad(out.square().sum(), at, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            grad.square().sum().backward()
            pytest.fail(f"{name}: a second derivative came out")
