"""A memory trunk in front of the CfC cell: residual norm, gated delta rule and
K loop together, in training and token by token.

Each block of the trunk reads the residual stream through the norm, projects it
to queries, keys, values and gates, runs the rule and projects back:

    y, s = norm(delta + s);   q, k, v, a, b = y W_in
    o = rule(q / |q|, k / |k|, v, g = -softplus(a + bias), beta = sigmoid(b));   delta = o W_out

The stream after the last norm is the cell's input.  The plain matrix products
and the elementwise gates are torch's; the rest are this library's calls, as
autograd functions (first derivatives: the gradient of a gradient is an error).
A sequence's whole state is one [v_heads, d_k, d_v] matrix a block and the cell's
hidden vector, so decoding takes a fixed amount of memory however long the
sequence is.

    python -m recurrent_cell_gb300.memory        (trains on recall, then decodes)
"""

from __future__ import annotations

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

from . import (GRAD_GEMM, MATH_BF16, MATH_FP32, cfc_gdr_backward, cfc_gdr_forward, cfc_gdr_step,
               cfc_gdr_workspace_bytes, cfc_kloop_backward, cfc_kloop_forward, cfc_kloop_workspace_bytes,
               cfc_rmsnorm_backward, cfc_rmsnorm_forward, cfc_rmsnorm_workspace_bytes)


def _math(dtype):
    return MATH_BF16 if dtype == torch.bfloat16 else MATH_FP32


def _workspace(size, device):
    return torch.empty(size, dtype=torch.uint8, device=device)


def _rows_of(t):
    return None if t is None else t.reshape(-1, t.shape[-1]).contiguous()


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        rows, d = x.shape
        y, s = torch.empty_like(x), torch.empty_like(x)
        rstd = torch.empty(rows, device=x.device)
        cfc_rmsnorm_forward(x, weight, y=y, residual=residual, residual_out=s, rstd=rstd, eps=eps, math=_math(x.dtype))
        ctx.save_for_backward(s, weight, rstd)
        ctx.residual = residual is not None
        return y, s

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_s):
        s, weight, rstd = ctx.saved_tensors
        grad_x, grad_w = torch.empty_like(s), torch.empty_like(weight)
        cfc_rmsnorm_backward(s, weight, rstd, grad_y.contiguous(), grad_x, grad_w,
                             _workspace(cfc_rmsnorm_workspace_bytes(*s.shape), s.device),
                             grad_residual_out=grad_s.contiguous(), math=_math(s.dtype))
        return grad_x, grad_x if ctx.residual else None, grad_w, None


def residual_norm(x, weight, residual=None, eps=1e-6):
    """(y, s): the norm of the stream s = x + residual, [rows, d], and s."""
    return _Norm.apply(x, residual, weight, eps)


class _Rule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, seq_offsets, initial_state, want_state):
        packed = seq_offsets is not None
        n = seq_offsets.numel() - 1 if packed else v.shape[0]
        hk, dk, hv, dv = *q.shape[-2:], *v.shape[-2:]
        rows, math = v[..., 0, 0].numel(), _math(q.dtype)
        save = any(ctx.needs_input_grad)
        ws = _workspace(cfc_gdr_workspace_bytes(rows, n, hk, hv, dk, dv, math, save), q.device)
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        state = torch.empty(n, hv, dk, dv, device=q.device) if want_state else None
        cfc_gdr_forward(q, k, v, g, beta, o, ws, seq_offsets=seq_offsets, initial_state=initial_state,
                        final_state=state, save=save, math=math)
        ctx.save_for_backward(q, k, v, g, beta, seq_offsets, initial_state)
        ctx.ws = ws
        ctx.set_materialize_grads(False)
        return o, state

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_o, grad_state):
        q, k, v, g, beta, seq_offsets, initial = ctx.saved_tensors
        like = lambda t: torch.empty(t.shape, dtype=q.dtype, device=q.device)  # noqa: E731
        grads = [like(t) for t in (q, k, v, g, beta)]
        grad_o = like(v).zero_() if grad_o is None else grad_o.contiguous()
        grad_init = torch.empty_like(initial) if initial is not None else None
        cfc_gdr_backward(q, k, v, g, beta, grad_o, *grads, ctx.ws, seq_offsets=seq_offsets,
                         grad_final_state=None if grad_state is None else grad_state.contiguous(),
                         grad_initial_state=grad_init, math=_math(q.dtype))
        return *grads[:3], grads[3].float(), grads[4].float(), None, grad_init, None


def gated_delta_rule(q, k, v, g, beta, seq_offsets=None, initial_state=None, want_state=False):
    """(o, final state or None) over whole sequences: q, k [sequences, tokens, k_heads, d_k],
    v [sequences, tokens, v_heads, d_v], g, beta [sequences, tokens, v_heads], or
    all of them packed [rows, ...] with seq_offsets.  scale = d_k ** -0.5."""
    return _Rule.apply(q, k, v, g, beta, seq_offsets, initial_state, want_state)


class _Cell(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, h0, W_in, W_rec, b, dt):
        B, K, n_in = x.shape
        H, math = h0.shape[1], _math(x.dtype)
        ws = _workspace(cfc_kloop_workspace_bytes(B, K, n_in, H, math, GRAD_GEMM), x.device)
        h_seq = torch.empty(B, K, H, dtype=x.dtype, device=x.device)
        cfc_kloop_forward(x, h0, W_in, W_rec, b, dt, h_seq, ws, math=math)
        ctx.save_for_backward(x, h0, W_in, W_rec, b, dt, h_seq)
        ctx.ws = ws
        return h_seq

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_h):
        x, h0, W_in, W_rec, b, dt, h_seq = ctx.saved_tensors
        f32 = lambda t: torch.empty(t.shape, device=t.device)  # noqa: E731
        gWi, gWr, gb, gh0, gx = (f32(t) for t in (W_in, W_rec, b, h0, x))
        cfc_kloop_backward(x, h0, W_in, W_rec, b, dt, h_seq, gWi, gWr, gb, ctx.ws, grad_h_seq=grad_h.float().contiguous(),
                           grad_h0=gh0, grad_x=gx, grad_path=GRAD_GEMM, math=_math(x.dtype))
        return tuple(g.to(t.dtype) for g, t in zip((gx, gh0, gWi, gWr, gb), (x, h0, W_in, W_rec, b))) + (None,)


class MemoryBlock(torch.nn.Module):
    """One block of the trunk; the norm and the gates' bias in fp32, the rest in ``dtype``."""

    def __init__(self, d, k_heads, v_heads, d_k, d_v, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.sizes = (k_heads, v_heads, d_k, d_v)
        width = 2 * k_heads * d_k + v_heads * d_v + 2 * v_heads
        width = (width + 7) // 8 * 8                    # rows of whole 16-byte vectors: v stays a part of the projection
        kw = dict(dtype=dtype, device=device)
        self.norm = torch.nn.Parameter(torch.ones(d, device=device))
        self.w_in = torch.nn.Parameter(torch.randn(d, width, **kw) * d ** -0.5)
        self.w_out = torch.nn.Parameter(torch.randn(v_heads * d_v, d, **kw) * (v_heads * d_v) ** -0.5)
        # forgetting times from a few tokens to thousands
        self.bias = torch.nn.Parameter(torch.linspace(-8, -1, v_heads, device=device))

    def _heads(self, y):
        """y [..., d] -> q, k [..., k_heads, d_k], v [..., v_heads, d_v], g, beta [..., v_heads]."""
        hk, hv, dk, dv = self.sizes
        p = y @ self.w_in
        parts = p.split([hk * dk, hk * dk, hv * dv, hv, hv, p.shape[-1] - 2 * hk * dk - hv * dv - 2 * hv], -1)
        q, k = (F.normalize(t.unflatten(-1, (hk, dk)).float(), dim=-1).to(y.dtype) for t in parts[:2])
        g = -F.softplus(parts[3].float() + self.bias)
        return q, k, parts[2].unflatten(-1, (hv, dv)), g, torch.sigmoid(parts[4].float())

    def forward(self, delta, stream, seq_offsets=None, state=None, want_state=False):
        """delta, stream (or None) [sequences, tokens, d] or packed [rows, d]
        -> delta of this block, the stream, the final state (or None)."""
        y, s = residual_norm(_rows_of(delta), self.norm, _rows_of(stream))
        o, state = gated_delta_rule(*self._heads(y.view_as(delta)), seq_offsets, state, want_state)
        return o.flatten(-2) @ self.w_out, s.view_as(delta), state

    @torch.no_grad()
    def step(self, delta, stream, pool, slots=None):
        """The next tokens [sequences, tokens, d]; sequence i's state is pool[slots[i]], updated in place."""
        x = _rows_of(delta)
        y, s = torch.empty_like(x), torch.empty_like(x)
        cfc_rmsnorm_forward(x, self.norm, y=y, residual=_rows_of(stream), residual_out=s, math=_math(x.dtype))
        q, k, v, g, beta = self._heads(y.view_as(delta))
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        cfc_gdr_step(q, k, v, g, beta, pool, o, slots=slots, math=_math(x.dtype))
        return o.flatten(-2) @ self.w_out, s.view_as(delta)


class MemoryCell(torch.nn.Module):
    """Blocks of memory, a last norm, and the CfC cell on what they give."""

    def __init__(self, d, hidden, blocks=2, k_heads=2, v_heads=2, d_k=32, d_v=32, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.blocks = torch.nn.ModuleList(MemoryBlock(d, k_heads, v_heads, d_k, d_v, dtype, device) for _ in range(blocks))
        self.norm = torch.nn.Parameter(torch.ones(d, device=device))
        kw = dict(dtype=dtype, device=device)
        scale = (d + hidden) ** -0.5
        self.W_in = torch.nn.Parameter(torch.randn(3, hidden, d, **kw) * scale)
        self.W_rec = torch.nn.Parameter(torch.randn(3, hidden, hidden, **kw) * scale)
        self.b = torch.nn.Parameter(torch.zeros(3, hidden, device=device))
        self.register_buffer("dt", torch.ones(1, device=device))

    def forward(self, x):
        """x [sequences, tokens, d] -> hidden states [sequences, tokens, hidden]."""
        delta, stream = x, None
        for block in self.blocks:
            delta, stream, _ = block(delta, stream)
        y, _ = residual_norm(delta.flatten(0, 1), self.norm, stream.flatten(0, 1))
        h0 = torch.zeros(x.shape[0], self.W_rec.shape[1], dtype=x.dtype, device=x.device)
        return _Cell.apply(y.view_as(x), h0, self.W_in, self.W_rec, self.b, self.dt)

    def empty_state(self, sequences):
        """Zero states: one pool a block, and the cell's hidden vectors."""
        pools = []
        for block in self.blocks:
            _, hv, dk, dv = block.sizes
            pools.append(torch.zeros(sequences, hv, dk, dv, device=self.norm.device))
        return pools, torch.zeros(sequences, self.W_rec.shape[1], dtype=self.W_rec.dtype, device=self.norm.device)

    @torch.no_grad()
    def step(self, x, state):
        """The next token x [sequences, d] -> (hidden [sequences, hidden], the next state)."""
        pools, h = state
        delta, stream = x[:, None], None
        for block, pool in zip(self.blocks, pools):
            delta, stream = block.step(delta, stream, pool)
        y = torch.empty_like(x)
        cfc_rmsnorm_forward(delta[:, 0].contiguous(), self.norm, y=y, residual=stream[:, 0].contiguous(), math=_math(x.dtype))
        B, d = x.shape
        H, math = h.shape[1], _math(x.dtype)
        ws = _workspace(cfc_kloop_workspace_bytes(B, 1, d, H, math, GRAD_GEMM), x.device)
        out = torch.empty(B, 1, H, dtype=x.dtype, device=x.device)
        cfc_kloop_forward(y[:, None], h, self.W_in, self.W_rec, self.b, self.dt, out, ws, math=math)
        return out[:, 0], (pools, out[:, 0].contiguous())


def recall_batch(gen, sequences, tokens, d, hidden, dtype, device="cuda"):
    """Pairs of a key and a value a token, and at the end one of the keys again:
    the hidden state there should be half of that key's value."""
    pairs = tokens - 1
    key = F.normalize(torch.randn(sequences, pairs, d // 2, generator=gen, device=device), dim=-1)
    value = torch.sign(torch.randn(sequences, pairs, d // 2, generator=gen, device=device))
    pick = torch.randint(pairs, (sequences,), generator=gen, device=device)
    at = torch.arange(sequences, device=device)
    x = torch.cat([key * (d // 2) ** 0.5, value], -1)
    last = torch.cat([key[at, pick] * (d // 2) ** 0.5, torch.zeros_like(value[:, 0])], -1)
    y = 0.5 * value[at, pick][:, :hidden]
    return torch.cat([x, last[:, None]], 1).to(dtype), y


def train_recall(steps=300, sequences=128, tokens=9, d=64, hidden=32, dtype=torch.float32, seed=0, report=None):
    """Trains a small model on recall_batch; the model and its losses."""
    gen = torch.Generator("cuda").manual_seed(seed)
    torch.manual_seed(seed)
    model = MemoryCell(d, hidden, blocks=2, k_heads=2, v_heads=2, d_k=32, d_v=32, dtype=dtype)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for i in range(steps):
        x, y = recall_batch(gen, sequences, tokens, d, hidden, dtype)
        loss = (model(x)[:, -1].float() - y).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if report and (i + 1) % report == 0:
            print(f"step {i + 1}: loss {float(losses[-1]):.4f} (0.25 without any memory)")
    return model, [float(v) for v in torch.stack(losses).cpu()]


def main():
    model, _ = train_recall(report=50)
    gen = torch.Generator("cuda").manual_seed(1)
    x, y = recall_batch(gen, 16, 9, 64, 32, torch.float32)
    whole = model(x).detach()
    state = model.empty_state(16)
    for t in range(x.shape[1]):
        h, state = model.step(x[:, t], state)
        diff = float((h - whole[:, t]).abs().max())
        print(f"token {t}: decoded against the whole sequence, largest difference {diff:.1e}")
    print(f"signs recalled: {float((torch.sign(h) == torch.sign(y)).float().mean()):.3f}")


if __name__ == "__main__":
    main()
