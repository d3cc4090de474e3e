"""What the trunk's autograd functions ask of the library and hand on, with the library's calls replaced by fakes (no GPU)."""

import pytest

torch = pytest.importorskip("torch")

from recurrent_cell_gb300 import memory  # noqa: E402

ROWS, USED, D, N = 11, 7, 8, 4


@pytest.fixture
def stale():
    """Memory that is allocated and not written holds NaN."""
    torch.use_deterministic_algorithms(True, warn_only=True)
    try:
        assert torch.empty(4).isnan().all()
        yield
    finally:
        torch.use_deterministic_algorithms(False)


def write(*tensors):
    """As the kernels do: the rows of sequences, and nothing behind them."""
    for t in tensors:
        if t is not None:
            t[:USED if t.shape[0] == ROWS else None] = 1


def test_rows_behind_the_last_sequence_are_zero(stale, monkeypatch):
    monkeypatch.setattr(memory, "cfc_conv_forward", lambda x, w, y, **kw: write(y, kw["final_state"]))
    monkeypatch.setattr(memory, "cfc_conv_workspace_bytes", lambda *a, **kw: 16)
    monkeypatch.setattr(memory, "cfc_conv_backward", lambda x, w, gy, gx, gw, ws, **kw: write(gx, gw, kw["grad_bias"]))
    monkeypatch.setattr(memory, "cfc_ssm_workspace_bytes", lambda *a, **kw: 16)
    monkeypatch.setattr(memory, "cfc_ssm_forward", lambda x, dl, A, B, C, y, ws, **kw: write(y, kw["final_state"]))
    monkeypatch.setattr(memory, "cfc_ssm_backward", lambda x, dl, A, B, C, gy, gx, gd, gA, gB, gC, ws, **kw: write(
        gx, gd, gA, gB, gC, kw["grad_D"], kw["grad_z"], kw["grad_delta_bias"]))
    off = torch.tensor([0, 3, USED], dtype=torch.int32)
    leaf = lambda *s: torch.zeros(*s, requires_grad=True)  # noqa: E731
    x, delta, z, B, C = leaf(ROWS, D), leaf(ROWS, D), leaf(ROWS, D), leaf(ROWS, 1, N), leaf(ROWS, 1, N)
    y, _ = memory.causal_conv(x, leaf(D, 3), leaf(D), off)
    o, _ = memory.selective_scan(y, delta, leaf(D, N), B, C, leaf(D), z, leaf(D), off)
    o.sum().backward()
    for t in (y, o, x.grad, delta.grad, z.grad, B.grad, C.grad):
        assert (t[:USED] == 1).all() and (t[USED:] == 0).all()


@pytest.fixture
def saves(monkeypatch):
    """What the workspaces and the forwards of the scan and the rule are told about a backward to come."""
    told = []
    for op in ("ssm", "gdr"):
        monkeypatch.setattr(memory, f"cfc_{op}_workspace_bytes", lambda *a: told.append(("size", bool(a[-1]))) or 16)
        monkeypatch.setattr(memory, f"cfc_{op}_forward", lambda *a, save, **kw: told.append(("call", save)))
    return told


def scan(of):
    return memory.selective_scan(of(2, 5, D), of(2, 5, D), of(D, N), of(2, 5, 1, N), of(2, 5, 1, N), of(D), of(2, 5, D), of(D))


def rule(of):
    return memory.gated_delta_rule(of(2, 5, 1, D), of(2, 5, 1, D), of(2, 5, 1, D), of(2, 5, 1), of(2, 5, 1))


@pytest.mark.parametrize("op", [scan, rule])
def test_a_forward_keeps_what_a_backward_needs_only_where_one_can_come(saves, op):
    leaf, plain = (lambda *s: torch.zeros(*s, requires_grad=True)), torch.zeros
    for of, mode, want in ((leaf, torch.enable_grad, True), (leaf, torch.no_grad, False), (leaf, torch.inference_mode, False),
                           (plain, torch.enable_grad, False), (plain, torch.no_grad, False)):
        saves.clear()
        with mode():
            out, _ = op(of)
        assert saves == [("size", want), ("call", want)], mode
        assert out.requires_grad == want
