"""The norm of many gradients together and clipping, on the GPU against 64 bits.

Tolerances.  A thread adds 128 squares in fp32, 32 of them in a row (32 x 2^-24 = 2e-6 of their sum at worst, 2e-7 in practice) and the
rest in 64 bits; the root halves it: 2e-6 on the norm.  The factor carries that and two roundings, the product one more:
2.5e-6 relative in fp32, in bf16 half a step, 2^-8, on top."""

import math

import numpy as np
import pytest

import recurrent_cell_gb300 as cfc

from gpu_common import require_gpu, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def tensors(sizes, kind="mixed", seed=0, size=1.0):
    torch = torch_mod()
    g = torch.Generator("cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        half = {"fp32": False, "bf16": True, "mixed": i % 2 == 1}[kind]
        out.append((size * 10.0 ** (i % 5 - 2) * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16 if half else torch.float32))
    return out


def exact_norm(grads):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))


def workspace(n):
    torch = torch_mod()
    return torch.full((cfc.cfc_grad_clip_workspace_bytes(n),), 255, dtype=torch.uint8, device="cuda")


def norm_of(grads):
    torch = torch_mod()
    norm = torch.full((1,), float("nan"), device="cuda")
    cfc.cfc_grad_norm(grads, norm, workspace(len(grads)))
    return float(norm)


def clip(grads, most, out=None):
    torch = torch_mod()
    norm = torch.full((1,), float("nan"), device="cuda")
    cfc.cfc_grad_clip(grads, most, norm, workspace(len(grads)), out=out)
    return float(norm)


def check(before, after, norm, most):
    want_norm = exact_norm(before)
    assert abs(norm - want_norm) <= 2e-6 * want_norm, (norm, want_norm)
    factor = min(1.0, most / (want_norm + 1e-6))
    for b, a in zip(before, after):
        want = b.double() * factor
        tol = 2.5e-6 + (2.0 ** -8 if a.element_size() == 2 else 0)
        assert bool(((a.double() - want).abs() <= tol * want.abs() + 1e-44).all())


SIZES = [[1], [5], [16384], [16385], [3, 0, 7, 0, 1 << 20], [8191, 16384, 16383, 40000, 3], [100] * 64, [100] * 65, [33] * 1100, [6_000_001]]


@pytest.mark.parametrize("kind", ["fp32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_clip(sizes, kind):
    torch = torch_mod()
    grads = tensors(sizes, kind, len(sizes))
    before = [g.clone() for g in grads]
    assert abs(norm_of(grads) - exact_norm(before)) <= 2e-6 * exact_norm(before)
    out = [torch.full_like(g, float("nan")) for g in grads]
    most = 0.3 * exact_norm(before)
    norm = clip(grads, most, out)
    for g, b in zip(grads, before):
        assert torch.equal(g, b)                                   # read only
    check(before, out, norm, most)
    assert clip(grads, most) == norm                               # in place: the same values
    for g, o in zip(grads, out):
        assert torch.equal(g, o)


def test_below_the_limit_nothing_changes():
    torch = torch_mod()
    grads = tensors([1000, 77, 40000])
    before = [g.clone() for g in grads]
    for most in (1.01 * exact_norm(before), 1e30, float("inf")):
        out = [torch.full_like(g, float("nan")) for g in grads]
        clip(grads, most, out)
        for g, o in zip(grads, out):
            assert torch.equal(g, o)
        clip(grads, most)
        for g, b in zip(grads, before):
            assert torch.equal(g, b)


def test_unaligned_parts_of_one_buffer():
    torch = torch_mod()
    for dt in (torch.float32, torch.bfloat16):
        flat = torch.randn(100_003, device="cuda").to(dt)
        parts = [flat[1:40_000], flat[40_000:40_003], flat[40_003:]]
        before = [p.clone() for p in parts]
        check(before, parts, clip(parts, 1.0), 1.0)
        assert flat[0] == flat[0].clone()


@pytest.mark.parametrize("size", [1e-43, 1e-38, 1e-30, 1e-20, 1e-15, 1e15, 1e19, 1e30])
def test_values_from_the_smallest_to_the_largest(size):
    """Squares that fp32 would lose or overflow are taken in 64 bits."""
    torch = torch_mod()
    for grads in (tensors([5000, 333], "fp32", 3, 1.0), tensors([5000, 333], "bf16", 3, 1.0)):
        grads = [(g.double() * size).to(g.dtype) for g in grads]
        want = exact_norm(grads)
        got = norm_of(grads)
        assert abs(got - want) <= 2e-6 * want + 1e-45, (got, want)
        mixed = grads + [torch.zeros(40000, device="cuda")]
        assert norm_of(mixed) == got


def test_what_is_not_finite():
    torch = torch_mod()
    grads = tensors([100, 40000, 7])
    grads[1][123] = float("nan")
    out = [torch.empty_like(g) for g in grads]
    assert math.isnan(clip(grads, 1.0, out)) and all(o.isnan().all() for o in out)
    grads[1][123] = float("inf")
    assert math.isinf(clip(grads, 1.0, out))
    assert not out[0].any() and not out[2].any() and out[1][123].isnan()        # factor 0


def test_nothing_and_zeros():
    torch = torch_mod()
    assert norm_of([]) == 0 and clip([], 1.0) == 0
    empty = torch.empty(0, device="cuda")
    assert clip([empty, empty], 1.0) == 0
    z = [torch.zeros(50000, device="cuda"), torch.zeros(3, dtype=torch.bfloat16, device="cuda")]
    assert clip(z, 1.0) == 0 and not z[0].any()
    g = tensors([64])
    assert clip(g, 0.0) > 0 and not g[0].any()


def test_the_same_bits_every_time_in_a_graph_and_on_another_stream():
    torch = torch_mod()
    grads = tensors([70000, 33, 16385] * 5)
    out, norm, ws = [torch.empty_like(g) for g in grads], torch.empty(1, device="cuda"), workspace(15)
    cfc.cfc_grad_clip(grads, 1.0, norm, ws, out=out)
    first, n0 = [o.clone() for o in out], norm.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cfc.cfc_grad_clip(grads, 1.0, norm, ws, out=out)
    side.synchronize()
    assert torch.equal(norm, n0) and all(torch.equal(a, b) for a, b in zip(first, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                                  # the table of tensors is kept by the graph
        cfc.cfc_grad_clip(grads, 1.0, norm, ws, out=out)
    for g in grads:
        g.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) - 2 * float(n0)) <= 1e-6 * float(n0) and torch.equal(out[0], first[0])


def test_more_than_2_32_bytes():
    torch = torch_mod()
    big = torch.full(((1 << 31) + 5,), 0.5, dtype=torch.bfloat16, device="cuda")
    want = math.sqrt(big.numel() * 0.25)
    assert abs(clip([big], want / 4) - want) <= 2e-6 * want
    assert float(big[-1]) == 0.125 and float(big[0]) == 0.125 and float(big[1 << 30]) == 0.125


@pytest.mark.parametrize("pieces", [3, 200])
def test_parts_of_one_buffer_and_a_gradient_named_twice(pieces):
    torch = torch_mod()
    flat = torch.randn(pieces * 37, device="cuda")
    before = flat.double()
    parts = [flat[i * 37:(i + 1) * 37] for i in range(pieces)][::-1]
    norm, ws = torch.empty(1, device="cuda"), workspace(pieces)
    cfc.cfc_grad_clip(parts, 1.0, norm, ws)
    want = float(before.norm())
    assert abs(float(norm) - want) <= 1e-6 * want
    assert (flat.double() - before / (want + 1e-6)).abs().max() <= 1e-6 * before.abs().max() / want
    out = [torch.empty_like(parts[0]) for _ in range(2)]
    cfc.cfc_grad_clip([parts[0], parts[0]], 1e-3, norm, workspace(2), out=out)
    assert torch.equal(out[0], out[1]) and abs(float(norm) - 2 ** 0.5 * float(parts[0].double().norm())) <= 1e-6 * float(norm)


def test_refusals_of_the_binding():
    torch = torch_mod()
    g = tensors([8, 8])
    ws, norm = workspace(2), torch.empty(1, device="cuda")
    for bad in (dict(out=[g[0]]), dict(out=[g[0], g[1][:4]]), dict(out=[g[0], g[0].to(g[1].dtype)[:4]]), dict(grads=[g[0], g[0]]),
                dict(grads=[g[0].expand(2, 8).t()]), dict(norm=torch.empty(2, device="cuda"))):
        with pytest.raises(ValueError):
            cfc.cfc_grad_clip(**{**dict(grads=g, max_norm=1.0, norm=norm, workspace=ws), **bad})
    with pytest.raises(TypeError):
        cfc.cfc_grad_clip([g[0].half()], 1.0, norm, ws)
    with pytest.raises(cfc.CfcError):
        cfc.cfc_grad_clip(g, -1.0, norm, ws)
    with pytest.raises(cfc.CfcError, match="overlap"):
        flat = torch.zeros(32, device="cuda")
        cfc.cfc_grad_clip([flat[:16]], 1.0, norm, ws, out=[flat[8:24]])
    assert np.isfinite(norm_of(g))


def test_infinity_never_clips():
    """max_norm infinite: gradients stay as they are, also where the norm itself is infinite or too large for a float."""
    torch = torch_mod()
    inf = float("inf")
    for grads in ([torch.full((300,), 1e38, device="cuda"), torch.randn(7, device="cuda")],
                  [torch.tensor([inf, 1.0, -2.0], device="cuda"), torch.randn(40000, device="cuda").to(torch.bfloat16)]):
        before = [g.clone() for g in grads]
        out = [torch.full_like(g, float("nan")) for g in grads]
        assert clip(grads, inf, out) == inf and clip(grads, inf) == inf
        for b, o, g in zip(before, out, grads):
            assert torch.equal(b, o) and torch.equal(b, g)
    grads = [torch.tensor([float("nan"), 1.0], device="cuda"), torch.ones(5, device="cuda")]
    assert math.isnan(clip(grads, inf)) and all(g.isnan().all() for g in grads)        # a NaN is not hidden


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_what_lies_beside_unaligned_parts_is_left_alone(dtype):
    """In place and into other tensors: nothing before, between or behind the parts is written."""
    torch = torch_mod()
    for into in (False, True):
        flat = torch.randn(100_011, device="cuda").to(getattr(torch, dtype))
        other = torch.randn(100_011, device="cuda").to(flat.dtype)
        kept, kept_other = flat.clone(), other.clone()
        spans = [(1, 40_000), (40_001, 40_004), (40_007, 100_003)]
        parts = [flat[a:b] for a, b in spans]
        before = [p.clone() for p in parts]
        after = [other[a:b] for a, b in spans] if into else parts
        check(before, after, clip(parts, 1.0, after if into else None), 1.0)
        beside = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
        for a, b in spans:
            beside[a:b] = False
        assert int(beside.sum()) == 1 + 1 + 3 + 8
        assert torch.equal(flat[beside], kept[beside]) and torch.equal(other[beside], kept_other[beside])
        if into:
            assert torch.equal(flat, kept)
