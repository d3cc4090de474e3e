"""Argument checks of the layer norm, the short convolution, the selective scan and gradient clipping at the C ABI:
what is refused, with which status, before anything is launched (no GPU; the addresses are never dereferenced)."""

import ctypes

import pytest

import recurrent_cell_gb300 as cfc
from recurrent_cell_gb300 import build as cfc_build

ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_MODE, ERR_OVERLAP = -1, -2, -3, -4, -5, -9
FP32, TF32, BF16 = cfc.MATH_FP32, cfc.MATH_TF32, cfc.MATH_BF16
BIG = 1 << 50


def far(i):
    """Fake addresses, aligned and far apart."""
    return 0x10_0000_0000 * (i + 1)


@pytest.fixture(scope="module")
def lib():
    cfc_build.build()
    return cfc.load_library()


def conv_in(**kw):
    a = dict(x=far(0), ldx=128, w=far(1), b=far(2), off=None, n_seq=3, rows=30, d=64, W=4, silu=1, math=BF16, init=far(3))
    a.update(kw)
    return a


def conv_forward(lib, y=far(4), final=far(5), **kw):
    return lib.cfc_conv_forward(*conv_in(**kw).values(), y, final, None)


def conv_backward(lib, gy=far(4), gfinal=far(5), gx=far(6), gw=far(7), gb=far(8), ginit=far(9), ws=far(10), ws_bytes=BIG, **kw):
    return lib.cfc_conv_backward(*conv_in(**kw).values(), gy, gfinal, gx, gw, gb, ginit, ws, ws_bytes, None)


def conv_step(lib, **kw):
    a = dict(x=far(0), ldx=128, w=far(1), b=far(2), n_seq=3, tokens=2, d=64, W=4, silu=1, math=BF16, state=far(3), n_slots=3,
             slots=None, y=far(4))
    a.update(kw)
    return lib.cfc_conv_step(*a.values(), None)


SCAN = dict(x=far(0), ldx=128, delta=far(1), ldd=64, A=far(2), B=far(3), ldb=40, C=far(4), ldc=40, D=far(5), z=far(6), ldz=128,
            bias=far(7))


def scan_forward(lib, y=far(8), final=far(9), save=0, ws=far(10), ws_bytes=BIG, **kw):
    a = dict(SCAN, off=None, n_seq=3, rows=30, d=64, groups=2, N=16, math=BF16, init=far(11))
    a.update(kw)
    return lib.cfc_ssm_forward(*a.values(), y, final, save, ws, ws_bytes, None)


def scan_backward(lib, ws=far(10), ws_bytes=BIG, **kw):
    a = dict(SCAN, off=None, n_seq=3, rows=30, d=64, groups=2, N=16, math=BF16, init=far(11), gy=far(12), gfinal=far(13),
             gx=far(14), gdelta=far(15), gA=far(16), gB=far(17), gC=far(18), gD=far(19), gz=far(20), gbias=far(21), ginit=far(22))
    a.update(kw)
    return lib.cfc_ssm_backward(*a.values(), ws, ws_bytes, None)


def scan_step(lib, **kw):
    a = dict(SCAN, n_seq=3, tokens=2, d=64, groups=2, N=16, math=BF16, state=far(8), n_slots=3, slots=None, y=far(9))
    a.update(kw)
    return lib.cfc_ssm_step(*a.values(), None)


CONVS, SCANS = [conv_forward, conv_backward, conv_step], [scan_forward, scan_backward, scan_step]


@pytest.mark.parametrize("call", CONVS)
@pytest.mark.parametrize("bad", [dict(d=60), dict(d=0), dict(d=-8), dict(d=(1 << 20) + 8, ldx=1 << 21), dict(W=1), dict(W=9),
                                 dict(ldx=56), dict(ldx=132), dict(ldx=-128)], ids=str)
def test_conv_refuses_shapes(lib, call, bad):
    assert call(lib, **bad) == ERR_SHAPE


@pytest.mark.parametrize("call", SCANS)
@pytest.mark.parametrize("bad", [dict(d=60), dict(d=0), dict(groups=0), dict(groups=3), dict(groups=16), dict(N=0), dict(N=65),
                                 dict(ldx=56), dict(ldx=132), dict(ldd=60), dict(ldz=68), dict(ldb=31), dict(ldc=31),
                                 dict(ldb=-40), dict(d=1 << 19, ldx=1 << 19, ldd=1 << 19, ldz=1 << 19, groups=1 << 16, N=2,
                                                     ldb=1 << 20, ldc=1 << 20)], ids=str)
def test_scan_refuses_shapes(lib, call, bad):
    assert call(lib, **bad) == ERR_SHAPE


@pytest.mark.parametrize("call", [conv_forward, conv_backward, scan_forward, scan_backward])
@pytest.mark.parametrize("bad", [dict(n_seq=0), dict(n_seq=(1 << 20) + 1, off=far(30)), dict(rows=-1), dict(rows=31),
                                 dict(rows=(1 << 30) + 3)], ids=str)
def test_sequences_refused(lib, call, bad):
    assert call(lib, **bad) == ERR_SHAPE


@pytest.mark.parametrize("call", [conv_step, scan_step])
@pytest.mark.parametrize("bad", [dict(n_seq=-1), dict(tokens=-1), dict(n_slots=-1, slots=far(30)), dict(n_slots=2),
                                 dict(n_seq=1 << 20, tokens=1 << 11, slots=far(30)), dict(n_seq=(1 << 20) + 1, slots=far(30))],
                         ids=str)
def test_steps_refuse_sizes(lib, call, bad):
    assert call(lib, **bad) == ERR_SHAPE


@pytest.mark.parametrize("call", CONVS + SCANS)
@pytest.mark.parametrize("math", [TF32, 3, -1])
def test_modes_refused(lib, call, math):
    assert call(lib, math=math) == ERR_MODE


@pytest.mark.parametrize("call,names", [
    (conv_forward, "x w y"), (conv_backward, "x w gy gx gw"), (conv_step, "x w y state"),
    (scan_forward, "x delta A B C y"), (scan_backward, "x delta A B C gy gx gdelta gA gB gC gz"),
    (scan_step, "x delta A B C y state")])
def test_null_refused(lib, call, names):
    for n in names.split():
        assert call(lib, **{n: None}) == ERR_NULL, n


@pytest.mark.parametrize("call,wide,narrow,two", [
    (conv_forward, "x w init y final", "b off", ""), (conv_backward, "x w init gy gfinal gx gw ginit ws", "b off gb", ""),
    (conv_step, "x w state y", "b slots", ""),
    (scan_forward, "x delta z y init final ws", "A D bias off", "B C"),
    (scan_backward, "x delta z init gy gfinal gx gdelta gz ginit ws", "A D bias off gA gB gC gD gbias", "B C"),
    (scan_step, "x delta z state y", "A D bias slots", "B C")])
def test_misaligned_refused(lib, call, wide, narrow, two):
    for names, by in ((wide, 8), (narrow, 2), (two, 1)):
        for n in names.split():
            assert call(lib, **{n: far(40) + by}) == ERR_ALIGN, n


def test_overlap_refused(lib):
    assert conv_forward(lib, y=far(0)) == ERR_OVERLAP                   # tiles read their neighbours' rows of x
    assert conv_forward(lib, y=far(0) + 29 * 128 * 2) == ERR_OVERLAP
    assert conv_forward(lib, final=far(3)) == ERR_OVERLAP and conv_step(lib, y=far(0)) == ERR_OVERLAP
    assert conv_backward(lib, gx=far(4)) == ERR_OVERLAP and conv_backward(lib, gx=far(0)) == ERR_OVERLAP
    assert conv_backward(lib, ginit=far(5)) == ERR_OVERLAP
    for y in (0, 1, 6):
        assert scan_forward(lib, y=far(y)) == ERR_OVERLAP and scan_step(lib, y=far(y)) == ERR_OVERLAP
    assert scan_forward(lib, final=far(11)) == ERR_OVERLAP
    assert scan_backward(lib, gx=far(12)) == ERR_OVERLAP and scan_backward(lib, gz=far(14)) == ERR_OVERLAP
    assert scan_backward(lib, ginit=far(13)) == ERR_OVERLAP


def test_small_workspaces_refused(lib):
    need = cfc.cfc_conv_workspace_bytes(30, 64, 4)
    assert conv_backward(lib, ws_bytes=need - 1) == ERR_WORKSPACE and conv_backward(lib, ws=None) == ERR_WORKSPACE
    for save, call in ((0, scan_forward), (1, scan_forward), (1, scan_backward)):
        need = cfc.cfc_ssm_workspace_bytes(30, 3, 64, 2, 16, BF16, save)
        kw = {"save": save} if call is scan_forward else {}
        assert call(lib, ws_bytes=need - 1, **kw) == ERR_WORKSPACE and call(lib, ws=None, **kw) == ERR_WORKSPACE


def test_workspace_sizes(lib):
    size = cfc.cfc_ssm_workspace_bytes
    for math in (FP32, BF16):
        assert 0 < size(0, 1, 8, 1, 1, math) <= size(1000, 4, 64, 2, 16, math) < size(1000, 4, 64, 2, 16, math, True)
    for bad in [(-1, 1, 8, 1, 1, BF16), ((1 << 30) + 1, 1, 8, 1, 1, BF16), (10, 0, 8, 1, 1, BF16), (10, 1, 12, 1, 1, BF16),
                (10, 1, 16, 4, 1, BF16), (10, 1, 8, 1, 65, BF16), (10, 1, 8, 1, 0, BF16), (10, 1, 8, 1, 1, TF32)]:
        assert size(*bad) == 0, bad
    assert size(1 << 30, 1, 4096, 1, 16, BF16, True) > 1 << 40          # sizes are 64-bit
    conv = cfc.cfc_conv_workspace_bytes
    assert conv(0, 8, 2) > 0 and conv(100000, 64, 4, FP32) > 0
    for bad in [(-1, 8, 2), (1, 12, 2), (1, 8, 1), (1, 8, 9), (1, 8, 2, TF32)]:
        assert conv(*bad) == 0, bad


def test_steps_of_nothing_are_ok(lib):
    for call in (conv_step, scan_step):
        assert call(lib, n_seq=0, n_slots=0, state=None, x=None) == 0
        assert call(lib, tokens=0, x=None) == 0


def norm(lib, **kw):
    a = dict(x=far(0), residual=None, weight=far(1), bias=None, rows=4, d=64, eps=1e-5, math=BF16, y=far(2), s=None, mean=None,
             rstd=None)
    a.update(kw)
    return lib.cfc_layernorm_forward(*a.values(), None)


def norm_back(lib, **kw):
    a = dict(s=far(0), weight=far(1), mean=far(2), rstd=far(3), gy=far(4), carry=None, rows=4, d=64, math=BF16, gx=far(5),
             gw=far(6), gb=None, ws=far(7), ws_bytes=BIG)
    a.update(kw)
    return lib.cfc_layernorm_backward(*a.values(), None)


def test_norm_refusals(lib):
    for call in (norm, norm_back):
        for math in (TF32, 5):
            assert call(lib, math=math) == ERR_MODE
        for bad in (dict(rows=-1), dict(d=0), dict(d=32769), dict(rows=(1 << 40) + 1)):
            assert call(lib, **bad) == ERR_SHAPE, bad
    for n in ("x", "weight", "y"):
        assert norm(lib, **{n: None}) == ERR_NULL, n
    for n in ("x", "residual", "weight", "bias", "y", "s"):
        assert norm(lib, **{n: far(9) + 8}) == ERR_ALIGN, n
    for n in ("mean", "rstd"):
        assert norm(lib, **{n: far(9) + 2}) == ERR_ALIGN, n
        assert norm_back(lib, **{n: far(9) + 2}) == ERR_ALIGN, n
    assert norm(lib, rows=0, x=None) == 0
    for n in ("s", "weight", "mean", "rstd", "gy", "gx", "gw"):
        assert norm_back(lib, **{n: None}) == ERR_NULL, n
    for n in ("s", "weight", "gy", "carry", "gx", "gw", "gb", "ws"):
        assert norm_back(lib, **{n: far(9) + 8}) == ERR_ALIGN, n
    assert norm_back(lib, ws_bytes=cfc.cfc_layernorm_workspace_bytes(4, 64) - 1) == ERR_WORKSPACE
    assert norm_back(lib, ws=None) == ERR_WORKSPACE
    assert cfc.cfc_layernorm_workspace_bytes(1 << 30, 64) == cfc.cfc_layernorm_workspace_bytes(1 << 20, 64)
    for bad in [(-1, 64), (1, 0), (1, 32769)]:
        assert cfc.cfc_layernorm_workspace_bytes(*bad) == 0


def grads(lib, clip, most=1.0, norm=far(50), ws=far(51), ws_bytes=BIG, count=None, ptrs=(far(0), far(1)), outs=None, n=(10, 3),
          math=(FP32, BF16)):
    k = len(ptrs)
    arr = [(ctypes.c_void_p * k)(*ptrs), (ctypes.c_longlong * k)(*n), (ctypes.c_int * k)(*math)]
    count = k if count is None else count
    if not clip:
        return lib.cfc_grad_norm(*arr, count, norm, ws, ws_bytes, None)
    o = (ctypes.c_void_p * k)(*(ptrs if outs is None else outs))
    return lib.cfc_grad_clip(arr[0], o, arr[1], arr[2], count, most, norm, ws, ws_bytes, None)


@pytest.mark.parametrize("clip", [False, True])
def test_grad_refusals(lib, clip):
    assert grads(lib, clip, count=-1) == ERR_SHAPE and grads(lib, clip, count=65537) == ERR_SHAPE
    assert grads(lib, clip, n=(-1, 3)) == ERR_SHAPE and grads(lib, clip, n=((1 << 35) + 1, 3)) == ERR_SHAPE
    assert grads(lib, clip, math=(FP32, TF32)) == ERR_MODE
    assert grads(lib, clip, ptrs=(far(0), None)) == ERR_NULL and grads(lib, clip, norm=None) == ERR_NULL
    assert grads(lib, clip, ptrs=(far(0) + 2, far(1))) == ERR_ALIGN and grads(lib, clip, ptrs=(far(0), far(1) + 1)) == ERR_ALIGN
    assert grads(lib, clip, norm=far(50) + 2) == ERR_ALIGN and grads(lib, clip, ws=far(51) + 8) == ERR_ALIGN
    assert grads(lib, clip, ws=None) == ERR_WORKSPACE
    assert grads(lib, clip, ws_bytes=cfc.cfc_grad_clip_workspace_bytes(2) - 1) == ERR_WORKSPACE
    if clip:
        for most in (-1.0, float("nan")):
            assert grads(lib, True, most=most) == ERR_SHAPE
        assert grads(lib, True, outs=(far(0) + 4, far(3))) == ERR_OVERLAP
        assert grads(lib, True, outs=(None, far(3))) == ERR_NULL
        assert grads(lib, True, ptrs=(far(0), far(1)), outs=(far(1), far(0))) == ERR_OVERLAP       # of each other
        assert grads(lib, True, ptrs=(far(0), far(1)), outs=(far(2), far(2))) == ERR_OVERLAP
        assert grads(lib, True, ptrs=(far(0), far(0)), outs=(far(0), far(0))) == ERR_OVERLAP       # in place twice
        assert grads(lib, True, ptrs=(far(0), far(0)), outs=(far(0), far(3))) == ERR_OVERLAP
    assert cfc.cfc_grad_clip_workspace_bytes(-1) == 0 and cfc.cfc_grad_clip_workspace_bytes(65537) == 0
    assert cfc.cfc_grad_clip_workspace_bytes(0) > 0


def test_the_binding_refuses_host_tensors_and_wrong_lists():
    torch = pytest.importorskip("torch")
    t = torch.zeros(2, 3, 8)
    with pytest.raises(TypeError, match="CUDA tensor"):
        cfc.cfc_conv_forward(t, torch.zeros(8, 4), t, math=FP32)
    with pytest.raises(ValueError, match="channels, width"):
        cfc.cfc_conv_forward(t, torch.zeros(8), t, math=FP32)
    with pytest.raises(TypeError, match="CUDA tensor"):
        cfc.cfc_layernorm_forward(t[0], torch.ones(8), t[0], math=FP32)
    with pytest.raises(ValueError, match="groups, states"):
        cfc.cfc_ssm_forward(t, t, torch.zeros(8, 4), t, t, t, t, math=FP32)
    with pytest.raises(TypeError, match=r"grads\[0\] must be a CUDA tensor"):
        cfc.cfc_grad_norm([t], torch.zeros(1), torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(TypeError, match="CUDA tensor"):
        cfc.cfc_grad_clip([3], 1.0, torch.zeros(1), torch.zeros(8, dtype=torch.uint8))


def test_a_trunk_of_an_unknown_kind_is_refused():
    pytest.importorskip("torch")
    from recurrent_cell_gb300.memory import MemoryCell
    with pytest.raises(ValueError, match="kind"):
        MemoryCell(16, 8, device="cpu", kind="other")


# (call, what it writes, a pool of states and the workspace among it, and what it only reads)
APART = [
    (conv_forward, "y final", "x w b off init"),
    (conv_backward, "gx gw gb ginit ws", "x w b off init gy gfinal"),
    (conv_step, "y state", "x w b slots"),
    (scan_forward, "y final ws", "x delta A B C D z bias off init"),
    (scan_backward, "gx gdelta gA gB gC gD gz gbias ginit ws", "x delta A B C D z bias off init gy gfinal"),
    (scan_step, "y state", "x delta A B C D z bias slots"),
]


@pytest.mark.parametrize("call,outs,ins", APART, ids=lambda v: getattr(v, "__name__", ""))
def test_no_output_may_overlap_anything(lib, call, outs, ins):
    """Every output against every input and every other output."""
    outs, ins = outs.split(), ins.split()
    where = {n: far(100 + i) for i, n in enumerate(outs + ins)}
    given = dict(where)
    if "slots" in ins:
        given["n_slots"] = 5                     # a pool of more slots than sequences
    for i, out in enumerate(outs):
        for other in ins + outs[:i]:
            for a, b in ((out, other), (other, out)):
                assert call(lib, **dict(given, **{a: where[b]})) == ERR_OVERLAP, (a, "at", b)


def test_the_last_rows_and_slots_count(lib):
    """Ranges end where the tensors do: in rows that are parts of wider ones, and in the last slot of a pool."""
    row = 2 * 40                                 # of B and C, in bytes; x's are 256 and hold 128, delta's 128
    for call in (scan_forward, scan_step):
        rows = 30 if call is scan_forward else 6
        for n in ("B", "C"):
            assert call(lib, y=SCAN[n] + (rows - 1) * row // 16 * 16) == ERR_OVERLAP
        assert call(lib, y=SCAN["z"] + (rows - 1) * 256 + 112) == ERR_OVERLAP
    slot = 64 * 16 * 4
    assert scan_step(lib, n_slots=9, y=far(8) + 9 * slot - 16) == ERR_OVERLAP
    assert scan_step(lib, n_slots=9, x=far(8) + 9 * slot - 16) == ERR_OVERLAP
    assert conv_step(lib, n_slots=9, y=far(3) + 9 * 3 * 64 * 2 - 16) == ERR_OVERLAP
    assert conv_step(lib, n_slots=1 << 62, slots=far(30), y=far(50)) == ERR_OVERLAP
    assert scan_backward(lib, gB=far(18) + 16, gC=far(18)) == ERR_OVERLAP and scan_backward(lib, gA=far(21)) == ERR_OVERLAP


@pytest.mark.parametrize("clip", [False, True])
def test_the_norm_and_the_sums_lie_in_no_tensor(lib, clip):
    need = cfc.cfc_grad_clip_workspace_bytes(2)
    assert grads(lib, clip, ws=far(0) + 32) == ERR_OVERLAP and grads(lib, clip, ws=far(1) - need + 16) == ERR_OVERLAP
    assert grads(lib, clip, ws=far(60), norm=far(60) + need - 4) == ERR_OVERLAP
    if clip:
        for at in (far(0), far(0) + 36, far(1) + 4):
            assert grads(lib, clip, outs=(far(2), far(3)), norm=at) == ERR_OVERLAP        # written while others are read
            assert grads(lib, clip, norm=at) == ERR_OVERLAP
        assert grads(lib, clip, outs=(far(2), far(3)), norm=far(2) + 36) == ERR_OVERLAP
        assert grads(lib, clip, outs=(far(2), far(3)), ws=far(3) - need + 16) == ERR_OVERLAP
