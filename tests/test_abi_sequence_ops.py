"""Argument checks of the gated delta rule and the residual norm at the C ABI:
what is refused, with which status, before anything is launched (no GPU; the
addresses are never dereferenced)."""

import pytest

import recurrent_cell_gb300 as cfc
from recurrent_cell_gb300 import build as cfc_build

ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_MODE = -1, -2, -3, -4, -5
FP32, TF32, BF16 = cfc.MATH_FP32, cfc.MATH_TF32, cfc.MATH_BF16
P = 0x100000          # fake and aligned
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    cfc_build.build()
    return cfc.load_library()


SIZES = dict(n_seq=3, rows=30, hk=2, hv=4, dk=64, dv=40, scale=1.0, math=BF16)


def forward(lib, **kw):
    a = dict(q=P, ldq=128, k=P, ldk=128, v=P, ldv=160, g=P, beta=P, off=None, **SIZES, init=None, o=P, final=None,
             save=0, ws=P, ws_bytes=BIG)
    a.update(kw)
    return lib.cfc_gdr_forward(*a.values(), None)


def backward(lib, **kw):
    a = dict(q=P, ldq=128, k=P, ldk=128, v=P, ldv=160, g=P, beta=P, off=None, **SIZES, go=P, gfinal=None, gq=P, gk=P,
             gv=P, gg=P, gb=P, ginit=None, ws=P, ws_bytes=BIG)
    a.update(kw)
    return lib.cfc_gdr_backward(*a.values(), None)


def step(lib, **kw):
    a = dict(q=P, ldq=128, k=P, ldk=128, v=P, ldv=160, g=P, beta=P, n_seq=3, tokens=1, hk=2, hv=4, dk=64, dv=40,
             scale=1.0, math=BF16, state=P, n_slots=3, slots=None, o=P)
    a.update(kw)
    return lib.cfc_gdr_step(*a.values(), None)


BAD_SHAPES = [dict(dk=60), dict(dk=0), dict(dk=136, ldq=512, ldk=512), dict(dv=44), dict(dv=264, ldv=2048), dict(hk=0),
              dict(hk=3), dict(hv=5), dict(hv=4098, hk=2, ldv=1 << 20), dict(ldq=120), dict(ldk=132), dict(ldv=152),
              dict(ldv=164), dict(ldq=-128)]


@pytest.mark.parametrize("call", [forward, backward, step])
@pytest.mark.parametrize("bad", BAD_SHAPES, ids=str)
def test_rule_refuses_shapes(lib, call, bad):
    assert call(lib, **bad) == ERR_SHAPE


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("bad", [dict(n_seq=0), dict(n_seq=(1 << 20) + 1, off=P), dict(rows=-1), dict(rows=31),
                                 dict(rows=(1 << 30) + 3), dict(rows=1 << 30, n_seq=1 << 20, hk=2048, hv=4096, ldq=1 << 17,
                                                                ldk=1 << 17, ldv=1 << 18)], ids=str)
def test_rule_refuses_sequences(lib, call, bad):
    assert call(lib, **bad) == ERR_SHAPE


@pytest.mark.parametrize("bad", [dict(n_seq=-1), dict(tokens=-1), dict(n_slots=-1, slots=P), dict(n_slots=2),
                                 dict(n_seq=1 << 30, tokens=2, slots=P)], ids=str)
def test_step_refuses_sizes(lib, bad):
    assert step(lib, **bad) == ERR_SHAPE


@pytest.mark.parametrize("call", [forward, backward, step])
@pytest.mark.parametrize("math", [TF32, 3, -1])
def test_rule_refuses_modes(lib, call, math):
    assert call(lib, math=math) == ERR_MODE


@pytest.mark.parametrize("call,names", [(forward, "q k v g beta o"), (backward, "q k v g beta go gq gk gv gg gb"),
                                        (step, "q k v g beta o state")])
def test_rule_refuses_null(lib, call, names):
    for n in names.split():
        assert call(lib, **{n: None}) == ERR_NULL, n


@pytest.mark.parametrize("call,wide,narrow", [
    (forward, "q k v o init final ws", "g beta off"),
    (backward, "q k v go gfinal gq gk gv ginit ws", "g beta off gg gb"),
    (step, "q k v o state", "g beta slots")])
def test_rule_refuses_misaligned(lib, call, wide, narrow):
    for n in wide.split():
        assert call(lib, **{n: P + 8}) == ERR_ALIGN, n
    for n in narrow.split():
        assert call(lib, **{n: P + 2}) == ERR_ALIGN, n


def test_rule_refuses_a_small_workspace(lib):
    for save, call in ((0, forward), (1, forward), (1, backward)):
        need = cfc.cfc_gdr_workspace_bytes(30, 3, 2, 4, 64, 40, BF16, save)
        kw = {"save": save} if call is forward else {}
        assert call(lib, ws_bytes=need - 1, **kw) == ERR_WORKSPACE
        assert call(lib, ws=None, **kw) == ERR_WORKSPACE


def test_rule_workspace(lib):
    size = cfc.cfc_gdr_workspace_bytes
    for math in (FP32, BF16):
        assert 0 < size(0, 1, 1, 1, 8, 8, math) <= size(1000, 4, 2, 4, 64, 64, math) < size(1000, 4, 2, 4, 64, 64, math, True)
    for bad in [(-1, 1, 1, 1, 8, 8, BF16), ((1 << 30) + 1, 1, 1, 1, 8, 8, BF16), (10, 0, 1, 1, 8, 8, BF16),
                (10, 1, 2, 3, 8, 8, BF16), (10, 1, 1, 1, 12, 8, BF16), (10, 1, 1, 1, 8, 12, BF16), (10, 1, 1, 1, 8, 8, TF32),
                (10, 1, 1, 1, 136, 8, BF16), (10, 1, 1, 1, 8, 264, BF16)]:
        assert size(*bad) == 0, bad
    assert size(1 << 30, 1, 64, 64, 128, 128, BF16, True) > 1 << 40          # sizes are 64-bit


def test_step_of_nothing_is_ok(lib):
    assert step(lib, n_seq=0, n_slots=0, state=None, q=None) == 0
    assert step(lib, tokens=0, q=None) == 0


def norm(lib, **kw):
    a = dict(x=P, residual=None, weight=P, rows=4, d=64, eps=1e-6, math=BF16, y=P, s=None, rstd=None, y8=None, scale=None,
             group=64)
    a.update(kw)
    return lib.cfc_rmsnorm_forward(*a.values(), None)


def norm_back(lib, **kw):
    a = dict(s=P, weight=P, rstd=P, gy=P, carry=None, rows=4, d=64, math=BF16, gx=P, gw=P, ws=P, ws_bytes=BIG)
    a.update(kw)
    return lib.cfc_rmsnorm_backward(*a.values(), None)


def test_norm_refusals(lib):
    for call in (norm, norm_back):
        for math in (TF32, 5):
            assert call(lib, math=math) == ERR_MODE
        for bad in (dict(rows=-1), dict(d=0), dict(d=32769), dict(rows=(1 << 40) + 1)):
            assert call(lib, **bad) == ERR_SHAPE, bad
    for group in (0, -1, 65, 48):
        assert norm(lib, y8=P, scale=P, group=group) == ERR_SHAPE
    for bad in (dict(x=None), dict(weight=None), dict(y=None), dict(y8=P)):
        assert norm(lib, **bad) == ERR_NULL, bad
    for n in ("x", "residual", "weight", "y", "s"):
        assert norm(lib, **{n: P + 8}) == ERR_ALIGN, n
    assert norm(lib, y8=P + 8, scale=P) == ERR_ALIGN
    assert norm(lib, rstd=P + 2) == ERR_ALIGN and norm(lib, y8=P, scale=P + 2) == ERR_ALIGN
    assert norm(lib, rows=0, x=None) == 0
    for n in ("s", "weight", "rstd", "gy", "gx", "gw"):
        assert norm_back(lib, **{n: None}) == ERR_NULL, n
    for n in ("s", "weight", "gy", "carry", "gx", "gw", "ws"):
        assert norm_back(lib, **{n: P + 8}) == ERR_ALIGN, n
    assert norm_back(lib, rstd=P + 2) == ERR_ALIGN
    assert norm_back(lib, ws_bytes=cfc.cfc_rmsnorm_workspace_bytes(4, 64) - 1) == ERR_WORKSPACE
    assert norm_back(lib, ws=None) == ERR_WORKSPACE


def test_norm_workspace(lib):
    size = cfc.cfc_rmsnorm_workspace_bytes
    assert size(0, 64) > 0 and size(10, 64) >= 10 * 64 * 4
    assert size(1 << 30, 64) == size(1 << 20, 64)            # a fixed number of partial sums
    for bad in [(-1, 64), (1, 0), (1, 32769)]:
        assert size(*bad) == 0


def test_current_stream_without_torchs_private_calls(monkeypatch):
    """The binding takes the current stream's handle from the public API where torch lacks the short way."""
    class Cuda:
        current_device = staticmethod(lambda: 3)
        current_stream = staticmethod(lambda d: type("Stream", (), {"cuda_stream": 1000 + d}))

    monkeypatch.setattr(cfc, "_torch_module", type("Torch", (), {"cuda": Cuda, "_C": object()}))
    monkeypatch.setattr(cfc, "_raw_stream", None)
    assert cfc._stream(None) == 1003
