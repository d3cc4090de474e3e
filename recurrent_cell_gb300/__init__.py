"""Python binding of libcfc (the C ABI in include/cfc.h).

The functions below carry the same names as the C entry points and do
argument marshalling only: they check dtypes/devices/shapes of torch tensors,
pass raw device pointers and the current CUDA stream, and raise on a non-zero
status.  All arithmetic runs in the library's CUDA kernels.  PyTorch is used
for device memory and streams.

There is no fallback: if libcfc.so is missing or cannot be loaded, every call
raises.
"""

from __future__ import annotations

import ctypes
import os
from array import array

from .workloads import (  # noqa: F401
    MATH_FP32, MATH_TF32, MATH_BF16, GRAD_SCRATCH, GRAD_GEMM,
)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcfc.so")

CFC_OK = 0
_lib = None


class CfcError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed with status {status}: {cfc_status_string(status)}")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libcfc.so (build it first with recurrent_cell_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libcfc.so not found at {path}: run `python -m recurrent_cell_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    lib.cfc_status_string.argtypes = [i32]
    lib.cfc_status_string.restype = ctypes.c_char_p
    lib.cfc_per_sample_length.argtypes = [i32, i32]
    lib.cfc_per_sample_length.restype = i64
    lib.cfc_kloop_workspace_bytes.argtypes = [i32] * 6
    lib.cfc_kloop_workspace_bytes.restype = sz
    lib.cfc_kloop_forward.argtypes = [vp] * 6 + [i32] * 6 + [vp, vp, sz, vp]
    lib.cfc_kloop_forward.restype = i32
    lib.cfc_kloop_backward.argtypes = ([vp] * 6 + [i32] * 6 + [vp] * 4 + [vp] * 5 + [vp, i32]
                                       + [vp, sz, vp])
    lib.cfc_kloop_backward.restype = i32
    lib.reduce_axis0.argtypes = [vp, i32, i64, vp, vp]
    lib.reduce_axis0.restype = i32
    lib.reduce_axis0_multi.argtypes = [vp, vp, vp, vp, i32, vp]
    lib.reduce_axis0_multi.restype = i32
    lib.cfc_tau_per_sample_length.argtypes = [i32, i32]
    lib.cfc_tau_per_sample_length.restype = i64
    lib.cfc_tau_kloop_workspace_bytes.argtypes = [i32] * 4
    lib.cfc_tau_kloop_workspace_bytes.restype = sz
    lib.cfc_tau_kloop_forward.argtypes = [vp] * 7 + [i32] * 5 + [vp, vp, sz, vp]
    lib.cfc_tau_kloop_forward.restype = i32
    lib.cfc_tau_kloop_backward.argtypes = [vp] * 7 + [i32] * 5 + [vp] * 4 + [vp] * 7 + [vp, sz, vp]
    lib.cfc_tau_kloop_backward.restype = i32
    lib.cfc_grn_param_length.argtypes = [i32, i32, i32]
    lib.cfc_grn_param_length.restype = i64
    lib.cfc_grn_saved_per_row.argtypes = [i32, i32]
    lib.cfc_grn_saved_per_row.restype = i64
    lib.cfc_grn_workspace_bytes.argtypes = [i32] * 5
    lib.cfc_grn_workspace_bytes.restype = sz
    lib.cfc_grn_forward.argtypes = [vp, i64, i32, i32, i32, vp, vp, vp, vp]
    lib.cfc_grn_forward.restype = i32
    lib.cfc_grn_backward.argtypes = [vp] + [i32] * 5 + [vp] * 9 + [vp, sz, vp]
    lib.cfc_grn_backward.restype = i32
    lib.cfc_kloop_forward_backward_static.argtypes = [vp] * 6 + [i32] * 6 + [vp] * 3 + [vp] * 6 + [vp]
    lib.cfc_kloop_forward_backward_static.restype = i32
    gdr_in = [vp, i64, vp, i64, vp, i64, vp, vp]
    lib.cfc_gdr_workspace_bytes.argtypes = [i64] + [i32] * 7
    lib.cfc_gdr_workspace_bytes.restype = sz
    lib.cfc_gdr_forward.argtypes = (gdr_in + [vp, i32, i64] + [i32] * 4 + [ctypes.c_float, i32] + [vp] * 3
                                    + [i32, vp, sz, vp])
    lib.cfc_gdr_forward.restype = i32
    lib.cfc_gdr_backward.argtypes = (gdr_in + [vp, i32, i64] + [i32] * 4 + [ctypes.c_float, i32] + [vp] * 9
                                     + [sz, vp])
    lib.cfc_gdr_backward.restype = i32
    lib.cfc_gdr_step.argtypes = gdr_in + [i32] * 6 + [ctypes.c_float, i32, vp, i64, vp, vp, vp]
    lib.cfc_gdr_step.restype = i32
    lib.cfc_rmsnorm_forward.argtypes = [vp] * 3 + [i64, i32, ctypes.c_float, i32] + [vp] * 5 + [i32, vp]
    lib.cfc_rmsnorm_forward.restype = i32
    lib.cfc_rmsnorm_workspace_bytes.argtypes = [i64, i32]
    lib.cfc_rmsnorm_workspace_bytes.restype = sz
    lib.cfc_rmsnorm_backward.argtypes = [vp] * 5 + [i64, i32, i32] + [vp] * 3 + [sz, vp]
    lib.cfc_rmsnorm_backward.restype = i32
    lib.cfc_layernorm_forward.argtypes = [vp] * 4 + [i64, i32, ctypes.c_float, i32] + [vp] * 5
    lib.cfc_layernorm_forward.restype = i32
    lib.cfc_layernorm_workspace_bytes.argtypes = [i64, i32]
    lib.cfc_layernorm_workspace_bytes.restype = sz
    lib.cfc_layernorm_backward.argtypes = [vp] * 6 + [i64, i32, i32] + [vp] * 4 + [sz, vp]
    lib.cfc_layernorm_backward.restype = i32
    conv_in = [vp, i64, vp, vp]
    lib.cfc_conv_forward.argtypes = conv_in + [vp, i32, i64] + [i32] * 4 + [vp] * 4
    lib.cfc_conv_forward.restype = i32
    lib.cfc_conv_workspace_bytes.argtypes = [i64] + [i32] * 3
    lib.cfc_conv_workspace_bytes.restype = sz
    lib.cfc_conv_backward.argtypes = conv_in + [vp, i32, i64] + [i32] * 4 + [vp] * 8 + [sz, vp]
    lib.cfc_conv_backward.restype = i32
    lib.cfc_conv_step.argtypes = conv_in + [i32] * 6 + [vp, i64, vp, vp, vp]
    lib.cfc_conv_step.restype = i32
    ssm_in = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, i64, vp]
    lib.cfc_ssm_workspace_bytes.argtypes = [i64] + [i32] * 6
    lib.cfc_ssm_workspace_bytes.restype = sz
    lib.cfc_ssm_forward.argtypes = ssm_in + [vp, i32, i64] + [i32] * 4 + [vp] * 3 + [i32, vp, sz, vp]
    lib.cfc_ssm_forward.restype = i32
    lib.cfc_ssm_backward.argtypes = ssm_in + [vp, i32, i64] + [i32] * 4 + [vp] * 13 + [sz, vp]
    lib.cfc_ssm_backward.restype = i32
    lib.cfc_ssm_step.argtypes = ssm_in + [i32] * 6 + [vp, i64, vp, vp, vp]
    lib.cfc_ssm_step.restype = i32
    lib.cfc_grad_clip_workspace_bytes.argtypes = [i32]
    lib.cfc_grad_clip_workspace_bytes.restype = sz
    lib.cfc_grad_norm.argtypes = [vp] * 3 + [i32, vp, vp, sz, vp]
    lib.cfc_grad_norm.restype = i32
    lib.cfc_grad_clip.argtypes = [vp] * 4 + [i32, ctypes.c_float, vp, vp, sz, vp]
    lib.cfc_grad_clip.restype = i32
    lib.cfc_kloop_grad_splits.argtypes = [i32] * 6
    lib.cfc_kloop_grad_splits.restype = i32
    lib.cfc_device_error.argtypes = [i32]
    lib.cfc_device_error.restype = i32
    lib.cfc_selftest_timeout.argtypes = [i32, vp]
    lib.cfc_selftest_timeout.restype = i32
    lib.cfc_trace_enable.argtypes = [i32]
    lib.cfc_trace_enable.restype = i32
    lib.cfc_trace_count.argtypes = []
    lib.cfc_trace_count.restype = i32
    lib.cfc_trace_get.argtypes = [i32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float)]
    lib.cfc_trace_get.restype = i32
    _lib = lib
    return lib


def cfc_status_string(status: int) -> str:
    return load_library().cfc_status_string(int(status)).decode()


def cfc_per_sample_length(n_in: int, n_hid: int) -> int:
    return int(load_library().cfc_per_sample_length(n_in, n_hid))


def cfc_kloop_workspace_bytes(B, K, n_in, n_hid, math, grad_path=GRAD_SCRATCH) -> int:
    return int(load_library().cfc_kloop_workspace_bytes(B, K, n_in, n_hid, math, grad_path))


def cfc_kloop_grad_splits(B, K, n_in, n_hid, math, grad_path=GRAD_SCRATCH) -> int:
    return int(load_library().cfc_kloop_grad_splits(B, K, n_in, n_hid, math, grad_path))


def cfc_device_error(clear: bool = False) -> int:
    """0 unless a kernel reported a device-side error (waits for the device)."""
    return int(load_library().cfc_device_error(1 if clear else 0))


def cfc_selftest_timeout(max_polls: int = 1000, stream=None) -> None:
    """Run one bounded wait that runs out (see include/cfc.h); afterwards
    cfc_device_error() reports 1 until cleared."""
    _check("cfc_selftest_timeout", load_library().cfc_selftest_timeout(int(max_polls), _stream(stream)))


_torch_module = None
_storage = {}


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_raw_stream = None


def _stream(stream):
    global _raw_stream
    if stream is None:
        # the current stream's handle without building a Stream object, where
        # torch has the two calls: the binding is most of a small call's time
        if _raw_stream is None:
            torch = _torch()
            torch.cuda.current_device()             # brings CUDA up
            get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            device = getattr(torch._C, "_cuda_getDevice", None)
            if get is None or device is None:       # not public names
                get, device = lambda d: torch.cuda.current_stream(d).cuda_stream, torch.cuda.current_device
            _raw_stream = get, device
        return _raw_stream[0](_raw_stream[1]())
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t, name, dtype=None, shape=None, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    try:        # the usual case in few steps: the checks are a good part of a small call
        if (dtype is None or t.dtype is dtype) and (shape is None or t.shape == shape) and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _storage_dtype(math):
    st = _storage.get(math)
    if st is None:
        torch = _torch()
        st = _storage[math] = torch.bfloat16 if math == MATH_BF16 else torch.float32
    return st


def _check(fn, status):
    if status != CFC_OK:
        raise CfcError(fn, status)


def cfc_kloop_forward(x, h0, W_in, W_rec, b, dt, h_seq, workspace, math=MATH_FP32, stream=None):
    """Forward K-loop: writes h_seq [B, K, n_hid] and the saved activations in
    ``workspace`` (a uint8 CUDA tensor of cfc_kloop_workspace_bytes bytes)."""
    torch = _torch()
    B, K, n_in = x.shape
    H = h0.shape[1]
    st = _storage_dtype(math)
    f32 = torch.float32
    dt_stride = 0 if dt.numel() == 1 else 1
    status = load_library().cfc_kloop_forward(
        _ptr(x, "x", st, (B, K, n_in)), _ptr(h0, "h0", st, (B, H)),
        _ptr(W_in, "W_in", st, (3, H, n_in)), _ptr(W_rec, "W_rec", st, (3, H, H)),
        _ptr(b, "b", f32, (3, H)), _ptr(dt, "dt", f32, (B,) if dt_stride else None),
        dt_stride, B, K, n_in, H, math,
        _ptr(h_seq, "h_seq", st, (B, K, H)), _ptr(workspace, "workspace", torch.uint8),
        workspace.numel(), _stream(stream))
    _check("cfc_kloop_forward", status)


def cfc_kloop_backward(x, h0, W_in, W_rec, b, dt, h_seq, grad_W_in, grad_W_rec, grad_b,
                       workspace, grad_h_seq=None, grad_h_last=None, y=None, grad_h0=None,
                       grad_x=None, per_sample_scratch=None, grad_path=GRAD_SCRATCH,
                       math=MATH_FP32, stream=None):
    """Backward through the K loop of the forward that filled ``workspace``."""
    torch = _torch()
    B, K, n_in = x.shape
    H = h0.shape[1]
    st = _storage_dtype(math)
    f32 = torch.float32
    N = 3 * (n_in + H + 1) * H
    dt_stride = 0 if dt.numel() == 1 else 1
    status = load_library().cfc_kloop_backward(
        _ptr(x, "x", st, (B, K, n_in)), _ptr(h0, "h0", st, (B, H)),
        _ptr(W_in, "W_in", st, (3, H, n_in)), _ptr(W_rec, "W_rec", st, (3, H, H)),
        _ptr(b, "b", f32, (3, H)), _ptr(dt, "dt", f32, (B,) if dt_stride else None),
        dt_stride, B, K, n_in, H, math,
        _ptr(h_seq, "h_seq", st, (B, K, H)),
        _ptr(grad_h_seq, "grad_h_seq", f32, (B, K, H), optional=True),
        _ptr(grad_h_last, "grad_h_last", f32, (B, H), optional=True),
        _ptr(y, "y", f32, (B, H), optional=True),
        _ptr(grad_W_in, "grad_W_in", f32, (3, H, n_in)),
        _ptr(grad_W_rec, "grad_W_rec", f32, (3, H, H)),
        _ptr(grad_b, "grad_b", f32, (3, H)),
        _ptr(grad_h0, "grad_h0", f32, (B, H), optional=True),
        _ptr(grad_x, "grad_x", f32, (B, K, n_in), optional=True),
        _ptr(per_sample_scratch, "per_sample_scratch", f32, (B, N),
             optional=(grad_path != GRAD_SCRATCH)),
        grad_path, _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("cfc_kloop_backward", status)


def reduce_axis0(per_batch, out, stream=None):
    """out[N] = column sums of per_batch[B, N] (overwrite, canonical order)."""
    torch = _torch()
    B, N = per_batch.shape
    status = load_library().reduce_axis0(
        _ptr(per_batch, "per_batch", torch.float32), B, N,
        _ptr(out, "out", torch.float32, (N,)), _stream(stream))
    _check("reduce_axis0", status)


def cfc_grn_param_length(hidden: int, head_mid: int, n_horizons: int) -> int:
    return int(load_library().cfc_grn_param_length(hidden, head_mid, n_horizons))


def cfc_grn_saved_per_row(head_mid: int, n_horizons: int) -> int:
    return int(load_library().cfc_grn_saved_per_row(head_mid, n_horizons))


def cfc_grn_workspace_bytes(B: int, K: int, hidden: int, head_mid: int, n_horizons: int) -> int:
    return int(load_library().cfc_grn_workspace_bytes(B, K, hidden, head_mid, n_horizons))


def cfc_grn_forward(h, params, probs, saved, head_mid: int, n_horizons: int, stream=None):
    """GRN heads forward over the rows of h [R, hidden] (float32): probs
    [R, n_horizons] and the saved intermediates [R, cfc_grn_saved_per_row]."""
    torch = _torch()
    f32 = torch.float32
    R, Hd = h.shape
    N = cfc_grn_param_length(Hd, head_mid, n_horizons)
    S = cfc_grn_saved_per_row(head_mid, n_horizons)
    status = load_library().cfc_grn_forward(
        _ptr(h, "h", f32, (R, Hd)), R, Hd, head_mid, n_horizons, _ptr(params, "params", f32, (N,)),
        _ptr(probs, "probs", f32, (R, n_horizons)), _ptr(saved, "saved", f32, (R, S)), _stream(stream))
    _check("cfc_grn_forward", status)


def cfc_grn_backward(h, params, probs, saved, grad_probs, lam, grad_h, per_sample_scratch, grad_params, workspace,
                     B: int, K: int, head_mid: int, n_horizons: int, grad_h_carry=None, stream=None):
    """GRN heads backward for h [B*K, hidden] rows (r = b*K + k): grad_h,
    the per-sample gradient rows and their batch sum (packed parameter order)."""
    R, Hd = h.shape
    if B < 1 or K < 1 or R != B * K:
        # the library reads B*K rows of every per-row tensor: a mismatch would
        # read past the tensors, so it is refused here
        raise ValueError(f"h has {R} rows; cfc_grn_backward needs B*K = {B}*{K} rows")
    torch = _torch()
    f32 = torch.float32
    N = cfc_grn_param_length(Hd, head_mid, n_horizons)
    S = cfc_grn_saved_per_row(head_mid, n_horizons)
    J = n_horizons
    status = load_library().cfc_grn_backward(
        _ptr(h, "h", f32, (R, Hd)), B, K, Hd, head_mid, J, _ptr(params, "params", f32, (N,)),
        _ptr(probs, "probs", f32, (R, J)), _ptr(saved, "saved", f32, (R, S)),
        _ptr(grad_probs, "grad_probs", f32, (R, J)), _ptr(lam, "lambda", f32, (J,)),
        _ptr(grad_h_carry, "grad_h_carry", f32, (R, Hd), optional=True), _ptr(grad_h, "grad_h", f32, (R, Hd)),
        _ptr(per_sample_scratch, "per_sample_scratch", f32, (B, N)), _ptr(grad_params, "grad_params", f32, (N,)),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("cfc_grn_backward", status)


def cfc_tau_per_sample_length(n_in: int, n_hid: int) -> int:
    return int(load_library().cfc_tau_per_sample_length(n_in, n_hid))


def cfc_tau_kloop_workspace_bytes(B: int, K: int, n_in: int, n_hid: int) -> int:
    return int(load_library().cfc_tau_kloop_workspace_bytes(B, K, n_in, n_hid))


def cfc_tau_kloop_forward(x, h0, W_in, W_rec, b, tau, dt, h_seq, workspace, stream=None):
    """tau-cell forward K loop (float32): writes h_seq [B, K, n_hid] and the
    saved activations in ``workspace``."""
    torch = _torch()
    f32 = torch.float32
    B, K, n_in = x.shape
    H = h0.shape[1]
    dt_stride = 0 if dt.numel() == 1 else 1
    status = load_library().cfc_tau_kloop_forward(
        _ptr(x, "x", f32, (B, K, n_in)), _ptr(h0, "h0", f32, (B, H)), _ptr(W_in, "W_in", f32, (H, n_in)),
        _ptr(W_rec, "W_rec", f32, (H, H)), _ptr(b, "b", f32, (H,)), _ptr(tau, "tau", f32, (H,)),
        _ptr(dt, "dt", f32, (B,) if dt_stride else None), dt_stride, B, K, n_in, H,
        _ptr(h_seq, "h_seq", f32, (B, K, H)), _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
        _stream(stream))
    _check("cfc_tau_kloop_forward", status)


def cfc_tau_kloop_backward(x, h0, W_in, W_rec, b, tau, dt, h_seq, grad_W_in, grad_W_rec, grad_b, grad_tau,
                           per_sample_scratch, workspace, grad_h_seq=None, grad_h_last=None, y=None,
                           grad_h0=None, grad_x=None, stream=None):
    """Backward through the tau-cell K loop of the forward that filled ``workspace``."""
    torch = _torch()
    f32 = torch.float32
    B, K, n_in = x.shape
    H = h0.shape[1]
    N = (n_in + H + 2) * H
    dt_stride = 0 if dt.numel() == 1 else 1
    status = load_library().cfc_tau_kloop_backward(
        _ptr(x, "x", f32, (B, K, n_in)), _ptr(h0, "h0", f32, (B, H)), _ptr(W_in, "W_in", f32, (H, n_in)),
        _ptr(W_rec, "W_rec", f32, (H, H)), _ptr(b, "b", f32, (H,)), _ptr(tau, "tau", f32, (H,)),
        _ptr(dt, "dt", f32, (B,) if dt_stride else None), dt_stride, B, K, n_in, H,
        _ptr(h_seq, "h_seq", f32, (B, K, H)),
        _ptr(grad_h_seq, "grad_h_seq", f32, (B, K, H), optional=True),
        _ptr(grad_h_last, "grad_h_last", f32, (B, H), optional=True),
        _ptr(y, "y", f32, (B, H), optional=True),
        _ptr(grad_W_in, "grad_W_in", f32, (H, n_in)), _ptr(grad_W_rec, "grad_W_rec", f32, (H, H)),
        _ptr(grad_b, "grad_b", f32, (H,)), _ptr(grad_tau, "grad_tau", f32, (H,)),
        _ptr(grad_h0, "grad_h0", f32, (B, H), optional=True),
        _ptr(grad_x, "grad_x", f32, (B, K, n_in), optional=True),
        _ptr(per_sample_scratch, "per_sample_scratch", f32, (B, N)),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("cfc_tau_kloop_backward", status)


def cfc_gdr_workspace_bytes(rows, n_seq, n_k_heads, n_v_heads, d_k, d_v, math=MATH_BF16, save=False) -> int:
    return int(load_library().cfc_gdr_workspace_bytes(rows, n_seq, n_k_heads, n_v_heads, d_k, d_v, math,
                                                      1 if save else 0))


def _rows(t, name, dtype, shape):
    """Pointer and row stride of t [..., heads, width], whose rows may be parts
    of wider ones (dense in heads and width, evenly spaced over the rest)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
            return t.data_ptr(), shape[-2] * shape[-1]
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    strides = t.stride()
    packed = len(shape) == 3
    ld = strides[-3] if packed or shape[-3] != 1 else strides[0]
    if (strides[-1] != 1 or (shape[-2] > 1 and strides[-2] != shape[-1])
            or (not packed and shape[0] > 1 and strides[0] != shape[1] * ld)):
        raise ValueError(f"{name} must be dense in its last two axes, with evenly spaced rows")
    return t.data_ptr(), ld


def _gdr_inputs(q, k, v, g, beta, packed, math):
    """What the three calls share: the stored type, the shapes of v, of q and of
    g, (k_heads, v_heads, d_k, d_v), and the leading C arguments."""
    st = _storage_dtype(math)
    vs, ks = v.shape, q.shape
    if len(vs) != (3 if packed else 4):
        raise ValueError("v must be [sequences, tokens, heads, d_v], or [rows, heads, d_v] with seq_offsets")
    if len(ks) != len(vs):
        raise ValueError("q and v must have the same number of axes")
    if packed:
        rows, hv, dv = vs
        _, hk, dk = ks
        ks, hs = (rows, hk, dk), (rows, hv)
    else:
        n, tokens, hv, dv = vs
        _, _, hk, dk = ks
        ks, hs = (n, tokens, hk, dk), (n, tokens, hv)
    qp, ldq = _rows(q, "q", st, ks)
    kp, ldk = _rows(k, "k", st, ks)
    vp, ldv = _rows(v, "v", st, vs)
    f32 = _torch().float32
    return st, vs, ks, hs, (hk, hv, dk, dv), (qp, ldq, kp, ldk, vp, ldv, _ptr(g, "g", f32, hs), _ptr(beta, "beta", f32, hs))


def _gdr_sequences(vs, seq_offsets):
    if seq_offsets is None:
        return None, vs[0], vs[0] * vs[1]
    if seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
        raise ValueError("seq_offsets must hold n_seq + 1 row numbers")
    return _ptr(seq_offsets, "seq_offsets", _torch().int32), seq_offsets.numel() - 1, vs[0]


def cfc_gdr_forward(q, k, v, g, beta, o, workspace, scale=None, seq_offsets=None, initial_state=None, final_state=None,
                    save=False, math=MATH_BF16, stream=None):
    """Gated delta rule over whole sequences: q, k [sequences, tokens, k_heads,
    d_k], v and o [sequences, tokens, v_heads, d_v], g, beta [sequences, tokens,
    v_heads]; or [rows, ...] packed, with int32 seq_offsets [sequences + 1] on
    the device.  scale: d_k ** -0.5 if None."""
    f32 = _torch().float32
    st, vs, _, _, sizes, args = _gdr_inputs(q, k, v, g, beta, seq_offsets is not None, math)
    off, n, rows = _gdr_sequences(vs, seq_offsets)
    hk, hv, dk, dv = sizes
    ss = (n, hv, dk, dv)
    status = load_library().cfc_gdr_forward(
        *args, off, n, rows, hk, hv, dk, dv, dk ** -0.5 if scale is None else scale, math,
        _ptr(initial_state, "initial_state", f32, ss, optional=True), _ptr(o, "o", st, vs),
        _ptr(final_state, "final_state", f32, ss, optional=True), 1 if save else 0,
        _ptr(workspace, "workspace", _torch().uint8), workspace.numel(), _stream(stream))
    _check("cfc_gdr_forward", status)


def cfc_gdr_backward(q, k, v, g, beta, grad_o, grad_q, grad_k, grad_v, grad_g, grad_beta, workspace, scale=None,
                     seq_offsets=None, grad_final_state=None, grad_initial_state=None, math=MATH_BF16, stream=None):
    """Backward of the cfc_gdr_forward(save=True) that filled ``workspace``;
    every gradient is overwritten, all in the type of q."""
    f32 = _torch().float32
    st, vs, ks, hs, sizes, args = _gdr_inputs(q, k, v, g, beta, seq_offsets is not None, math)
    off, n, rows = _gdr_sequences(vs, seq_offsets)
    hk, hv, dk, dv = sizes
    ss = (n, hv, dk, dv)
    status = load_library().cfc_gdr_backward(
        *args, off, n, rows, hk, hv, dk, dv, dk ** -0.5 if scale is None else scale, math,
        _ptr(grad_o, "grad_o", st, vs), _ptr(grad_final_state, "grad_final_state", f32, ss, optional=True),
        _ptr(grad_q, "grad_q", st, ks), _ptr(grad_k, "grad_k", st, ks), _ptr(grad_v, "grad_v", st, vs),
        _ptr(grad_g, "grad_g", st, hs), _ptr(grad_beta, "grad_beta", st, hs),
        _ptr(grad_initial_state, "grad_initial_state", f32, ss, optional=True),
        _ptr(workspace, "workspace", _torch().uint8), workspace.numel(), _stream(stream))
    _check("cfc_gdr_backward", status)


def cfc_gdr_step(q, k, v, g, beta, state, o, slots=None, scale=None, math=MATH_BF16, stream=None):
    """The next tokens of decoding sequences (shapes as for cfc_gdr_forward,
    [sequences, tokens, ...]): sequence i's state is ``state[slots[i]]``
    (int32 on the device; ``state[i]`` if None), updated in place."""
    torch = _torch()
    st, vs, _, _, sizes, args = _gdr_inputs(q, k, v, g, beta, False, math)
    n, tokens = vs[0], vs[1]
    dk, pool = sizes[2], state.shape
    if len(pool) != 4 or pool != (pool[0], sizes[1], dk, sizes[3]):
        raise ValueError(f"state must have shape (slots, {sizes[1]}, {dk}, {sizes[3]}), got {tuple(pool)}")
    status = load_library().cfc_gdr_step(
        *args, n, tokens, *sizes, dk ** -0.5 if scale is None else scale, math,
        _ptr(state, "state", torch.float32), pool[0], _ptr(slots, "slots", torch.int32, (n,), optional=True),
        _ptr(o, "o", st, vs), _stream(stream))
    _check("cfc_gdr_step", status)


def cfc_rmsnorm_workspace_bytes(rows: int, d: int) -> int:
    return int(load_library().cfc_rmsnorm_workspace_bytes(rows, d))


def cfc_rmsnorm_forward(x, weight, y=None, residual=None, residual_out=None, rstd=None, y8=None, y8_scale=None,
                        eps=1e-6, math=MATH_BF16, stream=None):
    """Norm of the stream x + residual [rows, d]: y in the stored type and/or
    y8 (float8_e4m3fn or uint8) with y8_scale [rows, groups], one scale for
    each d / groups columns."""
    torch = _torch()
    st, f32 = _storage_dtype(math), torch.float32
    rows, d = shape = x.shape
    group = d
    if y8 is not None:
        if y8.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise TypeError(f"y8 must be torch.float8_e4m3fn or torch.uint8, got {y8.dtype}")
        if y8_scale is None or y8_scale.dim() != 2 or y8_scale.shape[1] < 1 or d % y8_scale.shape[1]:
            raise ValueError("y8 needs y8_scale [rows, groups], with groups a divisor of d")
        group = d // y8_scale.shape[1]
    status = load_library().cfc_rmsnorm_forward(
        _ptr(x, "x", st), _ptr(residual, "residual", st, shape, optional=True), _ptr(weight, "weight", f32, (d,)),
        rows, d, eps, math, _ptr(y, "y", st, shape, optional=True),
        _ptr(residual_out, "residual_out", st, shape, optional=True), _ptr(rstd, "rstd", f32, (rows,), optional=True),
        _ptr(y8, "y8", None, shape, optional=True),
        _ptr(y8_scale, "y8_scale", f32, (rows, d // group), optional=True) if y8 is not None else None, group,
        _stream(stream))
    _check("cfc_rmsnorm_forward", status)


def cfc_rmsnorm_backward(s, weight, rstd, grad_y, grad_x, grad_weight, workspace, grad_residual_out=None,
                         math=MATH_BF16, stream=None):
    """Backward from the stream s (the forward's residual_out, or its x) and
    rstd: grad_x, the gradient of s, and grad_weight."""
    torch = _torch()
    st, f32 = _storage_dtype(math), torch.float32
    rows, d = shape = s.shape
    status = load_library().cfc_rmsnorm_backward(
        _ptr(s, "s", st), _ptr(weight, "weight", f32, (d,)), _ptr(rstd, "rstd", f32, (rows,)),
        _ptr(grad_y, "grad_y", st, shape), _ptr(grad_residual_out, "grad_residual_out", st, shape, optional=True),
        rows, d, math, _ptr(grad_x, "grad_x", st, shape), _ptr(grad_weight, "grad_weight", f32, (d,)),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("cfc_rmsnorm_backward", status)


def cfc_layernorm_workspace_bytes(rows: int, d: int) -> int:
    return int(load_library().cfc_layernorm_workspace_bytes(rows, d))


def cfc_layernorm_forward(x, weight, y, bias=None, residual=None, residual_out=None, mean=None, rstd=None, eps=1e-5,
                          math=MATH_BF16, stream=None):
    """Layer norm y of the stream x + residual [rows, d]; the backward needs the
    stream (residual_out, or x without a residual), mean and rstd [rows]."""
    st, f32 = _storage_dtype(math), _torch().float32
    rows, d = shape = x.shape
    status = load_library().cfc_layernorm_forward(
        _ptr(x, "x", st), _ptr(residual, "residual", st, shape, optional=True), _ptr(weight, "weight", f32, (d,)),
        _ptr(bias, "bias", f32, (d,), optional=True), rows, d, eps, math, _ptr(y, "y", st, shape),
        _ptr(residual_out, "residual_out", st, shape, optional=True), _ptr(mean, "mean", f32, (rows,), optional=True),
        _ptr(rstd, "rstd", f32, (rows,), optional=True), _stream(stream))
    _check("cfc_layernorm_forward", status)


def cfc_layernorm_backward(s, weight, mean, rstd, grad_y, grad_x, grad_weight, workspace, grad_bias=None,
                           grad_residual_out=None, math=MATH_BF16, stream=None):
    """Backward from the stream s, mean and rstd: grad_x, the gradient of s,
    grad_weight and (where given) grad_bias."""
    st, f32 = _storage_dtype(math), _torch().float32
    rows, d = shape = s.shape
    status = load_library().cfc_layernorm_backward(
        _ptr(s, "s", st), _ptr(weight, "weight", f32, (d,)), _ptr(mean, "mean", f32, (rows,)), _ptr(rstd, "rstd", f32, (rows,)),
        _ptr(grad_y, "grad_y", st, shape), _ptr(grad_residual_out, "grad_residual_out", st, shape, optional=True),
        rows, d, math, _ptr(grad_x, "grad_x", st, shape), _ptr(grad_weight, "grad_weight", f32, (d,)),
        _ptr(grad_bias, "grad_bias", f32, (d,), optional=True), _ptr(workspace, "workspace", _torch().uint8),
        workspace.numel(), _stream(stream))
    _check("cfc_layernorm_backward", status)


def _spaced(t, name, dtype, shape, tail=1):
    """Pointer and row stride of t of `shape`, whose rows (the last `tail` axes,
    dense) may be parts of wider ones, evenly spaced over the axes before them."""
    width = shape[-1] if tail == 1 else shape[-1] * shape[-2]
    try:
        if t.dtype is dtype and t.shape == shape and t.is_cuda:
            if t.is_contiguous():
                return t.data_ptr(), width
            s = t.stride()
            if s[-1] == 1 and (tail == 1 or s[-2] == shape[-1]):        # the usual part of a projection
                if len(shape) == tail + 1:
                    return t.data_ptr(), s[0] if shape[0] != 1 else width
                if shape[1] != 1 and (shape[0] == 1 or s[0] == shape[1] * s[1]):
                    return t.data_ptr(), s[1]
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    strides, lead = t.stride(), shape[:-tail]
    dense = shape[-1] == 1 or strides[-1] == 1
    if tail == 2:
        dense = dense and (shape[-2] == 1 or strides[-2] == shape[-1])
    many = [i for i in range(len(lead)) if lead[i] != 1]
    ld = strides[many[-1]] if many else width           # one row: its stride says nothing
    if not dense or (len(many) == 2 and strides[0] != lead[1] * ld):
        raise ValueError(f"{name} must be dense in its last {'axis' if tail == 1 else 'two axes'}, with evenly spaced rows")
    return t.data_ptr(), ld


def _row_sequences(shape, seq_offsets, name="x"):
    """(offsets, sequences, rows) of [sequences, tokens, channels], or [rows, channels] with seq_offsets."""
    if len(shape) != (3 if seq_offsets is None else 2):
        raise ValueError(f"{name} must be [sequences, tokens, channels], or [rows, channels] with seq_offsets")
    return _gdr_sequences(shape, seq_offsets)


def cfc_conv_workspace_bytes(rows: int, channels: int, width: int, math=MATH_BF16) -> int:
    return int(load_library().cfc_conv_workspace_bytes(rows, channels, width, math))


def _conv_inputs(x, weight, bias, math):
    st, f32, shape = _storage_dtype(math), _torch().float32, x.shape
    d = shape[-1]
    if len(weight.shape) != 2:
        raise ValueError("weight must be [channels, width]")
    w = weight.shape[1]
    return st, f32, shape, d, w, (*_spaced(x, "x", st, shape), _ptr(weight, "weight", f32, (d, w)),
                                  _ptr(bias, "bias", f32, (d,), optional=True))


def cfc_conv_forward(x, weight, y, bias=None, seq_offsets=None, initial_state=None, final_state=None, silu=True,
                     math=MATH_BF16, stream=None):
    """Short causal convolution of each channel of x [sequences, tokens, channels]
    (or [rows, channels] packed, with int32 seq_offsets [sequences + 1] on the
    device), weight [channels, width]; states [sequences, width - 1, channels]."""
    st, f32, shape, d, w, args = _conv_inputs(x, weight, bias, math)
    off, n, rows = _row_sequences(shape, seq_offsets)
    ss = (n, w - 1, d)
    status = load_library().cfc_conv_forward(
        *args, off, n, rows, d, w, 1 if silu else 0, math, _ptr(initial_state, "initial_state", st, ss, optional=True),
        _ptr(y, "y", st, shape), _ptr(final_state, "final_state", st, ss, optional=True), _stream(stream))
    _check("cfc_conv_forward", status)


def cfc_conv_backward(x, weight, grad_y, grad_x, grad_weight, workspace, bias=None, grad_bias=None, seq_offsets=None,
                      initial_state=None, grad_final_state=None, grad_initial_state=None, silu=True, math=MATH_BF16,
                      stream=None):
    """Backward of cfc_conv_forward from its inputs; every gradient is overwritten."""
    st, f32, shape, d, w, args = _conv_inputs(x, weight, bias, math)
    off, n, rows = _row_sequences(shape, seq_offsets)
    ss = (n, w - 1, d)
    status = load_library().cfc_conv_backward(
        *args, off, n, rows, d, w, 1 if silu else 0, math, _ptr(initial_state, "initial_state", st, ss, optional=True),
        _ptr(grad_y, "grad_y", st, shape), _ptr(grad_final_state, "grad_final_state", st, ss, optional=True),
        _ptr(grad_x, "grad_x", st, shape), _ptr(grad_weight, "grad_weight", f32, (d, w)),
        _ptr(grad_bias, "grad_bias", f32, (d,), optional=True),
        _ptr(grad_initial_state, "grad_initial_state", st, ss, optional=True),
        _ptr(workspace, "workspace", _torch().uint8), workspace.numel(), _stream(stream))
    _check("cfc_conv_backward", status)


def _pool(state, name, dtype, tail):
    shape = state.shape
    if len(shape) != len(tail) + 1 or shape[1:] != tail:
        raise ValueError(f"{name} must have shape (slots, {', '.join(map(str, tail))}), got {tuple(shape)}")
    return _ptr(state, name, dtype), shape[0]


def cfc_conv_step(x, weight, state, y, bias=None, slots=None, silu=True, math=MATH_BF16, stream=None):
    """The next tokens x [sequences, tokens, channels] of decoding sequences: sequence
    i's last inputs are ``state[slots[i]]`` (int32 on the device; ``state[i]`` if
    None), [slots, width - 1, channels], updated in place."""
    st, f32, shape, d, w, args = _conv_inputs(x, weight, bias, math)
    if len(shape) != 3:
        raise ValueError("x must be [sequences, tokens, channels]")
    n, tokens, _ = shape
    status = load_library().cfc_conv_step(
        *args, n, tokens, d, w, 1 if silu else 0, math, *_pool(state, "state", st, (w - 1, d)),
        _ptr(slots, "slots", _torch().int32, (n,), optional=True), _ptr(y, "y", st, shape), _stream(stream))
    _check("cfc_conv_step", status)


def cfc_ssm_workspace_bytes(rows, n_seq, channels, groups, n_states, math=MATH_BF16, save=False) -> int:
    return int(load_library().cfc_ssm_workspace_bytes(rows, n_seq, channels, groups, n_states, math, 1 if save else 0))


def _ssm_inputs(x, delta, A, B, C, D, z, delta_bias, math):
    """What the three calls share: the stored type, fp32, the shapes of x and of B,
    (channels, groups, states), and the leading C arguments."""
    st, f32, shape, bs = _storage_dtype(math), _torch().float32, x.shape, B.shape
    d = shape[-1]
    if len(bs) != len(shape) + 1 or bs[:-2] != shape[:-1]:
        raise ValueError("B must be [..., groups, states] with the leading axes of x")
    g, n = bs[-2:]
    zp, ldz = (None, d) if z is None else _spaced(z, "z", st, shape)
    args = (*_spaced(x, "x", st, shape), *_spaced(delta, "delta", st, shape), _ptr(A, "A", f32, (d, n)),
            *_spaced(B, "B", st, bs, 2), *_spaced(C, "C", st, bs, 2), _ptr(D, "D", f32, (d,), optional=True), zp, ldz,
            _ptr(delta_bias, "delta_bias", f32, (d,), optional=True))
    return st, f32, shape, bs, (d, g, n), args


def cfc_ssm_forward(x, delta, A, B, C, y, workspace, D=None, z=None, delta_bias=None, seq_offsets=None, initial_state=None,
                    final_state=None, save=False, math=MATH_BF16, stream=None):
    """Selective scan over whole sequences: x, delta, z and y [sequences, tokens,
    channels], B, C [sequences, tokens, groups, states], A [channels, states]; or
    [rows, ...] packed, with int32 seq_offsets [sequences + 1] on the device.
    States [sequences, channels, states] are fp32."""
    st, f32, shape, _, sizes, args = _ssm_inputs(x, delta, A, B, C, D, z, delta_bias, math)
    off, n, rows = _row_sequences(shape, seq_offsets)
    ss = (n, sizes[0], sizes[2])
    status = load_library().cfc_ssm_forward(
        *args, off, n, rows, *sizes, math, _ptr(initial_state, "initial_state", f32, ss, optional=True),
        _ptr(y, "y", st, shape), _ptr(final_state, "final_state", f32, ss, optional=True), 1 if save else 0,
        _ptr(workspace, "workspace", _torch().uint8), workspace.numel(), _stream(stream))
    _check("cfc_ssm_forward", status)


def cfc_ssm_backward(x, delta, A, B, C, grad_y, grad_x, grad_delta, grad_A, grad_B, grad_C, workspace, D=None, z=None,
                     delta_bias=None, grad_D=None, grad_z=None, grad_delta_bias=None, seq_offsets=None, initial_state=None,
                     grad_final_state=None, grad_initial_state=None, math=MATH_BF16, stream=None):
    """Backward of the cfc_ssm_forward(save=True) that filled ``workspace``; every gradient is overwritten:
    those of x, delta, z, B and C in their type, the others in fp32."""
    st, f32, shape, bs, sizes, args = _ssm_inputs(x, delta, A, B, C, D, z, delta_bias, math)
    off, n, rows = _row_sequences(shape, seq_offsets)
    d, _, N = sizes
    ss = (n, d, N)
    status = load_library().cfc_ssm_backward(
        *args, off, n, rows, *sizes, math, _ptr(initial_state, "initial_state", f32, ss, optional=True),
        _ptr(grad_y, "grad_y", st, shape), _ptr(grad_final_state, "grad_final_state", f32, ss, optional=True),
        _ptr(grad_x, "grad_x", st, shape), _ptr(grad_delta, "grad_delta", st, shape), _ptr(grad_A, "grad_A", f32, (d, N)),
        _ptr(grad_B, "grad_B", st, bs), _ptr(grad_C, "grad_C", st, bs), _ptr(grad_D, "grad_D", f32, (d,), optional=True),
        _ptr(grad_z, "grad_z", st, shape, optional=True),
        _ptr(grad_delta_bias, "grad_delta_bias", f32, (d,), optional=True),
        _ptr(grad_initial_state, "grad_initial_state", f32, ss, optional=True),
        _ptr(workspace, "workspace", _torch().uint8), workspace.numel(), _stream(stream))
    _check("cfc_ssm_backward", status)


def cfc_ssm_step(x, delta, A, B, C, state, y, D=None, z=None, delta_bias=None, slots=None, math=MATH_BF16, stream=None):
    """The next tokens of decoding sequences (shapes as for cfc_ssm_forward,
    [sequences, tokens, ...]): sequence i's state is ``state[slots[i]]`` (int32 on
    the device; ``state[i]`` if None), updated in place."""
    st, f32, shape, _, sizes, args = _ssm_inputs(x, delta, A, B, C, D, z, delta_bias, math)
    if len(shape) != 3:
        raise ValueError("x must be [sequences, tokens, channels]")
    n, tokens, d = shape
    status = load_library().cfc_ssm_step(
        *args, n, tokens, *sizes, math, *_pool(state, "state", f32, (d, sizes[2])),
        _ptr(slots, "slots", _torch().int32, (n,), optional=True), _ptr(y, "y", st, shape), _stream(stream))
    _check("cfc_ssm_step", status)


def cfc_grad_clip_workspace_bytes(count: int) -> int:
    return int(load_library().cfc_grad_clip_workspace_bytes(count))


_grad_kinds = {}


def _tensor_list(tensors, name):
    """Host arrays of the pointers, sizes and types of contiguous tensors."""
    if not _grad_kinds:
        torch = _torch()
        _grad_kinds.update({torch.float32: MATH_FP32, torch.bfloat16: MATH_BF16})
    try:        # many small tensors: a few list comprehensions, and the reasons only where something is wrong
        if all([t.is_cuda and t.is_contiguous() for t in tensors]):
            return (array("Q", [t.data_ptr() for t in tensors]), array("q", [t.numel() for t in tensors]),
                    array("i", [_grad_kinds[t.dtype] for t in tensors]))
    except (AttributeError, KeyError):
        pass
    torch = _torch()
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name}[{i}] must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")
        if t.dtype not in _grad_kinds:
            raise TypeError(f"{name}[{i}] must be torch.float32 or torch.bfloat16, got {t.dtype}")
    raise TypeError(f"{name} must be a list of CUDA tensors")


def _host(a):
    return a.buffer_info()[0]


def cfc_grad_norm(grads, norm, workspace, stream=None):
    """norm [1] = the square root of the sum of all squares of the tensors (float32 or bfloat16, in any mixture)."""
    grads = list(grads)
    ptrs, sizes, maths = _tensor_list(grads, "grads")
    torch = _torch()
    status = load_library().cfc_grad_norm(_host(ptrs), _host(sizes), _host(maths), len(grads), _ptr(norm, "norm", torch.float32, (1,)),
                                          _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("cfc_grad_norm", status)


def cfc_grad_clip(grads, max_norm, norm, workspace, out=None, stream=None):
    """norm [1] of the tensors together, and each scaled by min(1, max_norm / (norm + 1e-6)):
    in place, or into the tensors of out (each with as many values, of the same type)."""
    grads = list(grads)
    ptrs, sizes, maths = _tensor_list(grads, "grads")
    outs = ptrs
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError("out must have as many tensors as grads")
        outs, osizes, omaths = _tensor_list(out, "out")
        if osizes != sizes or omaths != maths:
            raise ValueError("out must have the sizes and types of grads")
    if len(set(outs)) != len(outs) and len(set(p for p, n in zip(outs, sizes) if n)) != len(sizes) - sizes.count(0):
        raise ValueError("a tensor is written twice")
    torch = _torch()
    status = load_library().cfc_grad_clip(_host(ptrs), _host(outs), _host(sizes), _host(maths), len(grads), max_norm, _ptr(norm, "norm", torch.float32, (1,)),
                                          _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("cfc_grad_clip", status)


def reduce_axis0_multi(per_batch, out, stream=None):
    """out[i][N_i] = column sums of per_batch[i][B_i, N_i] for every i, in few
    launches; the same bits as reduce_axis0 on each pair."""
    torch = _torch()
    per_batch, out = list(per_batch), list(out)
    if len(per_batch) != len(out):
        raise ValueError("per_batch and out must have the same length")
    n = len(per_batch)
    ins = (ctypes.c_void_p * max(n, 1))()
    outs = (ctypes.c_void_p * max(n, 1))()
    nb = (ctypes.c_int * max(n, 1))()
    nt = (ctypes.c_longlong * max(n, 1))()
    for i, (a, o) in enumerate(zip(per_batch, out)):
        if a.dim() != 2:
            raise ValueError(f"per_batch[{i}] must be 2-D")
        B, N = a.shape
        ins[i] = _ptr(a, f"per_batch[{i}]", torch.float32)
        outs[i] = _ptr(o, f"out[{i}]", torch.float32, (N,))
        nb[i], nt[i] = B, N
    status = load_library().reduce_axis0_multi(ins, nb, nt, outs, n, _stream(stream))
    _check("reduce_axis0_multi", status)


def cfc_kloop_forward_backward_static(x, h0, W_in, W_rec, b, dt, h_seq, grad_W_in, grad_W_rec,
                                      grad_b, grad_h_seq=None, grad_h_last=None, y=None,
                                      grad_h0=None, grad_x=None, math=MATH_FP32, stream=None):
    """Forward + backward with the library's fixed internal workspace, for
    callers that cannot allocate device memory.  Computes what
    cfc_kloop_forward + cfc_kloop_backward(grad_path=GRAD_GEMM) compute, always
    on the CUDA-core (SIMT) kernels, so the results agree with those calls
    within the parity tolerances, not bit for bit."""
    torch = _torch()
    B, K, n_in = x.shape
    H = h0.shape[1]
    st = _storage_dtype(math)
    f32 = torch.float32
    dt_stride = 0 if dt.numel() == 1 else 1
    status = load_library().cfc_kloop_forward_backward_static(
        _ptr(x, "x", st, (B, K, n_in)), _ptr(h0, "h0", st, (B, H)),
        _ptr(W_in, "W_in", st, (3, H, n_in)), _ptr(W_rec, "W_rec", st, (3, H, H)),
        _ptr(b, "b", f32, (3, H)), _ptr(dt, "dt", f32, (B,) if dt_stride else None),
        dt_stride, B, K, n_in, H, math,
        _ptr(grad_h_seq, "grad_h_seq", f32, (B, K, H), optional=True),
        _ptr(grad_h_last, "grad_h_last", f32, (B, H), optional=True),
        _ptr(y, "y", f32, (B, H), optional=True),
        _ptr(h_seq, "h_seq", st, (B, K, H)),
        _ptr(grad_W_in, "grad_W_in", f32, (3, H, n_in)),
        _ptr(grad_W_rec, "grad_W_rec", f32, (3, H, H)),
        _ptr(grad_b, "grad_b", f32, (3, H)),
        _ptr(grad_h0, "grad_h0", f32, (B, H), optional=True),
        _ptr(grad_x, "grad_x", f32, (B, K, n_in), optional=True),
        _stream(stream))
    _check("cfc_kloop_forward_backward_static", status)


def cfc_trace_enable(on: bool) -> None:
    """Start (clearing old records) or stop per-kernel event tracing."""
    _check("cfc_trace_enable", load_library().cfc_trace_enable(1 if on else 0))


def cfc_trace_records() -> list:
    """[(kernel name, device milliseconds)] for every traced launch."""
    lib = load_library()
    out = []
    for i in range(lib.cfc_trace_count()):
        name = ctypes.c_char_p()
        ms = ctypes.c_float()
        _check("cfc_trace_get", lib.cfc_trace_get(i, ctypes.byref(name), ctypes.byref(ms)))
        out.append((name.value.decode(), float(ms.value)))
    return out
