"""Python binding of the C ABI in include/jfa.h (argument marshalling only).

Every step of the attention runs in the library's CUDA kernels; this module only
checks tensors, allocates outputs and workspace through PyTorch's allocator, and
passes raw device pointers plus the current CUDA stream.  There is no CPU path:
without the built library, or with CPU tensors, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional, Tuple

import torch

from . import build as _build

JFA_OK = 0
STATUS_NAMES = {0: "JFA_OK", 1: "JFA_ERR_INVALID_ARG", 2: "JFA_ERR_UNSUPPORTED", 3: "JFA_ERR_WORKSPACE",
                4: "JFA_ERR_CUDA", 5: "JFA_ERR_BAD_OFFSETS", 6: "JFA_ERR_TIMEOUT", 7: "JFA_ERR_BAD_PAGES"}

# Every symbol include/jfa.h declares.
EXPORTED_SYMBOLS = ("jfa_workspace_size", "jfa_forward", "jfa_forward_noalloc", "jfa_backward", "jfa_check_status",
                    "jfa_status_string", "jfa_last_launch_count", "jfa_last_error", "jfa_timing_enable",
                    "jfa_timing_read", "jfa_trace_configure", "jfa_selftest_wait_timeout", "jfa_wait_limit_ns",
                    "jfa_set_nsp_max_tiles", "jfa_window_workspace_size", "jfa_window_forward", "jfa_window_backward",
                    "jfa_cache_workspace_size", "jfa_cache_append", "jfa_cache_attention")
KERNEL_KINDS = ("plan", "forward", "bwd_preprocess", "bwd_dkdv", "bwd_dq", "bwd_fused", "bwd_nsp", "bwd_join",
                "cache_append", "cache_attention")


class JfaError(RuntimeError):
    def __init__(self, status: int, what: str):
        detail = ""
        if status == 4:
            try:
                detail = " -- " + load_library(build_if_missing=False).jfa_last_error().decode()
            except Exception:
                pass
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status_string(status)}){detail}")
        self.status = status


class _Bias(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("table", ctypes.c_void_p), ("num_buckets", ctypes.c_int),
                ("center", ctypes.c_int), ("grad", ctypes.c_void_p), ("values", ctypes.c_void_p),
                ("block_offsets", ctypes.c_void_p), ("plane", ctypes.c_int64), ("values_grad", ctypes.c_void_p)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("H_kv", ctypes.c_int),
                ("page_size", ctypes.c_int), ("d", ctypes.c_int), ("page_table", ctypes.c_void_p),
                ("max_pages", ctypes.c_int), ("lengths", ctypes.c_void_p), ("B", ctypes.c_int)]


_LIB = None


def library_path() -> str:
    return _build.LIB_PATH


def load_library(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load the in-tree shared library (building it first if asked and needed)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = _build.LIB_PATH
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"jagged attention library not built ({path} missing); run build()")
    lib = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.jfa_workspace_size.argtypes = [i32, i32, i32, i64, i64, i32]
    lib.jfa_workspace_size.restype = sz
    lib.jfa_forward.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i64, i64, ctypes.POINTER(_Bias), f32, i32,
                                vp, vp, vp, sz, vp]
    lib.jfa_forward.restype = i32
    lib.jfa_forward_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i64, i64, ctypes.POINTER(_Bias), f32,
                                        i32, vp, vp, vp]
    lib.jfa_forward_noalloc.restype = i32
    lib.jfa_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i64, i64,
                                 ctypes.POINTER(_Bias), f32, i32, vp, vp, vp, vp, sz, vp]
    lib.jfa_backward.restype = i32
    lib.jfa_check_status.argtypes = [vp, vp]
    lib.jfa_check_status.restype = i32
    lib.jfa_status_string.argtypes = [i32]
    lib.jfa_status_string.restype = ctypes.c_char_p
    lib.jfa_last_launch_count.argtypes = []
    lib.jfa_last_launch_count.restype = i32
    lib.jfa_last_error.argtypes = []
    lib.jfa_last_error.restype = ctypes.c_char_p
    lib.jfa_timing_enable.argtypes = [i32]
    lib.jfa_timing_enable.restype = i32
    lib.jfa_timing_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int), i32]
    lib.jfa_timing_read.restype = i32
    lib.jfa_selftest_wait_timeout.argtypes = [vp, ctypes.c_uint64, vp]
    lib.jfa_selftest_wait_timeout.restype = i32
    lib.jfa_set_nsp_max_tiles.argtypes = [i32]
    lib.jfa_set_nsp_max_tiles.restype = i32
    lib.jfa_wait_limit_ns.argtypes = [i64, i32, i64]
    lib.jfa_wait_limit_ns.restype = ctypes.c_uint64
    lib.jfa_trace_configure.argtypes = [vp, sz, i32]
    lib.jfa_trace_configure.restype = i32
    lib.jfa_window_workspace_size.argtypes = [i32, i32, i32, i32, i64, i64, i32, i32]
    lib.jfa_window_workspace_size.restype = sz
    lib.jfa_window_forward.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i64, i32, i32, f32, vp, vp, vp, sz, vp]
    lib.jfa_window_forward.restype = i32
    lib.jfa_window_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i64, i32, i32, f32,
                                        vp, vp, vp, vp, sz, vp]
    lib.jfa_window_backward.restype = i32
    cache = ctypes.POINTER(_Cache)
    lib.jfa_cache_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.jfa_cache_workspace_size.restype = sz
    lib.jfa_cache_append.argtypes = [cache, vp, i64, vp, i64, vp, i64, i32, vp, i64, vp, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.jfa_cache_append.restype = i32
    lib.jfa_cache_attention.argtypes = [cache, vp, i32, i32, i32, f32, vp, vp, vp, sz, vp]
    lib.jfa_cache_attention.restype = i32
    _LIB = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load_library(build_if_missing=False).jfa_status_string(int(status)).decode()
    except Exception:  # library not loadable: fall back to the enum name
        return STATUS_NAMES.get(status, "unknown")


def _stream_handle(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _check_values(name, t, rows=None, H=None, d=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if t.dim() != 3 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [T, H, d] tensor")
    if H is not None and (t.shape[1] != H or t.shape[2] != d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [*, {H}, {d}]")
    if rows is not None and t.shape[0] != rows:
        raise ValueError(f"{name} has {t.shape[0]} rows, expected {rows}")


def _check_lse(t, H, Tq):
    if (not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 or tuple(t.shape) != (H, Tq)
            or not t.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 CUDA tensor [{H}, {Tq}]")


def _check_workspace(ws, nbytes, device):
    """A caller-given workspace: contiguous bytes on the inputs' device, at least `nbytes`
    long (its size is passed to the library in bytes, whatever its dtype)."""
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
    have = ws.numel() * ws.element_size()
    if have < nbytes:
        raise ValueError(f"workspace holds {have} bytes, the call needs {nbytes}")
    if ws.data_ptr() % 256:
        raise ValueError("workspace must start on a 256-byte boundary")
    return have


def _check_window(window, sinks):
    """`window` as the library's int (None: every key; longer than any sequence is the same)."""
    if int(sinks) < 0 or (window is not None and int(window) < 1):
        raise ValueError(f"window must be at least 1 and sinks at least 0, got {window} and {sinks}")
    return (1 << 31) - 1 if window is None else min(int(window), (1 << 31) - 1)


def _check_offsets(name, off):
    if not isinstance(off, torch.Tensor) or not off.is_cuda or off.dtype != torch.int64 or off.dim() != 1 \
            or not off.is_contiguous() or off.numel() < 2:
        raise ValueError(f"{name} must be a contiguous int64 CUDA tensor [B+1] with B >= 1")


def _bias_struct(bias, center, H, grad=None, jagged_bias=None, jagged_bias_grad=None):
    if jagged_bias is not None:
        if bias is not None or grad is not None:
            raise ValueError("a general jagged bias excludes the relative-position table and its gradient")
        values, boff = jagged_bias
        if (not values.is_cuda or values.dtype != torch.bfloat16 or values.dim() != 2 or values.shape[0] != H
                or not values.is_contiguous()):
            raise ValueError("jagged bias values must be a contiguous bf16 CUDA tensor [H, plane]")
        _check_offsets("jagged bias block offsets", boff)
        gptr = None
        if jagged_bias_grad is not None:
            if (jagged_bias_grad.dtype != torch.bfloat16 or tuple(jagged_bias_grad.shape) != tuple(values.shape)
                    or not jagged_bias_grad.is_contiguous() or jagged_bias_grad.device != values.device):
                raise ValueError("jagged_bias_grad must be a contiguous bf16 tensor shaped like the bias values")
            gptr = jagged_bias_grad.data_ptr()
        return (_Bias(2, None, 0, 0, None, values.data_ptr(), boff.data_ptr(), values.shape[1], gptr),
                (values, boff))
    if jagged_bias_grad is not None:
        raise ValueError("jagged_bias_grad needs a general jagged bias")
    if bias is None:
        if grad is not None:
            raise ValueError("bias_grad needs a bias table")
        return None, None
    if not bias.is_cuda or bias.dtype != torch.float32 or bias.dim() != 2 or bias.shape[0] != H:
        raise ValueError("bias must be a float32 CUDA tensor [H, num_buckets]")
    bias = bias.contiguous()
    gptr = None
    if grad is not None:
        if (grad.device != bias.device or grad.dtype != torch.float32 or tuple(grad.shape) != tuple(bias.shape)
                or not grad.is_contiguous()):
            raise ValueError("bias_grad must be a contiguous float32 tensor shaped like the bias table, on its device")
        gptr = grad.data_ptr()
    return _Bias(1, bias.data_ptr(), bias.shape[1], int(center), gptr), bias


def workspace_size(B, H, d, total_q, total_kv, backward) -> int:
    return int(load_library().jfa_workspace_size(B, H, d, total_q, total_kv, 1 if backward else 0))


def new_workspace(B, H, d, total_q, total_kv, backward, device) -> torch.Tensor:
    """A zero-initialised workspace for jfa_forward (backward=False) or jfa_backward."""
    return _workspace(workspace_size(B, H, d, total_q, total_kv, backward), device)


def _workspace(nbytes, device):
    # 256-byte alignment is guaranteed by the caching allocator; the status header must
    # start zeroed
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)


def jfa_forward(q, k, v, q_offsets, kv_offsets, bias=None, bias_center=0, scale=None, causal=False,
                out=None, lse=None, workspace=None, stream=None, jagged_bias=None):
    """out, lse = jfa_forward(...): the C-ABI forward on PyTorch-allocated device memory.

    q: bf16 [Tq, H, d]; k, v: bf16 [Tk, H, d]; offsets: int64 [B+1] on the device.
    bias: optional fp32 [H, num_buckets] relative-position table (bucket j - i + bias_center).
    jagged_bias: optional (values bf16 [H, plane], block offsets int64 [B+1]): a general
    bias, one Lq x Lk block per sequence with rows padded to 8 elements (see jfa.h).
    Returns out bf16 [Tq, H, d] and lse fp32 [H, Tq].  The call is asynchronous on
    the current stream; device-side errors are reported by jfa_check_status(workspace).
    """
    lib = load_library()
    _check_values("q", q)
    Tq, H, d = q.shape
    _check_values("k", k, H=H, d=d)
    _check_values("v", v, rows=k.shape[0], H=H, d=d)
    _check_offsets("q_offsets", q_offsets)
    _check_offsets("kv_offsets", kv_offsets)
    B = q_offsets.numel() - 1
    if kv_offsets.numel() != B + 1:
        raise ValueError("q_offsets and kv_offsets must have the same length")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    bstruct, bias_keep = _bias_struct(bias, bias_center, H, jagged_bias=jagged_bias)
    for name, t in (("k", k), ("v", v), ("q_offsets", q_offsets), ("kv_offsets", kv_offsets)):
        if t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_values("out", out, rows=Tq, H=H, d=d)
    if lse is None:
        lse = torch.empty((H, Tq), dtype=torch.float32, device=q.device)
    else:
        _check_lse(lse, H, Tq)
    nbytes = int(lib.jfa_workspace_size(B, H, d, Tq, k.shape[0], 0))
    if workspace is None:
        workspace = _workspace(nbytes, q.device)
    ws_bytes = _check_workspace(workspace, nbytes, q.device)
    st = lib.jfa_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_offsets.data_ptr(), kv_offsets.data_ptr(),
                         B, H, d, Tq, k.shape[0], ctypes.byref(bstruct) if bstruct is not None else None,
                         scale, 1 if causal else 0, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                         ws_bytes, _stream_handle(stream))
    if st != JFA_OK:
        raise JfaError(st, "jfa_forward")
    del bias_keep
    return out, lse, workspace


def jfa_backward(dout, q, k, v, out, lse, q_offsets, kv_offsets, bias=None, bias_center=0, scale=None,
                 causal=False, dq=None, dk=None, dv=None, workspace=None, stream=None, bias_grad=None,
                 jagged_bias=None, jagged_bias_grad=None):
    """dq, dk, dv, workspace = jfa_backward(...): gradients of sum(dout * out).  With
    `bias_grad` (a float32 tensor shaped like `bias`) the bias table's gradient is written
    into it as well; with `jagged_bias_grad` (a bf16 tensor shaped like a general bias's
    values) that bias's gradient (dS at every block element)."""
    lib = load_library()
    _check_values("q", q)
    Tq, H, d = q.shape
    for name, t, rows in (("dout", dout, Tq), ("out", out, Tq), ("k", k, None), ("v", v, k.shape[0])):
        _check_values(name, t, rows=rows, H=H, d=d)
    _check_lse(lse, H, Tq)
    _check_offsets("q_offsets", q_offsets)
    _check_offsets("kv_offsets", kv_offsets)
    B = q_offsets.numel() - 1
    if kv_offsets.numel() != B + 1:
        raise ValueError("q_offsets and kv_offsets must have the same length")
    for name, t in (("dout", dout), ("k", k), ("v", v), ("out", out), ("lse", lse), ("q_offsets", q_offsets),
                    ("kv_offsets", kv_offsets)):
        if t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    bstruct, bias_keep = _bias_struct(bias, bias_center, H, bias_grad, jagged_bias, jagged_bias_grad)
    for name, t, ref in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _check_values(name, t, rows=ref.shape[0], H=H, d=d)
            if t.device != q.device:
                raise ValueError(f"{name} is on {t.device}, q on {q.device}")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    nbytes = int(lib.jfa_workspace_size(B, H, d, Tq, k.shape[0], 1))
    if workspace is None:
        workspace = _workspace(nbytes, q.device)
    ws_bytes = _check_workspace(workspace, nbytes, q.device)
    st = lib.jfa_backward(dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                          lse.data_ptr(), q_offsets.data_ptr(), kv_offsets.data_ptr(), B, H, d, Tq, k.shape[0],
                          ctypes.byref(bstruct) if bstruct is not None else None, scale, 1 if causal else 0,
                          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), ws_bytes,
                          _stream_handle(stream))
    if st != JFA_OK:
        raise JfaError(st, "jfa_backward")
    del bias_keep
    return dq, dk, dv, workspace


# ---------------------------------------------------------------- sliding window with sinks
_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def _call(device, stream, run):
    """run(stream handle) with `stream` current (so that what the call allocates and clears is
    ordered with its kernels), else on `device`'s current stream.  As with any work on a stream of
    one's own, the inputs have to be ready on `stream` and alive until it has passed the call."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            return run(int(stream.cuda_stream))
    if device.index == torch.cuda.current_device():
        return run(torch._C._cuda_getCurrentRawStream(device.index))
    with torch.cuda.device(device):
        return run(torch._C._cuda_getCurrentRawStream(device.index))


def _rows_ok(t, shape, device):
    """Whether `t` is a contiguous bfloat16 CUDA tensor of that shape on `device`: the one test of
    the usual call.  A call takes microseconds, so only a tensor that fails it is looked at again,
    check by check, for the message."""
    return t.dtype is _BF16 and t.shape == shape and t.is_contiguous() and t.device == device


def _require_rows(name, t, shape, device):
    try:
        if _rows_ok(t, shape, device):
            return
    except AttributeError:
        pass
    _check_values(name, t, *shape)
    raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")


def _require_offsets(name, t, n, device):
    try:
        if t.dtype is _I64 and t.shape == (n,) and n > 1 and t.is_contiguous() and t.device == device:
            return
    except AttributeError:
        pass
    _check_offsets(name, t)
    raise ValueError(f"{name} must hold {n} offsets on {device}")


def _require_lse(t, H, rows, device):
    _check_lse(t, H, rows)
    if t.device != device:
        raise ValueError(f"lse is on {t.device}, the other tensors on {device}")


@functools.lru_cache(maxsize=256)
def _window_bytes(B, H, G, d, Tq, Tk, sinks, backward):
    return int(load_library().jfa_window_workspace_size(B, H, G, d, Tq, Tk, sinks, backward))


@functools.lru_cache(maxsize=256)
def _cache_bytes(B, H, G, d):
    return int(load_library().jfa_cache_workspace_size(B, H, G, d))


def window_workspace_size(B, H, H_kv, d, total_q, total_kv, sinks, backward) -> int:
    return int(load_library().jfa_window_workspace_size(B, H, H_kv, d, total_q, total_kv, sinks, 1 if backward else 0))


def new_window_workspace(B, H, H_kv, d, total_q, total_kv, sinks, backward, device) -> torch.Tensor:
    """A zero-initialised workspace for jfa_window_forward (backward=False) or jfa_window_backward."""
    nbytes = window_workspace_size(B, H, H_kv, d, total_q, total_kv, sinks, backward)
    if nbytes == 0:
        raise ValueError(f"no window workspace for B={B}, H={H}, H_kv={H_kv}, d={d}, sinks={sinks}")
    return _workspace(nbytes, device)


def _check_windowed(q, k, v, q_offsets, kv_offsets):
    """Checks of the inputs both directions share; returns (B, Tq, H, G, d, Tk)."""
    _check_values("q", q)
    Tq, H, d = q.shape
    if getattr(k, "ndim", 0) != 3 or k.shape[2] != d or k.shape[1] < 1 or H % k.shape[1]:
        _check_values("k", k)
        raise ValueError(f"k has shape {tuple(k.shape)}, expected [*, a divisor of {H}, {d}]")
    device, (Tk, G, _) = q.device, k.shape
    _require_rows("k", k, (Tk, G, d), device)
    _require_rows("v", v, (Tk, G, d), device)
    if not isinstance(q_offsets, torch.Tensor):
        _check_offsets("q_offsets", q_offsets)
    n = q_offsets.numel()
    _require_offsets("q_offsets", q_offsets, n, device)
    _require_offsets("kv_offsets", kv_offsets, n, device)
    return n - 1, Tq, H, G, d, Tk


def jfa_window_forward(q, k, v, q_offsets, kv_offsets, window=None, sinks=0, scale=None, out=None, lse=None,
                       workspace=None, stream=None):
    """out, lse, workspace = jfa_window_forward(...): causal jagged attention in a sliding window.

    q: bf16 [Tq, H, d]; k, v: bf16 [Tk, H_kv, d], H a multiple of H_kv; offsets: int64 [B+1] on the
    device.  Query i of a sequence, at position p = i + Lk - Lq, sees key j iff j <= p and
    (j > p - window or j < sinks); window None: every key up to p.  Returns out bf16 [Tq, H, d]
    and lse fp32 [H, Tq].  Asynchronous; device-side errors are reported by
    jfa_check_status(workspace).
    """
    lib = load_library()
    B, Tq, H, G, d, Tk = _check_windowed(q, k, v, q_offsets, kv_offsets)
    device, window, sinks = q.device, _check_window(window, sinks), int(sinks)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    nbytes = _window_bytes(B, H, G, d, Tq, Tk, sinks, 0)

    def run(handle):
        o = torch.empty_like(q) if out is None else out
        z = torch.empty((H, Tq), dtype=_F32, device=device) if lse is None else lse
        ws = _workspace(nbytes, device) if workspace is None else workspace
        if out is not None:
            _require_rows("out", o, (Tq, H, d), device)
        if lse is not None:
            _require_lse(z, H, Tq, device)
        st = lib.jfa_window_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_offsets.data_ptr(),
                                    kv_offsets.data_ptr(), B, H, G, d, Tq, Tk, window, sinks, scale, o.data_ptr(),
                                    z.data_ptr(), ws.data_ptr(), _check_workspace(ws, nbytes, device), handle)
        if st != JFA_OK:
            raise JfaError(st, "jfa_window_forward")
        return o, z, ws

    return _call(device, stream, run)


def jfa_window_backward(dout, q, k, v, out, lse, q_offsets, kv_offsets, window=None, sinks=0, scale=None, dq=None,
                        dk=None, dv=None, workspace=None, stream=None):
    """dq, dk, dv, workspace = jfa_window_backward(...): gradients of sum(dout * out), out and lse
    being jfa_window_forward's results for the same inputs.  dk and dv (shaped like k and v) sum
    over the query heads that share a key/value head."""
    lib = load_library()
    B, Tq, H, G, d, Tk = _check_windowed(q, k, v, q_offsets, kv_offsets)
    device, window, sinks = q.device, _check_window(window, sinks), int(sinks)
    _require_rows("dout", dout, (Tq, H, d), device)
    _require_rows("out", out, (Tq, H, d), device)
    _require_lse(lse, H, Tq, device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    nbytes = _window_bytes(B, H, G, d, Tq, Tk, sinks, 1)

    def run(handle):
        grads = [torch.empty_like(x) if g is None else g for g, x in ((dq, q), (dk, k), (dv, v))]
        for name, g, given, x in zip(("dq", "dk", "dv"), grads, (dq, dk, dv), (q, k, v)):
            if given is not None:
                _require_rows(name, g, tuple(x.shape), device)
        ws = _workspace(nbytes, device) if workspace is None else workspace
        st = lib.jfa_window_backward(dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                     lse.data_ptr(), q_offsets.data_ptr(), kv_offsets.data_ptr(), B, H, G, d, Tq, Tk,
                                     window, sinks, scale, grads[0].data_ptr(), grads[1].data_ptr(), grads[2].data_ptr(),
                                     ws.data_ptr(), _check_workspace(ws, nbytes, device), handle)
        if st != JFA_OK:
            raise JfaError(st, "jfa_window_backward")
        return (*grads, ws)

    return _call(device, stream, run)


# ---------------------------------------------------------------- paged key/value cache
def _check_int32(name, t, shape, device):
    if (not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.int32 or tuple(t.shape) != shape
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on {device}")


def _check_tokens(name, t, rows, heads, d, device):
    """Token rows [T, heads, d], each row contiguous; tokens may be strided.  Returns the rows, the
    address and the elements between tokens."""
    try:
        n, h, w = t.shape
        step, *inner = t.stride()
        ptr = t.data_ptr()
        if (t.dtype is _BF16 and w == d and t.device == device and (rows is None or n == rows)
                and (heads is None or h == heads) and n > 1 and h > 0 and inner == [d, 1]
                and step % 8 == 0 and step >= h * d and ptr % 16 == 0):
            return n, ptr, step
    except (AttributeError, ValueError, RuntimeError):
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device} (the library has no CPU path)")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if t.dim() != 3 or (rows is not None and t.shape[0] != rows) or t.shape[2] != d or \
            (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{rows}, {heads}, {d}]")
    if t.numel() and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d) or
                      (t.shape[0] > 1 and (t.stride(0) % 8 or t.stride(0) < t.shape[1] * d)) or t.data_ptr() % 16):
        raise ValueError(f"{name} needs contiguous 16-byte aligned rows, tokens a multiple of 8 elements apart")
    return t.shape[0], t.data_ptr(), t.stride(0)


def _cache_struct(k_cache, v_cache, page_table, lengths):
    try:
        device, shape = k_cache.device, k_cache.shape
        ok = (k_cache.is_cuda and len(shape) == 4 and page_table.dim() == 2 and _rows_ok(k_cache, shape, device)
              and _rows_ok(v_cache, shape, device) and page_table.dtype is _I32 and lengths.dtype is _I32
              and page_table.shape[0] > 0 and lengths.shape == page_table.shape[:1] and page_table.is_contiguous()
              and lengths.is_contiguous() and page_table.device == device and lengths.device == device)
    except AttributeError:
        ok = False
    if not ok:
        _explain_cache(k_cache, v_cache, page_table, lengths)
    P, G, page, d = shape
    B, width = page_table.shape
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), P, G, page, d, page_table.data_ptr(), width,
                  lengths.data_ptr(), B)


def _explain_cache(k_cache, v_cache, page_table, lengths):
    """Raises for the first thing wrong with a cache."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous() or t.shape != k_cache.shape or \
                t.device != k_cache.device:
            raise ValueError(f"{name} must be a contiguous bfloat16 tensor [num_pages, H_kv, page_size, d] "
                             "(both of one shape, on one device)")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or page_table.shape[0] < 1:
        raise ValueError("page_table must be an int32 CUDA tensor [B, max_pages]")
    B = page_table.shape[0]
    _check_int32("page_table", page_table, (B, page_table.shape[1]), k_cache.device)
    _check_int32("lengths", lengths, (B,), k_cache.device)
    raise ValueError("unusable cache")


def cache_workspace_size(B, H, H_kv, d) -> int:
    return int(load_library().jfa_cache_workspace_size(B, H, H_kv, d))


def new_cache_workspace(B, H, H_kv, d, device) -> torch.Tensor:
    """A zero-initialised workspace for jfa_cache_append and jfa_cache_attention, one call at a time.
    Zero it again after a timeout, or when forward or backward calls have used it: as long as its
    counters may not be zero, jfa_cache_attention reports JFA_ERR_WORKSPACE."""
    nbytes = cache_workspace_size(B, H, H_kv, d)
    if nbytes == 0:
        raise ValueError(f"no cache workspace for B={B}, H={H}, H_kv={H_kv}, d={d}")
    return _workspace(nbytes, device)


def rotary_frequencies(dim, base=10000.0) -> torch.Tensor:
    """The usual angles per position, base^(-2i/dim) for pairs i = 0 .. dim/2 - 1, as the
    float64 CPU tensor that jfa_cache_append takes."""
    return float(base) ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)


def jfa_cache_append(k, v, offsets, k_cache, v_cache, page_table, lengths, q=None, frequencies=None, interleaved=False,
                     q_out=None, k_out=None, lengths_out=None, workspace=None, stream=None):
    """q_out, k_out, lengths_out, workspace = jfa_cache_append(...): append new tokens to the
    paged cache, keys (and q) rotated by their positions on the way.

    k, v: bf16 [T, H_kv, d], q: bf16 [T, H, d] or None; tokens may be strided (slices of one
    projection).  offsets: int64 [B+1] on the device, sequence b's new tokens being rows
    offsets[b] .. offsets[b+1] - 1 (rows behind the last sequence are left alone).  k_cache,
    v_cache: bf16 [num_pages, H_kv, page_size, d]; page_table: int32 [B, max_pages]; lengths:
    int32 [B], tokens cached so far.  frequencies: float64 CPU tensor [rot_dim / 2], radians per
    position (rotary_frequencies), or None for no rotation.  Writes the caches; returns the
    rotated q (None without q), k_out (the rotated keys where a tensor was given for them) and
    the lengths after the call (lengths_out may be `lengths` itself).  Asynchronous; device-side
    errors are reported by jfa_check_status(workspace), and a sequence that they keep from being
    stored whole keeps its length.
    """
    lib = load_library()
    cache = _cache_struct(k_cache, v_cache, page_table, lengths)
    device, G, d, B = k_cache.device, cache.H_kv, cache.d, cache.B
    T, k_ptr, k_step = _check_tokens("k", k, None, G, d, device)
    _, v_ptr, v_step = _check_tokens("v", v, T, G, d, device)
    _require_offsets("offsets", offsets, B + 1, device)
    H, q_ptr, q_step = 0, None, 0
    if q is not None:
        _, q_ptr, q_step = _check_tokens("q", q, T, None, d, device)
        H = q.shape[1]
    elif q_out is not None:
        raise ValueError("q_out needs q")
    rot, freq_ptr = 0, None
    if frequencies is not None:
        if (not isinstance(frequencies, torch.Tensor) or frequencies.is_cuda or frequencies.dtype != torch.float64
                or frequencies.dim() != 1 or not frequencies.is_contiguous()):
            raise ValueError("frequencies must be a contiguous float64 CPU tensor [rot_dim / 2]")
        rot, freq_ptr = 2 * frequencies.numel(), frequencies.data_ptr()

    def run(handle):
        qo, ws = q_out, workspace
        if q is not None and qo is None:
            qo = torch.empty((T, H, d), dtype=_BF16, device=device)
        elif qo is not None:
            _require_rows("q_out", qo, (T, H, d), device)
        if k_out is not None:
            _require_rows("k_out", k_out, (T, G, d), device)
        if lengths_out is None:
            n = torch.empty_like(lengths)
        else:
            n = lengths_out
            _check_int32("lengths_out", n, (B,), device)
        if ws is None:
            ws = _workspace(256, device)
        st = lib.jfa_cache_append(ctypes.byref(cache), k_ptr, k_step, v_ptr, v_step, q_ptr if H else None,
                                  q_step if H else 0, H, offsets.data_ptr(), T,
                                  freq_ptr, rot, 1 if interleaved else 0, qo.data_ptr() if H else None,
                                  k_out.data_ptr() if k_out is not None else None, n.data_ptr(), ws.data_ptr(),
                                  _check_workspace(ws, 256, device), handle)
        if st != JFA_OK:
            raise JfaError(st, "jfa_cache_append")
        return qo, k_out, n, ws

    return _call(device, stream, run)


def jfa_cache_attention(q, k_cache, v_cache, page_table, lengths, window=None, sinks=0, scale=None, out=None, lse=None,
                        workspace=None, stream=None):
    """out, lse, workspace = jfa_cache_attention(...): attention of each sequence's newest token
    over the paged cache.

    q: bf16 [B, H, d], H a multiple of H_kv; lengths: int32 [B], the newest token included.  Key j
    is visible iff j < L and (j >= L - window or j < sinks); window None: every key.  Returns out
    bf16 [B, H, d] and lse fp32 [H, B] (0 and -inf for an empty sequence).  Asynchronous;
    device-side errors are reported by jfa_check_status(workspace).
    """
    lib = load_library()
    cache = _cache_struct(k_cache, v_cache, page_table, lengths)
    device, G, d, B = k_cache.device, cache.H_kv, cache.d, cache.B
    H = q.shape[1] if getattr(q, "ndim", 0) == 3 else 0
    if H < 1 or H % G:
        _check_values("q", q)
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [{B}, a multiple of {G}, {d}]")
    _require_rows("q", q, (B, H, d), device)
    window, sinks = _check_window(window, sinks), int(sinks)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    nbytes = _cache_bytes(B, H, G, d)

    def run(handle):
        o = torch.empty_like(q) if out is None else out
        z = torch.empty((H, B), dtype=_F32, device=device) if lse is None else lse
        ws = _workspace(nbytes, device) if workspace is None else workspace
        if out is not None:
            _require_rows("out", o, (B, H, d), device)
        if lse is not None:
            _require_lse(z, H, B, device)
        st = lib.jfa_cache_attention(ctypes.byref(cache), q.data_ptr(), H, window, sinks, scale, o.data_ptr(),
                                     z.data_ptr(), ws.data_ptr(), _check_workspace(ws, nbytes, device), handle)
        if st != JFA_OK:
            raise JfaError(st, "jfa_cache_attention")
        return o, z, ws

    return _call(device, stream, run)


def jfa_check_status(workspace, stream=None) -> int:
    """Synchronise `stream` (the workspace's device's current one) and return (and clear) the device
    status of the last call on that workspace."""
    lib = load_library()
    return _call(workspace.device, stream, lambda handle: int(lib.jfa_check_status(workspace.data_ptr(), handle)))


def jfa_set_nsp_max_tiles(max_tiles: int) -> int:
    """Sequences of 2 .. max_tiles query tiles take the non-sequence-parallel backward pass
    (0 or 1: none, the default); returns the previous setting.  Process-wide."""
    prev = int(load_library().jfa_set_nsp_max_tiles(int(max_tiles)))
    if prev < 0:
        raise ValueError(f"max_tiles must be in 0 .. 16, got {max_tiles}")
    return prev


def jfa_nsp_max_tiles() -> int:
    return int(load_library().jfa_set_nsp_max_tiles(-1))


def jfa_last_launch_count() -> int:
    return int(load_library().jfa_last_launch_count())


def jfa_timing_enable(on: bool) -> None:
    load_library().jfa_timing_enable(1 if on else 0)


def jfa_timing_read() -> dict:
    """{kind: (total_ms, launches)} for the launches recorded since the last read."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int * n)()
    st = load_library().jfa_timing_read(ms, cnt, n)
    if st != JFA_OK:
        raise JfaError(st, "jfa_timing_read")
    return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_KINDS)}


def jfa_trace_configure(buffer: Optional[torch.Tensor], kernel_kind: str = "forward") -> None:
    """Developer tracing: record pipeline events of the first CTA of every later launch of
    `kernel_kind` into `buffer` (a CUDA int64/uint8 tensor); None turns tracing off."""
    lib = load_library()
    if buffer is None:
        st = lib.jfa_trace_configure(None, 0, -1)
    else:
        st = lib.jfa_trace_configure(buffer.data_ptr(), buffer.numel() * buffer.element_size(),
                                     KERNEL_KINDS.index(kernel_kind))
    if st != JFA_OK:
        raise JfaError(st, "jfa_trace_configure")


def decode_trace(buffer: torch.Tensor):
    """Split a trace buffer into per-role lists of (sm_clock, event_id), dropping unused
    entries (the buffer should be zeroed before tracing)."""
    flat = buffer.detach().cpu().view(torch.int64).numpy()
    cap = flat.size // 5
    raw = flat[:5 * cap].reshape(5, cap)
    roles = []
    for r in range(5):
        ent = [int(x) & 0xFFFFFFFFFFFFFFFF for x in raw[r] if int(x) != 0]
        roles.append([(e >> 16, e & 0xFF) for e in ent])
    return roles


class JaggedAttention(torch.autograd.Function):
    """Differentiable jagged attention: out = JaggedAttention.apply(q, k, v, q_offsets,
    kv_offsets, bias, bias_center, scale, causal, jagged_bias_values, jagged_bias_offsets).
    lse is saved for the backward; the relative-position table and a general jagged bias's
    values get their gradients when they require them."""

    @staticmethod
    def forward(ctx, q, k, v, q_offsets, kv_offsets, bias=None, bias_center=0, scale=None, causal=False,
                jb_values=None, jb_offsets=None):
        jb = (jb_values, jb_offsets) if jb_values is not None else None
        out, lse, _ = jfa_forward(q, k, v, q_offsets, kv_offsets, bias, bias_center, scale, causal, jagged_bias=jb)
        ctx.save_for_backward(q, k, v, out, lse, q_offsets, kv_offsets, bias, jb_values, jb_offsets)
        ctx.cfg = (bias_center, scale, causal)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse, q_offsets, kv_offsets, bias, jb_values, jb_offsets = ctx.saved_tensors
        bias_center, scale, causal = ctx.cfg
        jb = (jb_values, jb_offsets) if jb_values is not None else None
        dbias = torch.empty_like(bias) if bias is not None and ctx.needs_input_grad[5] else None
        djb = torch.empty_like(jb_values) if jb_values is not None and ctx.needs_input_grad[9] else None
        dq, dk, dv, _ = jfa_backward(dout.contiguous(), q, k, v, out, lse, q_offsets, kv_offsets, bias,
                                     bias_center, scale, causal, bias_grad=dbias, jagged_bias=jb,
                                     jagged_bias_grad=djb)
        return dq, dk, dv, None, None, dbias, None, None, None, djb, None


def jagged_attention(q, k, v, q_offsets, kv_offsets, bias=None, bias_center=0, scale=None, causal=False,
                     jagged_bias=None):
    jb_values, jb_offsets = jagged_bias if jagged_bias is not None else (None, None)
    return JaggedAttention.apply(q, k, v, q_offsets, kv_offsets, bias, bias_center, scale, causal, jb_values,
                                 jb_offsets)


def _check_capture(*inputs):
    """Refuses to capture a step whose gradients would be accumulated outside the capture.

    While an eager graph of a leaf lives, the leaf's gradient is accumulated on the stream that
    this graph was made on.  Made on the default stream, that is work which a capture cannot hold,
    and a backward pass captured then ends the process.  So an eager call there marks its leaves'
    accumulators, and a captured call refuses a marked one.  (A graph made on a side stream joins
    the capture, and a mark is gone with its graph.)  Returns the accumulators, for the caller to
    hold until its own graph does."""
    leaves = [t for t in inputs if isinstance(t, torch.Tensor) and t.is_cuda and t.requires_grad and t.is_leaf]
    if not leaves:
        return ()
    capturing = torch.cuda.is_current_stream_capturing()
    if not capturing and torch.cuda.current_stream(leaves[0].device).cuda_stream != 0:
        return ()
    nodes = [torch.autograd.graph.get_gradient_edge(t).node for t in leaves]
    for node in nodes:
        if not capturing:
            node.metadata["jfa_default_stream"] = True
        elif node.metadata.get("jfa_default_stream"):
            raise RuntimeError("cannot capture this call: an eager graph of the same leaf tensors, made on the default "
                               "stream, is alive; drop its outputs first, or run eager steps on a side stream")
    return nodes


class WindowAttention(torch.autograd.Function):
    """Differentiable windowed attention: out = WindowAttention.apply(q, k, v, q_offsets,
    kv_offsets, window, sinks, scale).  lse is saved for the backward, which cannot be
    differentiated again.  A step may be captured in a CUDA graph (see _check_capture)."""

    @classmethod
    def apply(cls, q, k, v, *args):
        # no graph is made where no gradient is recorded (in inference mode neither): nothing to check
        marked = _check_capture(q, k, v) if torch.is_grad_enabled() else ()
        out = super().apply(q, k, v, *args)
        del marked  # the graph holds them now
        return out

    @staticmethod
    def forward(ctx, q, k, v, q_offsets, kv_offsets, window=None, sinks=0, scale=None):
        out, lse, _ = jfa_window_forward(q, k, v, q_offsets, kv_offsets, window, sinks, scale)
        ctx.save_for_backward(q, k, v, out, lse, q_offsets, kv_offsets)
        ctx.cfg = (window, sinks, scale)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, q_offsets, kv_offsets = ctx.saved_tensors
        dq, dk, dv, _ = jfa_window_backward(dout.contiguous(), q, k, v, out, lse, q_offsets, kv_offsets, *ctx.cfg)
        return dq, dk, dv, None, None, None, None, None


def window_attention(q, k, v, q_offsets, kv_offsets, window=None, sinks=0, scale=None):
    """Causal jagged attention in a sliding window with sinks (jfa_window_forward), differentiable."""
    return WindowAttention.apply(q, k, v, q_offsets, kv_offsets, window, sinks, scale)
