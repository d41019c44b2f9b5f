"""Causal Local Linear Attention (LLA) forward pass for GB300 (sm_103a).

Thin ctypes binding over liblla.so, whose C ABI is declared in include/lla.h.  The
binding only marshals arguments: every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and the current stream.

There is no CPU fallback: if liblla.so is missing or cannot load, every call
raises ``LLAError``.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from collections import namedtuple

__all__ = [
    "LLAError", "load_library", "library_path", "forward", "forward_host", "lla_forward", "lla_forward_ex",
    "lla_forward_host", "lla_forward_host_buffer_size",
    "lla_workspace_size", "lla_resolve_path", "lla_sync_status", "lla_selftest_device_timeout", "lla_last_error",
    "lla_version",
    "lla_profile_enable", "lla_profile_read", "lla_forward_noalloc", "lla_parallax_forward", "parallax_forward",
    "lla_decode", "lla_decode_ex", "lla_decode_max_n", "decode", "lla_backward", "lla_backward_workspace_size", "backward",
    "lla_backward_host", "lla_backward_host_buffer_size", "backward_host",
    "lla_paged_plan", "lla_paged_append", "lla_paged_parallax", "lla_paged_parallax_workspace_size",
    "PagedPlan", "paged_plan", "paged_append", "paged_parallax",
    "LLA_OK", "LLA_ERR_INVALID_ARG", "LLA_ERR_UNSUPPORTED", "LLA_ERR_CUDA", "LLA_ERR_DEVICE_TIMEOUT",
    "LLA_DTYPE_BF16", "LLA_DTYPE_FP32", "LLA_PATH_AUTO", "LLA_PATH_TENSOR", "LLA_PATH_FP32",
    "LLA_DECODE_AUTO", "LLA_DECODE_MOMENT", "LLA_DECODE_STREAM", "LLA_DECODE_CLUSTER",
    "EXPORTED_SYMBOLS",
]

LLA_OK, LLA_ERR_INVALID_ARG, LLA_ERR_UNSUPPORTED, LLA_ERR_CUDA, LLA_ERR_DEVICE_TIMEOUT = range(5)
LLA_DTYPE_BF16, LLA_DTYPE_FP32 = 0, 1
LLA_PATH_AUTO, LLA_PATH_TENSOR, LLA_PATH_FP32 = 0, 1, 2
LLA_DECODE_AUTO, LLA_DECODE_MOMENT, LLA_DECODE_STREAM, LLA_DECODE_CLUSTER = 0, 1, 2, 3

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

_c_int, _c_float, _c_size, _vp = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p
_c_ll = ctypes.c_longlong

# name -> (restype, argtypes); mirrors include/lla.h
_SIGNATURES = {
    "lla_forward": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_float, _c_float,
                             _c_int, _c_float, _vp]),
    "lla_forward_ex": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                _c_float, _c_float, _c_int, _c_float, _vp, _c_size, _vp]),
    "lla_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "lla_forward_host": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                  _c_float, _c_float, _c_int, _c_float, _c_int, _vp, _c_size, _vp]),
    "lla_forward_host_buffer_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "lla_resolve_path": (_c_int, [_c_int, _c_int, _c_int]),
    "lla_sync_status": (_c_int, [_vp]),
    "lla_selftest_device_timeout": (_c_int, [_vp]),
    "lla_last_error": (ctypes.c_char_p, []),
    "lla_forward_noalloc": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_float,
                                     _c_float, _c_int, _c_float, _vp]),
    "lla_parallax_forward": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                      _c_float, _vp, _c_size, _vp]),
    "lla_decode": (_c_int, [_c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                            _c_float, _c_float, _c_int, _c_float, _vp]),
    "lla_decode_ex": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                               _c_int, _c_float, _c_float, _c_int, _c_float, _vp]),
    "lla_decode_max_n": (_c_int, [_c_int]),
    "lla_backward": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int,
                              _c_int, _c_int, _c_float, _c_float, _c_int, _c_float, _vp, _c_size, _vp]),
    "lla_backward_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "lla_backward_host": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int,
                                   _c_int, _c_int, _c_float, _c_float, _c_int, _c_float, _c_int, _vp, _c_size, _vp]),
    "lla_backward_host_buffer_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "lla_paged_plan": (_c_int, [_vp, _vp, _c_int, _c_int, _vp, _c_int, _vp, _c_int, _vp, _c_int, _vp, _vp, _vp, _vp,
                                _vp, _vp, _vp]),
    "lla_paged_append": (_c_int, [_c_int, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_ll, _c_ll,
                                  _c_ll, _vp]),
    "lla_paged_parallax": (_c_int, [_c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                    _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_ll, _c_ll, _c_ll, _c_float,
                                    _c_int, _vp, _c_size, _vp]),
    "lla_paged_parallax_workspace_size": (_c_size, [_c_int] * 10),
    "lla_profile_enable": (_c_int, [_c_int]),
    "lla_profile_read": (_c_int, [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_float)]),
    "lla_version": (_c_int, []),
}
EXPORTED_SYMBOLS = tuple(_SIGNATURES)


class LLAError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"LLA status {status}: {message}")
        self.status = status


def library_path():
    return os.environ.get("LLA_LIBRARY", os.path.join(_HERE, "liblla.so"))


def load_library():
    """Load liblla.so (built by ``build.build()``); raises LLAError if it is absent."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise LLAError(-1, f"{path} not found: build it with local_linear_attention_flashlla_gb300.build.build()")
    try:
        lib = ctypes.CDLL(path)
    except OSError as e:
        raise LLAError(-1, f"cannot load {path}: {e}") from e
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def _check(status):
    if status != LLA_OK:
        raise LLAError(status, load_library().lla_last_error().decode(errors="replace"))


def lla_last_error():
    return load_library().lla_last_error().decode(errors="replace")


def lla_version():
    return load_library().lla_version()


def lla_resolve_path(dtype, path, d):
    return load_library().lla_resolve_path(dtype, path, d)


def lla_workspace_size(dtype, path, B, H, n, d):
    return load_library().lla_workspace_size(dtype, path, B, H, n, d)


def lla_profile_enable(on=True):
    """Record CUDA events around each later call's dominant kernel (measurement support)."""
    _check(load_library().lla_profile_enable(1 if on else 0))


def lla_profile_read():
    """(dominant-kernel ms, whole-call ms) of the most recent profiled call."""
    a, b = ctypes.c_float(), ctypes.c_float()
    _check(load_library().lla_profile_read(ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def lla_sync_status(stream=None):
    """Synchronise the stream and raise if a kernel recorded an error: a device-side wait timeout, no work done, or a
    paged call's length, slot or page id that its tensors do not hold (include/lla.h)."""
    _check(load_library().lla_sync_status(_stream_ptr(stream)))


def lla_selftest_device_timeout(stream=None):
    """Launch the library's timeout self-test kernel (a bounded wait that gives up after about two
    seconds); the next lla_sync_status(stream) raises LLAError with LLA_ERR_DEVICE_TIMEOUT."""
    _check(load_library().lla_selftest_device_timeout(_stream_ptr(stream)))


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def lla_forward(q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, B, H, n, d, tau, lam, cg_max_iters, cg_tol,
                stream_ptr):
    """Raw C entry point on device pointers (ints); raises LLAError on a non-zero status."""
    _check(load_library().lla_forward(q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, B, H, n, d, tau, lam,
                                      cg_max_iters, cg_tol, stream_ptr))


def lla_forward_noalloc(q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, B, H, n, d, tau, lam, cg_max_iters,
                        cg_tol, stream_ptr):
    """C entry point that uses the library's fixed device scratch instead of allocating."""
    _check(load_library().lla_forward_noalloc(q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, B, H, n, d, tau,
                                              lam, cg_max_iters, cg_tol, stream_ptr))


def lla_forward_ex(dtype, path, q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, iters_ptr, B, H, n, d, tau, lam,
                   cg_max_iters, cg_tol, ws_ptr, ws_bytes, stream_ptr):
    """Raw C entry point with dtype/path/iteration-count/workspace arguments."""
    _check(load_library().lla_forward_ex(dtype, path, q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, iters_ptr,
                                         B, H, n, d, tau, lam, cg_max_iters, cg_tol, ws_ptr, ws_bytes, stream_ptr))


def lla_forward_host(dtype, path, q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, iters_ptr, B, H, n, d, tau, lam,
                     cg_max_iters, cg_tol, chunk_slices, buf_ptr, buf_bytes, stream_ptr):
    """Raw C entry point of the host-buffer forward (pointers are host addresses, buf_ptr a device one)."""
    _check(load_library().lla_forward_host(dtype, path, q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, iters_ptr,
                                           B, H, n, d, tau, lam, cg_max_iters, cg_tol, chunk_slices, buf_ptr,
                                           buf_bytes, stream_ptr))


def lla_forward_host_buffer_size(dtype, path, B, H, n, d, chunk_slices=0):
    return load_library().lla_forward_host_buffer_size(dtype, path, B, H, n, d, chunk_slices)


def lla_parallax_forward(dtype, path, q_ptr, k_ptr, v_ptr, probe_ptr, out_ptr, B, H, n, d, tau, ws_ptr, ws_bytes,
                         stream_ptr):
    """Raw Parallax-form entry point on device pointers (ints); raises LLAError on failure."""
    _check(load_library().lla_parallax_forward(dtype, path, q_ptr, k_ptr, v_ptr, probe_ptr, out_ptr, B, H, n, d, tau,
                                               ws_ptr, ws_bytes, stream_ptr))


def lla_decode(dtype, q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, iters_ptr, B, H, n, n_cap, d, tau, lam,
               cg_max_iters, cg_tol, stream_ptr):
    """Raw decode-step entry point on device pointers (ints); raises LLAError on failure."""
    _check(load_library().lla_decode(dtype, q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, iters_ptr, B, H, n,
                                     n_cap, d, tau, lam, cg_max_iters, cg_tol, stream_ptr))


def lla_decode_ex(form, dtype, q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, iters_ptr, B, H, n, n_cap, d, tau,
                  lam, cg_max_iters, cg_tol, stream_ptr):
    """Raw decode-step entry point with the form chosen (an LLA_DECODE_* value); raises LLAError."""
    _check(load_library().lla_decode_ex(form, dtype, q_ptr, k_ptr, v_ptr, out_ptr, rho_ptr, denom_ptr, iters_ptr, B,
                                        H, n, n_cap, d, tau, lam, cg_max_iters, cg_tol, stream_ptr))


def lla_decode_max_n(d):
    return load_library().lla_decode_max_n(d)


def decode(q, k_cache, v_cache, n, tau, lam, cg_max_iters, cg_tol=0.0, *, return_iters=False, out=None, rho=None,
           denom=None, form=LLA_DECODE_AUTO, stream=None):
    """One decode step: q [B, H, d] against caches [B, H, n_cap, d] whose first n rows are valid.

    Returns (out [B, H, d], rho [B, H, d] fp32, denom [B, H] fp32) and, with return_iters, the
    CG iteration counts [B, H].  Equals row n-1 of forward() on the cached sequence.  form: an
    LLA_DECODE_* value (include/lla.h, lla_decode_ex).
    """
    import torch
    if not (q.is_cuda and k_cache.is_cuda and v_cache.is_cuda):
        raise LLAError(LLA_ERR_INVALID_ARG, "q and the caches must be CUDA tensors (there is no CPU path)")
    if q.dim() != 3 or k_cache.dim() != 4 or k_cache.shape != v_cache.shape or \
            tuple(k_cache.shape[:2]) != tuple(q.shape[:2]) or k_cache.shape[3] != q.shape[2]:
        raise LLAError(LLA_ERR_INVALID_ARG, f"q [B, H, d] and caches [B, H, n_cap, d] expected, got {tuple(q.shape)}, "
                                            f"{tuple(k_cache.shape)}, {tuple(v_cache.shape)}")
    if not (q.dtype == k_cache.dtype == v_cache.dtype) or q.dtype not in (torch.bfloat16, torch.float32):
        raise LLAError(LLA_ERR_INVALID_ARG, "q and the caches must all be bf16 or all fp32")
    q, k_cache, v_cache = q.contiguous(), k_cache.contiguous(), v_cache.contiguous()
    B, H, n_cap, d = k_cache.shape
    dtype = LLA_DTYPE_BF16 if q.dtype == torch.bfloat16 else LLA_DTYPE_FP32
    if out is None:
        out = torch.empty_like(q)
    if rho is None:
        rho = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    if denom is None:
        denom = torch.empty((B, H), dtype=torch.float32, device=q.device)
    iters = torch.empty((B, H), dtype=torch.int32, device=q.device) if return_iters else None
    lla_decode_ex(int(form), dtype, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                  rho.data_ptr(), denom.data_ptr(), None if iters is None else iters.data_ptr(), B, H, int(n), n_cap, d,
                  float(tau), float(lam), int(cg_max_iters), float(cg_tol), _stream_ptr(stream))
    if return_iters:
        return out, rho, denom, iters
    return out, rho, denom


def lla_backward(dtype, path, q_ptr, k_ptr, v_ptr, rho_ptr, denom_ptr, dout_ptr, dq_ptr, dk_ptr, dv_ptr, iters_ptr,
                 B, H, n, d, tau, lam, cg_max_iters, cg_tol, ws_ptr, ws_bytes, stream_ptr):
    """Raw backward entry point on device pointers (ints); raises LLAError on failure."""
    _check(load_library().lla_backward(dtype, path, q_ptr, k_ptr, v_ptr, rho_ptr, denom_ptr, dout_ptr, dq_ptr, dk_ptr,
                                       dv_ptr, iters_ptr, B, H, n, d, tau, lam, cg_max_iters, cg_tol, ws_ptr,
                                       ws_bytes, stream_ptr))


def lla_backward_workspace_size(dtype, path, B, H, n, d):
    return load_library().lla_backward_workspace_size(dtype, path, B, H, n, d)


def backward(q, k, v, rho, denom, dout, tau, lam, cg_max_iters, cg_tol=0.0, *, path=LLA_PATH_AUTO,
             return_iters=False, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) [B, H, n, d] fp32 of sum(dout * out) for the forward call that gave
    rho [B, H, n, d] and denom [B, H, n] on q, k, v (see include/lla.h).  With return_iters also
    the adjoint CG iteration counts [B, H, n].  Asynchronous on the current (or given) stream.
    """
    import torch
    _check_qkv(q, k, v)
    if tuple(dout.shape) != tuple(q.shape) or dout.dtype != q.dtype or not dout.is_cuda:
        raise LLAError(LLA_ERR_INVALID_ARG, f"dout must be a CUDA tensor of shape {tuple(q.shape)} and dtype {q.dtype}")
    B, H, n, d = q.shape
    if tuple(rho.shape) != (B, H, n, d) or tuple(denom.shape) != (B, H, n) or \
            rho.dtype != torch.float32 or denom.dtype != torch.float32:
        raise LLAError(LLA_ERR_INVALID_ARG, "rho [B, H, n, d] and denom [B, H, n] must be the forward's fp32 outputs")
    q, k, v, dout = q.contiguous(), k.contiguous(), v.contiguous(), dout.contiguous()
    rho, denom = rho.contiguous(), denom.contiguous()
    dtype = LLA_DTYPE_BF16 if q.dtype == torch.bfloat16 else LLA_DTYPE_FP32
    grads = []
    for t in (dq, dk, dv):
        grads.append(torch.empty((B, H, n, d), dtype=torch.float32, device=q.device) if t is None else t)
    iters = torch.empty((B, H, n), dtype=torch.int32, device=q.device) if return_iters else None
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    lla_backward(dtype, path, q.data_ptr(), k.data_ptr(), v.data_ptr(), rho.data_ptr(), denom.data_ptr(), dout.data_ptr(),
                 grads[0].data_ptr(), grads[1].data_ptr(), grads[2].data_ptr(),
                 None if iters is None else iters.data_ptr(), B, H, n, d, float(tau), float(lam), int(cg_max_iters),
                 float(cg_tol), ws_ptr, ws_bytes, _stream_ptr(stream))
    if return_iters:
        return (*grads, iters)
    return tuple(grads)


def lla_backward_host(dtype, path, q_ptr, k_ptr, v_ptr, rho_ptr, denom_ptr, dout_ptr, dq_ptr, dk_ptr, dv_ptr,
                      iters_ptr, B, H, n, d, tau, lam, cg_max_iters, cg_tol, chunk_slices, buf_ptr, buf_bytes,
                      stream_ptr):
    """Raw host-buffer backward entry point (host addresses; buf_ptr a device one)."""
    _check(load_library().lla_backward_host(dtype, path, q_ptr, k_ptr, v_ptr, rho_ptr, denom_ptr, dout_ptr, dq_ptr,
                                            dk_ptr, dv_ptr, iters_ptr, B, H, n, d, tau, lam, cg_max_iters, cg_tol,
                                            chunk_slices, buf_ptr, buf_bytes, stream_ptr))


def lla_backward_host_buffer_size(dtype, path, B, H, n, d, chunk_slices=0):
    return load_library().lla_backward_host_buffer_size(dtype, path, B, H, n, d, chunk_slices)


def backward_host(q, k, v, rho, denom, dout, tau, lam, cg_max_iters, cg_tol=0.0, *, path=LLA_PATH_AUTO,
                  chunk_slices=0, return_iters=False, dq=None, dk=None, dv=None, device_buffer=None, stream=None):
    """backward() on CPU tensors (pin them for overlapped copies): q, k, v, dout [B, H, n, d] bf16 or
    fp32, rho [B, H, n, d] and denom [B, H, n] fp32.  Returns CPU fp32 dq, dk, dv (pinned unless
    passed in).  Asynchronous on the current (or given) stream: synchronise before reading."""
    import torch
    ins = (q, k, v, dout, rho, denom)
    if any(t.is_cuda for t in ins):
        raise LLAError(LLA_ERR_INVALID_ARG, "backward_host takes CPU tensors; use backward() for CUDA tensors")
    if q.dim() != 4 or any(tuple(t.shape) != tuple(q.shape) for t in (k, v, dout, rho)):
        raise LLAError(LLA_ERR_INVALID_ARG, "q, k, v, dout, rho must share one [B, H, n, d] shape")
    B, H, n, d = q.shape
    if tuple(denom.shape) != (B, H, n) or rho.dtype != torch.float32 or denom.dtype != torch.float32:
        raise LLAError(LLA_ERR_INVALID_ARG, "rho [B, H, n, d] and denom [B, H, n] must be fp32")
    if not (q.dtype == k.dtype == v.dtype == dout.dtype) or q.dtype not in (torch.bfloat16, torch.float32):
        raise LLAError(LLA_ERR_INVALID_ARG, "q, k, v, dout must all be bf16 or all fp32")
    if not all(t.is_contiguous() for t in ins):
        raise LLAError(LLA_ERR_INVALID_ARG, "inputs must be contiguous (a copy would not stay alive for the call)")
    dtype = LLA_DTYPE_BF16 if q.dtype == torch.bfloat16 else LLA_DTYPE_FP32
    grads = []
    for t in (dq, dk, dv):
        if t is None:
            t = torch.empty((B, H, n, d), dtype=torch.float32).pin_memory()
        elif t.is_cuda or tuple(t.shape) != (B, H, n, d) or t.dtype != torch.float32 or not t.is_contiguous():
            raise LLAError(LLA_ERR_INVALID_ARG, "gradient outputs must be contiguous CPU fp32 [B, H, n, d] tensors")
        grads.append(t)
    iters = torch.empty((B, H, n), dtype=torch.int32).pin_memory() if return_iters else None
    if device_buffer is None:
        buf_ptr, buf_bytes = None, 0
    else:
        if not device_buffer.is_cuda:
            raise LLAError(LLA_ERR_INVALID_ARG, "device_buffer must be a CUDA tensor")
        buf_ptr, buf_bytes = device_buffer.data_ptr(), device_buffer.numel() * device_buffer.element_size()
    lla_backward_host(dtype, path, q.data_ptr(), k.data_ptr(), v.data_ptr(), rho.data_ptr(), denom.data_ptr(),
                      dout.data_ptr(), grads[0].data_ptr(), grads[1].data_ptr(), grads[2].data_ptr(),
                      None if iters is None else iters.data_ptr(), B, H, n, d, float(tau), float(lam),
                      int(cg_max_iters), float(cg_tol), int(chunk_slices), buf_ptr, buf_bytes, _stream_ptr(stream))
    if return_iters:
        return (*grads, iters)
    return tuple(grads)


def _check_qkv(q, k, v):
    import torch
    if not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise LLAError(LLA_ERR_INVALID_ARG, "q, k, v must be CUDA tensors (there is no CPU path)")
    if q.shape != k.shape or q.shape != v.shape or q.dim() != 4:
        raise LLAError(LLA_ERR_INVALID_ARG, f"q, k, v must share one [B, H, n, d] shape, got {tuple(q.shape)}, "
                                            f"{tuple(k.shape)}, {tuple(v.shape)}")
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in (torch.bfloat16, torch.float32):
        raise LLAError(LLA_ERR_INVALID_ARG, "q, k, v must all be bf16 or all fp32")


def parallax_forward(q, k, v, probe, tau, *, path=LLA_PATH_AUTO, out=None, workspace=None, stream=None):
    """Parallax-form causal attention: softmax output minus Sigma_KV probe (see include/lla.h).

    q, k, v: CUDA [B, H, n, d] bf16 or fp32; probe: [B, H, n, d] (converted to contiguous fp32).
    Returns out (dtype of q).  Asynchronous on the current (or given) stream.
    """
    import torch
    _check_qkv(q, k, v)
    if tuple(probe.shape) != tuple(q.shape) or not probe.is_cuda:
        raise LLAError(LLA_ERR_INVALID_ARG, f"probe must be a CUDA tensor of shape {tuple(q.shape)}")
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    probe = probe.to(torch.float32).contiguous()
    B, H, n, d = q.shape
    dtype = LLA_DTYPE_BF16 if q.dtype == torch.bfloat16 else LLA_DTYPE_FP32
    if out is None:
        out = torch.empty_like(q)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    lla_parallax_forward(dtype, path, q.data_ptr(), k.data_ptr(), v.data_ptr(), probe.data_ptr(), out.data_ptr(),
                         B, H, n, d, float(tau), ws_ptr, ws_bytes, _stream_ptr(stream))
    return out


def forward(q, k, v, tau, lam, cg_max_iters, cg_tol=0.0, *, path=LLA_PATH_AUTO, return_iters=False,
            out=None, rho=None, denom=None, workspace=None, stream=None):
    """Causal LLA forward on CUDA tensors q, k, v of shape [B, H, n, d] (bf16 or fp32).

    Returns (out, rho, denom) or, with return_iters, (out, rho, denom, cg_iters).
    Output tensors are allocated with torch unless passed in.  Asynchronous on the
    current (or given) stream.
    """
    import torch
    if not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise LLAError(LLA_ERR_INVALID_ARG, "q, k, v must be CUDA tensors (there is no CPU path)")
    if q.shape != k.shape or q.shape != v.shape or q.dim() != 4:
        raise LLAError(LLA_ERR_INVALID_ARG, f"q, k, v must share one [B, H, n, d] shape, got {tuple(q.shape)}, "
                                            f"{tuple(k.shape)}, {tuple(v.shape)}")
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in (torch.bfloat16, torch.float32):
        raise LLAError(LLA_ERR_INVALID_ARG, "q, k, v must all be bf16 or all fp32")
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    B, H, n, d = q.shape
    dtype = LLA_DTYPE_BF16 if q.dtype == torch.bfloat16 else LLA_DTYPE_FP32
    if out is None:
        out = torch.empty_like(q)
    if rho is None:
        rho = torch.empty((B, H, n, d), dtype=torch.float32, device=q.device)
    if denom is None:
        denom = torch.empty((B, H, n), dtype=torch.float32, device=q.device)
    iters = torch.empty((B, H, n), dtype=torch.int32, device=q.device) if return_iters else None
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    lla_forward_ex(dtype, path, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), rho.data_ptr(),
                   denom.data_ptr(), None if iters is None else iters.data_ptr(), B, H, n, d, float(tau), float(lam),
                   int(cg_max_iters), float(cg_tol), ws_ptr, ws_bytes, _stream_ptr(stream))
    if return_iters:
        return out, rho, denom, iters
    return out, rho, denom


def forward_host(q, k, v, tau, lam, cg_max_iters, cg_tol=0.0, *, path=LLA_PATH_AUTO, chunk_slices=0,
                 return_iters=False, out=None, rho=None, denom=None, device_buffer=None, stream=None):
    """forward() on CPU tensors q, k, v [B, H, n, d] (bf16 or fp32; pin them for overlapped copies).

    The library copies the (b, h) slices to the GPU in chunks, computes and copies the results
    back into CPU tensors (pinned unless passed in), overlapping the transfers with the compute.
    Asynchronous on the current (or given) stream: synchronise it before reading the results.
    device_buffer: optional uint8 CUDA tensor of lla_forward_host_buffer_size(...) bytes.
    """
    import torch
    if q.is_cuda or k.is_cuda or v.is_cuda:
        raise LLAError(LLA_ERR_INVALID_ARG, "forward_host takes CPU tensors; use forward() for CUDA tensors")
    if q.shape != k.shape or q.shape != v.shape or q.dim() != 4:
        raise LLAError(LLA_ERR_INVALID_ARG, f"q, k, v must share one [B, H, n, d] shape, got {tuple(q.shape)}, "
                                            f"{tuple(k.shape)}, {tuple(v.shape)}")
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in (torch.bfloat16, torch.float32):
        raise LLAError(LLA_ERR_INVALID_ARG, "q, k, v must all be bf16 or all fp32")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise LLAError(LLA_ERR_INVALID_ARG, "q, k, v must be contiguous (a copy would not stay alive for the call)")
    B, H, n, d = q.shape
    dtype = LLA_DTYPE_BF16 if q.dtype == torch.bfloat16 else LLA_DTYPE_FP32

    def host_out(t, shape, dt):
        if t is None:
            return torch.empty(shape, dtype=dt).pin_memory()
        if t.is_cuda or tuple(t.shape) != tuple(shape) or t.dtype != dt or not t.is_contiguous():
            raise LLAError(LLA_ERR_INVALID_ARG, f"output must be a contiguous CPU {dt} tensor of shape {tuple(shape)}")
        return t

    out = host_out(out, (B, H, n, d), q.dtype)
    rho = host_out(rho, (B, H, n, d), torch.float32)
    denom = host_out(denom, (B, H, n), torch.float32)
    iters = torch.empty((B, H, n), dtype=torch.int32).pin_memory() if return_iters else None
    if device_buffer is None:
        buf_ptr, buf_bytes = None, 0
    else:
        if not device_buffer.is_cuda:
            raise LLAError(LLA_ERR_INVALID_ARG, "device_buffer must be a CUDA tensor")
        buf_ptr, buf_bytes = device_buffer.data_ptr(), device_buffer.numel() * device_buffer.element_size()
    lla_forward_host(dtype, path, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), rho.data_ptr(),
                     denom.data_ptr(), None if iters is None else iters.data_ptr(), B, H, n, d, float(tau),
                     float(lam), int(cg_max_iters), float(cg_tol), int(chunk_slices), buf_ptr, buf_bytes,
                     _stream_ptr(stream))
    if return_iters:
        return out, rho, denom, iters
    return out, rho, denom


def lla_paged_plan(ctx_ptr, new_ptr, S, page_size, table_ptr, table_width, free_ptr, free_capacity, free_count_ptr, T,
                   kv_ptr, cu_ptr, slots_ptr, positions_ptr, granted_ptr, free_left_ptr, stream_ptr):
    """Raw page-planning entry point on device pointers (ints); raises LLAError on failure."""
    _check(load_library().lla_paged_plan(ctx_ptr, new_ptr, S, page_size, table_ptr, table_width, free_ptr, free_capacity,
                                         free_count_ptr, T, kv_ptr, cu_ptr, slots_ptr, positions_ptr, granted_ptr,
                                         free_left_ptr, stream_ptr))


def lla_paged_append(dtype, k_ptr, v_ptr, slots_ptr, k_cache_ptr, v_cache_ptr, T, Hkv, d, page_size, num_pages, k_stride,
                     v_stride, page_stride, stream_ptr):
    """Raw cache-append entry point on device pointers (ints); raises LLAError on failure."""
    _check(load_library().lla_paged_append(dtype, k_ptr, v_ptr, slots_ptr, k_cache_ptr, v_cache_ptr, T, Hkv, d, page_size,
                                           num_pages, k_stride, v_stride, page_stride, stream_ptr))


def lla_paged_parallax(dtype, path, q_ptr, probe_ptr, k_cache_ptr, v_cache_ptr, table_ptr, cu_ptr, kv_ptr, out_ptr, T, S,
                       Hq, Hkv, d, page_size, num_pages, table_width, max_new, q_stride, probe_stride, page_stride, tau,
                       causal, ws_ptr, ws_bytes, stream_ptr):
    """Raw paged Parallax entry point on device pointers (ints); raises LLAError on failure."""
    _check(load_library().lla_paged_parallax(dtype, path, q_ptr, probe_ptr, k_cache_ptr, v_cache_ptr, table_ptr, cu_ptr,
                                             kv_ptr, out_ptr, T, S, Hq, Hkv, d, page_size, num_pages, table_width, max_new,
                                             q_stride, probe_stride, page_stride, tau, causal, ws_ptr, ws_bytes,
                                             stream_ptr))


def lla_paged_parallax_workspace_size(dtype, path, T, S, Hq, Hkv, d, page_size, table_width, max_new):
    return load_library().lla_paged_parallax_workspace_size(dtype, path, T, S, Hq, Hkv, d, page_size, table_width, max_new)


PagedPlan = namedtuple("PagedPlan", "kv_lens cu_q slots positions granted free_left")


class _on_stream:
    """Makes `device` current and, where a stream is given, that stream: what a call allocates or copies
    inside belongs to the stream that its kernels run on."""

    def __init__(self, device, stream):
        self._device, self._stream, self._open = device, stream, ()

    def __enter__(self):
        import torch
        self._open = (torch.cuda.device(self._device),)
        self._open[0].__enter__()
        if self._stream is not None:
            self._open += (torch.cuda.stream(self._stream),)
            self._open[1].__enter__()

    def __exit__(self, *exc):
        for c in reversed(self._open):
            c.__exit__(*exc)


def _bad(message):
    return LLAError(LLA_ERR_INVALID_ARG, message)


def _ints(name, t, shape, dtype, device):
    """t's pointer, if it is a contiguous tensor of this shape, dtype and device."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise _bad(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}, got {t.dtype} "
                   f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _same(name, t, shape, dtype, device):
    _ints(name, t, shape, dtype, device)
    return t


def _check_caches(k_cache, v_cache):
    """(num_pages, Hkv, page_size, d, page stride, lla dtype) of two caches laid out alike."""
    import torch
    dt = k_cache.dtype
    if not k_cache.is_cuda or v_cache.device != k_cache.device:
        raise _bad("the caches must be CUDA tensors of one device (there is no CPU path)")
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or v_cache.dtype is not dt:
        raise _bad(f"caches [num_pages, Hkv, page_size, d] of one dtype expected, got {tuple(k_cache.shape)} "
                   f"{dt}, {tuple(v_cache.shape)} {v_cache.dtype}")
    if dt is torch.bfloat16:
        dtype = LLA_DTYPE_BF16
    elif dt is torch.float32:
        dtype = LLA_DTYPE_FP32
    else:
        raise _bad("the caches must be bf16 or fp32")
    P, Hkv, Z, d = k_cache.shape
    strides, inner = k_cache.stride(), (Z * d, d, 1)
    if strides[1:] != inner or v_cache.stride() != strides:
        for c in (k_cache, v_cache):
            if c.numel() and not c[0].is_contiguous():
                raise _bad("each page of a cache must be contiguous (a cache is written in place, so it is not copied)")
        if P > 1 and v_cache.stride(0) != strides[0]:
            raise _bad("the caches must have one page stride")
    return P, Hkv, Z, d, (strides[0] if P > 1 else Hkv * Z * d), dtype


def _token_rows(t, name, like, heads, d):
    """[T, heads, d] rows as the kernels take them: heads packed, any 16-byte token stride; else a copy."""
    if t.dim() != 3 or t.shape[1:] != (heads, d) or t.dtype is not like.dtype or t.device != like.device:
        raise _bad(f"{name} must be [T, {heads}, {d}] {like.dtype} on {like.device}, got {tuple(t.shape)} {t.dtype} on "
                   f"{t.device}")
    rows, most = t.shape[0], heads * d
    token, head, element = t.stride()
    if element == 1 and (head == d or heads == 1) and t.data_ptr() % 16 == 0:
        if rows <= 1:
            return t, most
        if token >= most and token * t.element_size() % 16 == 0:
            return t, token
    import torch
    t = t.contiguous() if t.data_ptr() % 16 == 0 and not t.is_contiguous() else t.clone(memory_format=torch.contiguous_format)
    return t, most


@functools.lru_cache(maxsize=256)
def _paged_workspace_bytes(device_index, dtype, path, Hq, Hkv, d, page_size, max_new):
    """Scratch of a paged attention call: a function of these sizes alone (0: the call will be refused)."""
    return lla_paged_parallax_workspace_size(dtype, path, 1, 1, Hq, Hkv, d, page_size, 1, max_new)


_BIND = None


def _bind():
    """The marshalling module (csrc/paged_bind.c), tied to the loaded library; False if it was not built."""
    global _BIND
    if _BIND is None:
        import torch
        lib = load_library()
        try:
            from . import _paged_bind as m
        except ImportError:
            _BIND = False
        else:
            m.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in (lib.lla_paged_plan, lib.lla_paged_append,
                                                                      lib.lla_paged_parallax)),
                   torch.bfloat16, torch.float32, torch.int32, torch.int64)
            _BIND = m
    return _BIND


# Scratch of eager attention calls by (device, stream, host thread): a thread's calls on one stream follow one
# another, so they can share it, and taking it from the allocator costs as much as all checks.  A thread keeps at
# most eight, and they go back to the allocator when it ends.
_SCRATCH = {}


class _ThreadKeys(list):
    """Keys of _SCRATCH that are one thread's, the oldest first."""

    def __del__(self, pop=_SCRATCH.pop):
        for key in self:
            pop(key, None)


class _Thread(threading.local):
    def __init__(self):
        self.keys = _ThreadKeys()


_THREAD = _Thread()


def _scratch(device, stream_ptr, nbytes):
    import torch
    # a call under graph capture takes its own (the graph keeps it), so that graphs never share scratch with anything
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    keys, key = _THREAD.keys, (device.index, stream_ptr, threading.get_ident())
    t = _SCRATCH.get(key)
    if t is None or t.numel() < nbytes:
        if _SCRATCH.pop(key, None) is not None:
            keys.remove(key)
        while len(keys) >= 8:
            _SCRATCH.pop(keys.pop(0), None)
        t = torch.empty(nbytes, dtype=torch.uint8, device=device)
        keys.append(key)
        _SCRATCH[key] = t
    return t


def paged_plan(ctx_lens, new_lens, block_table, free_pages, free_count, page_size, num_rows, *, kv_lens=None, cu_q=None,
               slots=None, positions=None, granted=None, free_left=None, stream=None):
    """Pages and slots for a step's new tokens, from the requests' lengths, on the GPU (include/lla.h,
    lla_paged_plan).

    ctx_lens, new_lens [S]; block_table [S, W], updated in place; free_pages [F] with free_count [1], a
    stack of free page ids; num_rows: token rows of the step's tensors.  All int32 CUDA tensors.
    Returns PagedPlan(kv_lens [S], cu_q [S+1], slots [num_rows] int64, positions [num_rows], granted [S],
    free_left [1]).  kv_lens=ctx_lens and free_left=free_count update a decode loop's state in place.
    A sequence is granted all of its tokens or none; what paged_parallax gives for the rows of a refused one
    (granted 0) is no answer for its tokens and has to be dropped.
    Asynchronous on the current (or given) stream.
    """
    import torch
    if not ctx_lens.is_cuda:
        raise _bad("paged_plan takes CUDA tensors (there is no CPU path)")
    dev, T, i32, i64 = ctx_lens.device, int(num_rows), torch.int32, torch.int64
    if stream is not None or dev.index != torch.cuda.current_device():
        with _on_stream(dev, stream):
            return paged_plan(ctx_lens, new_lens, block_table, free_pages, free_count, page_size, T, kv_lens=kv_lens,
                              cu_q=cu_q, slots=slots, positions=positions, granted=granted, free_left=free_left)
    if block_table.dim() != 2 or T < 1:
        raise _bad("block_table must be [S, W] and num_rows >= 1")
    stream_ptr = torch._C._cuda_getCurrentRawStream(dev.index)
    if kv_lens is cu_q is slots is positions is granted is free_left is None and _bind():
        S, empty, like = ctx_lens.shape[0] if ctx_lens.dim() else 0, torch.empty, torch.empty_like
        r = PagedPlan(like(ctx_lens), empty(S + 1, dtype=i32, device=dev), empty(T, dtype=i64, device=dev),
                      empty(T, dtype=i32, device=dev), like(ctx_lens), like(free_count))
        if _BIND.plan(dev.index, ctx_lens, new_lens, block_table, free_pages, free_count, page_size, T, r[0], r[1], r[2],
                      r[3], r[4], r[5], stream_ptr) == LLA_OK:
            return r
    S, W, F = ctx_lens.numel(), block_table.shape[1], free_pages.numel()
    ctx_ptr, new_ptr = _ints("ctx_lens", ctx_lens, (S,), i32, dev), _ints("new_lens", new_lens, (S,), i32, dev)
    table_ptr = _ints("block_table", block_table, (S, W), i32, dev)
    free_ptr, count_ptr = _ints("free_pages", free_pages, (F,), i32, dev), _ints("free_count", free_count, (1,), i32, dev)
    empty, like = torch.empty, torch.empty_like
    kv_lens = like(ctx_lens) if kv_lens is None else _same("kv_lens", kv_lens, (S,), i32, dev)
    granted = like(ctx_lens) if granted is None else _same("granted", granted, (S,), i32, dev)
    free_left = like(free_count) if free_left is None else _same("free_left", free_left, (1,), i32, dev)
    cu_q = empty(S + 1, dtype=i32, device=dev) if cu_q is None else _same("cu_q", cu_q, (S + 1,), i32, dev)
    slots = empty(T, dtype=i64, device=dev) if slots is None else _same("slots", slots, (T,), i64, dev)
    positions = empty(T, dtype=i32, device=dev) if positions is None else _same("positions", positions, (T,), i32, dev)
    status = load_library().lla_paged_plan(
        ctx_ptr, new_ptr, S, int(page_size), table_ptr, W, free_ptr, F, count_ptr, T, kv_lens.data_ptr(), cu_q.data_ptr(),
        slots.data_ptr(), positions.data_ptr(), granted.data_ptr(), free_left.data_ptr(), stream_ptr)
    if status != LLA_OK:
        _check(status)
    return PagedPlan(kv_lens, cu_q, slots, positions, granted, free_left)


def paged_append(k_new, v_new, slots, k_cache, v_cache, *, stream=None):
    """Write k_new, v_new [T, Hkv, d] into the paged caches [num_pages, Hkv, page_size, d] at slots [T]
    (int64, a plan's; rows with a negative slot are skipped).  In place, asynchronous on the current (or
    given) stream.  Rows may be slices of a fused projection (any 16-byte token stride)."""
    import torch
    if stream is None and k_cache.is_cuda and _bind():
        index = torch.cuda.current_device()
        if _BIND.append(index, k_new, v_new, slots, k_cache, v_cache, torch._C._cuda_getCurrentRawStream(index)) == LLA_OK:
            return
    P, Hkv, Z, d, page_stride, dtype = _check_caches(k_cache, v_cache)
    dev = k_cache.device
    if stream is not None or dev.index != torch.cuda.current_device():
        with _on_stream(dev, stream):
            return paged_append(k_new, v_new, slots, k_cache, v_cache)
    if k_new.shape != v_new.shape:
        raise _bad("k_new and v_new must have one shape")
    k_new, ks = _token_rows(k_new, "k_new", k_cache, Hkv, d)
    v_new, vs = _token_rows(v_new, "v_new", k_cache, Hkv, d)
    T = k_new.shape[0]
    status = load_library().lla_paged_append(
        dtype, k_new.data_ptr(), v_new.data_ptr(), _ints("slots", slots, (T,), torch.int64, dev), k_cache.data_ptr(),
        v_cache.data_ptr(), T, Hkv, d, Z, P, ks, vs, page_stride, torch._C._cuda_getCurrentRawStream(dev.index))
    if status != LLA_OK:
        _check(status)


def paged_parallax(q, probe, k_cache, v_cache, block_table, cu_q, kv_lens, tau, max_new, *, causal=True,
                   path=LLA_PATH_AUTO, out=None, workspace=None, stream=None):
    """Parallax-form attention of a step's token rows q, probe [T, Hq, d] over paged caches
    [num_pages, Hkv, page_size, d] (include/lla.h, lla_paged_parallax).

    block_table [S, W], cu_q [S+1], kv_lens [S]: int32 CUDA tensors (paged_plan's); max_new: the most
    tokens of one sequence in this step (it chooses the kernel for the whole batch: pass what the step needs, not what
    it could need).  causal=False: every row sees all of its sequence's keys.  path: LLA_PATH_AUTO takes bf16 with d 64
    or 128 to the tensor cores, where the weights are rounded to bf16 from 17 rows to a key head on; LLA_PATH_FP32 keeps
    them in fp32.
    Returns out [T, Hq, d]; rows behind the last sequence are left as they were.  Asynchronous on the
    current (or given) stream.  workspace: None (scratch kept per stream while the thread lives; under graph capture the
    graph's own), or a CUDA tensor of lla_paged_parallax_workspace_size(...) bytes that no other call uses at the
    same time.
    """
    import torch
    if stream is None and workspace is None and k_cache.is_cuda and _bind():
        index = torch.cuda.current_device()
        stream_ptr = torch._C._cuda_getCurrentRawStream(index)
        t = _SCRATCH.get((index, stream_ptr, threading.get_ident()))
        if t is not None and not torch.cuda.is_current_stream_capturing():
            res = torch.empty(q.shape, dtype=q.dtype, device=q.device) if out is None else out
            if _BIND.parallax(index, q, probe, k_cache, v_cache, block_table, cu_q, kv_lens, res, tau, max_new, causal, path,
                              t.data_ptr(), t.numel(), stream_ptr) == LLA_OK:
                return res
    P, Hkv, Z, d, page_stride, dtype = _check_caches(k_cache, v_cache)
    dev = k_cache.device
    if stream is not None or dev.index != torch.cuda.current_device():
        with _on_stream(dev, stream):
            return paged_parallax(q, probe, k_cache, v_cache, block_table, cu_q, kv_lens, tau, max_new, causal=causal,
                                  path=path, out=out, workspace=workspace)
    if q.dim() != 3:
        raise _bad(f"q must be [T, Hq, d], got {tuple(q.shape)}")
    if probe.shape != q.shape:
        raise _bad(f"probe must have q's shape {tuple(q.shape)}, got {tuple(probe.shape)}")
    if block_table.dim() != 2:
        raise _bad("block_table must be [S, W]")
    T, Hq, _ = q.shape
    S, W = block_table.shape
    i32, path, max_new = torch.int32, int(path), int(max_new)
    table_ptr = _ints("block_table", block_table, (S, W), i32, dev)
    cu_ptr, kv_ptr = _ints("cu_q", cu_q, (S + 1,), i32, dev), _ints("kv_lens", kv_lens, (S,), i32, dev)
    q, qs = _token_rows(q, "q", k_cache, Hq, d)
    probe, rs = _token_rows(probe, "probe", k_cache, Hq, d)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=q.dtype, device=dev)
    elif out.shape != q.shape or out.dtype is not q.dtype or out.device != dev or not out.is_contiguous():
        raise _bad(f"out must be a contiguous {q.dtype} tensor of shape {tuple(q.shape)} on {dev}")
    stream_ptr = torch._C._cuda_getCurrentRawStream(dev.index)
    if workspace is None:
        workspace = _scratch(dev, stream_ptr, _paged_workspace_bytes(dev.index, dtype, path, Hq, Hkv, d, Z, max_new))
        ws_bytes = workspace.numel()
    elif workspace.device != dev or not workspace.is_contiguous():
        raise _bad(f"workspace must be a contiguous tensor on {dev}")
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    status = load_library().lla_paged_parallax(
        dtype, path, q.data_ptr(), probe.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), table_ptr, cu_ptr, kv_ptr,
        out.data_ptr(), T, S, Hq, Hkv, d, Z, P, W, max_new, qs, rs, page_stride, float(tau), 1 if causal else 0,
        workspace.data_ptr(), ws_bytes, stream_ptr)
    if status != LLA_OK:
        _check(status)
    return out
