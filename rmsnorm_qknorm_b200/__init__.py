"""B200-native layerwise QK-Norm and FlashNorm: Python binding of libqknorm.so.

This module only marshals arguments: it checks tensor placement, reads
pointers, pitches and the current CUDA stream from torch, and calls the C ABI
declared in ``include/qknorm.h``.  Every step of the computation runs in the
library's sm_100a kernels; there is no CPU or PyTorch fallback, and a missing
library raises instead of degrading.

Entry points (same names as the C ABI):

* :func:`qknorm_fused` -- RMSNorm of every query row and key row (one launch for
  both wherever their kernels agree),
  statistics built from ``n_seg`` per-segment scalar partial sums combined in a
  fixed order (SwiftQK's tensor-parallel statistic, emulated on one GPU).
* :func:`rmsnorm_partial_stats` -- those per-segment partial sums on their own.
* :func:`flashnorm_fold_weights` -- FlashNorm's W' = diag(w) W.
* :func:`flashnorm_proj` -- y = (x W') * 1/rms(x), the deferred-normalisation
  GEMM with the scaling in the epilogue.
* :func:`rmsnorm_apply_partials` -- the apply step of tensor-parallel QK-Norm:
  normalise a shard from the gathered per-shard partial sums.
* :func:`rotary_apply` -- rotary positions on query and key rows (and back).
* :func:`qknorm_rotary`, :func:`qknorm_rotary_backward` -- QK-Norm and rotary
  positions in one pass, and the gradients of both.
* :func:`linear_fused`, :func:`linear_fused_backward` -- a linear layer with
  bias, activation and residual in its epilogue, and its gradients.
* :func:`qkv_norm_proj` -- QKV projection + QKV-normalisation with the
  pre-attention RMSNorm eliminated (FlashNorm's scale-invariance identity).
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from .rotary import rotary_inv_freq

__all__ = [
    "QKNormError",
    "load_library",
    "library_path",
    "qknorm_fused",
    "qknorm_fused_host",
    "qkv_proj_qknorm",
    "qkv_proj_qknorm_workspace_bytes",
    "rmsnorm_partial_stats",
    "flashnorm_fold_weights",
    "flashnorm_proj",
    "flashnorm_inv_rms",
    "rmsnorm_apply_partials",
    "qkv_norm_proj",
    "rotary_inv_freq",
    "rotary_apply",
    "qknorm_rotary",
    "qknorm_rotary_backward",
    "qknorm_rotary_backward_workspace_bytes",
    "linear_fused",
    "linear_fused_backward",
    "linear_fused_backward_workspace_bytes",
    "STATUS_NAMES",
    "QKN_MAX_SEG",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libqknorm.so")
_lock = threading.Lock()
_lib = None

QKN_MAX_SEG = 64
QKN_F32, QKN_BF16 = 0, 1
STATUS_NAMES = {
    0: "QKN_OK", 1: "QKN_ERR_NULL", 2: "QKN_ERR_SHAPE", 3: "QKN_ERR_DTYPE", 4: "QKN_ERR_EPS",
    5: "QKN_ERR_ALIGN", 6: "QKN_ERR_CUDA", 7: "QKN_ERR_TIMEOUT", 8: "QKN_ERR_UNSUPPORTED",
}


class QKNormError(RuntimeError):
    """A nonzero qkn_status from the library, with its message."""

    def __init__(self, fn: str, status: int, message: str):
        self.status = status
        self.status_name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{fn}: {self.status_name}: {message}")


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load libqknorm.so (built by ``python -m rmsnorm_qknorm_b200.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise ImportError(
                f"{_LIB_PATH} is missing: build it with `python -m rmsnorm_qknorm_b200.build` "
                "(there is no fallback implementation)")
        lib = ctypes.CDLL(_LIB_PATH)
        p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        lib.qknorm_fused.argtypes = [p, p, p, p, p, p, i64, i64, i64, i64, i64, i64, i64,
                                     i32, i32, f32, i32, p]
        lib.rmsnorm_partial_stats.argtypes = [p, i64, i64, i64, i32, i32, p, p]
        lib.flashnorm_fold_weights.argtypes = [p, p, p, i64, i64, i32, i32, p]
        lib.flashnorm_proj.argtypes = [p, p, p, i64, i64, i64, i32, f32, p, p, p]
        lib.rmsnorm_apply_partials.argtypes = [p, p, p, i64, i64, i64, i64, p, i32, i64, i64, i64,
                                               i32, i32, f32, p]
        lib.qkv_norm_proj.argtypes = [p, p, p, i64, i64, i64, i64, i64, p, p, p, i32, f32, i32, p]
        lib.qknorm_fused_host.argtypes = [p, p, p, p, p, p, i64, i64, i64, i32, i32, f32, i32,
                                          p, ctypes.c_size_t, p]
        lib.qkv_proj_qknorm.argtypes = [p, p, p, i64, i64, i64, i64, i64, p, p, i32, f32, f32, p, p,
                                        p, ctypes.c_size_t, p]
        lib.qkv_proj_qknorm_workspace_bytes.argtypes = [i64, i64, i64, i64]
        lib.qkv_proj_qknorm_workspace_bytes.restype = ctypes.c_size_t
        lib.flashnorm_inv_rms.argtypes = [p, p, i64, i64, f32, p]
        lib.rotary_apply.argtypes = [p, p, p, p] + [i64] * 8 + [p, i32, p, i64, i32, f32, i32, i32, p]
        lib.qknorm_rotary.argtypes = [p] * 6 + [i64] * 8 + [p, i32, p, i64, i32, f32, i32, i32, f32, p]
        lib.qknorm_rotary_backward.argtypes = ([p] * 10 + [i64] * 10 + [p, i32, p, i64, i32, f32, i32, i32, f32,
                                                                      p, ctypes.c_size_t, p])
        lib.qknorm_rotary_backward_workspace_bytes.argtypes = [i64, i64, i64]
        lib.qknorm_rotary_backward_workspace_bytes.restype = ctypes.c_size_t
        lib.linear_fused.argtypes = [p, p, p] + [i64] * 6 + [p, i32, i32, p, i64, p, p, i64, p]
        lib.linear_fused_backward.argtypes = [p] * 7 + [i64] * 9 + [i32, p, ctypes.c_size_t, p]
        lib.linear_fused_backward_workspace_bytes.argtypes = [i64, i64, i64, i32]
        lib.linear_fused_backward_workspace_bytes.restype = ctypes.c_size_t
        lib.qkn_check_device.argtypes = [p]
        for f in ("qknorm_fused", "qknorm_fused_host", "qkv_proj_qknorm", "rmsnorm_partial_stats", "flashnorm_fold_weights",
                  "flashnorm_proj", "flashnorm_inv_rms", "rmsnorm_apply_partials", "qkv_norm_proj", "rotary_apply", "qknorm_rotary",
                  "qknorm_rotary_backward", "linear_fused", "linear_fused_backward", "qkn_check_device"):
            getattr(lib, f).restype = ctypes.c_int
        lib.qkn_last_error.restype = ctypes.c_char_p
        lib.qkn_last_error.argtypes = []
        lib.qkn_version.restype = ctypes.c_char_p
        lib.qkn_version.argtypes = []
        _lib = lib
        return lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        msg = load_library().qkn_last_error().decode(errors="replace")
        raise QKNormError(fn, status, msg)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return QKN_F32
    if t == torch.bfloat16:
        return QKN_BF16
    raise TypeError(f"unsupported dtype {t}; expected torch.float32 or torch.bfloat16")


def _cuda(t: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    return t


def _rows(t: torch.Tensor, name: str):
    _cuda(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D with unit stride along the row")
    rows, cols = t.shape
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        raise ValueError(f"{name} must be 2-D with unit stride along the row")
    return rows, cols, max(s0, cols)


def _vec(t: torch.Tensor, name: str, n: int):
    _cuda(t, name)
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous 1-D tensor of length {n}")


def _out2d(t: torch.Tensor, name: str, rows: int, cols: int, dtype: torch.dtype) -> torch.Tensor:
    """A caller-provided output: the exact shape and dtype, unit stride along the row."""
    _cuda(t, name)
    if t.dim() != 2 or tuple(t.shape) != (rows, cols) or t.dtype != dtype or (cols > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a {dtype} [{rows}, {cols}] tensor with unit stride along the row")
    return t


def _device(ref: torch.Tensor, **tensors) -> torch.device:
    """Every CUDA tensor of a call lives on ref's device; the call is made there."""
    dev = ref.device
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device} but the call's inputs are on {dev}")
    return dev


class _On:
    """Makes the data's device current for the library call, only when it is not."""

    __slots__ = ("index", "prev")

    def __init__(self, dev: torch.device):
        self.index = dev.index

    def __enter__(self):
        self.prev = torch.cuda.current_device()
        if self.prev != self.index:
            torch.cuda.set_device(self.index)
        return self

    def __exit__(self, *exc):
        if self.prev != self.index:
            torch.cuda.set_device(self.prev)
        return False


# The current stream's raw handle without building a Stream object (the
# public route costs a few microseconds per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    """Handle of `stream`, or of the current device's current stream."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def qknorm_fused(q: torch.Tensor, k: torch.Tensor | None, wq: torch.Tensor,
                 wk: torch.Tensor | None, eps: float = 1e-6, n_seg: int = 1, *,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                 inplace: bool = False, stream=None):
    """QK-Norm of q [T, dq] and k [T, dk] (k may be None), one launch for both where
    their kernels agree (a row's result never depends on the other tensor).

    Returns ``(q_out, k_out)``.  With ``inplace=True`` the inputs are
    overwritten and returned; otherwise outputs are allocated unless given.
    Row pitches are taken from the tensors' strides (views of a fused QKV
    buffer work without copies).
    """
    T, dq, ldq = _rows(q, "q")
    act = _dtype_code(q.dtype)
    _vec(wq, "wq", dq)
    wdt = _dtype_code(wq.dtype)
    if k is not None:
        Tk, dk, ldk = _rows(k, "k")
        if Tk != T or k.dtype != q.dtype:
            raise ValueError("k must have q's row count and dtype")
        if wk is None:
            raise ValueError("wk is required with k")
        _vec(wk, "wk", dk)
        if wk.dtype != wq.dtype:
            raise ValueError("wk must have wq's dtype")
    else:
        dk, ldk = 0, 0
    if inplace:
        q_out_t, k_out_t = q, k
        q_ptr_out = k_ptr_out = None
        ldq_o, ldk_o = ldq, ldk
    else:
        q_out_t = q_out if q_out is not None else torch.empty((T, dq), dtype=q.dtype, device=q.device)
        _, _, ldq_o = _rows(_out2d(q_out_t, "q_out", T, dq, q.dtype), "q_out")
        q_ptr_out = q_out_t.data_ptr()
        if k is not None:
            k_out_t = k_out if k_out is not None else torch.empty((T, dk), dtype=k.dtype, device=k.device)
            _, _, ldk_o = _rows(_out2d(k_out_t, "k_out", T, dk, k.dtype), "k_out")
            k_ptr_out = k_out_t.data_ptr()
        else:
            k_out_t, k_ptr_out, ldk_o = None, None, 0
    dev = _device(q, k=k, wq=wq, wk=wk if k is not None else None, q_out=q_out_t, k_out=k_out_t)
    lib = load_library()
    with _On(dev):
        st = lib.qknorm_fused(q.data_ptr(), k.data_ptr() if k is not None else None,
                              wq.data_ptr(), wk.data_ptr() if k is not None else None,
                              q_ptr_out, k_ptr_out, T, dq, dk, ldq, ldk, ldq_o, ldk_o,
                              act, wdt, float(eps), int(n_seg), _stream(stream))
    _check("qknorm_fused", st)
    return q_out_t, k_out_t


HOST_WORKSPACE_BYTES = 3 * 64 * 1024 * 1024  # room for chunks up to 64 MiB


def qknorm_fused_host(q: torch.Tensor, k: torch.Tensor | None, wq: torch.Tensor,
                      wk: torch.Tensor | None, eps: float = 1e-6, n_seg: int = 1, *,
                      q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """QK-Norm of q [T, dq] and k [T, dk] held in HOST memory; results in host tensors.

    The rows stream through a device ``workspace`` (uint8 CUDA tensor,
    ``HOST_WORKSPACE_BYTES`` allocated when not given) in chunks whose upload,
    kernel and download overlap.  wq / wk live on the device.  Pinned host
    tensors let the copies run at link speed.  The call is asynchronous on
    ``stream``: synchronise it before reading the outputs.  Returns
    ``(q_out, k_out)``; ``q_out=q`` works in place.
    """
    def host_rows(t, name):
        if not isinstance(t, torch.Tensor) or t.is_cuda:
            raise ValueError(f"{name} must be a host (CPU) tensor")
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 2-D tensor")
        return t.shape
    T, dq = host_rows(q, "q")
    act = _dtype_code(q.dtype)
    _vec(wq, "wq", dq)
    wdt = _dtype_code(wq.dtype)
    if k is not None:
        Tk, dk = host_rows(k, "k")
        if Tk != T or k.dtype != q.dtype:
            raise ValueError("k must have q's row count and dtype")
        if wk is None:
            raise ValueError("wk is required with k")
        _vec(wk, "wk", dk)
        if wk.dtype != wq.dtype:
            raise ValueError("wk must have wq's dtype")
    else:
        dk = 0
    pin = q.is_pinned()
    if q_out is None:
        q_out = torch.empty((T, dq), dtype=q.dtype, pin_memory=pin)
    if host_rows(q_out, "q_out") != (T, dq) or q_out.dtype != q.dtype:
        raise ValueError("q_out must match q")
    if k is not None:
        if k_out is None:
            k_out = torch.empty((T, dk), dtype=k.dtype, pin_memory=pin)
        if host_rows(k_out, "k_out") != (T, dk) or k_out.dtype != k.dtype:
            raise ValueError("k_out must match k")
    if workspace is None:
        workspace = torch.empty(HOST_WORKSPACE_BYTES, dtype=torch.uint8, device=wq.device)
    _cuda(workspace, "workspace")
    dev = _device(wq, wk=wk if k is not None else None, workspace=workspace)
    lib = load_library()
    with _On(dev):
        st = lib.qknorm_fused_host(q.data_ptr(), k.data_ptr() if k is not None else None,
                                   wq.data_ptr(), wk.data_ptr() if k is not None else None,
                                   q_out.data_ptr(), k_out.data_ptr() if k is not None else None,
                                   T, dq, dk, act, wdt, float(eps), int(n_seg),
                                   workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   _stream(stream))
    _check("qknorm_fused_host", st)
    return q_out, (k_out if k is not None else None)


def rmsnorm_partial_stats(x: torch.Tensor, n_seg: int, *, out: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """Per-row sums of squares of n_seg contiguous segments: fp32 [rows, n_seg]."""
    rows, d, ld = _rows(x, "x")
    act = _dtype_code(x.dtype)
    if out is None:
        out = torch.empty((rows, n_seg), dtype=torch.float32, device=x.device)
    elif out.dtype != torch.float32 or not out.is_contiguous() or tuple(out.shape) != (rows, n_seg):
        raise ValueError("out must be a contiguous fp32 tensor of shape [rows, n_seg]")
    dev = _device(x, out=_cuda(out, "out"))
    with _On(dev):
        st = load_library().rmsnorm_partial_stats(x.data_ptr(), rows, d, ld, act, int(n_seg),
                                                  out.data_ptr(), _stream(stream))
    _check("rmsnorm_partial_stats", st)
    return out


def flashnorm_fold_weights(w: torch.Tensor, W: torch.Tensor, *, k_major: bool = True,
                           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """FlashNorm fold W' = diag(w) W of W [K, N] (bf16); [N, K] when k_major else [K, N]."""
    _cuda(W, "W")
    if W.dim() != 2 or not W.is_contiguous() or W.dtype != torch.bfloat16:
        raise ValueError("W must be a contiguous bf16 [K, N] tensor")
    K, N = W.shape
    _vec(w, "w", K)
    shape = (N, K) if k_major else (K, N)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=W.device)
    elif tuple(out.shape) != shape or not out.is_contiguous() or out.dtype != torch.bfloat16:
        raise ValueError(f"out must be a contiguous bf16 tensor of shape {shape}")
    dev = _device(W, w=w, out=_cuda(out, "out"))
    with _On(dev):
        st = load_library().flashnorm_fold_weights(w.data_ptr(), W.data_ptr(), out.data_ptr(),
                                                   K, N, _dtype_code(w.dtype), int(bool(k_major)),
                                                   _stream(stream))
    _check("flashnorm_fold_weights", st)
    return out


def flashnorm_proj(x: torch.Tensor, W_folded: torch.Tensor, eps: float = 1e-6, *,
                   inv_rms: torch.Tensor | None = None, inv_rms_out: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, k_major: bool = True, in_kernel_stats: bool = False,
                   stream=None) -> torch.Tensor:
    """y [M, N] = (x [M, K] @ W') * 1/rms(x), bf16 in/out, fp32 accumulate.

    W_folded is [N, K] (``k_major=True``, the layout the tensor cores read) or
    [K, N] (``k_major=False``: copied K-major inside the call first).  Without
    ``inv_rms`` the row statistics run as a separate pass overlapped with the
    projection, into ``inv_rms_out`` (allocated here when not given);
    ``in_kernel_stats=True`` computes them inside the projection kernel
    instead (no [M] workspace, slower).
    """
    _cuda(x, "x")
    _cuda(W_folded, "W_folded")
    if x.dim() != 2 or not x.is_contiguous() or x.dtype != torch.bfloat16:
        raise ValueError("x must be a contiguous bf16 [M, K] tensor")
    if W_folded.dim() != 2 or not W_folded.is_contiguous() or W_folded.dtype != torch.bfloat16:
        raise ValueError("W_folded must be a contiguous bf16 2-D tensor")
    M, K = x.shape
    N, K2 = W_folded.shape if k_major else (W_folded.shape[1], W_folded.shape[0])
    if K2 != K:
        raise ValueError(f"W_folded has K={K2} but x has K={K}")
    for name, t in (("inv_rms", inv_rms), ("inv_rms_out", inv_rms_out)):
        if t is not None:
            _vec(t, name, M)
            if t.dtype != torch.float32:
                raise ValueError(f"{name} must be fp32")
    if inv_rms is None and inv_rms_out is None and not in_kernel_stats:
        inv_rms_out = torch.empty(M, dtype=torch.float32, device=x.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    elif tuple(out.shape) != (M, N) or not out.is_contiguous() or out.dtype != torch.bfloat16:
        raise ValueError("out must be a contiguous bf16 [M, N] tensor")
    dev = _device(x, W_folded=W_folded, inv_rms=inv_rms, inv_rms_out=inv_rms_out, out=_cuda(out, "out"))
    with _On(dev):
        st = load_library().flashnorm_proj(
            x.data_ptr(), W_folded.data_ptr(), out.data_ptr(), M, N, K, 1 if k_major else 0, float(eps),
            inv_rms.data_ptr() if inv_rms is not None else None,
            inv_rms_out.data_ptr() if inv_rms_out is not None else None, _stream(stream))
    _check("flashnorm_proj", st)
    return out


def flashnorm_inv_rms(x: torch.Tensor, eps: float = 1e-6, *, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """FlashNorm's row statistic: fp32 [M] 1/rms of the rows of bf16 x [M, K]."""
    _cuda(x, "x")
    if x.dim() != 2 or not x.is_contiguous() or x.dtype != torch.bfloat16:
        raise ValueError("x must be a contiguous bf16 [M, K] tensor")
    M, K = x.shape
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=x.device)
    else:
        _vec(out, "out", M)
        if out.dtype != torch.float32:
            raise ValueError("out must be fp32")
    dev = _device(x, out=out)
    with _On(dev):
        st = load_library().flashnorm_inv_rms(x.data_ptr(), out.data_ptr(), M, K, float(eps), _stream(stream))
    _check("flashnorm_inv_rms", st)
    return out


def rmsnorm_apply_partials(x: torch.Tensor, w: torch.Tensor, partial: torch.Tensor, d_full: int,
                           eps: float = 1e-6, *, out: torch.Tensor | None = None,
                           inplace: bool = False, stream=None) -> torch.Tensor:
    """Normalise the shard x [rows, d] given every row's partial sums of squares.

    ``partial`` is fp32 and 2-D: [rows, n_part] (e.g. rmsnorm_partial_stats
    output) or [n_part, rows] (e.g. an all-gather of per-shard partials); the
    layout is read from its strides and its first dimension's length.
    ``d_full`` is the width of the whole row the partials cover.
    """
    rows, d, ld = _rows(x, "x")
    act = _dtype_code(x.dtype)
    _vec(w, "w", d)
    _cuda(partial, "partial")
    if partial.dtype != torch.float32 or partial.dim() != 2:
        raise ValueError("partial must be a 2-D fp32 tensor")
    if partial.shape[0] == rows:
        n_part, prs, ps = partial.shape[1], partial.stride(0), partial.stride(1)
    elif partial.shape[1] == rows:
        n_part, prs, ps = partial.shape[0], partial.stride(1), partial.stride(0)
    else:
        raise ValueError(f"partial {tuple(partial.shape)} does not match {rows} rows")
    if inplace:
        y, ldo = x, ld
    else:
        y = out if out is not None else torch.empty((rows, d), dtype=x.dtype, device=x.device)
        _, _, ldo = _rows(_out2d(y, "out", rows, d, x.dtype), "out")
    dev = _device(x, w=w, partial=partial, out=y)
    with _On(dev):
        st = load_library().rmsnorm_apply_partials(
            x.data_ptr(), w.data_ptr(), y.data_ptr(), rows, d, ld, ldo, partial.data_ptr(), int(n_part),
            int(prs), int(ps), int(d_full), act, _dtype_code(w.dtype), float(eps), _stream(stream))
    _check("rmsnorm_apply_partials", st)
    return y


def qkv_norm_proj(x: torch.Tensor, W_folded: torch.Tensor, nq: int, nk: int, nv: int,
                  wq: torch.Tensor, wk: torch.Tensor, wv: torch.Tensor | None, eps: float = 1e-6,
                  n_seg: int = 1, *, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """[q | k | v] = per-group RMSNorm of x W_folded^T; the pre-attention RMSNorm eliminated."""
    _cuda(x, "x")
    _cuda(W_folded, "W_folded")
    if x.dim() != 2 or not x.is_contiguous() or x.dtype != torch.bfloat16:
        raise ValueError("x must be a contiguous bf16 [M, K] tensor")
    M, K = x.shape
    N = nq + nk + nv
    if tuple(W_folded.shape) != (N, K) or not W_folded.is_contiguous() or W_folded.dtype != torch.bfloat16:
        raise ValueError(f"W_folded must be a contiguous bf16 [{N}, {K}] tensor")
    _vec(wq, "wq", nq)
    _vec(wk, "wk", nk)
    if nv > 0:
        _vec(wv, "wv", nv)
    for name, t in (("wk", wk), ("wv", wv if nv > 0 else None)):
        if t is not None and t.dtype != wq.dtype:
            raise ValueError(f"{name} must have wq's dtype")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    elif not out.is_contiguous():
        raise ValueError("out must be contiguous")
    _out2d(out, "out", M, N, torch.bfloat16)
    dev = _device(x, W_folded=W_folded, wq=wq, wk=wk, wv=wv if nv > 0 else None, out=out)
    with _On(dev):
        st = load_library().qkv_norm_proj(
            x.data_ptr(), W_folded.data_ptr(), out.data_ptr(), M, K, nq, nk, nv, wq.data_ptr(),
            wk.data_ptr(), wv.data_ptr() if (wv is not None and nv > 0) else None, _dtype_code(wq.dtype),
            float(eps), int(n_seg), _stream(stream))
    _check("qkv_norm_proj", st)
    return out


def qkv_proj_qknorm_workspace_bytes(M: int, nq: int, nk: int, nv: int) -> int:
    """Device scratch qkv_proj_qknorm needs for these sizes (bytes)."""
    return int(load_library().qkv_proj_qknorm_workspace_bytes(M, nq, nk, nv))


def qkv_proj_qknorm(x: torch.Tensor, W_folded: torch.Tensor, nq: int, nk: int, nv: int,
                    wq: torch.Tensor, wk: torch.Tensor, eps: float = 1e-6, eps_qk: float | None = None, *,
                    input_norm: bool = True, inv_rms: torch.Tensor | None = None,
                    inv_rms_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """[q | k | v] = QK-Norm of RMSNorm(x) W in one GEMM (q, k normalised in the epilogue).

    The input norm's weights are folded into ``W_folded`` ([nq+nk+nv, K],
    from ``flashnorm_fold_weights``).  Its 1/rms comes from ``inv_rms`` when
    given, else a statistics pass writes it to ``inv_rms_out`` (allocated when
    ``input_norm`` and not given); ``input_norm=False`` uses x unscaled.
    ``eps_qk`` defaults to ``eps``.  ``workspace`` (uint8 CUDA tensor of at
    least ``qkv_proj_qknorm_workspace_bytes``) avoids an allocation inside
    the call.
    """
    _cuda(x, "x")
    _cuda(W_folded, "W_folded")
    if x.dim() != 2 or not x.is_contiguous() or x.dtype != torch.bfloat16:
        raise ValueError("x must be a contiguous bf16 [M, K] tensor")
    M, K = x.shape
    N = nq + nk + nv
    if tuple(W_folded.shape) != (N, K) or not W_folded.is_contiguous() or W_folded.dtype != torch.bfloat16:
        raise ValueError(f"W_folded must be a contiguous bf16 [{N}, {K}] tensor")
    _vec(wq, "wq", nq)
    _vec(wk, "wk", nk)
    if wk.dtype != wq.dtype:
        raise ValueError("wk must have wq's dtype")
    if inv_rms is not None:
        _vec(inv_rms, "inv_rms", M)
        if inv_rms.dtype != torch.float32:
            raise ValueError("inv_rms must be fp32")
    elif input_norm and inv_rms_out is None:
        inv_rms_out = torch.empty(M, dtype=torch.float32, device=x.device)
    if inv_rms_out is not None:
        _vec(inv_rms_out, "inv_rms_out", M)
        if inv_rms_out.dtype != torch.float32:
            raise ValueError("inv_rms_out must be fp32")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    elif not out.is_contiguous():
        raise ValueError("out must be contiguous")
    _out2d(out, "out", M, N, torch.bfloat16)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _cuda(workspace, "workspace")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    dev = _device(x, W_folded=W_folded, wq=wq, wk=wk, inv_rms=inv_rms, inv_rms_out=inv_rms_out,
                  workspace=workspace, out=out)
    with _On(dev):
        st = load_library().qkv_proj_qknorm(
            x.data_ptr(), W_folded.data_ptr(), out.data_ptr(), M, K, nq, nk, nv,
            wq.data_ptr(), wk.data_ptr(), _dtype_code(wq.dtype), float(eps),
            float(eps if eps_qk is None else eps_qk),
            inv_rms.data_ptr() if inv_rms is not None else None,
            inv_rms_out.data_ptr() if (inv_rms is None and inv_rms_out is not None) else None,
            ws_ptr, ws_bytes, _stream(stream))
    _check("qkv_proj_qknorm", st)
    return out


class _AllocOn:
    """Allocations made for a call on `stream` come from that stream's memory pool.

    A tensor from the current stream's pool may still be in use by work queued
    there, which `stream` does not wait for.
    """

    __slots__ = ("ctx",)

    def __init__(self, stream, dev: torch.device):
        self.ctx = None
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                handle = int(stream)
                stream = torch.cuda.ExternalStream(handle, dev) if handle else torch.cuda.default_stream(dev)
            self.ctx = torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        return False


def _pitched(t: torch.Tensor, name: str):
    """(rows, width, pitch) of a 2-D CUDA tensor whose rows lie apart in memory."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _cuda(t, name)
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be 2-D with unit stride along the row")
    rows, cols = shape
    if rows <= 1:
        return rows, cols, cols
    if stride[0] < cols:
        raise ValueError(f"{name} has rows that overlap in memory (an expanded tensor?)")
    return rows, cols, stride[0]


def _not_over(out: torch.Tensor, name: str, inputs: tuple) -> None:
    """A result that the caller gives does not start where an input does."""
    p = out.data_ptr()
    for t in inputs:
        if t is not None and t.data_ptr() == p and out.numel() and t.numel():
            raise ValueError(f"{name} must not overlap the inputs")


_LAYOUTS = {"half": 0, "interleaved": 1}
_POS_BITS = {torch.int64: 64, torch.int32: 32}
_NO_ROTARY = (0, None, 64, None, 0, 0)


def _rotary_args(positions, inv_freq, head_dim: int, layout: str, T: int):
    """(head_dim, positions pointer, pos_bits, inv_freq pointer, rotary_dim, layout code) of a call."""
    lay = _LAYOUTS.get(layout)
    if lay is None:
        raise ValueError(f"layout must be 'half' or 'interleaved', not {layout!r}")
    _cuda(inv_freq, "inv_freq")
    if inv_freq.dim() != 1 or inv_freq.dtype is not torch.float64 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous 1-D float64 tensor")
    if positions is None:
        raise ValueError("positions is required with inv_freq")
    _vec(positions, "positions", T)
    bits = _POS_BITS.get(positions.dtype)
    if bits is None:
        raise TypeError("positions must be int32 or int64")
    return int(head_dim), positions.data_ptr(), bits, inv_freq.data_ptr(), 2 * inv_freq.shape[0], lay


def _rows_like(t: torch.Tensor, name: str, q: torch.Tensor, T: int):
    rows, d, ld = _pitched(t, name)
    if rows != T or t.dtype != q.dtype:
        raise ValueError(f"{name} must have q's row count and dtype")
    return d, ld


def _pair_weights(wq, wk, dq: int, dk: int, has_k: bool) -> int:
    _vec(wq, "wq", dq)
    if has_k:
        if wk is None:
            raise ValueError("wk is required with k")
        _vec(wk, "wk", dk)
        if wk.dtype != wq.dtype:
            raise ValueError("wk must have wq's dtype")
    return _dtype_code(wq.dtype)


_empty_like, _CONTIGUOUS = torch.empty_like, torch.contiguous_format


def _result(t: torch.Tensor, given: torch.Tensor | None, name: str, stream):
    """The output that takes the rows of t, its pointer and pitch: the one given, or a new contiguous one."""
    if given is None:
        if stream is None:
            given = _empty_like(t, memory_format=_CONTIGUOUS)
        else:
            with _AllocOn(stream, t.device):
                given = _empty_like(t, memory_format=_CONTIGUOUS)
        return given, given.data_ptr(), t.shape[1]
    rows, d, ld = _pitched(given, name)
    if (rows, d) != tuple(t.shape) or given.dtype != t.dtype:
        raise ValueError(f"{name} must be a {t.dtype} [{t.shape[0]}, {t.shape[1]}] tensor")
    return given, given.data_ptr(), ld


def _row_outputs(q, k, q_out, k_out, inplace: bool, stream):
    """Output tensors of a call on q and k, their pointers (None in place) and pitches."""
    if inplace:
        if q_out is not None or k_out is not None:
            raise ValueError("inplace=True takes no q_out or k_out")
        return q, None, 0, k, None, 0
    return *_result(q, q_out, "q_out", stream), *(_result(k, k_out, "k_out", stream) if k is not None else (None, None, 0))


_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_entry = {}  # C entry points by name, once the library is loaded


def _call(name: str, dev: torch.device, args: tuple, stream, given: tuple) -> None:
    """lib.name(*args, stream) with the data's device current.

    ``given`` are the (name, tensor or None) pairs of the call, which all have
    to live on ``dev``.
    """
    index = dev.index
    for _, t in given:
        if t is not None and t.get_device() != index:
            _device_mismatch(dev, given)
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(load_library(), name)
    if _get_device() == index:
        st = fn(*args, _raw_stream(index) if stream is None and _raw_stream is not None else _stream(stream))
    else:
        with _On(dev):
            st = fn(*args, _stream(stream))
    if st != 0:
        _check(name, st)


def _device_mismatch(dev: torch.device, given: tuple) -> None:
    for name, t in given:
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device} but the call's inputs are on {dev}")


def rotary_apply(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
                 head_dim: int, *, layout: str = "half", mscale: float = 1.0, inverse: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, inplace: bool = False,
                 stream=None):
    """Rotary positions on q [T, dq] and k [T, dk] (k may be None), one launch for both.

    Each head of ``head_dim`` elements has its first ``2 * len(inv_freq)``
    turned by ``positions[t] * inv_freq`` (``positions`` int32 or int64 [T],
    ``inv_freq`` float64, see :func:`rotary_inv_freq`), the rest copied.
    ``layout`` pairs element i with i + r/2 ("half") or 2i with 2i + 1
    ("interleaved").  ``inverse=True`` turns back, which is the call's own
    gradient.  Returns ``(q_out, k_out)``; pitches, outputs and ``inplace`` as
    in :func:`qknorm_fused`.
    """
    T, dq, ldq = _pitched(q, "q")
    dk, ldk = _rows_like(k, "k", q, T) if k is not None else (0, 0)
    act = _dtype_code(q.dtype)
    rot = _rotary_args(positions, inv_freq, head_dim, layout, T)
    q_out, qp, ldq_o, k_out, kp, ldk_o = _row_outputs(q, k, q_out, k_out, inplace, stream)
    _call("rotary_apply", q.device,
          (q.data_ptr(), k.data_ptr() if k is not None else None, qp, kp, T, dq, dk, ldq, ldk, ldq_o, ldk_o, *rot, mscale,
           1 if inverse else 0, act), stream,
          (("k", k), ("positions", positions), ("inv_freq", inv_freq), ("q_out", q_out), ("k_out", k_out)))
    return q_out, k_out


def qknorm_rotary(q: torch.Tensor, k: torch.Tensor | None, wq: torch.Tensor, wk: torch.Tensor | None,
                  positions: torch.Tensor | None, inv_freq: torch.Tensor | None, head_dim: int, eps: float = 1e-6, *,
                  layout: str = "half", mscale: float = 1.0, q_out: torch.Tensor | None = None,
                  k_out: torch.Tensor | None = None, inplace: bool = False, stream=None):
    """QK-Norm of the full rows of q and k, then rotary positions, in one pass over them.

    The statistic is :func:`qknorm_fused`'s with ``n_seg=1``; the normalised
    rows are not rounded before they are turned.  ``inv_freq=None`` leaves the
    rotation out.  Returns ``(q_out, k_out)``; arguments as in
    :func:`qknorm_fused` and :func:`rotary_apply`.
    """
    T, dq, ldq = _pitched(q, "q")
    has_k = k is not None
    dk, ldk = _rows_like(k, "k", q, T) if has_k else (0, 0)
    act = _dtype_code(q.dtype)
    wdt = _pair_weights(wq, wk, dq, dk, has_k)
    rot = _rotary_args(positions, inv_freq, head_dim, layout, T) if inv_freq is not None else _NO_ROTARY
    q_out, qp, ldq_o, k_out, kp, ldk_o = _row_outputs(q, k, q_out, k_out, inplace, stream)
    _call("qknorm_rotary", q.device,
          (q.data_ptr(), k.data_ptr() if has_k else None, wq.data_ptr(), wk.data_ptr() if has_k else None, qp, kp, T, dq,
           dk, ldq, ldk, ldq_o, ldk_o, *rot, mscale, act, wdt, eps), stream,
          (("k", k), ("wq", wq), ("wk", wk if has_k else None),
           ("positions", positions if inv_freq is not None else None), ("inv_freq", inv_freq), ("q_out", q_out),
           ("k_out", k_out)))
    return q_out, k_out


def qknorm_rotary_backward_workspace_bytes(T: int, dq: int, dk: int) -> int:
    """Device scratch qknorm_rotary_backward needs for these sizes (bytes)."""
    return int(load_library().qknorm_rotary_backward_workspace_bytes(T, dq, dk))


def _f32_vector(given: torch.Tensor | None, name: str, like: torch.Tensor) -> torch.Tensor:
    """The fp32 vector of like's length that takes a result: the one given, or a new one."""
    n = like.shape[0]
    if given is None:
        return like.new_empty(n, dtype=torch.float32)
    _vec(given, name, n)
    if given.dtype != torch.float32:
        raise ValueError(f"{name} must be fp32")
    return given


@functools.lru_cache(maxsize=256)
def _rotary_workspace(dev: torch.device, T: int, dq: int, dk: int) -> int:
    with _On(dev):  # the size goes by the device's number of SMs
        return qknorm_rotary_backward_workspace_bytes(T, dq, dk)


def qknorm_rotary_backward(gq: torch.Tensor, gk: torch.Tensor | None, q: torch.Tensor, k: torch.Tensor | None,
                           wq: torch.Tensor, wk: torch.Tensor | None, positions: torch.Tensor | None,
                           inv_freq: torch.Tensor | None, head_dim: int, eps: float = 1e-6, *, layout: str = "half",
                           mscale: float = 1.0, dq_out: torch.Tensor | None = None,
                           dk_out: torch.Tensor | None = None, dwq_out: torch.Tensor | None = None,
                           dwk_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients of :func:`qknorm_rotary` (of :func:`qknorm_fused` with ``inv_freq=None``).

    ``gq``, ``gk`` are the gradients of its two outputs, the other arguments
    those it was called with.  Returns ``(dq, dk, dwq, dwk)``: dq and dk in
    q's dtype, dwq and dwk in float32 (None for k when k is None).  The
    results must not overlap the inputs.  ``workspace`` (uint8 CUDA tensor of
    at least ``qknorm_rotary_backward_workspace_bytes``) avoids an allocation
    inside the call.
    """
    T, dq, ldq = _pitched(q, "q")
    act = _dtype_code(q.dtype)
    has_k = k is not None
    if has_k != (gk is not None):
        raise ValueError("gk is given with k, and only with k")
    dgq, ldgq = _rows_like(gq, "gq", q, T)
    dk, ldk = _rows_like(k, "k", q, T) if has_k else (0, 0)
    dgk, ldgk = _rows_like(gk, "gk", q, T) if has_k else (0, 0)
    if dgq != dq or dgk != dk:
        raise ValueError("gq and gk must have the widths of q and k")
    wdt = _pair_weights(wq, wk, dq, dk, has_k)
    rot = _rotary_args(positions, inv_freq, head_dim, layout, T) if inv_freq is not None else _NO_ROTARY
    for given, name in ((dq_out, "dq_out"), (dk_out, "dk_out")):
        if given is not None:
            _not_over(given, name, (q, k, gq, gk))
    dq_t, qp, ld_dq, dk_t, kp, ld_dk = _row_outputs(q, k, dq_out, dk_out, False, stream)
    dev = q.device
    with _AllocOn(stream, dev):
        dwq_out = _f32_vector(dwq_out, "dwq_out", wq)
        dwk_out = _f32_vector(dwk_out, "dwk_out", wk) if has_k else None
        if workspace is None:
            workspace = wq.new_empty(_rotary_workspace(dev, T, dq, dk), dtype=torch.uint8)
    _cuda(workspace, "workspace")
    _call("qknorm_rotary_backward", dev,
          (gq.data_ptr(), gk.data_ptr() if has_k else None, q.data_ptr(), k.data_ptr() if has_k else None,
           wq.data_ptr(), wk.data_ptr() if has_k else None, qp, kp, dwq_out.data_ptr(),
           dwk_out.data_ptr() if has_k else None, T, dq, dk, ldgq, ldgk, ldq, ldk, ld_dq, ld_dk, *rot, mscale, act, wdt,
           eps, workspace.data_ptr(), workspace.numel() * workspace.element_size()), stream,
          (("gq", gq), ("k", k), ("gk", gk), ("wq", wq), ("wk", wk if has_k else None),
           ("positions", positions if inv_freq is not None else None), ("inv_freq", inv_freq), ("dq_out", dq_t),
           ("dk_out", dk_t), ("dwq_out", dwq_out), ("dwk_out", dwk_out), ("workspace", workspace)))
    return dq_t, dk_t, dwq_out, dwk_out


_ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _activation(act: str) -> int:
    code = _ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(_ACTIVATIONS)}, not {act!r}")
    return code


def _bf16_rows(t: torch.Tensor, name: str):
    r = _pitched(t, name)
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bf16")
    return r


def _bf16_like(t: torch.Tensor, name: str, rows: int, cols: int) -> int:
    r, c, ld = _bf16_rows(t, name)
    if r != rows or c != cols:
        raise ValueError(f"{name} must be [{rows}, {cols}]")
    return ld


def _new(like: torch.Tensor, rows: int, cols: int, stream) -> torch.Tensor:
    if stream is None:
        return like.new_empty((rows, cols))
    with _AllocOn(stream, like.device):
        return like.new_empty((rows, cols))


def linear_fused(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
                 residual: torch.Tensor | None = None, *, inv_rms: torch.Tensor | None = None,
                 preact_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """y [M, N] = act(r * (x W^T) + bias) + residual, bf16 in and out, fp32 accumulate, one launch.

    x [M, K] and W [N, K] are bf16 (row pitches from their strides, multiples
    of 8), ``bias`` [N] bf16 or fp32, ``act`` one of "none", "relu", "silu",
    "gelu" (erf) and "gelu_tanh".  ``residual`` [M, N] may be ``out`` itself.
    ``inv_rms`` (fp32 [M]) scales the rows of the product: FlashNorm's
    deferred 1/rms, with W from :func:`flashnorm_fold_weights`.
    ``preact_out`` receives the pre-activation for :func:`linear_fused_backward`.
    """
    M, K, ldx = _bf16_rows(x, "x")
    N, K2, ldw = _bf16_rows(W, "W")
    if K2 != K:
        raise ValueError(f"W has K={K2} but x has K={K}")
    code = _activation(act)
    bias_dt = QKN_BF16
    if bias is not None:
        _vec(bias, "bias", N)
        bias_dt = _dtype_code(bias.dtype)
    ldr = _bf16_like(residual, "residual", M, N) if residual is not None else 0
    if inv_rms is not None:
        _vec(inv_rms, "inv_rms", M)
        if inv_rms.dtype != torch.float32:
            raise ValueError("inv_rms must be fp32")
    ldz = _bf16_like(preact_out, "preact_out", M, N) if preact_out is not None else 0
    if out is None:
        out, ldy = _new(x, M, N, stream), N
    else:
        ldy = _bf16_like(out, "out", M, N)
        _not_over(out, "out", (x, W, preact_out))
    _call("linear_fused", x.device,
          (x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K, ldx, ldw, ldy,
           bias.data_ptr() if bias is not None else None, bias_dt, code,
           residual.data_ptr() if residual is not None else None, ldr,
           inv_rms.data_ptr() if inv_rms is not None else None,
           preact_out.data_ptr() if preact_out is not None else None, ldz), stream,
          (("W", W), ("bias", bias), ("residual", residual), ("inv_rms", inv_rms), ("preact_out", preact_out),
           ("out", out)))
    return out


def linear_fused_backward_workspace_bytes(M: int, N: int, K: int, act: str = "none") -> int:
    """Device scratch linear_fused_backward needs for these sizes (bytes)."""
    return int(load_library().linear_fused_backward_workspace_bytes(M, N, K, _activation(act)))


@functools.lru_cache(maxsize=256)
def _linear_workspace(dev: torch.device, M: int, N: int, K: int, code: int) -> int:
    with _On(dev):  # the size goes by the device's number of SMs
        return int(load_library().linear_fused_backward_workspace_bytes(M, N, K, code))


def linear_fused_backward(dy: torch.Tensor, x: torch.Tensor | None, W: torch.Tensor | None,
                          preact: torch.Tensor | None = None, act: str = "none", *, need_dbias: bool = False,
                          dx_out: torch.Tensor | None = None, dW_out: torch.Tensor | None = None,
                          dbias_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients ``(dx, dW, dbias)`` of :func:`linear_fused` (called without ``inv_rms``) for dy [M, N].

    dx needs W and dW needs x: the one whose input is None is left out.
    dbias (fp32 [N]) is formed with ``need_dbias`` or ``dbias_out``.
    ``preact`` is what the forward call wrote to ``preact_out`` (not needed
    for act "none").  The residual's gradient is dy itself.  ``workspace``
    (uint8 CUDA tensor of at least ``linear_fused_backward_workspace_bytes``)
    avoids an allocation inside the call.
    """
    M, N, lddy = _bf16_rows(dy, "dy")
    code = _activation(act)
    if x is None and W is None and not need_dbias and dbias_out is None:
        raise ValueError("nothing to compute: x, W, need_dbias and dbias_out are all absent")
    K = 8
    if W is not None:
        n, K, ldw = _bf16_rows(W, "W")
        if n != N:
            raise ValueError(f"W has {n} rows but dy has {N} columns")
    if x is not None:
        m, kx, ldx = _bf16_rows(x, "x")
        if m != M or (W is not None and kx != K):
            raise ValueError("x must be [M, K]")
        K = kx
    if code != 0 and preact is None:
        raise ValueError("preact is required with an activation")
    if code == 0:
        preact = None
    ldz = _bf16_like(preact, "preact", M, N) if preact is not None else 0
    lddx = lddw = 0
    if W is not None:
        if dx_out is None:
            dx_out, lddx = _new(dy, M, K, stream), K
        else:
            lddx = _bf16_like(dx_out, "dx_out", M, K)
            _not_over(dx_out, "dx_out", (dy, W, x, preact))
    elif dx_out is not None:
        raise ValueError("dx_out needs W")
    if x is not None:
        if dW_out is None:
            dW_out, lddw = _new(dy, N, K, stream), K
        else:
            lddw = _bf16_like(dW_out, "dW_out", N, K)
            _not_over(dW_out, "dW_out", (dy, W, x, preact))
    elif dW_out is not None:
        raise ValueError("dW_out needs x")
    with _AllocOn(stream, dy.device):
        if need_dbias and dbias_out is None:
            dbias_out = torch.empty(N, dtype=torch.float32, device=dy.device)
        if workspace is None:
            workspace = torch.empty(_linear_workspace(dy.device, M, N, K, code), dtype=torch.uint8, device=dy.device)
    _cuda(workspace, "workspace")
    if dbias_out is not None:
        _vec(dbias_out, "dbias_out", N)
        if dbias_out.dtype != torch.float32:
            raise ValueError("dbias_out must be fp32")
    ptr = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
    _call("linear_fused_backward", dy.device,
          (dy.data_ptr(), ptr(preact), ptr(x), ptr(W), ptr(dx_out), ptr(dW_out), ptr(dbias_out), M, N, K, lddy, ldz,
           ldx if x is not None else 0, ldw if W is not None else 0, lddx, lddw, code, workspace.data_ptr(),
           workspace.numel() * workspace.element_size()), stream,
          (("x", x), ("W", W), ("preact", preact), ("dx_out", dx_out), ("dW_out", dW_out), ("dbias_out", dbias_out),
           ("workspace", workspace)))
    return dx_out, dW_out, dbias_out
