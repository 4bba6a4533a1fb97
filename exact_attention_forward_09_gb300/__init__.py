"""Fused exact attention forward for NVIDIA GB300 (sm_103a).

The product is the C library ``libfa.so`` (C ABI declared in
``include/fa.h``; hand-written CUDA kernels under ``csrc/``).  This package is
a thin ctypes binding with the same entry-point names: it checks tensor
shapes, allocates outputs with torch, passes raw device pointers and the
current CUDA stream, and turns status codes into exceptions.  Every step of
the computation runs in the library's kernels; there is no other code path.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import struct

import torch

from .build import LIB as _LIB_PATH

__all__ = ["fwd_host", "fwd_host_workspace_bytes", "bwd", "bwd_workspace_bytes", "fwd_splitkv", "splitkv_workspace_bytes", "fwd", "fwd_gqa", "fwd_window", "bwd_window", "bwd_window_workspace_bytes",
           "fwd_paged", "paged_workspace_bytes", "tree_plan", "fwd_tree", "cache_append", "rope", "rope_table", "pages_resize", "pages_fork",
           "cache_copy", "cache_compact", "fwd_fp8", "fwd_fp8_gqa", "quant_fp8", "quant_fp8_per_tensor_noalloc", "check_device_error", "lib",
           "FaError", "FA_OK", "FA_ERR_INVALID_ARG", "FA_ERR_UNSUPPORTED", "FA_ERR_CUDA", "FA_ERR_TIMEOUT",
           "FA_ERR_SCRATCH_LIMIT", "FA_ERR_INDEX", "FA_DTYPE_BF16", "FA_DTYPE_FP16", "FP8_BLOCK_ROWS",
           "FA_ROPE_INTERLEAVED", "FA_ROPE_HALF", "FA_ROPE_SCALE_NONE", "FA_ROPE_SCALE_LINEAR", "FA_ROPE_SCALE_BASE",
           "FA_ROPE_SCALE_TURNS", "FA_ROPE_SCALE_INDEX",
           "QUANT_NOALLOC_MAX_BLOCKS"]

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = 0, 1, 2, 3, 4
FA_ERR_SCRATCH_LIMIT = 5
FA_ERR_INDEX = 6
QUANT_NOALLOC_MAX_BLOCKS = 65536
FA_DTYPE_BF16, FA_DTYPE_FP16 = 0, 1
FA_ROPE_INTERLEAVED, FA_ROPE_HALF = 1, 2
FA_ROPE_SCALE_NONE, FA_ROPE_SCALE_LINEAR, FA_ROPE_SCALE_BASE, FA_ROPE_SCALE_TURNS, FA_ROPE_SCALE_INDEX = 0, 1, 2, 3, 4
FP8_BLOCK_ROWS = 128


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib().fa_status_string(status).decode()}")


class _KvCache(ctypes.Structure):
    """``fa_kv_cache``.  (The operators below pass its bytes, packed in one
    step: filling a ctypes structure field by field takes longer than their
    launch.)"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("heads", ctypes.c_int64), ("d", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


_KV_PACK = struct.Struct("@PPqqqqqqqi4x").pack
_ROPE_PACK = struct.Struct("@PPqqqqqqq").pack      # fa_rope_array
_SCALING_PACK = struct.Struct("@i4xddddd").pack    # fa_rope_scaling


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"libfa.so has not been built ({_LIB_PATH}); run "
                              "`python -c 'import __graft_entry__ as g; g.build()'` first")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, f32, i32, vp]
        lib.fa_fwd.restype = i32
        lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, f32, vp, vp, vp, vp]
        lib.fa_fwd_fp8.restype = i32
        lib.fa_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, f32, i32, vp]
        lib.fa_fwd_gqa.restype = i32
        lib.fa_fwd_fp8_gqa.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, f32, vp, vp, vp,
                                       vp]
        lib.fa_fwd_fp8_gqa.restype = i32
        lib.fa_quant_fp8.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, i32, vp, vp]
        lib.fa_quant_fp8.restype = i32
        lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, f32, i32, i32, vp,
                                       ctypes.c_size_t, vp]
        lib.fa_fwd_splitkv.restype = i32
        lib.fa_splitkv_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i64, i32, ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_splitkv_workspace_bytes.restype = i32
        lib.fa_quant_fp8_rope.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, vp, i32, vp, i32, vp, vp]
        lib.fa_quant_fp8_rope.restype = i32
        lib.fa_quant_fp8_qkv.argtypes = [vp] * 9 + [i64] * 6 + [vp, vp]
        lib.fa_quant_fp8_qkv.restype = i32
        lib.fa_quant_fp8_per_tensor_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, vp]
        lib.fa_quant_fp8_per_tensor_noalloc.restype = i32
        lib.fa_fwd_host.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, f32, i32, vp,
                                    ctypes.c_size_t, vp]
        lib.fa_fwd_host.restype = i32
        lib.fa_fwd_host_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i64, ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_fwd_host_workspace_bytes.restype = i32
        lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, f32, i32,
                               vp, ctypes.c_size_t, vp]
        lib.fa_bwd.restype = i32
        lib.fa_bwd_workspace_bytes.argtypes = [i64, i64, i64, i64, ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_bwd_workspace_bytes.restype = i32
        cache = ctypes.c_char_p  # the bytes of an fa_kv_cache
        lib.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp] + [i64] * 8 + [f32, i32, vp]
        lib.fa_fwd_window.restype = i32
        lib.fa_bwd_window.argtypes = [vp] * 9 + [i64] * 8 + [f32, i32, vp, ctypes.c_size_t, vp]
        lib.fa_bwd_window.restype = i32
        lib.fa_bwd_window_workspace_bytes.argtypes = [i64] * 8 + [ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_bwd_window_workspace_bytes.restype = i32
        lib.fa_paged_workspace_bytes.argtypes = [i64, ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_paged_workspace_bytes.restype = i32
        lib.fa_fwd_paged.argtypes = [vp, cache, vp, vp, vp, i64, i64, vp, vp] + [i64] * 7 + [f32, vp, ctypes.c_size_t, vp]
        lib.fa_fwd_paged.restype = i32
        lib.fa_tree_plan.argtypes = [vp, vp, vp, i64, i64, vp, i64, vp, vp]
        lib.fa_tree_plan.restype = i32
        lib.fa_tree_plan_window.argtypes = [vp, vp, vp, i64, i64, vp, i64, vp, i64, i64, vp]
        lib.fa_tree_plan_window.restype = i32
        lib.fa_fwd_tree.argtypes = [vp, cache, vp, vp, vp, i64, i64, vp, vp, vp, i64, vp] + [i64] * 7 + [f32, vp, ctypes.c_size_t, vp]
        lib.fa_fwd_tree.restype = i32
        lib.fa_cache_append.argtypes = [cache, vp, vp, vp, vp, i64, i64, i64, vp, i64, i64, vp, vp, i64, i64, i64, vp,
                                        vp, i64, i32, vp]
        lib.fa_cache_append.restype = i32
        lib.fa_cache_append_at.argtypes = [cache, vp, vp, vp, vp, i64, i64, i64, vp, i64, i64, vp, vp, i64, i64, i64, vp,
                                           vp, i64, i64, i32, vp, vp]
        lib.fa_cache_append_at.restype = i32
        packed = ctypes.c_char_p  # the bytes of fa_rope_array, fa_rope_scaling structures
        lib.fa_rope_table.argtypes = [vp, vp, i64, i64, ctypes.c_double, i64, packed, vp]
        lib.fa_rope_table.restype = i32
        lib.fa_rope.argtypes = [packed, i64, i64, i64, i64, vp, i64, i64, vp, vp, i64, i64, i32, i32, i32, vp]
        lib.fa_rope.restype = i32
        lib.fa_pages_resize.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, i64, vp]
        lib.fa_pages_resize.restype = i32
        lib.fa_pages_fork.argtypes = [cache, i64, i64, vp, vp, i64, i64, vp, i64, vp, vp, vp, i64, vp]
        lib.fa_pages_fork.restype = i32
        lib.fa_cache_copy.argtypes = [cache, i64, i64, vp, vp, i64, vp]
        lib.fa_cache_copy.restype = i32
        lib.fa_cache_compact.argtypes = [cache, i64, i64, vp, i64, i64, vp, vp, i64, i64, vp, vp, i64, vp]
        lib.fa_cache_compact.restype = i32
        lib.fa_status_string.argtypes = [i32]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_check_device_error.argtypes = [vp]
        lib.fa_check_device_error.restype = i32
        lib.fa_debug_inject.argtypes = [i32]
        lib.fa_debug_inject.restype = i32
        lib.fa_debug_exp2.argtypes = [vp, vp, i64, i32, vp]
        lib.fa_debug_exp2.restype = i32
        lib.fa_version.argtypes = []
        lib.fa_version.restype = i32
        _LIB = lib
    return _LIB


def lib():
    """The loaded ctypes library (raw C entry points)."""
    return _lib()


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _check(status: int, where: str):
    if status != FA_OK:
        raise FaError(status, where)


def _check_qkv(q, k, v, allowed):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, H, N, d] tensor")
        if t.dtype not in allowed:
            raise ValueError(f"{name} has dtype {t.dtype}; expected one of {allowed}")
    if not (q.shape == k.shape == v.shape and q.dtype == k.dtype == v.dtype and
            q.device == k.device == v.device):
        raise ValueError("q, k, v must share shape, dtype and device")


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
        scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None):
    """BF16/FP16 attention forward (``fa_fwd``).  Returns (O, LSE)."""
    _check_qkv(q, k, v, (torch.bfloat16, torch.float16))
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    dt = FA_DTYPE_BF16 if q.dtype == torch.bfloat16 else FA_DTYPE_FP16
    with torch.cuda.device(q.device):
        st = _lib().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                           B, H, N, d, int(bool(causal)), float(scale), dt, _stream(q))
    _check(st, "fa_fwd")
    return out, lse


def splitkv_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int, num_splits: int = 0) -> int:
    """Device workspace (bytes) ``fwd_splitkv`` needs on the current device."""
    n = ctypes.c_size_t(0)
    _check(_lib().fa_splitkv_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, int(num_splits), ctypes.byref(n)),
           "fa_splitkv_workspace_bytes")
    return int(n.value)


def fwd_splitkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
                scale: float | None = None, num_splits: int = 0, out: torch.Tensor | None = None,
                lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Split-KV forward for decode-like shapes (``fa_fwd_splitkv``): q [B, Hq,
    Nq, d], k/v [B, Hkv, Nk, d]; the query heads of a key/value group are
    packed together and the keys split into ``num_splits`` runs (0: chosen
    for the device).  Returns (O [B, Hq, Nq, d], LSE [B, Hq, Nq])."""
    _check_gqa(q, k, v, (torch.bfloat16, torch.float16))
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    dt = FA_DTYPE_BF16 if q.dtype == torch.bfloat16 else FA_DTYPE_FP16
    with torch.cuda.device(q.device):
        need = splitkv_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, num_splits)
        if workspace is None and need > 0:
            workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
        wp = workspace.data_ptr() if workspace is not None else None
        wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
        st = _lib().fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                   B, Hq, Hkv, Nq, Nk, d, int(bool(causal)), float(scale), dt, int(num_splits),
                                   wp, wb, _stream(q))
    _check(st, "fa_fwd_splitkv")
    return out, lse


def fwd_host_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int) -> int:
    """Bytes of device workspace ``fa_fwd_host`` needs for this shape."""
    n = ctypes.c_size_t(0)
    _check(_lib().fa_fwd_host_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, ctypes.byref(n)), "fa_fwd_host_workspace_bytes")
    return int(n.value)


def fwd_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False, scale: float | None = None,
             out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, device=None):
    """``fa_fwd_host``: q [B, Hq, Nq, d], k/v [B, Hkv, Nk, d] in HOST memory
    (page-locked for overlapped copies); the call copies them to the device,
    runs the kernel and copies O and LSE back, asynchronously on the current
    stream of ``device`` (default: the current CUDA device).  Returns
    (O, LSE) as host tensors, complete once that stream has synchronised."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.is_cuda or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D host tensor")
        if t.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"{name} has dtype {t.dtype}; expected bf16 or fp16")
    B, Hq, Nq, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d or q.dtype != k.dtype or k.dtype != v.dtype:
        raise ValueError("k and v must be [B, Hkv, Nk, d] with q's batch, head dimension and dtype")
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    pin = q.is_pinned()
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=pin)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, pin_memory=pin)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    dt = FA_DTYPE_BF16 if q.dtype == torch.bfloat16 else FA_DTYPE_FP16
    with torch.cuda.device(dev):
        need = fwd_host_workspace_bytes(B, Hq, Hkv, Nq, Nk, d)
        if workspace is None:
            workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
        st = _lib().fa_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                B, Hq, Hkv, Nq, Nk, d, int(bool(causal)), float(scale), dt,
                                workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                torch.cuda.current_stream(dev).cuda_stream)
    _check(st, "fa_fwd_host")
    return out, lse


def bwd_workspace_bytes(B: int, Hq: int, Nq: int, d: int) -> int:
    """Bytes of device workspace ``fa_bwd`` needs for this shape."""
    n = ctypes.c_size_t(0)
    _check(_lib().fa_bwd_workspace_bytes(B, Hq, Nq, d, ctypes.byref(n)), "fa_bwd_workspace_bytes")
    return int(n.value)


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
        dout: torch.Tensor, causal: bool = False, scale: float | None = None, dq: torch.Tensor | None = None,
        dk: torch.Tensor | None = None, dv: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Gradients of sum(dout * O) (``fa_bwd``): q, out, dout [B, Hq, Nq, d],
    k/v [B, Hkv, Nk, d], lse [B, Hq, Nq] fp32 from the forward with the same
    causal flag and scale.  Returns (dq, dk, dv)."""
    _check_gqa(q, k, v, (torch.bfloat16, torch.float16))
    for name, t in (("out", out), ("dout", dout)):
        if not isinstance(t, torch.Tensor) or t.shape != q.shape or t.dtype != q.dtype or not t.is_contiguous() \
                or t.device != q.device:
            raise ValueError(f"{name} must be a contiguous tensor with q's shape, dtype and device")
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if not isinstance(lse, torch.Tensor) or lse.shape != (B, Hq, Nq) or lse.dtype != torch.float32 \
            or not lse.is_contiguous() or lse.device != q.device:
        raise ValueError("lse must be a contiguous fp32 [B, Hq, Nq] tensor on q's device")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    dt = FA_DTYPE_BF16 if q.dtype == torch.bfloat16 else FA_DTYPE_FP16
    with torch.cuda.device(q.device):
        need = bwd_workspace_bytes(B, Hq, Nq, d)
        if workspace is None:
            workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=q.device)
        st = _lib().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                           dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                           B, Hq, Hkv, Nq, Nk, d, int(bool(causal)), float(scale), dt,
                           workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(q))
    _check(st, "fa_bwd")
    return dq, dk, dv


def _check_gqa(q, k, v, allowed):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D CUDA tensor")
        if t.dtype not in allowed:
            raise ValueError(f"{name} has dtype {t.dtype}; expected one of {allowed}")
    B, Hq, Nq, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d or q.dtype != k.dtype or k.dtype != v.dtype:
        raise ValueError("k and v must be [B, Hkv, Nk, d] with q's batch, head dimension and dtype")
    if k.shape[1] == 0 or Hq % k.shape[1] != 0:
        raise ValueError("the number of query heads must be a multiple of the number of key/value heads")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on one device")


def fwd_gqa(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
            scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None):
    """Grouped/multi-query attention with Nq != Nk allowed (``fa_fwd_gqa``):
    q [B, Hq, Nq, d], k/v [B, Hkv, Nk, d]; causal masks are bottom-right
    aligned.  Returns (O [B, Hq, Nq, d], LSE [B, Hq, Nq])."""
    _check_gqa(q, k, v, (torch.bfloat16, torch.float16))
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    dt = FA_DTYPE_BF16 if q.dtype == torch.bfloat16 else FA_DTYPE_FP16
    with torch.cuda.device(q.device):
        st = _lib().fa_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                               B, Hq, Hkv, Nq, Nk, d, int(bool(causal)), float(scale), dt, _stream(q))
    _check(st, "fa_fwd_gqa")
    return out, lse


# The calls below are often small, and then the time on the host counts: they
# ask for the current stream and switch devices only as far as needed.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device  # (asked with CUDA tensors in hand)
_NO_GUARD = contextlib.nullcontext()


def _current_stream(index: int) -> int:
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _guard(index: int):
    return _NO_GUARD if _raw_device() == index else torch.cuda.device(index)


_TYPES = {torch.bfloat16: FA_DTYPE_BF16, torch.float16: FA_DTYPE_FP16}
_I32, _F32, _U8, _empty = torch.int32, torch.float32, torch.uint8, torch.empty


def _count(x) -> int:
    """x as a whole number that 64 bits hold (one beyond them would reach the
    library as what is left of it): the nearest one."""
    x = int(x)
    return x if -1 << 63 <= x < 1 << 63 else ((1 << 63) - 1 if x > 0 else -1 << 63)


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def _check_out(name, t, shape, dtype, index):
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype is not dtype or t.get_device() != index \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on cuda:{index}")


def _workspace(t, index):
    """The address and size of a caller's workspace."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{index}")
    return t.data_ptr(), t.nbytes


def _dense(q, k, v):
    """(B, Hq, Nq, d, Hkv, Nk, device index) of checked dense q, k, v."""
    if isinstance(q, torch.Tensor) and isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor):
        sq, sk, dt, index = q.shape, k.shape, q.dtype, q.get_device()
        if len(sq) == 4 and len(sk) == 4 and v.shape == sk and dt in _TYPES and k.dtype is dt and v.dtype is dt \
                and index >= 0 and k.get_device() == index and v.get_device() == index and q.is_contiguous() \
                and k.is_contiguous() and v.is_contiguous():
            B, Hq, Nq, d = sq
            Bk, Hkv, Nk, dk = sk
            if Bk == B and dk == d and Hkv > 0 and Hq % Hkv == 0:
                return B, Hq, Nq, d, Hkv, Nk, index
    _check_gqa(q, k, v, (torch.bfloat16, torch.float16))  # says what is wrong
    raise ValueError("q, k and v are not dense 16-bit CUDA tensors of one device")


def fwd_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, sinks: int = 0,
               scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None):
    """Attention under a sliding window with sinks (``fa_fwd_window``): q [B,
    Hq, Nq, d], k/v [B, Hkv, Nk, d]; query i at position p = i + Nk - Nq sees
    key j iff j <= p and (j > p - window or j < sinks).  Returns
    (O [B, Hq, Nq, d], LSE [B, Hq, Nq])."""
    B, Hq, Nq, d, Hkv, Nk, index = _dense(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out("out", out, (B, Hq, Nq, d), q.dtype, index)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    else:
        _check_out("lse", lse, (B, Hq, Nq), torch.float32, index)
    with _guard(index):
        st = _lib().fa_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                  B, Hq, Hkv, Nq, Nk, d, _count(window), _count(sinks), _scale(scale, d), _TYPES[q.dtype],
                                  _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_window")
    return out, lse


@functools.lru_cache(maxsize=256)
def _bwd_window_bytes(*sizes: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib().fa_bwd_window_workspace_bytes(*sizes, ctypes.byref(n)), "fa_bwd_window_workspace_bytes")
    return n.value


def bwd_window_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int, window: int, sinks: int = 0) -> int:
    """Bytes of device workspace ``bwd_window`` needs for this shape, on any device."""
    return _bwd_window_bytes(B, Hq, Hkv, Nq, Nk, d, _count(window), _count(sinks))


def bwd_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
               dout: torch.Tensor, window: int, sinks: int = 0, scale: float | None = None,
               dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None):
    """Gradients of sum(dout * O) for ``fwd_window`` (``fa_bwd_window``): q,
    out, dout [B, Hq, Nq, d], k/v [B, Hkv, Nk, d], lse [B, Hq, Nq] fp32 from
    the forward with the same window, sinks and scale; d 64 or 128.  Returns
    (dq, dk, dv)."""
    B, Hq, Nq, d, Hkv, Nk, index = _dense(q, k, v)
    window, sinks = _count(window), _count(sinks)
    dt = q.dtype
    _check_out("out", out, q.shape, dt, index)
    _check_out("dout", dout, q.shape, dt, index)
    _check_out("lse", lse, (B, Hq, Nq), torch.float32, index)
    if dq is None:
        dq = torch.empty_like(q)
    else:
        _check_out("dq", dq, q.shape, dt, index)
    if dk is None:
        dk = torch.empty_like(k)
    else:
        _check_out("dk", dk, k.shape, dt, index)
    if dv is None:
        dv = torch.empty_like(v)
    else:
        _check_out("dv", dv, v.shape, dt, index)
    with _guard(index):
        if workspace is None:
            need = _bwd_window_bytes(B, Hq, Hkv, Nq, Nk, d, window, sinks)
            workspace = torch.empty((need or 1,), dtype=torch.uint8, device=q.device)
        st = _lib().fa_bwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                  dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Nq, Nk, d,
                                  window, sinks, _scale(scale, d), _TYPES[dt],
                                  *_workspace(workspace, index), _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_window")
    return dq, dk, dv


def _cache(k_pages, v_pages):
    """The ``fa_kv_cache`` of two [num_pages, heads, page_size, d] tensors (or
    views of that shape with other strides), their heads, head dimension,
    dtype and device index."""
    if isinstance(k_pages, torch.Tensor) and isinstance(v_pages, torch.Tensor):
        shape, stride, dt, index = k_pages.shape, k_pages.stride(), k_pages.dtype, k_pages.get_device()
        if len(shape) == 4 and index >= 0 and dt in _TYPES and stride[3] == 1 and v_pages.shape == shape \
                and v_pages.stride() == stride and v_pages.dtype is dt and v_pages.get_device() == index:
            n, h, ps, d = shape
            return _KV_PACK(k_pages.data_ptr(), v_pages.data_ptr(), n, ps, h, d, stride[0], stride[1], stride[2],
                            _TYPES[dt]), h, d, dt, index
    raise ValueError("k_pages and v_pages must be bf16 or fp16 [num_pages, heads, page_size, d] CUDA tensors of one shape, "
                     "dtype, device and strides, their last dimension contiguous")


def _check_batch(block_table, cu_q, seq_k, index):
    """(B, table stride, table width) of a ragged batch's index tensors."""
    if isinstance(block_table, torch.Tensor) and isinstance(cu_q, torch.Tensor) and isinstance(seq_k, torch.Tensor):
        i32, st, sc, sk = torch.int32, block_table.shape, cu_q.shape, seq_k.shape
        if len(st) == 2 and len(sc) == 1 and len(sk) == 1 and block_table.dtype is i32 and cu_q.dtype is i32 \
                and seq_k.dtype is i32 and block_table.get_device() == index and cu_q.get_device() == index \
                and seq_k.get_device() == index and st[0] == sk[0] and sc[0] == sk[0] + 1 and cu_q.is_contiguous() \
                and seq_k.is_contiguous() and (st[1] < 2 or block_table.stride(1) == 1):
            return sk[0], block_table.stride(0), st[1]
    raise ValueError(f"block_table [B, max_pages], cu_q [B + 1] and seq_k [B] must be int32 tensors on cuda:{index}, "
                     "cu_q and seq_k contiguous, and so each row of block_table")


def _check_tokens(name, t, T, heads, d, dtype, index):
    """The token stride of a packed [T, heads, d] tensor."""
    if isinstance(t, torch.Tensor):
        shape = t.shape
        if len(shape) == 3 and t.dtype is dtype and t.get_device() == index and shape[0] == T and shape[1] == heads \
                and shape[2] == d:
            stride = t.stride()
            if t.numel() == 0 or (stride[2] == 1 and (heads == 1 or stride[1] == d)):
                return stride[0]
    raise ValueError(f"{name} must be a {dtype} [{T}, {heads}, {d}] tensor on cuda:{index}, the heads of a token contiguous")


_PAGED_BYTES = {}  # by device index and head dimension


def paged_workspace_bytes(d: int) -> int:
    """Bytes of device workspace ``fwd_paged`` needs on the current device."""
    n = ctypes.c_size_t(0)
    _check(_lib().fa_paged_workspace_bytes(d, ctypes.byref(n)), "fa_paged_workspace_bytes")
    return n.value


def fwd_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
              cu_q: torch.Tensor, seq_k: torch.Tensor, window: int | None = None, sinks: int = 0,
              scale: float | None = None, max_q: int = 0, out: torch.Tensor | None = None,
              lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Attention of the new tokens of a ragged batch over a paged cache
    (``fa_fwd_paged``): q [T, Hq, d] (sequence b has rows cu_q[b] to
    cu_q[b+1]), pages [num_pages, Hkv, page_size, d], block_table [B,
    max_pages], seq_k [B] keys per sequence with the new tokens' last.
    ``window`` None: every key up to a query's own.  ``max_q``: the most new
    tokens of any sequence, if known.  Returns (O [T, Hq, d], LSE [T, Hq]);
    rows outside every sequence are left as they were."""
    return _fwd_paged(q, k_pages, v_pages, block_table, cu_q, seq_k, None, None, window, sinks, scale, max_q, out, lse, workspace)


def _fwd_paged(q, k_pages, v_pages, block_table, cu_q, seq_k, mask, positions, window, sinks, scale, max_q, out, lse, workspace):
    # The checks of _cache, _check_tokens and _check_batch in one place, as a
    # call's time on the host counts; what fails goes to them, which say what is wrong.
    try:
        pages, heads, page_size, d = shape = k_pages.shape
        s0, s1, s2, s3 = strides = k_pages.stride()
        dt, index = k_pages.dtype, k_pages.get_device()
        T, Hq, c = q.shape
        q_stride, qh, qc = q.stride()
        B, max_pages = block_table.shape
        table_stride, tc = block_table.stride()
        good = s3 == 1 and index >= 0 and dt in _TYPES and v_pages.shape == shape and v_pages.stride() == strides \
            and v_pages.dtype is dt and v_pages.get_device() == index and c == d and q.dtype is dt and q.get_device() == index \
            and qc == 1 and (qh == d or Hq == 1) and block_table.dtype is _I32 and cu_q.dtype is _I32 and seq_k.dtype is _I32 \
            and block_table.get_device() == index and cu_q.get_device() == index and seq_k.get_device() == index \
            and cu_q.shape == (B + 1,) and seq_k.shape == (B,) and cu_q.is_contiguous() and seq_k.is_contiguous() \
            and (tc == 1 or max_pages < 2) and isinstance(q, torch.Tensor)
    except (AttributeError, TypeError, ValueError):
        good = False
    if good:
        cache = _KV_PACK(k_pages.data_ptr(), v_pages.data_ptr(), pages, page_size, heads, d, s0, s1, s2, _TYPES[dt])
    else:
        cache, heads, d, dt, index = _cache(k_pages, v_pages)
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a [T, Hq, d] CUDA tensor")
        T, Hq, _ = q.shape
        q_stride = _check_tokens("q", q, T, Hq, d, dt, index)
        B, table_stride, max_pages = _check_batch(block_table, cu_q, seq_k, index)
    if heads == 0 or Hq % heads != 0:
        raise ValueError("the number of query heads must be a multiple of the number of key/value heads")
    dev = k_pages.device
    if out is None:
        out = _empty((T, Hq, d), dtype=dt, device=dev)
    else:
        _check_out("out", out, (T, Hq, d), dt, index)
    if lse is None:
        lse = _empty((T, Hq), dtype=_F32, device=dev)
    else:
        _check_out("lse", lse, (T, Hq), _F32, index)
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or len(mask.shape) != 2:
            raise ValueError("mask must be an int32 [T, words] tensor")
        words = mask.shape[1]
        _check_out("mask", mask, (T, words), _I32, index)
        pp = None if positions is None else _check_ints("positions", positions, T, index)
    if workspace is None:
        need = _PAGED_BYTES.get((index, d))
        if need is None:
            with torch.cuda.device(index):
                need = _PAGED_BYTES[index, d] = paged_workspace_bytes(d)
        workspace = _empty((need,), dtype=_U8, device=dev)
        wp = workspace.data_ptr()
    else:
        wp, need = _workspace(workspace, index)
    lib = _LIB or _lib()
    with _guard(index):
        if mask is None:
            st = lib.fa_fwd_paged(q.data_ptr(), cache, out.data_ptr(), lse.data_ptr(), block_table.data_ptr(), table_stride,
                                  max_pages, cu_q.data_ptr(), seq_k.data_ptr(), B, T, Hq, q_stride, _count(max_q),
                                  1 << 30 if window is None else _count(window), _count(sinks), _scale(scale, d), wp, need,
                                  _current_stream(index))
        else:
            st = lib.fa_fwd_tree(q.data_ptr(), cache, out.data_ptr(), lse.data_ptr(), block_table.data_ptr(), table_stride,
                                 max_pages, cu_q.data_ptr(), seq_k.data_ptr(), mask.data_ptr(), words, pp, B, T, Hq, q_stride,
                                 _count(max_q), 1 << 30 if window is None else _count(window), _count(sinks), _scale(scale, d),
                                 wp, need, _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_paged" if mask is None else "fa_fwd_tree")
    return out, lse


def tree_plan(parents: torch.Tensor, cu_q: torch.Tensor, seq_k: torch.Tensor, max_tree: int,
              mask: torch.Tensor | None = None, positions: torch.Tensor | None = None, window: int | None = None, sinks: int = 0):
    """Lays out trees of drafted tokens (``fa_tree_plan_window``): parents int32
    [T], each a node's parent by its number within its sequence, or -1; cu_q and
    seq_k as in ``fwd_paged``; ``max_tree``: the most nodes of a tree, up to 1024
    (sequences of more tokens than its next multiple of 32 are chunks of a
    prompt); ``window`` and ``sinks`` those of ``fwd_tree``, so that nodes do not see
    the nodes above them that have left the window.  Returns (mask int32 [T,
    ceil(max_tree / 32)], positions int32 [T]) for ``fwd_tree`` and ``cache_append``."""
    T, index = _ints("parents", parents)
    B, words = _ints("seq_k", seq_k)[0], (_count(max_tree) + 31) // 32
    cp, sp = _check_ints("cu_q", cu_q, B + 1, index), _check_ints("seq_k", seq_k, B, index)
    if not 1 <= words <= 32:
        raise ValueError("max_tree must be 1 to 1024")
    if mask is None:
        mask = torch.empty((T, words), dtype=torch.int32, device=parents.device)
    else:
        _check_out("mask", mask, (T, words), torch.int32, index)
    if positions is None:
        positions = torch.empty_like(parents)
    else:
        _check_out("positions", positions, (T,), torch.int32, index)
    with _guard(index):
        st = _lib().fa_tree_plan_window(parents.data_ptr(), cp, sp, B, T, mask.data_ptr(), words, positions.data_ptr(),
                                        1 << 30 if window is None else _count(window), _count(sinks), _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_tree_plan_window")
    return mask, positions


def fwd_tree(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
             cu_q: torch.Tensor, seq_k: torch.Tensor, mask: torch.Tensor, positions: torch.Tensor | None = None,
             window: int | None = None, sinks: int = 0, scale: float | None = None, max_q: int = 0,
             out: torch.Tensor | None = None, lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """``fwd_paged`` where the new tokens of a sequence are the nodes of a tree
    (``fa_fwd_tree``): each sees the cached keys (under a window by its own
    position, from ``positions`` int32 [T]) and the new tokens up to itself that
    its row of ``mask`` (int32 [T, words], 32 tokens of its sequence to a word)
    has a bit for, whatever the window: give ``tree_plan`` the same window and
    sinks.  Sequences of more than 32 * words new tokens are plain chunks."""
    if mask is None:
        raise ValueError("mask must be an int32 [T, words] tensor")
    return _fwd_paged(q, k_pages, v_pages, block_table, cu_q, seq_k, mask, positions, window, sinks, scale, max_q, out, lse, workspace)


def _check_rope(rope, d, index):
    """(cos, sin, positions, rotated columns, layout) of a rope = (cos, sin, layout) for rows of d."""
    cos, sin, layout = rope
    if layout not in (FA_ROPE_INTERLEAVED, FA_ROPE_HALF):
        raise ValueError("rope layout must be FA_ROPE_INTERLEAVED or FA_ROPE_HALF")
    if isinstance(cos, torch.Tensor) and isinstance(sin, torch.Tensor):
        shape, f32 = cos.shape, torch.float32
        if len(shape) == 2 and sin.shape == shape and cos.dtype is f32 and sin.dtype is f32 and cos.get_device() == index \
                and sin.get_device() == index and cos.is_contiguous() and sin.is_contiguous():
            n, half = shape
            if 8 <= half <= d // 2 and half % 8 == 0:
                return cos.data_ptr(), sin.data_ptr(), n, 2 * half, int(layout)
    raise ValueError(f"rope cos and sin must be contiguous fp32 [positions, rope_dim/2] tensors on cuda:{index}, rope_dim a "
                     f"multiple of 16 up to d = {d}")


def cache_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 block_table: torch.Tensor, cu_q: torch.Tensor, seq_k: torch.Tensor, q: torch.Tensor | None = None,
                 rope=None, q_out: torch.Tensor | None = None, positions: torch.Tensor | None = None):
    """Writes the new tokens' keys and values, [T, heads, d], into their pages
    (``fa_cache_append_at``; the batch as in ``fwd_paged``).  ``rope``: None, or
    (cos, sin, layout) with cos / sin contiguous fp32 [length, rope_dim/2] and
    layout FA_ROPE_INTERLEAVED or FA_ROPE_HALF: the first rope_dim columns of
    keys, and of the queries q [T, Hq, d] if given, are rotated first, by the
    tokens' positions in their sequences or by ``positions`` (int32 [T], as
    ``tree_plan`` gives them).  k, v and q may be slices of one projection.
    Returns the rotated queries (``q_out``), or None without q."""
    # (checked in one place, as in _fwd_paged)
    Hq, qs, qp, op = 0, 0, None, None
    try:
        pages, heads, page_size, d = shape = k_pages.shape
        s0, s1, s2, s3 = strides = k_pages.stride()
        dt, index = k_pages.dtype, k_pages.get_device()
        T = k.shape[0]
        ks, kh, kc = k.stride()
        vs, vh, vc = v.stride()
        B, max_pages = block_table.shape
        table_stride, tc = block_table.stride()
        good = s3 == 1 and index >= 0 and dt in _TYPES and v_pages.shape == shape and v_pages.stride() == strides \
            and v_pages.dtype is dt and v_pages.get_device() == index and k.shape == (T, heads, d) and v.shape == (T, heads, d) \
            and k.dtype is dt and v.dtype is dt and k.get_device() == index and v.get_device() == index and kc == 1 and vc == 1 \
            and (heads == 1 or (kh == d and vh == d)) and block_table.dtype is _I32 and cu_q.dtype is _I32 and seq_k.dtype is _I32 \
            and block_table.get_device() == index and cu_q.get_device() == index and seq_k.get_device() == index \
            and cu_q.shape == (B + 1,) and seq_k.shape == (B,) and cu_q.is_contiguous() and seq_k.is_contiguous() \
            and (tc == 1 or max_pages < 2)
        if good and q is not None:
            t, Hq, c = q.shape
            qs, qh, qc = q.stride()
            good = t == T and c == d and q.dtype is dt and q.get_device() == index and qc == 1 and (qh == d or Hq == 1)
    except (AttributeError, TypeError, ValueError):
        good = False
    if good:
        cache = _KV_PACK(k_pages.data_ptr(), v_pages.data_ptr(), pages, page_size, heads, d, s0, s1, s2, _TYPES[dt])
    else:
        cache, heads, d, dt, index = _cache(k_pages, v_pages)
        if not isinstance(k, torch.Tensor) or k.dim() != 3:
            raise ValueError("k must be a [T, heads, d] CUDA tensor")
        T = k.shape[0]
        ks = _check_tokens("k", k, T, heads, d, dt, index)
        vs = _check_tokens("v", v, T, heads, d, dt, index)
        B, table_stride, max_pages = _check_batch(block_table, cu_q, seq_k, index)
        if q is not None:
            Hq = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1
            qs = _check_tokens("q", q, T, Hq, d, dt, index)
    if q is not None:
        if q_out is None:
            q_out = _empty((T, Hq, d), dtype=dt, device=q.device)
        else:
            _check_out("q_out", q_out, (T, Hq, d), dt, index)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    cp, sp, n, r, layout, pp = None, None, 0, 0, 0, None
    if rope is not None:
        cp, sp, n, r, layout = _check_rope(rope, d, index)
        if positions is not None:
            pp = _check_ints("positions", positions, T, index)
    elif positions is not None:
        raise ValueError("positions need rope")
    with _guard(index):
        st = _lib().fa_cache_append_at(cache, qp, k.data_ptr(), v.data_ptr(), op, qs, ks, vs, block_table.data_ptr(),
                                       table_stride, max_pages, cu_q.data_ptr(), seq_k.data_ptr(), B, T, Hq, cp, sp, n,
                                       r, layout, pp, _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_cache_append_at")
    return q_out


_SCALE_KINDS = {"none": FA_ROPE_SCALE_NONE, "linear": FA_ROPE_SCALE_LINEAR, "base": FA_ROPE_SCALE_BASE,
                "turns": FA_ROPE_SCALE_TURNS, "index": FA_ROPE_SCALE_INDEX}


def rope_table(length: int, rope_dim: int, theta: float = 10000.0, scaling=None, start: int = 0, device=None, out=None):
    """Angle tables of the positions start .. start + length - 1
    (``fa_rope_table``): (cos, sin), fp32 [length, rope_dim/2] on ``device``
    (default: the current CUDA device), or written to ``out`` = (cos, sin).
    ``scaling``: None, or a dict with ``kind`` ("none", "linear", "base",
    "turns" or "index"), ``factor``, for the last two ``original``, ``low`` and
    ``high``, and ``amplitude`` (1 unless given)."""
    sc = None
    if scaling is not None:
        more = set(scaling) - {"kind", "factor", "original", "low", "high", "amplitude"}
        if scaling.get("kind") not in _SCALE_KINDS or more:
            raise ValueError(f"scaling kind must be one of {sorted(_SCALE_KINDS)}" if not more else f"scaling has no {sorted(more)}")
        sc = _SCALING_PACK(_SCALE_KINDS[scaling["kind"]], float(scaling.get("factor", 1.0)), float(scaling.get("original", 0.0)),
                           float(scaling.get("low", 0.0)), float(scaling.get("high", 0.0)), float(scaling.get("amplitude", 1.0)))
    length, rope_dim = _count(length), _count(rope_dim)
    if out is None:
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if length < 0 or rope_dim < 0:
            raise ValueError("length and rope_dim must not be negative")
        cos = torch.empty((length, rope_dim // 2), dtype=torch.float32, device=dev)
        sin = torch.empty((length, rope_dim // 2), dtype=torch.float32, device=dev)
        index = cos.get_device()
    else:
        cos, sin = out
        index = cos.get_device() if isinstance(cos, torch.Tensor) else -1
        _check_out("cos", cos, (length, rope_dim // 2), torch.float32, index)
        _check_out("sin", sin, (length, rope_dim // 2), torch.float32, index)
    if index < 0:
        raise ValueError("rope tables are CUDA tensors")
    with _guard(index):
        st = _lib().fa_rope_table(cos.data_ptr(), sin.data_ptr(), length, rope_dim, float(theta), _count(start), sc,
                                  _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_rope_table")
    return cos, sin


def _rope_array(name, x, y, four, B, N, d, dt, index):
    """(the result, the bytes of an ``fa_rope_array``) of one array and its
    result, where one is given."""
    if isinstance(x, torch.Tensor):
        shape, st = x.shape, x.stride()
        if x.dtype is dt and x.get_device() == index and len(shape) == 3 + four:
            if four:
                b, heads, n, c = shape
                xb, xh, xn, xc = st
            else:
                n, heads, c = shape
                xn, xh, xc = st
                b, xb = 1, 0
            if b == B and n == N and c == d and (xc == 1 or x.numel() == 0):
                if y is None:
                    y = torch.empty(shape, dtype=dt, device=x.device)
                    yb, yh, yn = (heads * N * d, N * d, d) if four else (0, d, heads * d)
                elif isinstance(y, torch.Tensor) and y.shape == shape and y.dtype is dt and y.get_device() == index \
                        and (y.stride(-1) == 1 or y.numel() == 0):
                    yb, yh, yn = y.stride()[:3] if four else (0, y.stride(1), y.stride(0))
                else:
                    raise ValueError(f"{name}_out must be a {dt} {list(shape)} tensor on cuda:{index}, its last dimension contiguous")
                return y, _ROPE_PACK(x.data_ptr(), y.data_ptr(), heads, xb, xh, xn, yb, yh, yn)
    raise ValueError(f"{name} must be a {dt} {'[B, heads, N, d]' if four else '[N, heads, d]'} tensor on cuda:{index} with "
                     "q's B, N and d, its last dimension contiguous")


def rope(q: torch.Tensor, k: torch.Tensor | None, rope, positions: torch.Tensor | None = None, offset: int = 0,
         inverse: bool = False, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None):
    """Rotary positions of q and k (None: q alone) in one launch
    (``fa_rope``): both [B, heads, N, d], or both [N, heads, d], bf16 or fp16,
    with any strides but of d.  ``rope`` = (cos, sin, layout) as in
    ``cache_append``: the first rope_dim columns of a row are rotated, the others
    copied.  Token n is at ``offset`` + n, or at ``positions`` (int32 [N], or
    [B, N]).  ``inverse`` turns back, which takes gradients of the results to
    those of q and k.  Returns (q_out, k_out), contiguous unless given; q_out = q
    works in place."""
    shape = q.shape if isinstance(q, torch.Tensor) else ()
    four = len(shape) == 4
    if not (four or len(shape) == 3) or q.dtype not in _TYPES or q.get_device() < 0:
        raise ValueError("q must be a bf16 or fp16 [B, heads, N, d] or [N, heads, d] CUDA tensor")
    index, dt = q.get_device(), q.dtype
    if four:
        B, _, N, d = shape
    else:
        N, _, d = shape
        B = 1
    cp, sp, length, r, layout = _check_rope(rope, d, index)
    q_out, arrays = _rope_array("q", q, q_out, four, B, N, d, dt, index)
    if k is not None:
        k_out, more = _rope_array("k", k, k_out, four, B, N, d, dt, index)
        arrays += more
    elif k_out is not None:
        raise ValueError("k_out needs k")
    pp, ps = None, 0
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int32 or positions.get_device() != index \
                or positions.shape not in ((N,), (B, N)) or not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous int32 [{N}] or [{B}, {N}] tensor on cuda:{index}")
        pp, ps = positions.data_ptr(), N if len(positions.shape) == 2 else 0
    with _guard(index):
        st = _lib().fa_rope(arrays, 1 if k is None else 2, B, N, d, pp, ps, _count(offset), cp, sp, length, r, layout,
                            1 if inverse else 0, _TYPES[dt], _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_rope")
    return q_out, k_out


def _layers(k_pages, v_pages):
    """The ``fa_kv_cache`` of the first layer, the number of layers, the
    elements between them and the device index, of pages [num_pages, heads,
    page_size, d] or [layers, num_pages, heads, page_size, d]."""
    if isinstance(k_pages, torch.Tensor) and isinstance(v_pages, torch.Tensor) and len(k_pages.shape) == 5:
        shape, stride, dt, index = k_pages.shape, k_pages.stride(), k_pages.dtype, k_pages.get_device()
        if index >= 0 and dt in _TYPES and stride[4] == 1 and shape[0] > 0 and v_pages.shape == shape and v_pages.stride() == stride \
                and v_pages.dtype is dt and v_pages.get_device() == index:
            layers, n, h, ps, d = shape
            return _KV_PACK(k_pages.data_ptr(), v_pages.data_ptr(), n, ps, h, d, stride[1], stride[2], stride[3],
                            _TYPES[dt]), layers, stride[0], index
        raise ValueError("k_pages and v_pages must be bf16 or fp16 [layers, num_pages, heads, page_size, d] CUDA tensors of one "
                         "shape, dtype, device and strides, their last dimension contiguous")
    cache, _, _, _, index = _cache(k_pages, v_pages)
    return cache, 1, 0, index


def _check_ints(name, t, n, index):
    """The address of a contiguous int32 [n] tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _I32 or t.shape != (n,) or t.get_device() != index \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor on cuda:{index}")
    return t.data_ptr()


def _ints(name, t):
    """(entries, device index) of the 1-D int32 CUDA tensor that others are checked against."""
    if isinstance(t, torch.Tensor) and len(t.shape) == 1 and t.dtype is torch.int32 and t.get_device() >= 0 and t.is_contiguous():
        return t.shape[0], t.get_device()
    raise ValueError(f"{name} must be a contiguous 1-D int32 CUDA tensor")


def _check_table(block_table, rows, index):
    """(address, row stride, width) of a block table with ``rows`` rows."""
    if isinstance(block_table, torch.Tensor) and block_table.dtype is torch.int32 and block_table.get_device() == index:
        shape, st = block_table.shape, block_table.stride()
        if len(shape) == 2 and shape[0] == rows and (st[1] == 1 or shape[1] < 2):
            return block_table.data_ptr(), st[0], shape[1]
    raise ValueError(f"block_table must be an int32 [{rows}, max_pages] tensor on cuda:{index}, each row contiguous")


def pages_resize(refs: torch.Tensor, block_table: torch.Tensor, seq_k: torch.Tensor, want: torch.Tensor, page_size: int):
    """Rows of a block table give back pages or get free ones
    (``fa_pages_resize``), in place: refs [num_pages] (0: a free page),
    block_table [B, max_pages], seq_k [B] the tokens that a row holds pages for,
    want [B] those that it shall, all int32.  Afterwards seq_k is want, or less
    where the pages ran out."""
    pages, index = _ints("refs", refs)
    B, _ = _ints("seq_k", seq_k)
    sp, wp = _check_ints("seq_k", seq_k, B, index), _check_ints("want", want, B, index)
    tp, stride, width = _check_table(block_table, B, index)
    with _guard(index):
        st = _lib().fa_pages_resize(refs.data_ptr(), pages, _count(page_size), tp, stride, width, sp, wp, B, _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_pages_resize")


def pages_fork(k_pages: torch.Tensor, v_pages: torch.Tensor, refs: torch.Tensor, block_table: torch.Tensor,
               seq_k: torch.Tensor, src: torch.Tensor, dst: torch.Tensor):
    """Row dst[i] becomes a second copy of the sequence in row src[i]
    (``fa_pages_fork``), in place: it shares the full pages and gets a copy of the
    last, partly filled one.  Pages as in ``fwd_paged``, or of all layers [layers,
    num_pages, heads, page_size, d]; refs [num_pages], block_table [rows,
    max_pages], seq_k [rows], src and dst [n], int32.  Rows dst are empty before
    (seq_k 0), not among src and given once.  Returns fresh [n]: the page that a
    fork got, -1: none was needed, -2: refused, -3: no page was left."""
    cache, layers, layer_stride, index = _layers(k_pages, v_pages)
    n, rows = _ints("src", src)[0], _ints("seq_k", seq_k)[0]
    rp = _check_ints("refs", refs, k_pages.shape[-4], index)
    kp, ap, bp = _check_ints("seq_k", seq_k, rows, index), _check_ints("src", src, n, index), _check_ints("dst", dst, n, index)
    tp, stride, width = _check_table(block_table, rows, index)
    fresh = torch.empty_like(src)
    with _guard(index):
        st = _lib().fa_pages_fork(cache, layers, layer_stride, rp, tp, stride, width, kp, rows, ap, bp, fresh.data_ptr(), n,
                                  _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_pages_fork")
    return fresh


def cache_copy(k_pages: torch.Tensor, v_pages: torch.Tensor, src: torch.Tensor, dst: torch.Tensor):
    """Copies page src[i] to page dst[i] (``fa_cache_copy``), keys and values of
    all layers (pages as in ``pages_fork``); src and dst int32 [n], no page twice
    in dst or in both."""
    cache, layers, layer_stride, index = _layers(k_pages, v_pages)
    n, _ = _ints("src", src)
    ap, bp = _check_ints("src", src, n, index), _check_ints("dst", dst, n, index)
    with _guard(index):
        st = _lib().fa_cache_copy(cache, layers, layer_stride, ap, bp, n, _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_cache_copy")


def cache_compact(k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, first: torch.Tensor,
                  keep: torch.Tensor, keep_n: torch.Tensor):
    """Moves the kept tokens of each sequence together (``fa_cache_compact``), in
    place: for i < keep_n[b], position keep[b, i] goes to position first[b] + i,
    in all layers (pages as in ``pages_fork``).  block_table [B, max_pages], first
    [B], keep [B, max_keep] with keep[b, i] >= first[b] + i (any ascending list
    from first[b] on), keep_n [B], int32.  Returns the new lengths first + keep_n."""
    cache, layers, layer_stride, index = _layers(k_pages, v_pages)
    B, _ = _ints("first", first)
    fp, np = _check_ints("first", first, B, index), _check_ints("keep_n", keep_n, B, index)
    tp, stride, width = _check_table(block_table, B, index)
    try:
        kp, kept, most = _check_table(keep, B, index)
    except ValueError:
        raise ValueError(f"keep must be an int32 [{B}, max_keep] tensor on cuda:{index}, each row contiguous") from None
    seq_k = torch.empty_like(first)
    with _guard(index):
        st = _lib().fa_cache_compact(cache, layers, layer_stride, tp, stride, width, fp, kp, kept, most, np, seq_k.data_ptr(), B,
                                     _current_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_cache_compact")
    return seq_k


def fwd_fp8_gqa(q8, k8, v8, q_descale, k_descale, v_descale, causal: bool = False,
                scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None):
    """FP8 E4M3 version of ``fwd_gqa`` (``fa_fwd_fp8_gqa``); descales are
    [B, Hq, ceil(Nq/128)] for Q and [B, Hkv, ceil(Nk/128)] for K and V."""
    _check_gqa(q8, k8, v8, (torch.uint8, torch.float8_e4m3fn))
    B, Hq, Nq, d = q8.shape
    Hkv, Nk = k8.shape[1], k8.shape[2]
    nq, nk = (Nq + FP8_BLOCK_ROWS - 1) // FP8_BLOCK_ROWS, (Nk + FP8_BLOCK_ROWS - 1) // FP8_BLOCK_ROWS
    for name, t, shape in (("q_descale", q_descale, (B, Hq, nq)), ("k_descale", k_descale, (B, Hkv, nk)),
                           ("v_descale", v_descale, (B, Hkv, nk))):
        if t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous() or t.device != q8.device:
            raise ValueError(f"{name} must be a contiguous fp32 {list(shape)} tensor on {q8.device}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, Hq, Nq, d), dtype=torch.bfloat16, device=q8.device)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q8.device)
    with torch.cuda.device(q8.device):
        st = _lib().fa_fwd_fp8_gqa(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                   B, Hq, Hkv, Nq, Nk, d, int(bool(causal)), float(scale), q_descale.data_ptr(),
                                   k_descale.data_ptr(), v_descale.data_ptr(), _stream(q8))
    _check(st, "fa_fwd_fp8_gqa")
    return out, lse


def fwd_fp8(q8: torch.Tensor, k8: torch.Tensor, v8: torch.Tensor, q_descale: torch.Tensor,
            k_descale: torch.Tensor, v_descale: torch.Tensor, causal: bool = False,
            scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None):
    """FP8 E4M3 attention forward (``fa_fwd_fp8``).  q8/k8/v8 hold E4M3 codes
    (uint8 or float8_e4m3fn), descales are [B, H, ceil(N/128)] fp32.
    Returns (O bf16, LSE fp32)."""
    _check_qkv(q8, k8, v8, (torch.uint8, torch.float8_e4m3fn))
    B, H, N, d = q8.shape
    nblk = (N + FP8_BLOCK_ROWS - 1) // FP8_BLOCK_ROWS
    for name, t in (("q_descale", q_descale), ("k_descale", k_descale), ("v_descale", v_descale)):
        if t.dtype != torch.float32 or tuple(t.shape) != (B, H, nblk) or not t.is_contiguous() or \
                t.device != q8.device:
            raise ValueError(f"{name} must be a contiguous fp32 [B, H, {nblk}] tensor on {q8.device}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    with torch.cuda.device(q8.device):
        st = _lib().fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), out.data_ptr(), lse.data_ptr(),
                               B, H, N, d, int(bool(causal)), float(scale), q_descale.data_ptr(),
                               k_descale.data_ptr(), v_descale.data_ptr(), _stream(q8))
    _check(st, "fa_fwd_fp8")
    return out, lse


def quant_fp8(x: torch.Tensor, signs=None, per_tensor: bool = False, workspace: torch.Tensor | None = None,
              rope=None):
    """fp32 [B, H, N, d] -> (E4M3 codes uint8 [B, H, N, d], descale fp32
    [B, H, ceil(N/128)]) via ``fa_quant_fp8``.  ``signs``: d entries of +-1
    (host sequence / numpy / CPU tensor) for the Hadamard rotation, or None.
    ``rope``: None, or (cos, sin, layout) with cos / sin contiguous fp32 CUDA
    tensors [N, d/2] and layout FA_ROPE_INTERLEAVED or FA_ROPE_HALF: the
    rotary embedding is applied first, in the same pass (``fa_quant_fp8_rope``)."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.float32 or x.dim() != 4 \
            or not x.is_contiguous():
        raise ValueError("x must be a contiguous fp32 [B, H, N, d] CUDA tensor")
    B, H, N, d = x.shape
    nblk = (N + FP8_BLOCK_ROWS - 1) // FP8_BLOCK_ROWS
    x8 = torch.empty((B, H, N, d), dtype=torch.uint8, device=x.device)
    ds = torch.empty((B, H, nblk), dtype=torch.float32, device=x.device)
    sp = None
    keep = None
    if signs is not None:
        keep = (ctypes.c_int8 * d)(*[int(s) for s in (signs.tolist() if hasattr(signs, "tolist") else signs)])
        sp = ctypes.cast(keep, ctypes.c_void_p)
    ws = None
    if per_tensor:
        if workspace is None:
            workspace = torch.empty((1,), dtype=torch.float32, device=x.device)
        ws = workspace.data_ptr()
    with torch.cuda.device(x.device):
        if rope is None:
            st = _lib().fa_quant_fp8(x.data_ptr(), x8.data_ptr(), ds.data_ptr(), B, H, N, d, sp,
                                     int(bool(per_tensor)), ws, _stream(x))
            name = "fa_quant_fp8"
        else:
            cos, sin, layout = rope
            for nm, t in (("cos", cos), ("sin", sin)):
                if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 \
                        or not t.is_contiguous() or tuple(t.shape) != (N, d // 2) or t.device != x.device:
                    raise ValueError(f"rope {nm} must be a contiguous fp32 [N, d/2] tensor on x's device")
            st = _lib().fa_quant_fp8_rope(x.data_ptr(), x8.data_ptr(), ds.data_ptr(), B, H, N, d,
                                          cos.data_ptr(), sin.data_ptr(), int(layout), sp,
                                          int(bool(per_tensor)), ws, _stream(x))
            name = "fa_quant_fp8_rope"
    _check(st, name)
    del keep
    return x8, ds


def quant_fp8_qkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, signs=None, out=None):
    """The FP8 inputs of one attention call (``fa_quant_fp8_qkv``): Q and K
    with block scales after the rotation given by ``signs`` (or none), V with
    block scales, the three on internal streams joined back into the current
    stream.  q: fp32 [B, Hq, Nq, d]; k, v: fp32 [B, Hkv, Nk, d].  Returns
    (q8, k8, v8, q_descale, k_descale, v_descale), each as ``quant_fp8``
    would give it; ``out`` may supply those six tensors (written in place)."""
    for nm, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 or t.dim() != 4 \
                or not t.is_contiguous() or t.device != q.device:
            raise ValueError(f"{nm} must be a contiguous fp32 [B, H, N, d] CUDA tensor on q's device")
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Bk != B or dk != d:
        raise ValueError("k and v must be [B, Hkv, Nk, d] with q's B and d")
    shapes_ds = [(B, Hq, (Nq + FP8_BLOCK_ROWS - 1) // FP8_BLOCK_ROWS)] + \
                [(B, Hkv, (Nk + FP8_BLOCK_ROWS - 1) // FP8_BLOCK_ROWS)] * 2
    if out is None:
        outs = [torch.empty(t.shape, dtype=torch.uint8, device=q.device) for t in (q, k, v)]
        ds = [torch.empty(sh, dtype=torch.float32, device=q.device) for sh in shapes_ds]
    else:
        outs, ds = list(out[:3]), list(out[3:])
        for t, ref in zip(outs, (q, k, v)):
            if t.dtype != torch.uint8 or tuple(t.shape) != tuple(ref.shape) or not t.is_contiguous() \
                    or t.device != q.device:
                raise ValueError("code outputs must be contiguous uint8 tensors shaped like q, k, v")
        for t, sh in zip(ds, shapes_ds):
            if t.dtype != torch.float32 or tuple(t.shape) != sh or not t.is_contiguous() or t.device != q.device:
                raise ValueError(f"descale outputs must be contiguous fp32 {sh}")
    sp = None
    keep = None
    if signs is not None:
        keep = (ctypes.c_int8 * d)(*[int(s) for s in (signs.tolist() if hasattr(signs, "tolist") else signs)])
        sp = ctypes.cast(keep, ctypes.c_void_p)
    with torch.cuda.device(q.device):
        st = _lib().fa_quant_fp8_qkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), *[t.data_ptr() for t in outs],
                                     *[t.data_ptr() for t in ds], B, Hq, Hkv, Nq, Nk, d, sp, _stream(q))
    _check(st, "fa_quant_fp8_qkv")
    del keep
    return outs[0], outs[1], outs[2], ds[0], ds[1], ds[2]


def quant_fp8_per_tensor_noalloc(x: torch.Tensor, signs=None, x8: torch.Tensor | None = None,
                                 descale: torch.Tensor | None = None):
    """Per-tensor FP8 quantisation through ``fa_quant_fp8_per_tensor_noalloc``:
    the library uses its own static device scratch, so the call itself needs
    no allocation (pass ``x8`` and ``descale`` to avoid torch allocating the
    outputs too).  Same result as ``quant_fp8(x, signs, per_tensor=True)``.
    Calls that overlap on the GPU share the scratch and race."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.float32 or x.dim() != 4 \
            or not x.is_contiguous():
        raise ValueError("x must be a contiguous fp32 [B, H, N, d] CUDA tensor")
    B, H, N, d = x.shape
    nblk = (N + FP8_BLOCK_ROWS - 1) // FP8_BLOCK_ROWS
    if x8 is None:
        x8 = torch.empty((B, H, N, d), dtype=torch.uint8, device=x.device)
    if descale is None:
        descale = torch.empty((B, H, nblk), dtype=torch.float32, device=x.device)
    keep = None
    sp = None
    if signs is not None:
        keep = (ctypes.c_int8 * d)(*[int(s) for s in (signs.tolist() if hasattr(signs, "tolist") else signs)])
        sp = ctypes.cast(keep, ctypes.c_void_p)
    with torch.cuda.device(x.device):
        st = _lib().fa_quant_fp8_per_tensor_noalloc(x.data_ptr(), x8.data_ptr(), descale.data_ptr(),
                                                    B, H, N, d, sp, _stream(x))
    _check(st, "fa_quant_fp8_per_tensor_noalloc")
    del keep
    return x8, descale


def check_device_error(device=None):
    """Synchronise the current stream and raise FaError if a kernel reported a
    pipeline timeout (FA_ERR_TIMEOUT), or an index out of range in device memory
    (FA_ERR_INDEX), that no check has reported yet."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        st = _lib().fa_check_device_error(torch.cuda.current_stream(dev).cuda_stream)
    _check(st, "fa_check_device_error")
