"""Thin ctypes binding over ``libsage.so`` (declared in ``include/sage.h``).

The binding marshals torch tensors into pointers, sizes and the current CUDA
stream; every step of the computation runs in the library's CUDA kernels.
There is no fallback: if the library is missing or a call fails, a
``SageError`` is raised.

Accepted inputs mirror the kernel contract of diffusers issue #15014
("gfx1201 (RDNA4) SageAttention attention backend", kernel contract bullets):
BF16 Q/K/V of equal shape [B, S, H, 128], no mask, non-causal.  Anything else
(another dtype, head dim, layout or device) is rejected with a clear error, as
that issue's "Describe the solution you'd like" asks.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libsage.so")
HEAD_DIM = 128

_STATUS = {
    0: "SAGE_OK", 1: "SAGE_ERR_INVALID_ARG", 2: "SAGE_ERR_UNSUPPORTED", 3: "SAGE_ERR_MISALIGNED",
    4: "SAGE_ERR_CUDA", 5: "SAGE_ERR_NO_MEMORY", 6: "SAGE_ERR_TIMEOUT", 7: "SAGE_ERR_WORKSPACE",
    8: "SAGE_ERR_BAD_PAGE", 9: "SAGE_ERR_NO_PAGES",
}
EXPORTED = (
    "sage_padded_len", "sage_workspace_bytes", "sage_quantize_qkv", "sage_attn_fwd",
    "sage_attn_fwd_ws", "sage_attn_fwd_quantized", "sage_debug_qk_int32",
    "sage_debug_wait_timeout", "sage_sync_status", "sage_set_wait_timeout_ns",
    "sage_last_error", "sage_status_string", "sage_set_attention_events",
    "sage_quantize_qkv_noalloc", "sage_attn_fwd_lse", "sage_attn_fwd_cross",
    "sage_debug_fused_q", "sage_attn_fwd_fused_q", "sage_quantize_qkv_smooth_k",
    "sage_attn_fwd_smooth_k", "sage_attn_fwd_launches", "sage_debug_staging_codes",
    "sage_debug_inject_fault", "sage_debug_pool_state", "sage_plan_create", "sage_plan_launch",
    "sage_plan_destroy", "sage_plan_create_ex", "sage_kv_cache_write", "sage_kv_cache_read",
    "sage_attn_fwd_cache", "sage_attn_fwd_cache_prefix", "sage_attn_fwd_cache_workspace_bytes",
    "sage_kv4_cache_write", "sage_kv4_cache_read", "sage_attn_fwd_kv4_cache", "sage_attn_fwd_kv4_cache_prefix",
    "sage_rope_frequencies", "sage_rope_frequency", "sage_qk_norm_rope", "sage_kv_cache_append",
    "sage_kv4_cache_append", "sage_kv_pages_reserve", "sage_kv_pages_release",
)

# Options of sage_plan_create_ex (include/sage.h).
PLAN_SMOOTH_K, PLAN_FUSED_Q = 1, 2

# Fault sites of sage_debug_inject_fault (include/sage.h).
FAULT_NONE, FAULT_POOL_ALLOC, FAULT_QUANT_LAUNCH, FAULT_ATTN_LAUNCH = 0, 1, 2, 3


# Page sizes of the quantised KV cache (include/sage.h).
KV_PAGE_SIZES = (16, 32, 64, 128, 256)


class _KVCache(ctypes.Structure):
    """sage_kv_cache (include/sage.h)."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("H", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class _KV4Cache(ctypes.Structure):
    """sage_kv4_cache (include/sage.h)."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_block", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_block", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("H", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    """sage_rope (include/sage.h)."""
    _fields_ = [("freq", ctypes.c_void_p), ("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4), ("factor", ctypes.c_float)]


class SageError(RuntimeError):
    """A non-zero sage_status, with the library's message."""

    def __init__(self, status: int, message: str):
        self.status = status
        self.name = _STATUS.get(status, f"status {status}")
        super().__init__(f"{self.name}: {message}")


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load libsage.so and declare its signatures (no CUDA call is made)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m quantized_attention_diffusion_gb300.build`")
        lib = ctypes.CDLL(path)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        S, L, D = ctypes.c_int, ctypes.c_int64, ctypes.c_double
        sigs = {
            "sage_padded_len": (ctypes.c_int64, [I]),
            "sage_attn_fwd_launches": (I, [I, I, I, I, I]),
            "sage_workspace_bytes": (Z, [I, I, I, I]),
            "sage_quantize_qkv": (S, [P, P, P, I, I, I, I, P, P, P, P, P, P, P]),
            "sage_quantize_qkv_noalloc": (S, [P, P, P, I, I, I, I, P, P, P, P, P, P, P]),
            "sage_attn_fwd": (S, [P, P, P, P, I, I, I, I, F, P]),
            "sage_attn_fwd_ws": (S, [P, P, P, P, I, I, I, I, F, P, Z, P]),
            "sage_attn_fwd_lse": (S, [P, P, P, P, P, I, I, I, I, F, P]),
            "sage_attn_fwd_cross": (S, [P, P, P, P, P, I, I, I, I, I, F, P]),
            "sage_plan_create": (S, [P, P, P, P, P, I, I, I, I, I, F, P]),
            "sage_plan_create_ex": (S, [P, P, P, P, P, I, I, I, I, I, F, ctypes.c_uint, P]),
            "sage_plan_launch": (S, [P, P]),
            "sage_plan_destroy": (S, [P]),
            "sage_debug_fused_q": (S, [P, P, P, P, I, I, I, I, F, P, P, P]),
            "sage_attn_fwd_fused_q": (S, [P, P, P, P, I, I, I, I, F, P]),
            "sage_quantize_qkv_smooth_k": (S, [P, P, P, I, I, I, I, P, P, P, P, P, P, P, P]),
            "sage_attn_fwd_smooth_k": (S, [P, P, P, P, I, I, I, I, F, P]),
            "sage_attn_fwd_quantized": (S, [P, P, P, P, P, P, P, I, I, I, I, F, P, Z, P]),
            "sage_debug_qk_int32": (S, [P, P, P, P, P, P, P, P, I, I, I, I, F, P, Z, P]),
            "sage_debug_wait_timeout": (S, [ctypes.c_uint64, P]),
            "sage_debug_staging_codes": (S, [P, P, I, I, I, I, P, P, P, P, P]),
            "sage_debug_inject_fault": (S, [I, I]),
            "sage_debug_pool_state": (S, [P, P]),
            "sage_kv_cache_write": (S, [P, P, P, L, L, L, L, I, I, I, P, I, L, P, P, P]),
            "sage_kv_cache_read": (S, [P, P, I, L, P, P, P, I, I, I, P]),
            "sage_attn_fwd_cache": (S, [P, L, L, P, P, I, L, P, P, P, I, I, I, I, F, I, P, Z, P]),
            "sage_attn_fwd_cache_prefix": (S, [P, L, L, P, P, I, P, I, L, P, P, P, I, I, I, I, F, I, P, Z, P]),
            "sage_attn_fwd_cache_workspace_bytes": (Z, [I, I, I, I, I]),
            "sage_kv4_cache_write": (S, [P, P, P, L, L, L, L, I, I, I, P, I, L, P, P, P]),
            "sage_kv4_cache_read": (S, [P, P, I, L, P, P, P, I, I, I, P]),
            "sage_attn_fwd_kv4_cache": (S, [P, L, L, P, P, I, L, P, P, P, I, I, I, I, F, I, P, Z, P]),
            "sage_attn_fwd_kv4_cache_prefix": (S, [P, L, L, P, P, I, P, I, L, P, P, P, I, I, I, I, F, I, P, Z, P]),
            "sage_rope_frequencies": (S, [I, D, I, D, D, D, D, P, P]),
            "sage_rope_frequency": (ctypes.c_uint64, [D]),
            "sage_qk_norm_rope": (S, [P, P, L, L, L, L, I, I, I, I, I, P, P, L, L, P, P, F, P, P, P]),
            "sage_kv_cache_append": (S, [P, P, P, P, L, L, L, L, L, L, I, I, I, I, P, P, L, L, P, P, F, P, P, P]),
            "sage_kv4_cache_append": (S, [P, P, P, P, L, L, L, L, L, L, I, I, I, I, P, P, L, L, P, P, F, P, P, P]),
            "sage_kv_pages_reserve": (S, [P, P, I, I, P, P, I, P, I, L, I, I, P, P, P, P, P, P, P, P]),
            "sage_kv_pages_release": (S, [P, P, I, I, P, P, I, P, I, L, P]),
            "sage_sync_status": (S, [P]),
            "sage_set_wait_timeout_ns": (None, [ctypes.c_uint64]),
            "sage_set_attention_events": (None, [P, P]),
            "sage_last_error": (ctypes.c_char_p, []),
            "sage_status_string": (ctypes.c_char_p, [S]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _check(status: int):
    if status != 0:
        msg = _lib.sage_last_error().decode(errors="replace")
        raise SageError(status, msg)


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _check_qkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bfloat16 (got {t.dtype})")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [B, S, H, D] (got {tuple(t.shape)})")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous in [B, S, H, D] order")
    if not (q.shape == k.shape == v.shape):
        raise ValueError(f"Q, K and V must have equal shapes (got {tuple(q.shape)}, "
                         f"{tuple(k.shape)}, {tuple(v.shape)})")
    if not (q.device == k.device == v.device):
        raise ValueError("Q, K and V must be on one device")
    B, S, H, D = q.shape
    return B, S, H, D


def padded_len(S: int) -> int:
    return int(load_library().sage_padded_len(S))


def attn_fwd_launches(B: int, Sq: int, H: int, Skv: int | None = None, smooth_k: bool = False) -> int:
    """Kernels one sage_attn_fwd (or _lse, _cross, _fused_q; _smooth_k with
    smooth_k) call launches for this shape."""
    n = int(load_library().sage_attn_fwd_launches(B, Sq, Sq if Skv is None else Skv, H, int(smooth_k)))
    if n < 0:
        raise ValueError(f"invalid shape B={B} Sq={Sq} Skv={Skv} H={H}")
    return n


def workspace_bytes(B: int, S: int, H: int, D: int = HEAD_DIM) -> int:
    return int(load_library().sage_workspace_bytes(B, S, H, D))


def attn_fwd(q, k, v, softmax_scale: float | None = None, out=None, workspace=None, fused_q=False,
             smooth_k=False):
    """Quantized attention forward: bf16 [B, S, H, 128] -> bf16 [B, S, H, 128].

    ``workspace`` (optional uint8 CUDA tensor of >= workspace_bytes) selects
    sage_attn_fwd_ws; otherwise the library's stream-ordered pool is used.
    ``fused_q`` selects sage_attn_fwd_fused_q (Q quantised in the attention
    kernel; same result); ``smooth_k`` selects sage_attn_fwd_smooth_k (K loses
    its per-channel mean before quantisation).
    """
    lib = load_library()
    B, S, H, D = _check_qkv(q, k, v)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    with torch.cuda.device(q.device):
        st = _stream(q.device)
        if smooth_k:
            _check(lib.sage_attn_fwd_smooth_k(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, S, H, D,
                                              float(softmax_scale), st))
        elif fused_q:
            _check(lib.sage_attn_fwd_fused_q(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, S, H, D,
                                             float(softmax_scale), st))
        elif workspace is None:
            _check(lib.sage_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, S, H, D,
                                     float(softmax_scale), st))
        else:
            _check(lib.sage_attn_fwd_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, S, H, D,
                                        float(softmax_scale), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), st))
    return out


def attn_fwd_lse(q, k, v, softmax_scale: float | None = None, out=None, lse=None):
    """attn_fwd that also returns each query row's log-sum-exp.

    Returns (out bf16 [B, S, H, 128], lse fp32 [B, H, S]); ``out`` and
    ``lse`` may be given to be filled (sage_attn_fwd_lse).
    """
    lib = load_library()
    B, S, H, D = _check_qkv(q, k, v)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, S) or not lse.is_contiguous() \
            or lse.device != q.device:
        raise ValueError("lse must be a contiguous float32 [B, H, S] tensor on q's device")
    with torch.cuda.device(q.device):
        _check(lib.sage_attn_fwd_lse(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, S, H, D,
                                     float(softmax_scale), _stream(q.device)))
    return out, lse


def attn_fwd_cross(q, k, v, softmax_scale: float | None = None, out=None, lse=None,
                   return_lse: bool = False):
    """Cross-attention: q bf16 [B, Sq, H, 128], k and v bf16 [B, Skv, H, 128]
    -> out bf16 [B, Sq, H, 128] (and lse fp32 [B, H, Sq] with return_lse or
    when ``lse`` is given), through sage_attn_fwd_cross."""
    lib = load_library()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda \
                or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor [B, S, H, D]")
    B, Sq, H, D = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[2] != H or k.shape[3] != D:
        raise ValueError(f"k and v must be [B, Skv, H, D] with B, H, D of q; got {tuple(k.shape)}, "
                         f"{tuple(v.shape)} for q {tuple(q.shape)}")
    if k.device != q.device or v.device != q.device:
        raise ValueError("q, k and v must be on one device")
    Skv = k.shape[1]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Sq)
                            or not lse.is_contiguous() or lse.device != q.device):
        raise ValueError("lse must be a contiguous float32 [B, H, Sq] tensor on q's device")
    with torch.cuda.device(q.device):
        _check(lib.sage_attn_fwd_cross(_ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                       _ptr(lse) if lse is not None else None, B, Sq, Skv, H, D,
                                       float(softmax_scale), _stream(q.device)))
    return (out, lse) if lse is not None else out


class Plan:
    """One fixed attention call recorded as a CUDA graph (sage_plan_create_ex):
    q bf16 [B, Sq, H, 128], k and v bf16 [B, Skv, H, 128] (Skv = Sq for
    self-attention), out bf16 [B, Sq, H, 128] and optionally lse fp32
    [B, H, Sq], all fixed at creation.  ``smooth_k`` records attn_fwd_smooth_k
    instead and ``fused_q`` attn_fwd_fused_q (self-attention without lse, one
    at a time).  ``launch()`` replays the call on the current stream, reading
    q, k and v as they are then; launches of one plan must not overlap (one
    stream, or ordered).  ``close()`` (or leaving a ``with`` block) releases
    the graph and its workspace."""

    def __init__(self, q, k, v, softmax_scale: float | None = None, out=None, lse=None, smooth_k: bool = False,
                 fused_q: bool = False):
        lib = load_library()
        for name, t in (("q", q), ("k", k), ("v", v)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda \
                    or not t.is_contiguous() or t.dim() != 4:
                raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor [B, S, H, D]")
        B, Sq, H, D = q.shape
        if k.shape != v.shape or k.shape[0] != B or k.shape[2] != H or k.shape[3] != D:
            raise ValueError(f"k and v must be [B, Skv, H, D] with B, H, D of q; got {tuple(k.shape)}, "
                             f"{tuple(v.shape)} for q {tuple(q.shape)}")
        if k.device != q.device or v.device != q.device:
            raise ValueError("q, k and v must be on one device")
        if softmax_scale is None:
            softmax_scale = 1.0 / math.sqrt(D)
        if out is None:
            out = torch.empty_like(q)
        if out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous() or out.device != q.device:
            raise ValueError("out must be a contiguous bf16 tensor of q's shape on q's device")
        if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Sq)
                                or not lse.is_contiguous() or lse.device != q.device):
            raise ValueError("lse must be a contiguous float32 [B, H, Sq] tensor on q's device")
        self.q, self.k, self.v, self.out, self.lse = q, k, v, out, lse   # kept alive with the graph
        self.device = q.device
        self._lib = lib
        self._h = ctypes.c_void_p(0)
        with torch.cuda.device(q.device):
            flags = (PLAN_SMOOTH_K if smooth_k else 0) | (PLAN_FUSED_Q if fused_q else 0)
            _check(lib.sage_plan_create_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                           _ptr(lse) if lse is not None else None, B, Sq, k.shape[1], H, D,
                                           float(softmax_scale), flags, ctypes.byref(self._h)))

    def launch(self):
        if not self._h:
            raise RuntimeError("plan is closed")
        with torch.cuda.device(self.device):
            _check(self._lib.sage_plan_launch(self._h, _stream(self.device)))
        return self.out

    def close(self):
        if self._h:
            with torch.cuda.device(self.device):
                st = self._lib.sage_plan_destroy(self._h)
            self._h = ctypes.c_void_p(0)
            _check(st)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            if self._h and self._lib is not None:
                self._lib.sage_plan_destroy(self._h)
                self._h = ctypes.c_void_p(0)
        except Exception:
            pass


def debug_fused_q(q, k, v, softmax_scale: float | None = None):
    """Run sage_attn_fwd's path and return (out, q_i8 [B,H,S_pad,D],
    q_scale [B,H,nb]): the Q codes and scales the attention kernel computed."""
    lib = load_library()
    B, S, H, D = _check_qkv(q, k, v)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    Sp = padded_len(S)
    nb = (S + 31) // 32
    out = torch.empty_like(q)
    q_i8 = torch.zeros((B, H, Sp, D), dtype=torch.int8, device=q.device)
    q_scale = torch.zeros((B, H, nb), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        _check(lib.sage_debug_fused_q(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, S, H, D, float(softmax_scale),
                                      _ptr(q_i8), _ptr(q_scale), _stream(q.device)))
    return out, q_i8, q_scale


def quantize_qkv(q, k, v, out=None, noalloc=False):
    """Returns (q_i8 [B,H,S_pad,D], q_scale [B,H,nb], k_i8, k_scale,
    vt_fp8 uint8 [B,H,D,S_pad], v_scale [B,H,D]).

    ``out`` (optional) is a tuple of those six tensors to fill.  With
    ``noalloc`` the call goes to sage_quantize_qkv_noalloc, which uses the
    library's built-in scratch instead of allocating (B*H <= 8192)."""
    lib = load_library()
    if out is not None:
        B, S, H, D = _check_qkv(q, k, v)
        q_i8, q_sc, k_i8, k_sc, vt, v_sc = out
        fn = lib.sage_quantize_qkv_noalloc if noalloc else lib.sage_quantize_qkv
        with torch.cuda.device(q.device):
            _check(fn(_ptr(q), _ptr(k), _ptr(v), B, S, H, D, _ptr(q_i8), _ptr(q_sc), _ptr(k_i8),
                      _ptr(k_sc), _ptr(vt), _ptr(v_sc), _stream(q.device)))
        return out
    B, S, H, D = _check_qkv(q, k, v)
    Sp = padded_len(S)
    nb = (S + 31) // 32
    dev = q.device
    q_i8 = torch.empty((B, H, Sp, D), dtype=torch.int8, device=dev)
    k_i8 = torch.empty_like(q_i8)
    q_sc = torch.empty((B, H, nb), dtype=torch.float32, device=dev)
    k_sc = torch.empty_like(q_sc)
    vt = torch.empty((B, H, D, Sp), dtype=torch.uint8, device=dev)
    v_sc = torch.empty((B, H, D), dtype=torch.float32, device=dev)
    fn = lib.sage_quantize_qkv_noalloc if noalloc else lib.sage_quantize_qkv
    with torch.cuda.device(dev):
        _check(fn(_ptr(q), _ptr(k), _ptr(v), B, S, H, D, _ptr(q_i8), _ptr(q_sc),
                  _ptr(k_i8), _ptr(k_sc), _ptr(vt), _ptr(v_sc), _stream(dev)))
    return q_i8, q_sc, k_i8, k_sc, vt, v_sc


def quantize_qkv_smooth_k(q, k, v):
    """sage_quantize_qkv_smooth_k: returns (q_i8, q_scale, k_i8, k_scale,
    vt_fp8, v_scale, k_mean [B,H,D]) with K smoothed before quantisation."""
    lib = load_library()
    B, S, H, D = _check_qkv(q, k, v)
    Sp = padded_len(S)
    nb = (S + 31) // 32
    dev = q.device
    q_i8 = torch.empty((B, H, Sp, D), dtype=torch.int8, device=dev)
    k_i8 = torch.empty_like(q_i8)
    q_sc = torch.empty((B, H, nb), dtype=torch.float32, device=dev)
    k_sc = torch.empty_like(q_sc)
    vt = torch.empty((B, H, D, Sp), dtype=torch.uint8, device=dev)
    v_sc = torch.empty((B, H, D), dtype=torch.float32, device=dev)
    k_mean = torch.empty((B, H, D), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(lib.sage_quantize_qkv_smooth_k(_ptr(q), _ptr(k), _ptr(v), B, S, H, D, _ptr(q_i8), _ptr(q_sc),
                                              _ptr(k_i8), _ptr(k_sc), _ptr(vt), _ptr(v_sc), _ptr(k_mean),
                                              _stream(dev)))
    return q_i8, q_sc, k_i8, k_sc, vt, v_sc, k_mean


def _quant_shape(q_i8, S):
    B, H, Sp, D = q_i8.shape
    if q_i8.dtype != torch.int8 or not q_i8.is_cuda or not q_i8.is_contiguous():
        raise ValueError("q_i8 must be a contiguous int8 CUDA tensor [B, H, S_pad, D]")
    if Sp != padded_len(S):
        raise ValueError(f"S_pad {Sp} does not match S {S}")
    return B, H, D


def attn_fwd_quantized(quant, S: int, softmax_scale: float, out=None, workspace=None,
                       s_out=None):
    """Attention from sage_quantize_qkv outputs.  quant = (q_i8, q_scale,
    k_i8, k_scale, vt_fp8, v_scale).  With ``s_out`` (int32 [B,H,S,S]) the
    debug entry also dumps the integer QK^T accumulators."""
    lib = load_library()
    q_i8, q_sc, k_i8, k_sc, vt, v_sc = quant
    B, H, D = _quant_shape(q_i8, S)
    dev = q_i8.device
    if out is None:
        out = torch.empty((B, S, H, D), dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = torch.empty(workspace_bytes(B, S, H, D), dtype=torch.uint8, device=dev)
    nbytes = workspace.numel() * workspace.element_size()
    with torch.cuda.device(dev):
        st = _stream(dev)
        if s_out is None:
            _check(lib.sage_attn_fwd_quantized(_ptr(q_i8), _ptr(q_sc), _ptr(k_i8), _ptr(k_sc),
                                               _ptr(vt), _ptr(v_sc), _ptr(out), B, S, H, D,
                                               float(softmax_scale), _ptr(workspace), nbytes, st))
        else:
            _check(lib.sage_debug_qk_int32(_ptr(q_i8), _ptr(q_sc), _ptr(k_i8), _ptr(k_sc),
                                           _ptr(vt), _ptr(v_sc), _ptr(out), _ptr(s_out), B, S, H,
                                           D, float(softmax_scale), _ptr(workspace), nbytes, st))
    return out


def debug_qk_int32(quant, S: int, softmax_scale: float):
    """(out bf16 [B,S,H,D], s int32 [B,H,S,S]) from the debug entry point."""
    q_i8 = quant[0]
    B, H, _, D = q_i8.shape
    s_out = torch.empty((B, H, S, S), dtype=torch.int32, device=q_i8.device)
    out = attn_fwd_quantized(quant, S, softmax_scale, s_out=s_out)
    return out, s_out


def debug_wait_timeout(timeout_ns: int, device=None):
    """Launch the bounded-wait probe; returns the status sync_status() reports."""
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        st = _stream(dev)
        _check(lib.sage_debug_wait_timeout(int(timeout_ns), st))
        return int(lib.sage_sync_status(st))


def sync_status(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device error status."""
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return int(lib.sage_sync_status(_stream(dev)))


def set_wait_timeout_ns(ns: int):
    load_library().sage_set_wait_timeout_ns(int(ns))


def set_attention_events(before=None, after=None):
    """Install (or with no arguments clear) the attention-kernel timing hook.

    ``before``/``after`` are ``torch.cuda.Event`` objects that have been
    recorded at least once (so that their CUDA handles exist)."""
    lib = load_library()
    if before is None or after is None:
        lib.sage_set_attention_events(None, None)
    else:
        lib.sage_set_attention_events(ctypes.c_void_p(before.cuda_event), ctypes.c_void_p(after.cuda_event))


def debug_staging_codes(q, k):
    """The Q/K quantisation exactly as sage_attn_fwd feeds the attention
    kernel: (q16 fp16 [B,H,S_pad,D], q_scale [B,H,nb], k16, k_scale)."""
    lib = load_library()
    B, S, H, D = _check_qkv(q, k, k)
    Sp = padded_len(S)
    nb = (S + 31) // 32
    dev = q.device
    q16 = torch.empty((B, H, Sp, D), dtype=torch.float16, device=dev)
    k16 = torch.empty_like(q16)
    q_sc = torch.empty((B, H, nb), dtype=torch.float32, device=dev)
    k_sc = torch.empty_like(q_sc)
    with torch.cuda.device(dev):
        _check(lib.sage_debug_staging_codes(_ptr(q), _ptr(k), B, S, H, D, _ptr(q16), _ptr(q_sc), _ptr(k16),
                                            _ptr(k_sc), _stream(dev)))
    return q16, q_sc, k16, k_sc


def debug_inject_fault(site: int, skip: int = 0):
    """Arm the library's host-side fault injection (FAULT_* sites)."""
    _check(load_library().sage_debug_inject_fault(int(site), int(skip)))


def debug_pool_state(device=None):
    """(created, used_bytes) of the library's private memory pool on a device."""
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    created, used = ctypes.c_int(0), ctypes.c_uint64(0)
    with torch.cuda.device(dev):
        _check(lib.sage_debug_pool_state(ctypes.byref(created), ctypes.byref(used)))
    return bool(created.value), int(used.value)


def kv_cache_alloc(num_pages: int, H: int, page_size: int = 64, device=None, bits: int = 8):
    """Tensors of an empty paged KV cache: (k_codes int8 [num_pages, H,
    page_size, 128], k_scale fp32 [num_pages, H, page_size], v_codes
    float8_e4m3fn like k_codes, v_scale like k_scale), or with ``bits`` 4
    (k_codes uint8 [num_pages, H, page_size, 64], k_block float8_e4m3fn
    [num_pages, H, page_size, 8], k_scale, and the same for v): the tuple that the
    other kv_cache_* and attn_fwd_cache* functions take, of either kind.
    Contents are undefined until they are written."""
    if page_size not in KV_PAGE_SIZES:
        raise ValueError(f"page_size must be one of {KV_PAGE_SIZES} (got {page_size})")
    if num_pages < 1 or H < 1:
        raise ValueError(f"num_pages and H must be >= 1 (got {num_pages}, {H})")
    if bits not in (4, 8):
        raise ValueError(f"bits must be 8 or 4 (got {bits})")
    dev = torch.device("cuda") if device is None else torch.device(device)
    scales = (num_pages, H, page_size)

    def tensor(n, dtype):
        return torch.empty(scales + (n,) if n else scales, dtype=dtype, device=dev)

    if bits == 4:
        return tuple(tensor(n, t) for _ in "kv" for n, t in ((64, torch.uint8), (8, torch.float8_e4m3fn), (0, torch.float32)))
    return (tensor(HEAD_DIM, torch.int8), tensor(0, torch.float32), tensor(HEAD_DIM, torch.float8_e4m3fn),
            tensor(0, torch.float32))


# The checks below run on every generation step, so they ask each tensor for as
# little as they need: device numbers instead of devices, and no context manager
# where the device is the current one.

_INT8, _UINT8, _FP32, _BF16, _INT32 = torch.int8, torch.uint8, torch.float32, torch.bfloat16, torch.int32
_FP8 = (torch.float8_e4m3fn, torch.uint8)


def _check_kv4_cache(cache):
    """The tuple of a 4-bit cache as a sage_kv4_cache, and its device number."""
    kc, kb, ks, vc, vb, vs = cache
    if kc.dtype is not _UINT8 or vc.dtype is not _UINT8 or kb.dtype not in _FP8 or vb.dtype not in _FP8 \
            or ks.dtype is not _FP32 or vs.dtype is not _FP32:
        for name, t, want in (("k_codes", kc, (_UINT8,)), ("k_block", kb, _FP8), ("k_scale", ks, (_FP32,)),
                              ("v_codes", vc, (_UINT8,)), ("v_block", vb, _FP8), ("v_scale", vs, (_FP32,))):
            if t.dtype not in want:
                raise ValueError(f"{name} must be {want[0]} (got {t.dtype})")
    dev = kc.get_device()
    if dev < 0 or kb.get_device() != dev or ks.get_device() != dev or vc.get_device() != dev or vb.get_device() != dev \
            or vs.get_device() != dev or not kc.is_cuda:
        raise ValueError("the cache must be CUDA tensors on one device")
    if not (kc.is_contiguous() and kb.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vb.is_contiguous()
            and vs.is_contiguous()):
        raise ValueError("the cache's tensors must be contiguous")
    shape, blocks, scales = kc.shape, kb.shape, ks.shape
    if len(shape) != 4 or len(blocks) != 4 or shape[3] != 64 or blocks[3] != 8 or scales != shape[:3] or blocks[:3] != scales \
            or vc.shape != shape or vb.shape != blocks or vs.shape != scales:
        raise ValueError("a cache of 4 bits is codes [num_pages, H, page_size, 64], blocks [.., 8] and scales [num_pages, H, "
                         f"page_size] (got {[tuple(t.shape) for t in cache]})")
    pages, H, page = scales
    if page not in KV_PAGE_SIZES or pages < 1 or H < 1:
        raise ValueError(f"a cache has pages of {KV_PAGE_SIZES} tokens (got {tuple(scales)})")
    return _KV4Cache(kc.data_ptr(), kb.data_ptr(), ks.data_ptr(), vc.data_ptr(), vb.data_ptr(), vs.data_ptr(), pages, H, page), dev


def _check_cache(cache):
    """The cache tuple as a sage_kv_cache or a sage_kv4_cache, and its device number."""
    if isinstance(cache, (tuple, list)) and len(cache) == 6:
        return _check_kv4_cache(cache)
    if not isinstance(cache, (tuple, list)) or len(cache) != 4:
        raise TypeError("cache must be (k_codes, k_scale, v_codes, v_scale)")
    kc, ks, vc, vs = cache
    if kc.dtype is not _INT8 or ks.dtype is not _FP32 or vc.dtype not in _FP8 or vs.dtype is not _FP32:
        for name, t, want in (("k_codes", kc, _INT8), ("k_scale", ks, _FP32), ("v_codes", vc, _FP8[0]), ("v_scale", vs, _FP32)):
            if t.dtype is not want:
                raise ValueError(f"{name} must be {want} (got {t.dtype})")
    dev = kc.get_device()
    if dev < 0 or ks.get_device() != dev or vc.get_device() != dev or vs.get_device() != dev or not kc.is_cuda:
        raise ValueError("the cache must be CUDA tensors on one device")
    if not (kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()):
        raise ValueError("the cache's tensors must be contiguous")
    shape, scales = kc.shape, ks.shape
    if len(shape) != 4 or vc.shape != shape or scales != shape[:3] or vs.shape != scales:
        raise ValueError(f"a cache is codes [num_pages, H, page_size, 128] and scales [num_pages, H, page_size] "
                         f"(got {tuple(kc.shape)}, {tuple(ks.shape)}, {tuple(vc.shape)}, {tuple(vs.shape)})")
    pages, H, page, D = shape
    if D != HEAD_DIM or page not in KV_PAGE_SIZES or pages < 1 or H < 1:
        raise ValueError(f"a cache has 128 channels and pages of {KV_PAGE_SIZES} tokens (got {tuple(shape)})")
    return _KVCache(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), pages, H, page), dev


def _check_rows(name, t, dev, H=None):
    """bf16 [B, S, H, 128] whose tokens' heads are dense: the shape, batch stride
    and token stride (in elements; 0 where there is one)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be bfloat16 (got {t.dtype})")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the cache's device cuda:{dev} (got {t.device})")
    shape = t.shape
    if len(shape) != 4 or shape[3] != HEAD_DIM or 0 in shape or (H is not None and shape[2] != H):
        raise ValueError(f"{name} must be [B, S, {'H' if H is None else H}, 128] (got {tuple(shape)})")
    sb, ss, sh, sd = t.stride()
    if sd != 1 or (sh != HEAD_DIM and shape[2] > 1):
        raise ValueError(f"the heads of a token of {name} must be dense (strides {t.stride()})")
    return shape, sb if shape[0] > 1 else 0, ss if shape[1] > 1 else 0


def _check_table(table, B, dev, name="block_table"):
    shape = table.shape
    if table.dtype is not _INT32 or table.get_device() != dev or len(shape) != 2 or shape[0] != B or shape[1] < 1:
        raise ValueError(f"{name} must be an int32 [{B}, pages] tensor on cuda:{dev}")
    sb, se = table.stride()
    if se != 1 and shape[1] > 1:
        raise ValueError(f"the rows of {name} must be dense")
    return shape[1], sb if B > 1 else 0


def _check_ints(name, t, n, dev):
    if t.dtype is not _INT32 or t.get_device() != dev or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor on cuda:{dev}")


def _call(fn, dev, *args):
    """fn(*args, the current stream of device `dev`), with that device current."""
    if torch.cuda.current_device() == dev:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        _check(status)


def kv_cache_write(k, v, cache, block_table, start, count=None):
    """Quantise k and v, bf16 [B, S, H, 128] (slices of a projection are
    taken as they are), and put token i of sequence b at position start[b] + i of
    the cache, through sage_kv_cache_write.  ``block_table`` int32 [B, pages]
    names the pages of each sequence, ``start`` int32 [B]; with ``count`` int32
    [B] only the first count[b] tokens of a padded sequence are written.
    Returns ``cache``."""
    lib = _lib or load_library()
    c, dev = _check_cache(cache)
    shape, k_sb, k_ss = _check_rows("k", k, dev, c.H)
    v_shape, v_sb, v_ss = _check_rows("v", v, dev, c.H)
    if shape != v_shape:
        raise ValueError(f"k and v must have equal shapes (got {tuple(k.shape)}, {tuple(v.shape)})")
    B, S = shape[0], shape[1]
    width, stride = _check_table(block_table, B, dev)
    _check_ints("start", start, B, dev)
    if count is not None:
        _check_ints("count", count, B, dev)
    _call(lib.sage_kv_cache_write if len(cache) == 4 else lib.sage_kv4_cache_write, dev, ctypes.byref(c), k.data_ptr(), v.data_ptr(), k_sb, k_ss, v_sb, v_ss, B, S,
          HEAD_DIM, block_table.data_ptr(), width, stride, start.data_ptr(), None if count is None else count.data_ptr())
    return cache


def kv_cache_read(cache, block_table, lens, S: int, out=None):
    """The first S positions of each sequence in the cache as bf16 (k, v),
    each [B, S, H, 128], zeros from position lens[b] on (sage_kv_cache_read).
    ``out`` (optional) is the pair of tensors to fill."""
    lib = _lib or load_library()
    c, dev = _check_cache(cache)
    if lens.dim() != 1:
        raise ValueError("lens must be an int32 [B] tensor")
    B, S = lens.shape[0], int(S)
    if B < 1 or S < 1:
        raise ValueError(f"B and S must be >= 1 (got {B}, {S})")
    width, stride = _check_table(block_table, B, dev)
    _check_ints("lens", lens, B, dev)
    shape = (B, S, c.H, HEAD_DIM)
    if out is None:
        k = torch.empty(shape, dtype=_BF16, device=cache[0].device)
        out = k, torch.empty_like(k)
    else:
        if len(out) != 2 or out[0].data_ptr() == out[1].data_ptr():
            raise ValueError("out must be two tensors, one for k and one for v")
        for t in out:
            if t.shape != shape or t.dtype is not _BF16 or t.get_device() != dev or not t.is_contiguous():
                raise ValueError(f"out must be two contiguous bf16 tensors {shape} on cuda:{dev}")
    _call(lib.sage_kv_cache_read if len(cache) == 4 else lib.sage_kv4_cache_read, dev, ctypes.byref(c), block_table.data_ptr(), width, stride, lens.data_ptr(),
          out[0].data_ptr(), out[1].data_ptr(), B, S, HEAD_DIM)
    return out


def attn_fwd_cache_workspace_bytes(B: int, Sq: int, Hq: int, H: int, prefix_len: int = 0) -> int:
    return int(load_library().sage_attn_fwd_cache_workspace_bytes(B, Sq, Hq, H, prefix_len))


def _attn_fwd_cache(q, cache, prefix, block_table, lens, softmax_scale, causal, out, lse, return_lse, workspace):
    lib = _lib or load_library()
    c, dev = _check_cache(cache)
    shape, q_sb, q_ss = _check_rows("q", q, dev)
    B, Sq, Hq, D = shape
    if Hq % c.H:
        raise ValueError(f"q's heads ({Hq}) must be a multiple of the cache's ({c.H})")
    width, stride = _check_table(block_table, B, dev)
    _check_ints("lens", lens, B, dev)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty(shape, dtype=_BF16, device=q.device)
    elif out.shape != shape or out.dtype is not _BF16 or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError("out must be a contiguous bf16 tensor of q's shape on its device")
    if lse is None:
        if return_lse:
            lse = torch.empty((B, Hq, Sq), dtype=_FP32, device=q.device)
    elif lse.dtype is not _FP32 or lse.shape != (B, Hq, Sq) or not lse.is_contiguous() or lse.get_device() != dev:
        raise ValueError("lse must be a contiguous float32 [B, Hq, Sq] tensor on q's device")
    ws_bytes = 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's device")
        ws_bytes = workspace.numel() * workspace.element_size()
    tail = (block_table.data_ptr(), width, stride, lens.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
            B, Sq, Hq, D, softmax_scale, 1 if causal else 0, None if workspace is None else workspace.data_ptr(), ws_bytes)
    if prefix is None:
        _call(lib.sage_attn_fwd_cache if len(cache) == 4 else lib.sage_attn_fwd_kv4_cache, dev, q.data_ptr(), q_sb, q_ss, ctypes.byref(c), *tail)
    else:
        table, length = prefix
        if length < 1 or table.dim() != 1 or table.shape[0] < -(-length // c.page_size):
            raise ValueError(f"prefix_table must name the pages of prefix_len >= 1 positions (got "
                             f"{tuple(table.shape)} for {length})")
        _check_ints("prefix_table", table, table.shape[0], dev)
        _call(lib.sage_attn_fwd_cache_prefix if len(cache) == 4 else lib.sage_attn_fwd_kv4_cache_prefix, dev, q.data_ptr(), q_sb, q_ss, ctypes.byref(c), table.data_ptr(), length, *tail)
    return (out, lse) if lse is not None else out


def attn_fwd_cache(q, cache, block_table, lens, softmax_scale: float | None = None, causal: bool = True, out=None,
                   lse=None, return_lse: bool = False, workspace=None):
    """Attention of q, bf16 [B, Sq, Hq, 128], the newest Sq tokens of each
    sequence, over the lens[b] positions that each has in the cache (their own
    among them), through sage_attn_fwd_cache: query head h reads key/value head
    h // (Hq // H).  Returns out bf16 [B, Sq, Hq, 128], and lse fp32 [B, Hq, Sq]
    with ``return_lse`` or when ``lse`` is given.  With ``causal`` query i sees
    positions up to lens[b] - Sq + i; a query that sees nothing gives zeros and
    -inf.  A sequence with fewer than Sq new tokens has its queries at the end,
    q[b, Sq - c:], behind padding (kv_cache_write has its tokens at the front).
    A length behind what ``block_table`` has room for is reported by sync_status
    (SAGE_ERR_BAD_PAGE), except that 2**30 or more means all of it.
    ``workspace`` (optional uint8 CUDA tensor of >=
    attn_fwd_cache_workspace_bytes) replaces the library's pool; few short
    sequences need none."""
    return _attn_fwd_cache(q, cache, None, block_table, lens, softmax_scale, causal, out, lse, return_lse, workspace)


def attn_fwd_cache_prefix(q, cache, prefix_table, prefix_len: int, block_table, lens,
                          softmax_scale: float | None = None, causal: bool = True, out=None, lse=None,
                          return_lse: bool = False, workspace=None):
    """attn_fwd_cache for sequences that all begin with the same prefix_len
    positions, pages ``prefix_table`` (int32 [pages]): sequence b is the prefix
    and then the lens[b] positions of its row of ``block_table``.  The prefix is
    read and multiplied once for all sequences (above 256, for every 256), unless
    a few and a short prefix are done sooner without (sage_attn_fwd_cache_prefix)."""
    return _attn_fwd_cache(q, cache, (prefix_table, int(prefix_len)), block_table, lens, softmax_scale, causal, out,
                           lse, return_lse, workspace)


# Scaling of positions and where tokens stand (include/sage.h).
ROPE_SCALINGS = ("plain", "linear", "ntk", "yarn", "bands")
TOKEN_LAYOUTS = ("packed", "front", "end")


class Rope:
    """Rotary positions of the first ``dim`` channels (32, 64, 96 or 128) of a head
    (sage_rope): pairs (2i, 2i + 1) with ``interleaved``, else (i, i + dim / 2).

    ``sections`` names the pairs of each of up to four axes (for images and videos),
    which have frequencies base ** (-2i / (2 * pairs)) of their own; without it there is
    one axis.  ``scaling``: None, ("linear", factor), ("ntk", factor), ("yarn", factor,
    original_len[, low, high]) or ("bands", factor, original_len[, low, high]).
    ``freqs`` (dim / 2 radians a position, at most 3) replaces base and scaling.
    ``freq`` is the table on the device, ``factor`` what sine and cosine are
    multiplied by (given, it replaces the scaling's)."""

    def __init__(self, dim: int = HEAD_DIM, base: float = 10000.0, interleaved: bool = False, sections=None, scaling=None,
                 freqs=None, factor: float | None = None, device=None):
        lib = load_library()
        if dim not in (32, 64, 96, 128):
            raise ValueError(f"dim must be 32, 64, 96 or 128 (got {dim})")
        self.dim, self.interleaved = int(dim), bool(interleaved)
        self.sections = (self.dim // 2,) if sections is None else tuple(int(n) for n in sections)
        if not 1 <= len(self.sections) <= 4 or min(self.sections) < 1 or sum(self.sections) != self.dim // 2:
            raise ValueError(f"sections must be 1 to 4 numbers >= 1 that add up to {self.dim // 2} (got {self.sections})")
        table, own = [], ctypes.c_double(1.0)
        if freqs is not None:
            freqs = [float(f) for f in freqs]
            if scaling is not None or len(freqs) != self.dim // 2 or not all(abs(f) <= 3.0 for f in freqs):
                raise ValueError(f"freqs must be {self.dim // 2} numbers of at most 3, without scaling")
            table = [lib.sage_rope_frequency(f) for f in freqs]
        else:
            kind, *rest = scaling if scaling is not None else ("plain",)
            if kind not in ROPE_SCALINGS or len(rest) not in {"plain": (0,), "linear": (1,), "ntk": (1,)}.get(kind, (2, 4)):
                raise ValueError(f"scaling must be (kind, factor[, original_len[, low, high]]), kind one of {ROPE_SCALINGS} (got {scaling})")
            rest = [float(x) for x in rest] + [1.0, 0.0, 1.0, 32.0 if kind == "yarn" else 4.0][len(rest):]
            for n in self.sections:
                part = (ctypes.c_uint64 * n)()
                _check(lib.sage_rope_frequencies(2 * n, float(base), ROPE_SCALINGS.index(kind), *rest, part, ctypes.byref(own)))
                table += list(part)
        self.factor = own.value if factor is None else float(factor)
        dev = torch.device("cuda") if device is None else torch.device(device)
        signed = [f - (1 << 64) if f >> 63 else f for f in table]
        self.freq = torch.tensor(signed, dtype=torch.int64, device=dev)
        self._c = _Rope(self.freq.data_ptr(), self.dim, int(self.interleaved), len(self.sections),
                        (ctypes.c_int32 * 4)(*self.sections), self.factor)


def _check_turn(rope, positions, q_weight, k_weight, eps, B, S, dev):
    """The arguments of norm and rotation: (rope, positions, their strides, weights, eps)."""
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype is not _BF16 or w.shape != (HEAD_DIM,) or not w.is_contiguous() or w.get_device() != dev):
            raise ValueError(f"{name} must be a contiguous bf16 [128] tensor on cuda:{dev}")
    if eps is None and not (q_weight is None and k_weight is None):
        raise ValueError("weights without a norm: give eps")
    if eps is not None and not 0.0 <= eps < math.inf:
        raise ValueError(f"eps must be finite and >= 0 (got {eps})")
    tail = (None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
            -1.0 if eps is None else eps)
    if rope is None:
        if positions is not None:
            raise ValueError("positions without rope")
        return (None, None, 0, 0) + tail
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    if rope.freq.get_device() != dev:
        raise ValueError(f"rope must be on cuda:{dev}")
    if not isinstance(positions, torch.Tensor):
        raise TypeError("rope needs positions, a torch.Tensor")
    axes = len(rope.sections)
    shape, strides = positions.shape, positions.stride()
    if axes == 1 and (len(shape) != 3) and (len(shape) == 1 or shape[-1] != 1 or shape == (B, S)):
        shape, strides = (*shape, 1), (*strides, 1)      # one axis may be left out
    if len(shape) == 2:
        # [S, axes] for all batches, or, for packed tokens or one token of each sequence, [B * S, axes]
        if shape[0] == S:
            shape, strides = (B, *shape), (0, *strides)
        elif shape[0] == B * S:
            shape, strides = (B, S, shape[1]), (S * strides[0], *strides)
    if positions.dtype is not _INT32 or positions.get_device() != dev or shape != (B, S, axes):
        raise ValueError(f"positions must be int32 [{B}, {S}{', ' + str(axes) if axes > 1 else ''}] on cuda:{dev} "
                         f"(got {positions.dtype} {tuple(positions.shape)})")
    sb, ss, sa = strides
    if axes > 1 and sa != 1:
        raise ValueError("the axes of a position must be dense")
    return (ctypes.byref(rope._c), positions.data_ptr(), sb if B > 1 else 0, ss if S > 1 else 0) + tail


def _check_out(name, t, shape, dev):
    if t.shape != shape or t.dtype is not _BF16 or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous bf16 tensor {tuple(shape)} on cuda:{dev}")
    return t


def qk_norm_rope(q, k=None, rope=None, positions=None, q_weight=None, k_weight=None, eps: float | None = None, out=None):
    """RMS norm of each head of q, bf16 [B, S, Hq, 128], and k, bf16 [B, S, Hk,
    128] (slices of a projection are taken as they are), with ``eps`` and the
    weights bf16 [128] of each if given, then the rotation by ``rope`` at
    ``positions``, int32 [B, S] ([B, S, axes] for several axes, [S] or [S, axes]
    the same for all of the batch), in one pass (sage_qk_norm_rope).  Returns the
    dense (q, k), or q alone without k.  ``out``: the pair (or the tensor) to fill,
    which may be q and k themselves."""
    lib = _lib or load_library()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dev = q.get_device()
    shape, q_sb, q_ss = _check_rows("q", q, dev)
    B, S, Hq, D = shape
    Hk = k_sb = k_ss = 0
    if k is not None:
        k_shape, k_sb, k_ss = _check_rows("k", k, dev)
        Hk = k_shape[2]
        if k_shape[:2] != shape[:2]:
            raise ValueError(f"q and k must have equal batches and lengths (got {tuple(q.shape)}, {tuple(k.shape)})")
    turn = _check_turn(rope, positions, q_weight, k_weight, eps, B, S, dev)
    if out is None:
        q_out = torch.empty(shape, dtype=_BF16, device=q.device)
        k_out = None if k is None else torch.empty(k_shape, dtype=_BF16, device=q.device)
    else:
        q_out, k_out = (out, None) if k is None else out
        _check_out("out", q_out, shape, dev)
        if k is not None:
            _check_out("out", k_out, k_shape, dev)
            if k_out.data_ptr() == q_out.data_ptr():
                raise ValueError("out must be two tensors, one for q and one for k")
    _call(lib.sage_qk_norm_rope, dev, q.data_ptr(), None if k is None else k.data_ptr(), q_sb, q_ss, k_sb, k_ss, B, S, Hq, Hk, D,
          *turn, q_out.data_ptr(), None if k is None else k_out.data_ptr())
    return q_out if k is None else (q_out, k_out)


def kv_cache_append(q, k, v, cache, slots, rope=None, positions=None, q_weight=None, k_weight=None, eps: float | None = None,
                    out=None):
    """qk_norm_rope of q, bf16 [B, S, Hq, 128], and k, with k and v, bf16 [B, S, H,
    128], quantised and put into ``cache`` (of 8 or 4 bits) in the same pass: token (b,
    s) goes to ``slots``, int32 [B, S] (kv_pages_reserve makes them; a negative one is
    not written).  Tokens may be packed as [1, T, ...] with slots and positions [T].
    Returns the dense q (``out`` if given); q None: None (sage_kv_cache_append)."""
    lib = _lib or load_library()
    c, dev = _check_cache(cache)
    shape, k_sb, k_ss = _check_rows("k", k, dev, c.H)
    v_shape, v_sb, v_ss = _check_rows("v", v, dev, c.H)
    if shape != v_shape:
        raise ValueError(f"k and v must have equal shapes (got {tuple(k.shape)}, {tuple(v.shape)})")
    B, S, _, D = shape
    Hq = q_sb = q_ss = 0
    if q is not None:
        q_shape, q_sb, q_ss = _check_rows("q", q, dev)
        Hq = q_shape[2]
        if q_shape[:2] != shape[:2]:
            raise ValueError(f"q and k must have equal batches and lengths (got {tuple(q.shape)}, {tuple(k.shape)})")
        out = torch.empty(q_shape, dtype=_BF16, device=q.device) if out is None else _check_out("out", out, q_shape, dev)
    elif out is not None or q_weight is not None:
        raise ValueError("out and q_weight without q")
    turn = _check_turn(rope, positions, q_weight, k_weight, eps, B, S, dev)
    if slots.dtype is not _INT32 or slots.get_device() != dev or slots.numel() != B * S or not slots.is_contiguous():
        raise ValueError(f"slots must be a contiguous int32 [{B}, {S}] tensor on cuda:{dev}")
    _call(lib.sage_kv_cache_append if len(cache) == 4 else lib.sage_kv4_cache_append, dev, ctypes.byref(c),
          None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), q_sb, q_ss, k_sb, k_ss, v_sb, v_ss, B, S, Hq, D,
          *turn, slots.data_ptr(), None if q is None else out.data_ptr())
    return out


class PagePlan(NamedTuple):
    """What kv_pages_reserve gives, int32 tensors: ``start``, ``taken``, ``lens`` and
    ``first`` [B], ``free_count`` [1], ``slots`` and ``positions`` [tokens] (packed) or
    [B, tokens]."""
    start: torch.Tensor
    taken: torch.Tensor
    lens: torch.Tensor
    first: torch.Tensor
    free_count: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor


def _check_free(free_pages, free_count, lens, page_size):
    """(num_pages, B, device) of a free list and lengths."""
    dev = free_pages.get_device()
    if not free_pages.is_cuda or free_pages.dim() != 1 or free_pages.shape[0] < 1:
        raise ValueError("free_pages must be an int32 [num_pages] CUDA tensor")
    _check_ints("free_pages", free_pages, free_pages.shape[0], dev)
    _check_ints("free_count", free_count, 1, dev)
    if page_size not in KV_PAGE_SIZES:
        raise ValueError(f"page_size must be one of {KV_PAGE_SIZES} (got {page_size})")
    if lens.dim() != 1 or lens.shape[0] < 1:
        raise ValueError("lens must be an int32 [B] tensor")
    _check_ints("lens", lens, lens.shape[0], dev)
    return free_pages.shape[0], lens.shape[0], dev


def kv_pages_reserve(free_pages, free_count, lens, counts, block_table, page_size: int, tokens: int, layout: str = "packed",
                     out: PagePlan | None = None):
    """Pages for counts[b] more tokens of each sequence of lens[b], off the stack
    ``free_pages`` (int32 [num_pages], the first free_count[0] free): fills
    ``block_table`` (int32 [B, pages]) and returns a PagePlan with the tokens' slots
    and positions (sage_kv_pages_reserve).  ``layout``: "packed" tokens one behind
    another, ``tokens`` in all, or [B, tokens] with a sequence's at the "front" or
    the "end" of its row.  Sequences for which there are too few pages get none (taken
    0), and sync_status reports SAGE_ERR_NO_PAGES; those for whose tokens there are too
    few rows SAGE_ERR_BAD_PAGE.  ``out``: the PagePlan to fill, of which lens and
    free_count may be the arguments."""
    lib = _lib or load_library()
    num_pages, B, dev = _check_free(free_pages, free_count, lens, page_size)
    _check_ints("counts", counts, B, dev)
    width, stride = _check_table(block_table, B, dev)
    tokens = int(tokens)
    if layout not in TOKEN_LAYOUTS:
        raise ValueError(f"layout must be one of {TOKEN_LAYOUTS} (got {layout!r})")
    if tokens < 1:
        raise ValueError(f"tokens must be >= 1 (got {tokens})")
    packed = layout == "packed"
    rows = (tokens,) if packed else (B, tokens)
    if out is None:
        n = tokens if packed else B * tokens
        flat = torch.empty(4 * B + 1 + 2 * n, dtype=_INT32, device=free_pages.device)
        start, taken, new_lens, first, left, slots, positions = flat.split_with_sizes((B, B, B, B, 1, n, n))
        out = PagePlan(start, taken, new_lens, first, left, slots if packed else slots.view(rows), positions if packed else positions.view(rows))
        at, b = flat.data_ptr(), 4 * B
        ptrs = (at, at + b, at + 2 * b, at + 3 * b, at + 4 * b, at + 4 * b + 4, at + 4 * b + 4 + 4 * n)
    else:
        for name, t, shape in zip(PagePlan._fields, out, ((B,),) * 4 + ((1,), rows, rows)):
            if t.dtype is not _INT32 or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
                raise ValueError(f"out.{name} must be a contiguous int32 {shape} tensor on cuda:{dev}")
        ptrs = [t.data_ptr() for t in out]
    _call(lib.sage_kv_pages_reserve, dev, free_pages.data_ptr(), free_count.data_ptr(), num_pages, page_size, lens.data_ptr(),
          counts.data_ptr(), B, block_table.data_ptr(), width, stride, TOKEN_LAYOUTS.index(layout), tokens, *ptrs)
    return out


def kv_pages_release(free_pages, free_count, lens, keep, block_table, page_size: int):
    """Cut sequences to keep[b] tokens (0: all of a finished one), in place: their
    pages behind that go back to the free list (sage_kv_pages_release)."""
    lib = _lib or load_library()
    num_pages, B, dev = _check_free(free_pages, free_count, lens, page_size)
    _check_ints("keep", keep, B, dev)
    width, stride = _check_table(block_table, B, dev)
    _call(lib.sage_kv_pages_release, dev, free_pages.data_ptr(), free_count.data_ptr(), num_pages, page_size, lens.data_ptr(),
          keep.data_ptr(), B, block_table.data_ptr(), width, stride)
