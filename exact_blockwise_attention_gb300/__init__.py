"""Exact blockwise attention for long video-token sequences on GB300 (sm_103a).

A thin Python binding over the C ABI of ``libattn.so`` (include/attn.h). Every
step of the computation runs in the library's CUDA kernels; this module only
checks tensors, allocates outputs with PyTorch (device memory and the current
stream are all PyTorch provides here) and passes raw pointers through ctypes.
There is no fallback: if the library is missing, importing the functions
raises.

Entry points (same names as the C ABI):
  fwd(q, k, v, scale=None)                      -> (o, lse)
  bwd(q, k, v, o, do, lse, scale=None)          -> (dq, dk, dv)
  partial_fwd(q, k, v, k0, k1, scale=None)      -> (o_part fp32, lse_part)
  split_fwd(q, k, v, bounds, scale=None)        -> (o_parts fp32, lse_parts)
  merge(o_parts, lse_parts)                     -> (o, lse)
  attention(q, k, v, scale=None)                -> o   (autograd-aware)
  attention_varlen(q, k, v, cu_q, cu_k, scale=None) -> o   (autograd-aware, packed)
  fwd_varlen(q, k, v, cu_q, cu_k, scale=None)   -> (o, lse)      packed sequences
  fwd_fp8(q8, k8, vt8, q_scale, k_scale, v_scale, scale=None) -> (o, lse)   e4m3, d = 128
  bwd_varlen(q, k, v, o, do, lse, cu_q, cu_k, scale=None) -> (dq, dk, dv)
  fwd_window(q, k, v, left, right=0, sinks=0, scale=None, rest=False) -> (o, lse)   a sliding window and first tokens
  bwd_window(q, k, v, o, do, lse, left, right=0, sinks=0, scale=None) -> (dq, dk, dv)
  attention_window(q, k, v, left, right=0, sinks=0, scale=None) -> o   (autograd-aware)
  rope_fwd(q, k, positions, plan), rope_bwd(dq, dk, positions, plan) -> (q, k)   rotary positions
  rope(q, k, positions, plan)                   -> (q, k)   (autograd-aware)
  cache_append(cache, k, v, page_table, seq_lens, cu_new=None, rope=None, positions=None)
  decode(cache, q, page_table, seq_lens, scale=None, rope=None, positions=None, window=None, sinks=0)
      -> (o, lse)
  decode_tree(cache, q, page_table, seq_lens, cu_q=None, mask=None, window=None, sinks=0) -> (o, lse)
  pages_release(pool, page_table, first, last), pages_reserve(pool, page_table, seq_lens, new_lens),
  pages_fork(pool, page_table, seq_lens, src, dst) -> (from_pages, to_pages)   page tables kept on the GPU
  cache_copy(cache, from_pages, to_pages)       whole pages within a cache
  cache_gather(cache, page_table, places, cu, to_table=None, to_start=None)   chosen tokens together
with the handles Rope (a rotation: axes, frequencies, pairs), PagedCache (key and value pages) and
PagePool (which pages are free).
Tensors are CUDA, contiguous, [B, H, L, d] with d in {64, 128}; q, k, v, o,
do are bfloat16, lse and partials float32. The default scale is 1/sqrt(d).
fwd, bwd and attention also take k, v with fewer heads H_kv dividing H
(grouped-query attention: query head h reads K/V head h // (H // H_kv);
attn_fwd_gqa / attn_bwd_gqa).
Packed sequences are token-major [T, H, d] with lse [H, Tq]; cu_q, cu_k are
host-side cumulative lengths (n_seqs + 1 ints, first 0). The rotation and the
cache calls also take views whose heads are contiguous rows on 16-byte
boundaries; their positions, page tables and lengths are int32 device tensors.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from . import _build

__all__ = [
    "AttnError", "lib", "fwd", "bwd", "bwd_noalloc", "partial_fwd", "split_fwd", "merge", "attention",
    "bwd_workspace_size", "poll_device_status", "set_wait_limit_ns", "status_string",
    "MAX_CHUNKS", "MAX_SEQS", "fwd_varlen", "bwd_varlen", "bwd_varlen_workspace_size", "fwd_fp8",
    "attention_varlen", "Rope", "rope_fwd", "rope_bwd", "rope", "PagedCache", "cache_append",
    "decode", "decode_workspace_size", "PagePool", "pages_release", "pages_fork", "pages_reserve",
    "cache_copy", "cache_gather", "fwd_window", "bwd_window", "bwd_window_workspace_size",
    "attention_window", "decode_tree", "decode_tree_workspace_size",
]

ATTN_OK = 0
MAX_CHUNKS = 64
MAX_SEQS = 1024
MAX_AXES = 4
MAX_PAIRS = 64
MAX_MASK_WORDS = 16
_LIB = None


class _RopeStruct(ctypes.Structure):
    """attn_rope_t"""
    _fields_ = [("n_pairs", ctypes.c_int), ("n_axes", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("axis", ctypes.c_ubyte * MAX_PAIRS), ("turns", ctypes.c_ulonglong * MAX_PAIRS)]


class _CacheStruct(ctypes.Structure):
    """attn_cache_t"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_strides", ctypes.c_longlong * 3), ("v_strides", ctypes.c_longlong * 3),
                ("n_pages", ctypes.c_longlong), ("page_size", ctypes.c_int),
                ("H_kv", ctypes.c_int), ("d", ctypes.c_int), ("type", ctypes.c_int),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class _PoolStruct(ctypes.Structure):
    """attn_pool_t"""
    _fields_ = [("refs", ctypes.c_void_p), ("scratch", ctypes.c_void_p),
                ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int)]


class AttnError(RuntimeError):
    """A non-zero status returned by the C ABI."""

    def __init__(self, fn: str, status: int):
        self.status = status
        msg = f"{fn} failed: {status_string(status)} (status {status})"
        if status == 4:
            self.cuda_error = int(lib().attn_last_cuda_error())
            msg += f", cudaError {self.cuda_error}"
        super().__init__(msg)


def _declare(L):
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    L.attn_bwd_workspace_size.argtypes = [i, i, i, i, i]
    L.attn_bwd_workspace_size.restype = sz
    L.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, sz, vp]
    L.attn_partial_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp]
    L.attn_split_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, ctypes.POINTER(i), i, f, vp]
    L.attn_merge.argtypes = [vp, vp, i, vp, vp, i, i, i, i, vp]
    L.attn_status_string.argtypes = [i]
    L.attn_status_string.restype = ctypes.c_char_p
    L.attn_poll_device_status.argtypes = [vp]
    L.attn_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    L.attn_bwd_noalloc.restype = ctypes.c_int
    L.attn_last_cuda_error.argtypes = []
    L.attn_last_cuda_error.restype = ctypes.c_int
    L.attn_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    L.attn_set_wait_limit_ns.restype = ctypes.c_ulonglong
    L.attn_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
    L.attn_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, f, f, f, vp]
    L.attn_bwd_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp, sz,
                               vp]
    L.attn_fwd_window.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp]
    L.attn_fwd_window.restype = ctypes.c_int
    L.attn_bwd_window_workspace_size.argtypes = [i, i, i, i, i, i, i, i, i]
    L.attn_bwd_window_workspace_size.restype = sz
    L.attn_bwd_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp,
                                  sz, vp]
    L.attn_bwd_window.restype = ctypes.c_int
    ip = ctypes.POINTER(i)
    L.attn_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, ip, ip, i, i, i, f, vp]
    L.attn_bwd_varlen_workspace_size.argtypes = [i, i, i, i]
    L.attn_bwd_varlen_workspace_size.restype = sz
    L.attn_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ip, ip, i, i, i, f, vp, sz,
                                  vp]
    L.attn_fwd_varlen_gqa.argtypes = [vp, vp, vp, vp, vp, ip, ip, i, i, i, i, f, vp]
    L.attn_bwd_varlen_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ip, ip, i, i, i, i, f,
                                      vp, sz, vp]
    ll, rp, cp = ctypes.c_longlong, ctypes.POINTER(_RopeStruct), ctypes.POINTER(_CacheStruct)
    lp = ctypes.POINTER(ll)
    L.attn_rope_init.argtypes = [rp, i, i, ip, ctypes.POINTER(ctypes.c_double), i]
    L.attn_rope.argtypes = [rp, vp, lp, vp, lp, vp, lp, vp, lp, vp, lp, i, i, i, i, i, i, vp]
    L.attn_cache_append.argtypes = [cp, vp, lp, vp, lp, vp, ll, i, vp, i, vp, i, rp, vp, ll, vp]
    L.attn_decode_workspace_size.argtypes = [i, i, i, i, i, ll]
    L.attn_decode_workspace_size.restype = sz
    L.attn_decode.argtypes = [cp, vp, lp, vp, ll, i, vp, i, i, f, rp, vp, ll, vp, vp, vp, sz, vp]
    L.attn_decode_window_workspace_size.argtypes = [i, i, i, i, i, ll, i, i]
    L.attn_decode_window_workspace_size.restype = sz
    L.attn_decode_window.argtypes = [cp, vp, lp, vp, ll, i, vp, i, i, i, i, f, rp, vp, ll, vp, vp, vp,
                                     sz, vp]
    pp = ctypes.POINTER(_PoolStruct)
    L.attn_pages_release.argtypes = [pp, vp, ll, i, vp, vp, i, vp]
    L.attn_pages_fork.argtypes = [pp, vp, ll, i, vp, i, vp, vp, i, vp, vp, vp]
    L.attn_pages_reserve.argtypes = [pp, vp, ll, i, vp, vp, i, vp]
    L.attn_cache_copy.argtypes = [cp, vp, vp, i, vp]
    L.attn_cache_gather.argtypes = [cp, vp, ll, i, i, vp, vp, i, vp, ll, i, vp, vp]
    L.attn_decode_tree_workspace_size.argtypes = [i, i, i, i, i]
    L.attn_decode_tree_workspace_size.restype = sz
    L.attn_decode_tree.argtypes = [cp, vp, lp, vp, ll, i, vp, i, vp, i, i, vp, ll, i, i, i, f, vp, vp,
                                   vp, sz, vp]
    for name in ("attn_rope_init", "attn_rope", "attn_cache_append", "attn_decode", "attn_decode_window",
                 "attn_decode_tree",
                 "attn_pages_release", "attn_pages_fork", "attn_pages_reserve", "attn_cache_copy",
                 "attn_cache_gather"):
        getattr(L, name).restype = ctypes.c_int
    for name in ("attn_fwd", "attn_bwd", "attn_partial_fwd", "attn_split_fwd", "attn_merge",
                 "attn_poll_device_status", "attn_fwd_varlen", "attn_bwd_varlen", "attn_fwd_gqa",
                 "attn_bwd_gqa", "attn_fwd_fp8", "attn_fwd_varlen_gqa", "attn_bwd_varlen_gqa"):
        getattr(L, name).restype = ctypes.c_int
    return L


def lib():
    """The loaded libattn.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(_build.LIB):
            raise ImportError(
                f"{_build.LIB} is missing: build it with "
                "`python -c 'import exact_blockwise_attention_gb300._build as b; b.build()'`")
        _LIB = _declare(ctypes.CDLL(_build.LIB))
    return _LIB


def status_string(status: int) -> str:
    return lib().attn_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != ATTN_OK:
        raise AttnError(fn, status)


def _ptr(t: torch.Tensor) -> int:
    return t.data_ptr()


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _require(t, name, dtype, ndim=4, device_type="cuda"):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.device.type != device_type:
        raise ValueError(f"{name} must be a {device_type.upper()} tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _qkv(q, k, v, gqa=False, device_type="cuda"):
    for n, t in (("q", q), ("k", k), ("v", v)):
        _require(t, n, torch.bfloat16, device_type=device_type)
    B, H, Lq, d = q.shape
    Hkv = k.shape[1]
    heads_ok = Hkv == H or (gqa and Hkv >= 1 and H % Hkv == 0)
    if k.shape[0] != B or not heads_ok or k.shape[3] != d or v.shape != k.shape:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on the same device")
    if gqa:
        return B, H, Hkv, Lq, k.shape[2], d
    return B, H, Lq, k.shape[2], d


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def fwd(q, k, v, scale=None):
    """Exact attention forward: returns (o bf16 [B,H,Lq,d], lse fp32 [B,H,Lq]).
    k, v may have H_kv < H heads (grouped-query attention)."""
    B, H, Hkv, Lq, Lk, d = _qkv(q, k, v, gqa=True)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Lq), device=q.device, dtype=torch.float32)
    with torch.cuda.device(q.device):
        if Hkv == H:
            _check("attn_fwd", lib().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H,
                                              Lq, Lk, d, _scale(scale, d), _stream()))
        else:
            _check("attn_fwd_gqa", lib().attn_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                                      _ptr(lse), B, H, Hkv, Lq, Lk, d,
                                                      _scale(scale, d), _stream()))
    return o, lse


def bwd_workspace_size(B, H, Lq, Lk, d) -> int:
    return int(lib().attn_bwd_workspace_size(B, H, Lq, Lk, d))


def _bwd_inputs(q, k, v, o, do, lse, gqa, device_type="cuda"):
    """Checks shared by the backward entry points: q, k, v as for the forward,
    o and do shaped like q (bf16, contiguous, same device), lse [B, H, Lq] fp32."""
    dims = _qkv(q, k, v, gqa=gqa, device_type=device_type)
    B, H, Lq = q.shape[0], q.shape[1], q.shape[2]
    _require(o, "o", torch.bfloat16, device_type=device_type)
    _require(do, "do", torch.bfloat16, device_type=device_type)
    _require(lse, "lse", torch.float32, ndim=3, device_type=device_type)
    if o.shape != q.shape or do.shape != q.shape or lse.shape != (B, H, Lq):
        raise ValueError("o/do must match q and lse must be [B,H,Lq]")
    if not (o.device == do.device == lse.device == q.device):
        raise ValueError("o, do and lse must be on q's device")
    return dims


def _noalloc_out(q, k, v, out, device_type="cuda"):
    """The caller's (dq, dk, dv) for bwd_noalloc: bf16, contiguous, on q's
    device and shaped like q, k and v, so the kernels never write past them."""
    if not isinstance(out, (tuple, list)) or len(out) != 3:
        raise ValueError("out must be a (dq, dk, dv) tuple")
    for name, t, src, like in zip(("dq", "dk", "dv"), out, "qkv", (q, k, v)):
        _require(t, name, torch.bfloat16, device_type=device_type)
        if t.shape != like.shape or t.device != q.device:
            raise ValueError(f"{name} must be shaped like {src} {tuple(like.shape)} on {q.device}, "
                             f"got {tuple(t.shape)} on {t.device}")
    return tuple(out)


def bwd(q, k, v, o, do, lse, scale=None, workspace=None):
    """Gradients (dq, dk, dv) of sum(o * do); P is recomputed from lse. With
    grouped-query k, v (H_kv < H heads), dk and dv sum over each group."""
    B, H, Hkv, Lq, Lk, d = _bwd_inputs(q, k, v, o, do, lse, gqa=True)
    need = bwd_workspace_size(B, H, Lq, Lk, d)
    if workspace is None:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    elif workspace.numel() * workspace.element_size() < need or not workspace.is_cuda:
        raise ValueError(f"workspace must be a CUDA tensor of at least {need} bytes")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ptrs = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv))
    with torch.cuda.device(q.device):
        if Hkv == H:
            _check("attn_bwd", lib().attn_bwd(*ptrs, B, H, Lq, Lk, d, _scale(scale, d),
                                              _ptr(workspace), need, _stream()))
        else:
            _check("attn_bwd_gqa", lib().attn_bwd_gqa(*ptrs, B, H, Hkv, Lq, Lk, d,
                                                      _scale(scale, d), _ptr(workspace), need,
                                                      _stream()))
    return dq, dk, dv


def bwd_noalloc(q, k, v, o, do, lse, scale=None, out=None):
    """bwd() for callers that cannot allocate device memory: the scratch comes
    from a 64 MiB buffer built into the library (see attn_bwd_noalloc in
    include/attn.h). Pass preallocated ``out=(dq, dk, dv)`` to allocate
    nothing at all from Python either; they are checked (bf16, contiguous,
    on q's device, shaped like q, k, v) before the library is called."""
    B, H, Lq, Lk, d = _bwd_inputs(q, k, v, o, do, lse, gqa=False)
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    dq, dk, dv = _noalloc_out(q, k, v, out)
    with torch.cuda.device(q.device):
        _check("attn_bwd_noalloc", lib().attn_bwd_noalloc(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
            B, H, Lq, Lk, d, _scale(scale, d), _stream()))
    return dq, dk, dv


def partial_fwd(q, k, v, k0, k1, scale=None):
    """Attention over keys [k0, k1): (o_part fp32 [B,H,Lq,d], lse_part fp32 [B,H,Lq])."""
    B, H, Lq, Lk, d = _qkv(q, k, v)
    o = torch.empty((B, H, Lq, d), device=q.device, dtype=torch.float32)
    lse = torch.empty((B, H, Lq), device=q.device, dtype=torch.float32)
    with torch.cuda.device(q.device):
        _check("attn_partial_fwd", lib().attn_partial_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Lq, Lk, d, int(k0), int(k1),
            _scale(scale, d), _stream()))
    return o, lse


def split_fwd(q, k, v, bounds, scale=None):
    """Partial attention for every chunk [bounds[c], bounds[c+1]) in one launch."""
    B, H, Lq, Lk, d = _qkv(q, k, v)
    bounds = [int(b) for b in bounds]
    C = len(bounds) - 1
    if C < 1:
        raise ValueError("bounds needs at least two entries")
    arr = (ctypes.c_int * len(bounds))(*bounds)
    o = torch.empty((C, B, H, Lq, d), device=q.device, dtype=torch.float32)
    lse = torch.empty((C, B, H, Lq), device=q.device, dtype=torch.float32)
    with torch.cuda.device(q.device):
        _check("attn_split_fwd", lib().attn_split_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Lq, Lk, d, arr, C,
            _scale(scale, d), _stream()))
    return o, lse


def merge(o_parts, lse_parts):
    """Exact merge of partials: (o bf16 [B,H,Lq,d], lse fp32 [B,H,Lq])."""
    _require(o_parts, "o_parts", torch.float32, ndim=5)
    _require(lse_parts, "lse_parts", torch.float32, ndim=4)
    C, B, H, Lq, d = o_parts.shape
    if lse_parts.shape != (C, B, H, Lq):
        raise ValueError("lse_parts must be [C,B,H,Lq] matching o_parts")
    o = torch.empty((B, H, Lq, d), device=o_parts.device, dtype=torch.bfloat16)
    lse = torch.empty((B, H, Lq), device=o_parts.device, dtype=torch.float32)
    with torch.cuda.device(o_parts.device):
        _check("attn_merge", lib().attn_merge(_ptr(o_parts), _ptr(lse_parts), C, _ptr(o),
                                              _ptr(lse), B, H, Lq, d, _stream()))
    return o, lse


def fwd_fp8(q8, k8, vt8, q_scale, k_scale, v_scale, scale=None):
    """Forward with e4m3 operands (d = 128): q8 [B,H,Lq,128], k8 [B,H,Lk,128] and
    vt8 = V transposed [B,H,128,Lk], torch.float8_e4m3fn, with per-tensor
    dequantisation scales (real value = stored value * scale). Returns
    (o bf16 [B,H,Lq,128], lse fp32 [B,H,Lq])."""
    f8 = getattr(torch, "float8_e4m3fn")
    for n, t in (("q8", q8), ("k8", k8), ("vt8", vt8)):
        _require(t, n, f8)
    B, H, Lq, d = q8.shape
    Lk = k8.shape[2]
    if k8.shape != (B, H, Lk, d) or vt8.shape != (B, H, d, Lk):
        raise ValueError(f"shape mismatch: q8 {tuple(q8.shape)} k8 {tuple(k8.shape)} "
                         f"vt8 {tuple(vt8.shape)} (vt8 is V transposed, [B,H,d,Lk])")
    o = torch.empty((B, H, Lq, d), device=q8.device, dtype=torch.bfloat16)
    lse = torch.empty((B, H, Lq), device=q8.device, dtype=torch.float32)
    with torch.cuda.device(q8.device):
        _check("attn_fwd_fp8", lib().attn_fwd_fp8(
            _ptr(q8), _ptr(k8), _ptr(vt8), _ptr(o), _ptr(lse), B, H, Lq, Lk, d, _scale(scale, d),
            float(q_scale), float(k_scale), float(v_scale), _stream()))
    return o, lse


def _cu(cu, name):
    """Host int array of cumulative lengths (a sequence of ints or a CPU tensor)."""
    if isinstance(cu, torch.Tensor):
        if cu.device.type != "cpu":
            raise ValueError(f"{name} must be on the host (cumulative lengths are read by the CPU)")
        cu = cu.tolist()
    vals = [int(x) for x in cu]
    if len(vals) < 2:
        raise ValueError(f"{name} needs at least two entries")
    return vals, (ctypes.c_int * len(vals))(*vals)


def _varlen_qkv(q, k, v, cu_q, cu_k):
    for n, t in (("q", q), ("k", k), ("v", v)):
        _require(t, n, torch.bfloat16, ndim=3)
    Tq, H, d = q.shape
    Hkv = k.shape[1]
    if k.shape[2] != d or not (Hkv >= 1 and H % Hkv == 0) or v.shape != k.shape:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    cq, aq = _cu(cu_q, "cu_q")
    ck, ak = _cu(cu_k, "cu_k")
    if len(cq) != len(ck):
        raise ValueError("cu_q and cu_k must have the same length")
    if cq[-1] != Tq or ck[-1] != k.shape[0]:
        raise ValueError("cu_q[-1] / cu_k[-1] must equal the packed token counts")
    return Tq, H, Hkv, d, aq, ak, len(cq) - 1


def fwd_varlen(q, k, v, cu_q, cu_k, scale=None):
    """Exact attention within each packed sequence: (o bf16 [Tq,H,d], lse fp32 [H,Tq]).
    k, v may have H_kv < H heads (grouped-query attention)."""
    Tq, H, Hkv, d, aq, ak, n = _varlen_qkv(q, k, v, cu_q, cu_k)
    o = torch.empty_like(q)
    lse = torch.empty((H, Tq), device=q.device, dtype=torch.float32)
    with torch.cuda.device(q.device):
        _check("attn_fwd_varlen_gqa", lib().attn_fwd_varlen_gqa(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), aq, ak, n, H, Hkv, d, _scale(scale, d),
            _stream()))
    return o, lse


def bwd_varlen_workspace_size(Tq, H, d, n_seqs) -> int:
    return int(lib().attn_bwd_varlen_workspace_size(Tq, H, d, n_seqs))


def bwd_varlen(q, k, v, o, do, lse, cu_q, cu_k, scale=None, workspace=None):
    """Gradients (dq, dk, dv) of sum(o * do) over packed sequences (dk, dv summed
    over each group of query heads when k, v have fewer heads)."""
    Tq, H, Hkv, d, aq, ak, n = _varlen_qkv(q, k, v, cu_q, cu_k)
    _require(o, "o", torch.bfloat16, ndim=3)
    _require(do, "do", torch.bfloat16, ndim=3)
    _require(lse, "lse", torch.float32, ndim=2)
    if o.shape != q.shape or do.shape != q.shape or lse.shape != (H, Tq):
        raise ValueError("o/do must match q and lse must be [H,Tq]")
    need = bwd_varlen_workspace_size(Tq, H, d, n)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    elif workspace.numel() * workspace.element_size() < need or not workspace.is_cuda:
        raise ValueError(f"workspace must be a CUDA tensor of at least {need} bytes")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    with torch.cuda.device(q.device):
        _check("attn_bwd_varlen_gqa", lib().attn_bwd_varlen_gqa(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
            aq, ak, n, H, Hkv, d, _scale(scale, d), _ptr(workspace), need, _stream()))
    return dq, dk, dv


def poll_device_status() -> int:
    """Synchronise the current stream; return the status word (0 ok, 5 a wait timed
    out, 7 a cached length or page was out of range)."""
    return int(lib().attn_poll_device_status(_stream()))


def set_wait_limit_ns(ns: int) -> int:
    return int(lib().attn_set_wait_limit_ns(int(ns)))


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, scale):
        o, lse = fwd(q, k, v, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.scale = scale
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv = bwd(q, k, v, o, do.contiguous(), lse, ctx.scale)
        return dq, dk, dv, None


def attention(q, k, v, scale=None):
    """Autograd-aware exact attention; only o and lse are saved for backward."""
    return _Attention.apply(q, k, v, scale)


def _sides(left, right, sinks):
    """left, right and sinks as the C ABI takes them (None: no end to that side)."""
    out = []
    for name, x in (("left", left), ("right", right), ("sinks", sinks)):
        if x is None and name != "sinks":
            x = -1
        elif not isinstance(x, int) or not 0 <= x < 1 << 31:
            raise ValueError(f"{name} must be an int of at least 0, got {x!r}")
        out.append(x)
    return out


def _few_keys(Lq, Lk, left, right, sinks):
    """Whether no row sees more than 512 keys, sinks among them (left, right -1: no end), or 1024
    where the first or the last row sees fewer than 8, as plain causal attention's does; a
    training step then keeps what rounding took from o. The error of dq and dk goes from
    0.0038 to 0.0025 with 2 keys a row, 0.0027 to 0.0024 with 8, 0.00243 to 0.00238 with 61,
    from 0.00250 to 0.00240 for 600 and 1000 causal tokens (steps of 189 and 226 us take 201 and
    240), 0.00248 to 0.00240 for 1500, and a step of 12544 tokens that see 1568 each would take
    838 us instead of 808."""
    left, right = (Lq + Lk if x < 0 else x for x in (left, right))

    def seen(place):
        first = max(place - left, 0)
        return min(place + right, Lk - 1) - first + 1 + min(sinks, first)

    fewest = min(seen(max(Lk - Lq, -right)), seen(Lk - 1))
    return min(Lk, left + right + 1 + sinks) <= (1024 if fewest < 8 else 512)


_WINDOW_LAYOUTS = None  # _Layouts, below


def _window_layout(q, k, v, left, right, sinks):
    """A windowed call's sizes and window as the C ABI takes them, the bytes of the
    backward's workspace, and whether a training step keeps what rounding took from o;
    its checks are made once for each form of tensors."""
    try:
        key = (_form(q), _form(k), _form(v), left, right, sinks, type(left), type(right), type(sinks))
        lay = _WINDOW_LAYOUTS.get(key)
    except AttributeError:
        lay = key = None
    if lay is None:
        sizes = _qkv(q, k, v, gqa=True)
        window = _sides(left, right, sinks)
        lay = ((*sizes, *window), int(lib().attn_bwd_window_workspace_size(*sizes, *window)),
               _few_keys(*sizes[3:5], *window))
        _WINDOW_LAYOUTS.add(key, lay)
    return lay


def _fwd_window(q, k, v, sizes, scale, rest):
    o = torch.empty_like(q)
    rest = torch.empty_like(q) if rest else None
    lse = torch.empty(sizes[0:2] + sizes[3:4], device=q.device, dtype=torch.float32)
    _launch(q.device, lib().attn_fwd_window, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
            None if rest is None else rest.data_ptr(), lse.data_ptr(), *sizes, _scale(scale, sizes[5]))
    return o, lse, rest


def _bwd_window(q, k, v, o, do, lse, sizes, need, scale, workspace, rest):
    if workspace is None:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    elif workspace.numel() * workspace.element_size() < need or workspace.device != q.device or \
            not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor of at least {need} bytes on {q.device}")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    _launch(q.device, lib().attn_bwd_window, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
            None if rest is None else rest.data_ptr(), do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), *sizes, _scale(scale, sizes[5]), workspace.data_ptr(), need)
    return dq, dk, dv


def fwd_window(q, k, v, left, right=0, sinks=0, scale=None, rest=False):
    """Attention within a sliding window and to the first tokens: (o bf16 [B,H,Lq,d],
    lse fp32 [B,H,Lq]).

    Query i stands at the place p = i + Lk - Lq, the last query at the last key, and
    sees the keys p - left to p + right and, up to p + right, the first ``sinks``. left
    or right None: no end to that side (left=None is plain causal attention). ``decode``'s
    and ``decode_tree``'s window of W keys is left = W - 1. A query that sees no key gives
    o = 0 and lse = -inf. k, v may have H_kv < H heads.

    With ``rest`` a third tensor, of o's shape and type: what rounding took from o, for
    bwd_window."""
    out = _fwd_window(q, k, v, _window_layout(q, k, v, left, right, sinks)[0], scale, rest)
    return out if rest else out[:2]


def bwd_window_workspace_size(B, H, H_kv, Lq, Lk, d, left, right=0, sinks=0) -> int:
    return int(lib().attn_bwd_window_workspace_size(B, H, H_kv, Lq, Lk, d, *_sides(left, right, sinks)))


def bwd_window(q, k, v, o, do, lse, left, right=0, sinks=0, scale=None, workspace=None, rest=None):
    """Gradients (dq, dk, dv) of sum(o * do) for fwd_window; P is recomputed from lse.
    Keys that no query sees, and queries that see no key, have zero gradients. With
    fwd_window's ``rest`` dq and dk are more exact where rows see few keys."""
    sizes, need, _ = _window_layout(q, k, v, left, right, sinks)
    _bwd_inputs(q, k, v, o, do, lse, gqa=True)
    if rest is not None:
        _bwd_inputs(q, k, v, rest, do, lse, gqa=True)
    return _bwd_window(q, k, v, o, do, lse, sizes, need, scale, workspace, rest)


class _AttentionWindow(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, left, right, sinks, scale):
        sizes, need, few = _window_layout(q, k, v, left, right, sinks)
        o, lse, rest = _fwd_window(q, k, v, sizes, scale, few and any(ctx.needs_input_grad[:2]))
        ctx.save_for_backward(q, k, v, o, lse, rest)
        ctx.call = sizes, need, scale
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, rest = ctx.saved_tensors
        do = do.contiguous()
        if do.data_ptr() & 15:  # autograd also hands over views
            do = do.clone()
        grads = _bwd_window(q, k, v, o, do, lse, *ctx.call, None, rest)
        need = ctx.needs_input_grad
        return (grads[0] if need[0] else None, grads[1] if need[1] else None, grads[2] if need[2] else None,
                None, None, None, None)


def attention_window(q, k, v, left, right=0, sinks=0, scale=None):
    """Autograd-aware fwd_window; only o and lse are saved for backward, and where no row
    sees more than 512 keys, or some fewer than 8 and none more than 1024, what rounding
    took from o."""
    return _AttentionWindow.apply(q, k, v, left, right, sinks, scale)


class _AttentionVarlen(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k, scale):
        o, lse = fwd_varlen(q, k, v, cu_q, cu_k, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.cu = (cu_q, cu_k)
        ctx.scale = scale
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv = bwd_varlen(q, k, v, o, do.contiguous(), lse, *ctx.cu, ctx.scale)
        return dq, dk, dv, None, None, None


def attention_varlen(q, k, v, cu_q, cu_k, scale=None):
    """Autograd-aware exact attention over packed sequences (token-major
    [T, H, d]; cu_q, cu_k host cumulative lengths)."""
    return _AttentionVarlen.apply(q, k, v, cu_q, cu_k, scale)


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

_Strides2, _Strides3 = ctypes.c_longlong * 2, ctypes.c_longlong * 3


def _rows(t, name, ndim, device_type="cuda"):
    """Checks a bf16 tensor of rows (the last dimension contiguous, every row on
    a 16-byte boundary) and returns the strides of its other dimensions, 0 for
    those of size 1."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.device.type != device_type:
        raise ValueError(f"{name} must be a {device_type.upper()} tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    shape = t.shape
    if len(shape) != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {len(shape)}")
    if shape[-1] not in (64, 128):
        raise ValueError(f"{name}'s head dimension must be 64 or 128, got {shape[-1]}")
    strides = t.stride()
    if strides[-1] != 1:
        raise ValueError(f"{name}'s heads must be contiguous rows")
    out = [s if n != 1 else 0 for s, n in zip(strides[:-1], shape)]
    if any(s & 7 for s in out) or t.data_ptr() & 15:
        raise ValueError(f"{name}'s rows must start on 16-byte boundaries")
    return out


def _int32(t, name, device, ndim=None):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
        raise ValueError(f"{name} must be an int32 tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


class Rope:
    """A rotation by position over one or several axes (attn_rope_t).

    axis_pairs   pairs of a head's elements that each axis turns, e.g. (8, 12, 12)
                 for time, height and width of a 64-element head, or (64,) for
                 text positions of a 128-element one; together a multiple of 8.
                 The first 2 * sum(axis_pairs) elements of a head are rotated.
    theta        pair i of an axis with n pairs turns by theta ** (-i / n) radians
                 a position
    pairing      "half": pair i is elements (i, i + sum(axis_pairs));
                 "interleaved": elements (2 i, 2 i + 1)
    frequencies  the pairs' radians a position instead of theta's (scaled long
                 contexts, one spectrum over all axes, 0 for a pair that stays)
    """

    def __init__(self, axis_pairs, theta=10000.0, pairing="half", frequencies=None):
        axis_pairs = [int(n) for n in axis_pairs]
        if not axis_pairs or min(axis_pairs) < 1 or len(axis_pairs) > MAX_AXES:
            raise ValueError(f"axis_pairs must hold 1 to {MAX_AXES} positive numbers")
        n = sum(axis_pairs)
        if n % 8 or n > MAX_PAIRS:
            raise ValueError(f"axis_pairs must add up to a multiple of 8, at most {MAX_PAIRS}, got {n}")
        if pairing not in ("half", "interleaved"):
            raise ValueError(f"pairing must be 'half' or 'interleaved', got {pairing!r}")
        if frequencies is None:
            theta = float(theta)
            if not (math.isfinite(theta) and theta > 0):
                raise ValueError("theta must be finite and positive")
            frequencies = [theta ** (-i / m) for m in axis_pairs for i in range(m)]
        frequencies = [float(x) for x in frequencies]
        if len(frequencies) != n or not all(map(math.isfinite, frequencies)):
            raise ValueError(f"frequencies must be {n} finite numbers")
        axes = [a for a, m in enumerate(axis_pairs) for _ in range(m)]
        self.axis_pairs, self.n_axes, self.n_pairs = tuple(axis_pairs), len(axis_pairs), n
        self.pairing, self.frequencies = pairing, tuple(frequencies)
        self._struct = _RopeStruct()
        _check("attn_rope_init", lib().attn_rope_init(
            self._struct, n, self.n_axes, (ctypes.c_int * n)(*axes),
            (ctypes.c_double * n)(*frequencies), int(pairing == "interleaved")))

    def _positions(self, t, device, tokens):
        """Positions [n_axes, *tokens] (one axis: tokens alone); returns the axis' stride."""
        _int32(t, "positions", device)
        shape = tuple(t.shape)
        if self.n_axes == 1 and shape == tokens:
            return 0
        if shape != (self.n_axes, *tokens):
            raise ValueError(f"positions must be {(self.n_axes, *tokens)}, got {shape}")
        return t.stride(0)


def _launch(device, fn, *args):
    """Call an entry point on the current stream of ``device``. (The raw handle:
    building a Stream object takes longer than the launch.)"""
    index = device.index
    if index == torch.cuda.current_device():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != ATTN_OK:
        raise AttnError(fn.__name__, st)


class _Layouts(dict):
    """What a call's checks made of its tensors' shapes, strides, types and
    devices, by those alone: calls of the same form skip the checks, which take
    longer than a small launch. Addresses are checked in every call."""

    def add(self, key, value):
        if len(self) >= 1024:
            self.clear()
        self[key] = value
        return value


def _form(t):
    """What a tensor's checks depend on (None stays None)."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _off_boundary(name):
    return ValueError(f"{name}'s rows must start on 16-byte boundaries")


_ROPE_LAYOUTS = _Layouts()
_WINDOW_LAYOUTS = _Layouts()


def _rope_layout(q, k, positions, plan):
    """Checks a rotation's arguments: sizes, strides (batch, head, token) and the
    output's strides, as the C ABI takes them."""
    if not isinstance(plan, Rope):
        raise ValueError("plan must be a Rope")
    nd = q.dim() if isinstance(q, torch.Tensor) else 0
    if nd not in (3, 4):
        raise ValueError("q must be a [B, H, L, d] or [T, H, d] tensor")
    packed = nd == 3
    sq = _rows(q, "q", nd)
    d = q.shape[-1]
    if 2 * plan.n_pairs > d:
        raise ValueError(f"the plan rotates {2 * plan.n_pairs} elements of a head of {d}")
    B, H, L = (1, q.shape[1], q.shape[0]) if packed else q.shape[:3]

    def order(s):
        return _Strides3(0, s[1], s[0]) if packed else _Strides3(*s)

    def fresh(heads):
        return _Strides3(0, d, heads * d) if packed else _Strides3(heads * L * d, L * d, d)

    Hk, sk, sko = 0, None, None
    if k is not None:
        sk = order(_rows(k, "k", nd))
        Hk = k.shape[1]
        like = (L, Hk, d) if packed else (B, Hk, L, d)
        if tuple(k.shape) != like or k.device != q.device:
            raise ValueError(f"k must be {like} on {q.device}, got {tuple(k.shape)} on {k.device}")
        sko = fresh(Hk)
    per_batch = (not packed and isinstance(positions, torch.Tensor)
                 and positions.dim() == (2 if plan.n_axes == 1 and positions.dim() < 3 else 3)
                 and positions.shape[-2] == B)
    if per_batch:
        axis, batch = plan._positions(positions, q.device, (B, L)), positions.stride(-2)
    else:
        axis, batch = plan._positions(positions, q.device, (L,)), 0
    return (order(sq), fresh(H), sk, sko, _Strides2(axis, batch), B, H, Hk, L, d)


def _rope(q, k, positions, plan, inverse):
    try:
        key = (_form(q), _form(k), _form(positions), plan.n_axes, plan.n_pairs)
        lay = _ROPE_LAYOUTS.get(key)
    except AttributeError:
        lay = key = None
    if lay is None:
        lay = _rope_layout(q, k, positions, plan)
        _ROPE_LAYOUTS.add(key, lay)
    sq, sqo, sk, sko, sp, B, H, Hk, L, d = lay
    qp = q.data_ptr()
    if qp & 15:
        raise _off_boundary("q")
    qo = torch.empty_like(q, memory_format=torch.contiguous_format)
    ko = kp = kop = None
    if k is not None:
        kp = k.data_ptr()
        if kp & 15:
            raise _off_boundary("k")
        ko = torch.empty_like(k, memory_format=torch.contiguous_format)
        kop = ko.data_ptr()
    _launch(q.device, lib().attn_rope, plan._struct, qp, sq, qo.data_ptr(), sqo, kp, sk, kop, sko,
            positions.data_ptr(), sp, B, H, Hk, L, d, inverse)
    return qo, ko


def rope_fwd(q, k, positions, plan):
    """q and k (or None) rotated by their tokens' positions: new contiguous tensors.

    q [B, H, L, d] with k [B, H_k, L, d], or token-major q [T, H, d] with k
    [T, H_k, d]; positions int32 on the device, [n_axes, L] (shared by the batch),
    [n_axes, B, L] or [n_axes, T]; with one axis its dimension may be left out."""
    return _rope(q, k, positions, plan, False)


def rope_bwd(dq, dk, positions, plan):
    """Gradients of rope_fwd's inputs from those of its outputs (the rotation back)."""
    return _rope(dq, dk, positions, plan, True)


class _Rotation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, plan, inverse):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions)
        ctx.plan, ctx.inverse = plan, inverse
        return _rope(q, k, positions, plan, inverse)

    @staticmethod
    def backward(ctx, dq, dk):
        (positions,) = ctx.saved_tensors
        # (under create_graph the gradient is a rotation with a gradient of its own)
        turn = _Rotation.apply if torch.is_grad_enabled() else _rope
        plan, back = ctx.plan, not ctx.inverse
        # (an output's gradient comes also where its input wants none)
        need_q, need_k = ctx.needs_input_grad[:2]
        dq, dk = dq if need_q else None, dk if need_k else None
        try:
            if dq is not None:
                dq, dk = turn(dq, dk, positions, plan, back)
            elif dk is not None:
                dk, dq = turn(dk, None, positions, plan, back)
        except ValueError:  # autograd also hands over expanded and transposed gradients
            dq, dk = (g if g is None else g.clone(memory_format=torch.contiguous_format)
                      for g in (dq, dk))
            if dq is not None:
                dq, dk = turn(dq, dk, positions, plan, back)
            else:
                dk, dq = turn(dk, None, positions, plan, back)
        return dq, dk, None, None, None


def rope(q, k, positions, plan):
    """Autograd-aware rope_fwd; only the positions are saved for backward."""
    return _Rotation.apply(q, k, positions, plan, False)


# ---------------------------------------------------------------------------
# The paged key-value cache
# ---------------------------------------------------------------------------

_CACHE_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}


class PagedCache:
    """Pages of keys and values, [n_pages, page_size, H_kv, d] each, bf16 or
    float8_e4m3fn (a stored value then stands for itself times k_scale or
    v_scale). The dimensions before d may be strided, so pages laid out
    [n_pages, H_kv, page_size, d] are passed as a transposed view. The tensors
    stay the caller's; the handle keeps their layout and the scales."""

    def __init__(self, k, v, k_scale=1.0, v_scale=1.0):
        s = _CacheStruct()
        for name, t in (("k", k), ("v", v)):
            if not isinstance(t, torch.Tensor) or t.dim() != 4:
                raise ValueError(f"{name} must be a [n_pages, page_size, H_kv, d] tensor")
            if t.dtype not in _CACHE_TYPES:
                raise ValueError(f"{name} must be bfloat16 or float8_e4m3fn, got {t.dtype}")
            if t.shape != k.shape or t.dtype != k.dtype or t.device != k.device:
                raise ValueError("k and v must have the same shape, type and device")
            if t.numel() == 0 or t.shape[3] not in (64, 128):
                raise ValueError(f"{name} must hold pages of heads of 64 or 128, got {tuple(t.shape)}")
            if t.stride(3) != 1:
                raise ValueError(f"{name}'s heads must be contiguous rows")
            strides = [st if n != 1 else 0 for st, n in zip(t.stride()[:3], t.shape)]
            if any(st * t.element_size() % 16 for st in strides) or t.data_ptr() % 16:
                raise ValueError(f"{name}'s rows must start on 16-byte boundaries")
            reach = t.shape[3]  # rows must not overlap: each is written by itself
            for st, n in sorted((st, n) for st, n in zip(strides, t.shape) if n != 1):
                if st < reach:
                    raise ValueError(f"{name}'s rows must not overlap")
                reach += st * (n - 1)
            getattr(s, name + "_strides")[:] = strides
        if k.data_ptr() == v.data_ptr():
            raise ValueError("k and v must be different tensors")
        for name, x in (("k_scale", k_scale), ("v_scale", v_scale)):
            if not (math.isfinite(x) and x > 0):
                raise ValueError(f"{name} must be finite and positive")
            if k.dtype == torch.bfloat16 and x != 1:
                raise ValueError(f"{name} must be 1 for a bfloat16 cache")
        s.n_pages, s.page_size, s.H_kv, s.d = k.shape
        s.type, s.k_scale, s.v_scale = _CACHE_TYPES[k.dtype], float(k_scale), float(v_scale)
        self.k, self.v, self.k_scale, self.v_scale = k, v, float(k_scale), float(v_scale)
        self.n_pages, self.page_size, self.H_kv, self.d = k.shape
        self.device = k.device
        # what the checks of a call depend on
        self._key = (self.H_kv, self.d, self.page_size, k.dtype, self.device)
        self._struct = s

    def _at(self):
        if self.device.type != "cuda":
            raise ValueError("the cache must be on a CUDA device")
        self._struct.k, self._struct.v = self.k.data_ptr(), self.v.data_ptr()
        return self._struct

    def _batch(self, page_table, seq_lens):
        """Checks a batch's page table and lengths; returns the number of sequences."""
        _int32(page_table, "page_table", self.device, 2)
        _int32(seq_lens, "seq_lens", self.device, 1)
        n = seq_lens.shape[0]
        if page_table.shape[0] != n or n < 1 or page_table.shape[1] < 1:
            raise ValueError(f"page_table must be [n_seqs, max_pages] for {n} sequences, "
                             f"got {tuple(page_table.shape)}")
        return n

    def _turn(self, rope, positions, tokens):
        """The rotation's arguments: its struct, the positions' address and axis stride."""
        if rope is None:
            if positions is not None:
                raise ValueError("positions are used with a rope only")
            return None, None, 0
        if not isinstance(rope, Rope):
            raise ValueError("rope must be a Rope")
        if 2 * rope.n_pairs > self.d:
            raise ValueError(f"the rope rotates {2 * rope.n_pairs} elements of a head of {self.d}")
        if positions is None:
            if rope.n_axes != 1:
                raise ValueError("positions are needed for a rope with several axes")
            return rope._struct, None, 0
        stride = rope._positions(positions, self.device, (tokens,))
        return rope._struct, positions.data_ptr(), stride


def cache_append(cache, k, v, page_table, seq_lens, cu_new=None, rope=None, positions=None):
    """Write new keys (rotated by ``rope``) and values, [T, H_kv, d] bf16, into the
    cache's pages.

    page_table int32 [n_seqs, max_pages] and seq_lens int32 [n_seqs] on the
    device; seq_lens counts the new tokens, the last ones of their sequences.
    cu_new int32 [n_seqs + 1] on the device: sequence b's new tokens are rows
    cu_new[b] .. cu_new[b + 1]; without it each sequence has one. Rows outside
    cu_new and those of a sequence of length 0 are left out. positions int32
    [n_axes, T]; without them (one axis) a token's place in its sequence. The
    pages written must not be shared. Lengths and pages out of range write
    nothing and are reported by poll_device_status."""
    try:
        key = (_form(k), _form(v), _form(page_table), _form(seq_lens), _form(cu_new), _form(positions),
               cache._key, None if rope is None else (rope.n_axes, rope.n_pairs))
        lay = _APPEND_LAYOUTS.get(key)
    except AttributeError:
        lay = key = None
    if lay is None:
        lay = _append_layout(cache, k, v, page_table, seq_lens, cu_new, rope, positions)
        _APPEND_LAYOUTS.add(key, lay)
    sk, sv, row, wide, n, T, stride = lay
    kp, vp = k.data_ptr(), v.data_ptr()
    if (kp | vp) & 15:
        raise _off_boundary("k's or v")
    _launch(cache.device, lib().attn_cache_append, cache._at(), kp, sk, vp, sv,
            page_table.data_ptr(), row, wide, seq_lens.data_ptr(), n,
            None if cu_new is None else cu_new.data_ptr(), T, None if rope is None else rope._struct,
            None if positions is None else positions.data_ptr(), stride)


_APPEND_LAYOUTS = _Layouts()


def _append_layout(cache, k, v, page_table, seq_lens, cu_new, rope, positions):
    """Checks an append's arguments: strides and sizes as the C ABI takes them."""
    if not isinstance(cache, PagedCache):
        raise ValueError("cache must be a PagedCache")
    sk, sv = _rows(k, "k", 3), _rows(v, "v", 3)
    T = k.shape[0]
    if k.shape != v.shape or k.shape[1] != cache.H_kv or k.shape[2] != cache.d:
        raise ValueError(f"k and v must be [T, {cache.H_kv}, {cache.d}], got {tuple(k.shape)} "
                         f"and {tuple(v.shape)}")
    if k.device != cache.device or v.device != cache.device:
        raise ValueError(f"k and v must be on {cache.device}")
    n = cache._batch(page_table, seq_lens)
    if cu_new is not None:
        _int32(cu_new, "cu_new", cache.device, 1)
        if cu_new.shape[0] != n + 1:
            raise ValueError(f"cu_new must have {n + 1} entries, got {cu_new.shape[0]}")
    elif T != n:
        raise ValueError(f"without cu_new there is one new token per sequence: {n}, got {T}")
    stride = cache._turn(rope, positions, T)[2]
    return (_Strides2(*sk), _Strides2(*sv), page_table.stride(0), page_table.shape[1], n, T, stride)


def decode_workspace_size(cache, B, H, max_pages, window=None, sinks=0) -> int:
    """Scratch bytes of decode for B sequences of H query heads and a page table of
    max_pages columns; 0 where none is needed."""
    if window is not None:
        return int(lib().attn_decode_window_workspace_size(
            B, H, cache.H_kv, cache.d, cache._struct.type, max_pages * cache.page_size, window, sinks))
    return int(lib().attn_decode_workspace_size(B, H, cache.H_kv, cache.d, cache._struct.type,
                                                max_pages * cache.page_size))


def _window(window, sinks):
    """Checks the window and sinks of a cache call: ints; (None, 0) without a window,
    where the sinks are seen as all other keys are."""
    for name, x, least in (("window", window, 1), ("sinks", sinks, 0)):
        if (name == "sinks" or x is not None) and (not isinstance(x, int) or not least <= x < 1 << 31):
            raise ValueError(f"{name} must be an int of at least {least}, got {x!r}")
    return window, 0 if window is None else sinks


def decode(cache, q, page_table, seq_lens, scale=None, rope=None, positions=None, workspace=None,
           window=None, sinks=0):
    """Attention of one new token per sequence, q [B, H, d] bf16, over the
    seq_lens[b] keys and values its sequence has in the cache: (o bf16 [B, H, d],
    lse fp32 [B, H]); a sequence of length 0 gives o = 0 and lse = -inf.

    H is a multiple of the cache's heads (grouped-query attention). With ``rope``
    q is rotated on the way (and rounded to bf16, as rope_fwd gives it) by
    positions, int32 [n_axes, B], or, with one axis and none given, by
    seq_lens - 1. page_table and seq_lens as for cache_append; the GPU reads
    them, so a captured call follows their contents.

    With a ``window`` the token sees the last that many of its sequence's keys (its own
    among them: fwd_window's left is one less) and the first ``sinks``; pages that hold
    none of these need not be there. Without one ``sinks`` is of no effect: all keys are
    seen."""
    try:
        key = (_form(q), _form(page_table), _form(seq_lens), _form(positions), cache._key, window, sinks,
               type(window), type(sinks),
               None if rope is None else (rope.n_axes, rope.n_pairs))
        lay = _DECODE_LAYOUTS.get(key)
    except AttributeError:
        lay = key = None
    if lay is None:
        lay = _decode_layout(cache, q, page_table, seq_lens, rope, positions, window, sinks)
        _DECODE_LAYOUTS.add(key, lay)
    sq, row, wide, B, H, d, stride, need = lay
    dev = cache.device
    qp = q.data_ptr()
    if qp & 15:
        raise _off_boundary("q")
    if not need:
        workspace = None
    elif workspace is None:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    elif workspace.numel() * workspace.element_size() < need or workspace.device != dev or \
            not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor of at least {need} bytes on {dev}")
    o = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = torch.empty((B, H), device=dev, dtype=torch.float32)
    args = (_scale(scale, d), None if rope is None else rope._struct,
            None if positions is None else positions.data_ptr(), stride, o.data_ptr(),
            lse.data_ptr(), None if workspace is None else workspace.data_ptr(), need)
    if window is None:
        _launch(dev, lib().attn_decode, cache._at(), qp, sq, page_table.data_ptr(), row, wide,
                seq_lens.data_ptr(), B, H, *args)
    else:
        _launch(dev, lib().attn_decode_window, cache._at(), qp, sq, page_table.data_ptr(), row, wide,
                seq_lens.data_ptr(), B, H, window, sinks, *args)
    return o, lse


_DECODE_LAYOUTS = _Layouts()


def _decode_layout(cache, q, page_table, seq_lens, rope, positions, window, sinks):
    """Checks a decode's arguments: strides and sizes as the C ABI takes them, and
    the bytes of workspace."""
    if not isinstance(cache, PagedCache):
        raise ValueError("cache must be a PagedCache")
    sq = _rows(q, "q", 3)
    B, H, d = q.shape
    if d != cache.d or H < 1 or H % cache.H_kv:
        raise ValueError(f"q must be [B, a multiple of {cache.H_kv}, {cache.d}], got {tuple(q.shape)}")
    if q.device != cache.device:
        raise ValueError(f"q must be on {cache.device}")
    n = cache._batch(page_table, seq_lens)
    if n != B:
        raise ValueError(f"q holds {B} sequences, seq_lens {n}")
    stride = cache._turn(rope, positions, B)[2]
    window, sinks = _window(window, sinks)
    return (_Strides2(*sq), page_table.stride(0), page_table.shape[1], B, H, d, stride,
            decode_workspace_size(cache, B, H, page_table.shape[1], window, sinks))


# ---------------------------------------------------------------------------
# Several drafted tokens per sequence
# ---------------------------------------------------------------------------

def decode_tree_workspace_size(cache, T, B, H) -> int:
    """Scratch bytes of decode_tree for T tokens of B sequences with H query heads."""
    return int(lib().attn_decode_tree_workspace_size(T, B, H, cache.H_kv, cache.d))


def decode_tree(cache, q, page_table, seq_lens, cu_q=None, mask=None, window=None, sinks=0, scale=None,
                workspace=None):
    """Attention of several drafted tokens per sequence, q [T, H, d] bf16, over the
    cached keys and values of its sequence, the drafted ones among them: (o bf16
    [T, H, d], lse fp32 [T, H]).

    cu_q int32 [B + 1] on the device: sequence b's tokens are rows cu_q[b] ..
    cu_q[b + 1], and the last ones of its seq_lens[b] keys; without it each sequence
    has one. A token sees the keys before its sequence's drafted ones and, of these,
    those that its mask names, int64 [T] or [T, words] on the device: bit x % 64 of
    word x // 64 for the sequence's x-th drafted token, its own bit among them;
    without a mask those up to itself (a chain of drafts, or the next tokens of a
    prompt).

    With a ``window`` a token at place p sees of the keys before the drafts (without a
    mask: of all) those after p - window and the first ``sinks``; its place is that
    of the drafts' first key plus its place in the chain, or plus the number of its
    mask's bits less one. (The window cuts nothing off a mask: leave out the bits of
    ancestors ``window`` or more places back for what ``decode`` would see.) Pages
    between the sinks and the window of a token at the drafts' first key need not be
    there. Without a window ``sinks`` is of no effect.
    q is taken as it is: rotate it with rope_fwd, the new keys in cache_append.

    A token that sees nothing, or whose sequence has length 0, gives o = 0 and
    lse = -inf; rows of no sequence are not written. The GPU reads lengths, offsets,
    masks and tables, so a captured call follows their contents."""
    try:
        key = (_form(q), _form(page_table), _form(seq_lens), _form(cu_q), _form(mask), cache._key, window,
               sinks, type(window), type(sinks))
        lay = _TREE_LAYOUTS.get(key)
    except AttributeError:
        lay = key = None
    if lay is None:
        lay = _tree_layout(cache, q, page_table, seq_lens, cu_q, mask, window, sinks)
        _TREE_LAYOUTS.add(key, lay)
    sq, row, wide, B, T, H, d, mask_row, words, need = lay
    dev = cache.device
    qp = q.data_ptr()
    if qp & 15:
        raise _off_boundary("q")
    if workspace is None:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    elif workspace.numel() * workspace.element_size() < need or workspace.device != dev or \
            not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor of at least {need} bytes on {dev}")
    o = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = torch.empty((T, H), device=dev, dtype=torch.float32)
    _launch(dev, lib().attn_decode_tree, cache._at(), qp, sq, page_table.data_ptr(), row, wide,
            seq_lens.data_ptr(), B, None if cu_q is None else cu_q.data_ptr(), T, H,
            None if mask is None else mask.data_ptr(), mask_row, words, window or 0, sinks,
            _scale(scale, d), o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), need)
    return o, lse


_TREE_LAYOUTS = _Layouts()


def _tree_layout(cache, q, page_table, seq_lens, cu_q, mask, window, sinks):
    """Checks a tree decode's arguments: strides and sizes as the C ABI takes them, and
    the bytes of workspace."""
    if not isinstance(cache, PagedCache):
        raise ValueError("cache must be a PagedCache")
    sq = _rows(q, "q", 3)
    T, H, d = q.shape
    if T < 1 or d != cache.d or H < 1 or H % cache.H_kv:
        raise ValueError(f"q must be [T, a multiple of {cache.H_kv}, {cache.d}], got {tuple(q.shape)}")
    if q.device != cache.device:
        raise ValueError(f"q must be on {cache.device}")
    B = cache._batch(page_table, seq_lens)
    if cu_q is not None:
        _int32(cu_q, "cu_q", cache.device, 1)
        if cu_q.shape[0] != B + 1:
            raise ValueError(f"cu_q must have {B + 1} entries, got {cu_q.shape[0]}")
    elif T != B:
        raise ValueError(f"without cu_q there is one token per sequence: {B}, got {T}")
    mask_row = words = 0
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dtype != torch.int64 or mask.dim() not in (1, 2):
            raise ValueError("mask must be an int64 [T] or [T, words] tensor")
        words = mask.shape[1] if mask.dim() == 2 else 1
        if mask.device != cache.device or mask.shape[0] != T or not 1 <= words <= MAX_MASK_WORDS:
            raise ValueError(f"mask must be [{T}] or [{T}, 1 to {MAX_MASK_WORDS}] on {cache.device}, "
                             f"got {tuple(mask.shape)} on {mask.device}")
        if words > 1 and mask.stride(1) != 1:
            raise ValueError("mask must be contiguous in its last dimension")
        mask_row = mask.stride(0)
        if mask_row < 0:
            raise ValueError("mask's rows must not run backwards")
    window, sinks = _window(window, sinks)
    return (_Strides2(*sq), page_table.stride(0), page_table.shape[1], B, T, H, d, mask_row, words,
            decode_tree_workspace_size(cache, T, B, H))


# ---------------------------------------------------------------------------
# The cache's pages
# ---------------------------------------------------------------------------

class PagePool:
    """The pages of a cache (or of several that go by one page table, as a model's
    layers do) and how many table entries name each: refs, int32 [n_pages] on the
    device, 0 for a free page. A fresh pool's are all 0; the tensor stays the
    caller's, and pages_release, pages_fork and pages_reserve keep it. They take the
    lowest free pages, in order of the sequences, so what they give depends on the
    counts and tables alone. Calls on one pool run one after the other."""

    def __init__(self, refs, page_size):
        if not isinstance(refs, torch.Tensor) or refs.dtype != torch.int32 or refs.dim() != 1:
            raise ValueError("refs must be an int32 [n_pages] tensor")
        if refs.numel() < 1 or refs.numel() > 1 << 30 or not refs.is_contiguous():
            raise ValueError("refs must be contiguous, for 1 to 2^30 pages")
        page_size = int(page_size)
        if not 1 <= page_size < 1 << 31:
            raise ValueError("page_size must be positive")
        self.refs, self.page_size, self.n_pages, self.device = refs, page_size, refs.numel(), refs.device
        self._scratch = torch.empty_like(refs)
        self._stream = self._here() if refs.is_cuda else None
        self._struct = _PoolStruct(0, self._scratch.data_ptr(), self.n_pages, page_size)

    def _here(self):
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    def _at(self):
        if self.device.type != "cuda":
            raise ValueError("the pool must be on a CUDA device")
        if self._here() != self._stream:  # a pool that goes leaves its scratch to that stream's work
            self._scratch.record_stream(torch.cuda.current_stream(self.device))
        self._struct.refs = self.refs.data_ptr()
        return self._struct


_POOL_LAYOUTS = _Layouts()


def _pool_layout(pool, page_table, lengths, pairs):
    """Checks a pool call's arguments: the table's row stride and columns, the
    sequences, the pairs."""
    if not isinstance(pool, PagePool):
        raise ValueError("pool must be a PagePool")
    _int32(page_table, "page_table", pool.device, 2)
    n, wide = page_table.shape
    if n < 1 or wide < 1 or n * wide >= 1 << 31:
        raise ValueError(f"page_table must be [n_seqs, max_pages], got {tuple(page_table.shape)}")
    if n > 1 and page_table.stride(0) < wide:
        raise ValueError("page_table's rows must not overlap")
    for name, t in lengths:
        _int32(t, name, pool.device, 1)
        if t.shape[0] != n:
            raise ValueError(f"{name} must hold {n} sequences, got {t.shape[0]}")
    for name, t in pairs:
        _int32(t, name, pool.device, 1)
        if t.shape != pairs[0][1].shape:
            raise ValueError("src and dst must have the same length")
    return page_table.stride(0), wide, n


def _pool_call(pool, page_table, lengths, pairs=()):
    try:
        key = (pool.device, _form(page_table), *((name, _form(t)) for name, t in (*lengths, *pairs)))
        lay = _POOL_LAYOUTS.get(key)
    except AttributeError:
        lay = key = None
    if lay is None:
        lay = _pool_layout(pool, page_table, lengths, pairs)
        _POOL_LAYOUTS.add(key, lay)
    return lay


def pages_release(pool, page_table, first, last):
    """Give back the pages that lie wholly within the keys first[b] .. last[b] - 1 of
    each sequence (int32 [n_seqs] on the device): their entries become -1. A page is
    free once no entry names it."""
    row, wide, n = _pool_call(pool, page_table, (("first", first), ("last", last)))
    _launch(pool.device, lib().attn_pages_release, pool._at(), page_table.data_ptr(), row, wide,
            first.data_ptr(), last.data_ptr(), n)


def pages_fork(pool, page_table, seq_lens, src, dst):
    """Sequence dst[i] becomes a copy of sequence src[i] (int32 [n] on the device), its
    length too: they share the pages that src fills, and the last one, where it is
    not full, dst has of its own. Returns the pages to copy for that, (from_pages,
    to_pages), for cache_copy of each cache that goes by this table; -1 where there
    is nothing to copy. dst's former pages are not given back here. Pairs out of
    range, or whose dst is used twice or forked from, are left out and reported by
    poll_device_status, as is a pool without a free page."""
    row, wide, n = _pool_call(pool, page_table, (("seq_lens", seq_lens),), (("src", src), ("dst", dst)))
    old, new = torch.empty_like(src), torch.empty_like(src)
    if src.shape[0]:
        _launch(pool.device, lib().attn_pages_fork, pool._at(), page_table.data_ptr(), row, wide,
                seq_lens.data_ptr(), n, src.data_ptr(), dst.data_ptr(), src.shape[0], old.data_ptr(),
                new.data_ptr())
    return old, new


def pages_reserve(pool, page_table, seq_lens, new_lens):
    """Room for each sequence to grow from seq_lens[b] to new_lens[b] keys (int32
    [n_seqs] on the device): the entries for them that hold no page get a free one.
    An entry for which none is left stays -1, and poll_device_status reports it."""
    row, wide, n = _pool_call(pool, page_table, (("seq_lens", seq_lens), ("new_lens", new_lens)))
    _launch(pool.device, lib().attn_pages_reserve, pool._at(), page_table.data_ptr(), row, wide,
            seq_lens.data_ptr(), new_lens.data_ptr(), n)


def cache_copy(cache, from_pages, to_pages):
    """Copy the cache's pages from_pages[i] to pages to_pages[i], keys and values
    (int32 [n] on the device; a pair with an index below 0 is skipped). No page may be
    written twice, or both written and read."""
    if not isinstance(cache, PagedCache):
        raise ValueError("cache must be a PagedCache")
    _int32(from_pages, "from_pages", cache.device, 1)
    _int32(to_pages, "to_pages", cache.device, 1)
    n = from_pages.shape[0]
    if to_pages.shape[0] != n:
        raise ValueError("from_pages and to_pages must have the same length")
    if n:
        _launch(cache.device, lib().attn_cache_copy, cache._at(), from_pages.data_ptr(),
                to_pages.data_ptr(), n)


_GATHER_LAYOUTS = _Layouts()


def cache_gather(cache, page_table, places, cu, to_table=None, to_start=None):
    """Move chosen tokens' keys and values together: sequence b's tokens at places[cu[b]]
    .. places[cu[b + 1] - 1] go to its places to_start[b], to_start[b] + 1, .. (without
    to_start 0, 1, ..). places int32 [T], cu int32 [n_seqs + 1] and to_start int32
    [n_seqs] on the device.

    Without to_table within the sequence's own pages, as the accepted tokens of a
    draft move up behind their context: no token may move to a later place. With
    to_table, int32 [n_seqs, to_max_pages], into the pages of that table, none of
    which this call reads. What is out of range or order is left out and reported by
    poll_device_status. The pages written must not be shared."""
    try:
        key = (cache._key, _form(page_table), _form(places), _form(cu), _form(to_table), _form(to_start))
        lay = _GATHER_LAYOUTS.get(key)
    except AttributeError:
        lay = key = None
    if lay is None:
        lay = _gather_layout(cache, page_table, places, cu, to_table, to_start)
        _GATHER_LAYOUTS.add(key, lay)
    row, wide, n, T, to_row, to_wide = lay
    if T:
        _launch(cache.device, lib().attn_cache_gather, cache._at(), page_table.data_ptr(), row, wide, n,
                places.data_ptr(), cu.data_ptr(), T, None if to_table is None else to_table.data_ptr(),
                to_row, to_wide, None if to_start is None else to_start.data_ptr())


def _gather_layout(cache, page_table, places, cu, to_table, to_start):
    """Checks a gather's arguments: the tables' row strides and columns, the sequences
    and the tokens."""
    if not isinstance(cache, PagedCache):
        raise ValueError("cache must be a PagedCache")
    _int32(page_table, "page_table", cache.device, 2)
    n, wide = page_table.shape
    if n < 1 or wide < 1:
        raise ValueError(f"page_table must be [n_seqs, max_pages], got {tuple(page_table.shape)}")
    _int32(places, "places", cache.device, 1)
    if places.shape[0] > 1 << 30:
        raise ValueError("places must hold at most 2^30 tokens")
    _int32(cu, "cu", cache.device, 1)
    if cu.shape[0] != n + 1:
        raise ValueError(f"cu must have {n + 1} entries, got {cu.shape[0]}")
    to_row = to_wide = 0
    if to_table is not None:
        _int32(to_table, "to_table", cache.device, 2)
        if to_table.shape[0] != n or to_table.shape[1] < 1:
            raise ValueError(f"to_table must be [{n}, to_max_pages], got {tuple(to_table.shape)}")
        to_row, to_wide = to_table.stride(0), to_table.shape[1]
    if to_start is not None:
        _int32(to_start, "to_start", cache.device, 1)
        if to_start.shape[0] != n:
            raise ValueError(f"to_start must hold {n} sequences, got {to_start.shape[0]}")
    return page_table.stride(0), wide, n, places.shape[0], to_row, to_wide
