"""Thin ctypes binding of libesa (include/esa.h).

Argument marshalling only: every step of the path runs in libesa's CUDA kernels.
Outputs and workspaces are torch tensors (the caller's device memory); a function
allocates them when the caller passes none. There is no CPU fallback: without the
built library, or without a CUDA device, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libesa.so")

ESA_OK, ESA_ERR_INVALID_ARG, ESA_ERR_UNSUPPORTED, ESA_ERR_CUDA, ESA_ERR_TIMEOUT, ESA_ERR_WORKSPACE = range(6)
ESA_F32, ESA_BF16 = 0, 1

# Every exported function of include/esa.h: name -> (restype, argtypes)
_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class EsaParams(ctypes.Structure):
    """esa_params_t: n_init, window, topk, eps, clamp_c (+inf = no clamp)."""

    _fields_ = [("n_init", ctypes.c_int32), ("window", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("eps", ctypes.c_int32), ("clamp_c", ctypes.c_float)]


class EsaCacheQ8(ctypes.Structure):
    """esa_cache_q8_t: the buffers, sizes and format of an 8-bit key/value cache."""

    _fields_ = [("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_cap", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("block", ctypes.c_int32),
                ("format", ctypes.c_int32)]


SIGNATURES = {
    "esa_compress": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i32, _i32, _i32, _vp, _i32, _vp, _i64, _vp]),
    "esa_compress_pack_size": (_sz, [_i32, _i32, _i32]),
    "esa_compress_pack": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _vp, _sz, _vp]),
    "esa_compress_packed": (ctypes.c_int, [_vp, _i64, _i64, _i32, _i32, _vp, _i32, _vp, _i64, _vp]),
    "esa_score_select": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i64, _i64, _i32, EsaParams, _vp, _vp, _vp,
                                        _vp, _sz, _vp]),
    "esa_score_select_workspace_size": (_sz, [_i32, _i32, _i64, _i64, _i32, EsaParams]),
    "esa_sparse_attn": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _i32, _i32, _i64, _i64, _i32, _i32, _i32,
                                       _vp, _vp, EsaParams, _f32, _vp, _vp, _vp, _sz, _vp]),
    "esa_sparse_attn_workspace_size": (_sz, [_i32, _i32, _i64, _i32, _i32, _i32, ctypes.c_int, EsaParams]),
    "moba_block_gate": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i32, _i64, _i32, _i32, _i32, _i32, _vp, _vp,
                                       _sz, _vp]),
    "moba_block_attn": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _i32, _i64, _i32, _i32, _i32, _i32, _vp,
                                       _f32, _vp, _vp, _vp, _sz, _vp]),
    "moba_block_gate_attn": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _i32, _i64, _i32, _i32, _i32, _i32,
                                            _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moba_workspace_size": (_sz, [_i32, _i32, _i64, _i32, _i32, _i32, _i32]),
    "esa_last_error": (ctypes.c_char_p, []),
    "esa_device_status": (ctypes.c_int, [_vp]),
    "esa_version": (ctypes.c_char_p, []),
    "esa_launch_count": (ctypes.c_uint64, []),
    "esa_score_select_noalloc": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i64, _i64, _i32, EsaParams, _vp, _vp, _vp,
                                                _vp]),
    "esa_score_select_noalloc_capacity": (_sz, []),
    "moba_block_means": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "moba_decode_attn": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _i32, _i64, _i64, _i32, _i32, _i32, _i32, _vp,
                                        _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moba_decode_workspace_size": (_sz, [_i32, _i64, _i64, _i32, _i32, _i32, _i32]),
    "esa_score_select_heads": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i64, _i64, _i32, _i32, EsaParams, _vp, _vp,
                                              _vp, _vp, _sz, _vp]),
    "esa_score_select_heads_workspace_size": (_sz, [_i32, _i32, _i64, _i64, _i32, _i32, EsaParams]),
    "esa_sparse_attn_heads": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _i32, _i32, _i64, _i64, _i32, _i32,
                                             _i32, _vp, _vp, EsaParams, _f32, _vp, _vp, _vp, _sz, _vp]),
    "esa_sparse_attn_heads_workspace_size": (_sz, [_i32, _i32, _i64, _i32, _i32, _i32, ctypes.c_int, EsaParams]),
    "esa_wait_selftest": (ctypes.c_int, [ctypes.c_uint64, _vp]),
    "cca_attn": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _i32, _i64, _i32, _i32, _i32, _i32, _i32, _f32, _vp,
                                _vp, _vp, _sz, _vp]),
    "cca_workspace_size": (_sz, [_i32, _i64, _i32, _i32, _i32]),
    "esa_gram": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i32, _vp, _vp, _sz, _vp]),
    "esa_gram_workspace_size": (_sz, [_i64, _i32]),
    "esa_fit_maps": (ctypes.c_int, [_vp, _i64, _vp, _i64, ctypes.c_int, _i32, _i32, _i32, _i32, _i32,
                                    ctypes.c_double, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "esa_fit_workspace_size": (_sz, [_i64, _i64, _i32, _i32, _i32, _i32, _i32]),
    "esa_compress_packed_varlen": (ctypes.c_int, [_vp, _i32, _i64, _i32, _i32, _vp, _i32, _vp, _i64, _vp, _vp]),
    "esa_score_select_varlen": (ctypes.c_int, [_vp, _vp, _i32, _i64, _vp, _i32, _i32, EsaParams, _vp, _vp, _vp,
                                               _vp, _sz, _vp]),
    "esa_score_select_varlen_workspace_size": (_sz, [_i32, _i64, _i32, _i32, EsaParams]),
    "esa_sparse_attn_varlen": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _i32, _i64, _vp, _i32, _i32, _i32, _vp,
                                              _vp, _i32, EsaParams, _f32, _vp, _vp, _vp, _sz, _vp]),
    "esa_sparse_attn_varlen_workspace_size": (_sz, [_i32, _i64, _i32, _i32, _i32, ctypes.c_int, _i32, EsaParams]),
    "esa_cache_write_q8": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i64, _i64, _i64, _i64, _i64, EsaCacheQ8, _i64,
                                          _vp]),
    "esa_cache_write_q8_varlen": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i64, _i64, _i64, _i64, _i64, EsaCacheQ8,
                                                 _vp, _vp, _vp]),
    "esa_cache_read_q8": (ctypes.c_int, [EsaCacheQ8, _i64, _i64, _vp, _vp, _vp, ctypes.c_int, _vp]),
    "esa_sparse_attn_q8": (ctypes.c_int, [_vp, ctypes.c_int, EsaCacheQ8, _i32, _i64, _i32, _vp, _vp, _i32, EsaParams,
                                          _f32, _vp, _vp, _vp, _sz, _vp]),
    "esa_sparse_attn_q8_workspace_size": (_sz, [_i32, _i32, _i64, _i32, _i32, _i32, ctypes.c_int, EsaParams]),
    "esa_sparse_attn_q8_varlen": (ctypes.c_int, [_vp, ctypes.c_int, EsaCacheQ8, _vp, _i32, _vp, _vp, _i32, EsaParams,
                                                 _f32, _vp, _vp, _vp]),
}

_lib = None


class EsaError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: status {status}: {message}")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libesa and declare every signature. Raises if the library is missing."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libesa is not built ({path} missing); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(status: int, where: str):
    if status != ESA_OK:
        raise EsaError(status, where, load().esa_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return ESA_F32
    if t.dtype == torch.bfloat16:
        return ESA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("libesa takes CUDA tensors (no CPU path)")
            if not t.is_contiguous():
                raise ValueError("libesa takes contiguous tensors")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _workspace(nbytes: int, device, ws: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return ws
    if ws is not None and ws.numel() * ws.element_size() >= nbytes:
        return ws
    return torch.empty(nbytes + 256, dtype=torch.uint8, device=device)


def _ws_ptr(ws: Optional[torch.Tensor]) -> tuple:
    if ws is None:
        return None, 0
    p = ws.data_ptr()
    pad = (-p) % 256
    return p + pad, ws.numel() * ws.element_size() - pad


def params(n_init: int, window: int, topk: int, eps: int, clamp_c: float = math.inf) -> EsaParams:
    return EsaParams(n_init, window, topk, eps, clamp_c)


def compress(x: torch.Tensor, w: torch.Tensor, n_heads_out: int, out: Optional[torch.Tensor] = None,
             out_row_stride: Optional[int] = None) -> torch.Tensor:
    """esa_compress. x: [rows, Hin, D] (f32 or bf16; each row contiguous, rows may be
    strided); w: [Hout*D, d'] f32 -> [rows, d'] f32. With `out` given, rows are written
    at out + r * out_row_stride (default d')."""
    if not x.is_cuda or not w.is_cuda or not w.is_contiguous():
        raise ValueError("libesa takes CUDA tensors (no CPU path); w must be contiguous")
    rows, hin, d = x.shape
    if x.stride(2) != 1 or x.stride(1) != d:
        raise ValueError("each row of x must be contiguous [Hin, D]")
    dout = w.shape[1]
    if out is None:
        out = torch.empty((rows, dout), dtype=torch.float32, device=x.device)
        stride = dout
    else:
        stride = out_row_stride or dout
    _check(load().esa_compress(_ptr(x), _dtype_code(x), rows, x.stride(0) if rows > 1 else hin * d, hin,
                               n_heads_out, d, _ptr(w), dout, _ptr(out), stride, _stream()), "esa_compress")
    return out


def compress_pack_size(n_heads_in: int, head_dim: int, d_out: int) -> int:
    """esa_compress_pack_size: bytes of the packed weight, 0 if the packed path does
    not take the shape."""
    return load().esa_compress_pack_size(n_heads_in, head_dim, d_out)


def compress_pack(w: torch.Tensor, n_heads_in: int, n_heads_out: int, head_dim: int,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """esa_compress_pack: w [Hout*D, d'] f32 -> packed weight (uint8 device tensor)."""
    if not w.is_cuda or not w.is_contiguous():
        raise ValueError("libesa takes contiguous CUDA tensors (no CPU path)")
    dout = w.shape[1]
    n = compress_pack_size(n_heads_in, head_dim, dout)
    if n == 0:
        raise EsaError(ESA_ERR_UNSUPPORTED, "esa_compress_pack", "shape not supported by the packed path")
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=w.device)
    _check(load().esa_compress_pack(_ptr(w), n_heads_in, n_heads_out, head_dim, dout, _ptr(out),
                                    out.numel() * out.element_size(), _stream()), "esa_compress_pack")
    return out


def compress_packed(x: torch.Tensor, packed: torch.Tensor, d_out: int = 128, out: Optional[torch.Tensor] = None,
                    out_row_stride: Optional[int] = None) -> torch.Tensor:
    """esa_compress_packed. x: [rows, Hin, D] bf16 (each row contiguous, rows may be
    strided); packed from compress_pack -> [rows, d_out] f32 (or written into `out`
    with row stride out_row_stride)."""
    if not x.is_cuda or not packed.is_cuda:
        raise ValueError("libesa takes CUDA tensors (no CPU path)")
    rows, hin, d = x.shape
    if x.stride(2) != 1 or x.stride(1) != d:
        raise ValueError("each row of x must be contiguous [Hin, D]")
    if out is None:
        out = torch.empty((rows, d_out), dtype=torch.float32, device=x.device)
        stride = d_out
    else:
        stride = out_row_stride or d_out
    _check(load().esa_compress_packed(_ptr(x), rows, x.stride(0) if rows > 1 else hin * d, hin, d, _ptr(packed),
                                      d_out, _ptr(out), stride, _stream()), "esa_compress_packed")
    return out


def score_select_workspace_size(batch, lq, n_cap, c0, d_c, p: EsaParams) -> int:
    return load().esa_score_select_workspace_size(batch, lq, n_cap, c0, d_c, p)


def score_select(q_c: torch.Tensor, k_c: torch.Tensor, c0: int, p: EsaParams, want_scores: bool = False,
                 idx: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None,
                 scores: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """esa_score_select. q_c [B, Lq, d'] f32, k_c [B, n_cap, d'] f32.
    Returns (idx [B, topk] int32, count [B] int32, s' [B, n_mid] f32 or None)."""
    _dev(q_c, k_c)
    b, lq, dc = q_c.shape
    n_cap = k_c.shape[1]
    dev = q_c.device
    if idx is None:
        idx = torch.empty((b, p.topk), dtype=torch.int32, device=dev)
    if count is None:
        count = torch.empty((b,), dtype=torch.int32, device=dev)
    if want_scores and scores is None:
        lo = min(c0, max(p.n_init, c0 - p.window))
        scores = torch.empty((b, max(0, lo - p.n_init)), dtype=torch.float32, device=dev)
    ws = _workspace(score_select_workspace_size(b, lq, n_cap, c0, dc, p), dev, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().esa_score_select(_ptr(q_c), _ptr(k_c), b, lq, n_cap, c0, dc, p, _ptr(idx), _ptr(count),
                                   _ptr(scores) if want_scores else None, wp, wn, _stream()), "esa_score_select")
    return idx, count, (scores if want_scores else None)


def score_select_noalloc(q_c: torch.Tensor, k_c: torch.Tensor, c0: int, p: EsaParams, want_scores: bool = False,
                         idx: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None,
                         scores: Optional[torch.Tensor] = None):
    """esa_score_select_noalloc: the same selection, with the library's fixed scratch
    instead of a workspace (for callers that cannot allocate device memory)."""
    _dev(q_c, k_c)
    b, lq, dc = q_c.shape
    dev = q_c.device
    if idx is None:
        idx = torch.empty((b, p.topk), dtype=torch.int32, device=dev)
    if count is None:
        count = torch.empty((b,), dtype=torch.int32, device=dev)
    if want_scores and scores is None:
        lo = min(c0, max(p.n_init, c0 - p.window))
        scores = torch.empty((b, max(0, lo - p.n_init)), dtype=torch.float32, device=dev)
    _check(load().esa_score_select_noalloc(_ptr(q_c), _ptr(k_c), b, lq, k_c.shape[1], c0, dc, p, _ptr(idx),
                                           _ptr(count), _ptr(scores) if want_scores else None, _stream()),
           "esa_score_select_noalloc")
    return idx, count, (scores if want_scores else None)


def score_select_heads_workspace_size(batch, lq, n_cap, c0, d_c, n_groups, p: EsaParams) -> int:
    return load().esa_score_select_heads_workspace_size(batch, lq, n_cap, c0, d_c, n_groups, p)


def score_select_heads(q_c: torch.Tensor, k_c: torch.Tensor, c0: int, n_groups: int, p: EsaParams,
                       want_scores: bool = False, idx: Optional[torch.Tensor] = None,
                       count: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """esa_score_select_heads (per-head selection: one per group of compressed columns).
    Returns (idx [B, G, topk] int32, count [B, G] int32, s' [B, G, n_mid] f32 or None)."""
    _dev(q_c, k_c)
    b, lq, dc = q_c.shape
    n_cap = k_c.shape[1]
    dev = q_c.device
    if idx is None:
        idx = torch.empty((b, n_groups, p.topk), dtype=torch.int32, device=dev)
    if count is None:
        count = torch.empty((b, n_groups), dtype=torch.int32, device=dev)
    if want_scores and scores is None:
        lo = min(c0, max(p.n_init, c0 - p.window))
        scores = torch.empty((b, n_groups, max(0, lo - p.n_init)), dtype=torch.float32, device=dev)
    ws = _workspace(score_select_heads_workspace_size(b, lq, n_cap, c0, dc, n_groups, p), dev, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().esa_score_select_heads(_ptr(q_c), _ptr(k_c), b, lq, n_cap, c0, dc, n_groups, p, _ptr(idx),
                                         _ptr(count), _ptr(scores) if want_scores else None, wp, wn, _stream()),
           "esa_score_select_heads")
    return idx, count, (scores if want_scores else None)


def sparse_attn_heads_workspace_size(batch, lq, c0, hq, hkv, d, dtype_code, p: EsaParams) -> int:
    return load().esa_sparse_attn_heads_workspace_size(batch, lq, c0, hq, hkv, d, dtype_code, p)


def sparse_attn_heads(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, c0: int, idx: torch.Tensor,
                      count: torch.Tensor, p: EsaParams, scale: float = 0.0, want_lse: bool = False,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None):
    """esa_sparse_attn_heads: idx [B, Hkv, >=topk], count [B, Hkv] (one list per KV head).
    Returns (o [B, Lq, Hq, D], lse [B, Lq, Hq] f32 or None)."""
    _dev(q, k, v, idx, count)
    b, lq, hq, d = q.shape
    n_cap, hkv = k.shape[1], k.shape[2]
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((b, lq, hq), dtype=torch.float32, device=q.device)
    ws = _workspace(sparse_attn_heads_workspace_size(b, lq, c0, hq, hkv, d, dt, p), q.device, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().esa_sparse_attn_heads(_ptr(q), _ptr(k), _ptr(v), dt, b, lq, n_cap, c0, hq, hkv, d, _ptr(idx),
                                        _ptr(count), p, scale, _ptr(out), _ptr(lse) if want_lse else None, wp, wn,
                                        _stream()), "esa_sparse_attn_heads")
    return out, (lse if want_lse else None)


def sparse_attn_workspace_size(batch, lq, c0, hq, hkv, d, dtype_code, p: EsaParams) -> int:
    return load().esa_sparse_attn_workspace_size(batch, lq, c0, hq, hkv, d, dtype_code, p)


def sparse_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, c0: int, idx: torch.Tensor,
                count: torch.Tensor, p: EsaParams, scale: float = 0.0, want_lse: bool = False,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None):
    """esa_sparse_attn. q [B, Lq, Hq, D]; k, v [B, n_cap, Hkv, D]; idx [B, >=topk] int32.
    Returns (o [B, Lq, Hq, D], lse [B, Lq, Hq] f32 or None)."""
    _dev(q, k, v, idx, count)
    b, lq, hq, d = q.shape
    n_cap, hkv = k.shape[1], k.shape[2]
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((b, lq, hq), dtype=torch.float32, device=q.device)
    ws = _workspace(sparse_attn_workspace_size(b, lq, c0, hq, hkv, d, dt, p), q.device, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().esa_sparse_attn(_ptr(q), _ptr(k), _ptr(v), dt, b, lq, n_cap, c0, hq, hkv, d, _ptr(idx),
                                  _ptr(count), p, scale, _ptr(out), _ptr(lse) if want_lse else None, wp, wn,
                                  _stream()), "esa_sparse_attn")
    return out, (lse if want_lse else None)


def _seq_len(seq_len: torch.Tensor, batch: int) -> torch.Tensor:
    if not seq_len.is_cuda or seq_len.dtype != torch.int64 or seq_len.shape != (batch,) or not seq_len.is_contiguous():
        raise ValueError("seq_len must be a contiguous CUDA int64 tensor of shape [batch]")
    return seq_len


def compress_packed_varlen(x: torch.Tensor, packed: torch.Tensor, k_c: torch.Tensor, seq_len: torch.Tensor) -> None:
    """esa_compress_packed_varlen: x [B, Hin, D] bf16 (one new key row per sequence, each
    row contiguous) -> k_c[b, seq_len[b] - 1] of k_c [B, n_cap, d_out] f32."""
    if not x.is_cuda or not packed.is_cuda or not k_c.is_cuda:
        raise ValueError("libesa takes CUDA tensors (no CPU path)")
    b, hin, d = x.shape
    if x.stride(2) != 1 or x.stride(1) != d:
        raise ValueError("each row of x must be contiguous [Hin, D]")
    if not k_c.is_contiguous():
        raise ValueError("k_c must be contiguous")
    _check(load().esa_compress_packed_varlen(_ptr(x), b, x.stride(0) if b > 1 else hin * d, hin, d, _ptr(packed),
                                             k_c.shape[2], _ptr(k_c), k_c.shape[1], _ptr(_seq_len(seq_len, b)),
                                             _stream()), "esa_compress_packed_varlen")


def score_select_varlen_workspace_size(batch, n_cap, d_c, n_groups, p: EsaParams) -> int:
    return load().esa_score_select_varlen_workspace_size(batch, n_cap, d_c, n_groups, p)


def score_select_varlen(q_c: torch.Tensor, k_c: torch.Tensor, seq_len: torch.Tensor, p: EsaParams, n_groups: int = 1,
                        want_scores: bool = False, idx: Optional[torch.Tensor] = None,
                        count: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None):
    """esa_score_select_varlen: one query per sequence at position seq_len[b] - 1.
    q_c [B, 1, d_c], k_c [B, n_cap, d_c] f32. Returns (idx [B, G, topk] int32,
    count [B, G] int32, s' [B, G, n_mid_max] f32 or None); G = n_groups."""
    _dev(q_c, k_c)
    b, lq, dc = q_c.shape
    if lq != 1:
        raise ValueError("one query per sequence")
    n_cap = k_c.shape[1]
    dev = q_c.device
    if idx is None:
        idx = torch.empty((b, n_groups, p.topk), dtype=torch.int32, device=dev)
    if count is None:
        count = torch.empty((b, n_groups), dtype=torch.int32, device=dev)
    if want_scores and scores is None:
        c0 = n_cap - 1
        lo = min(c0, max(p.n_init, c0 - p.window))
        scores = torch.full((b, n_groups, max(0, lo - p.n_init)), float("nan"), dtype=torch.float32, device=dev)
    ws = _workspace(score_select_varlen_workspace_size(b, n_cap, dc, n_groups, p), dev, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().esa_score_select_varlen(_ptr(q_c), _ptr(k_c), b, n_cap, _ptr(_seq_len(seq_len, b)), dc, n_groups,
                                          p, _ptr(idx), _ptr(count), _ptr(scores) if want_scores else None, wp, wn,
                                          _stream()), "esa_score_select_varlen")
    return idx, count, (scores if want_scores else None)


def sparse_attn_varlen_workspace_size(batch, n_cap, hq, hkv, d, dtype_code, lists, p: EsaParams) -> int:
    return load().esa_sparse_attn_varlen_workspace_size(batch, n_cap, hq, hkv, d, dtype_code, lists, p)


def sparse_attn_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seq_len: torch.Tensor, idx: torch.Tensor,
                       count: torch.Tensor, p: EsaParams, scale: float = 0.0, want_lse: bool = False,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """esa_sparse_attn_varlen: q [B, 1, Hq, D]; k, v [B, n_cap, Hkv, D]; idx [B, L, >=topk],
    count [B, L] with L = 1 (shared list) or Hkv (one per KV head), or idx [B, topk] and
    count [B]. Returns (o [B, 1, Hq, D], lse [B, 1, Hq] f32 or None)."""
    _dev(q, k, v, idx, count)
    b, lq, hq, d = q.shape
    if lq != 1:
        raise ValueError("one query per sequence")
    n_cap, hkv = k.shape[1], k.shape[2]
    lists = count.shape[1] if count.dim() == 2 else 1
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((b, lq, hq), dtype=torch.float32, device=q.device)
    ws = _workspace(sparse_attn_varlen_workspace_size(b, n_cap, hq, hkv, d, dt, lists, p), q.device, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().esa_sparse_attn_varlen(_ptr(q), _ptr(k), _ptr(v), dt, b, n_cap, _ptr(_seq_len(seq_len, b)), hq,
                                         hkv, d, _ptr(idx), _ptr(count), lists, p, scale, _ptr(out),
                                         _ptr(lse) if want_lse else None, wp, wn, _stream()),
           "esa_sparse_attn_varlen")
    return out, (lse if want_lse else None)


Q8_FORMATS = {torch.float8_e4m3fn: 0, torch.int8: 1}     # code dtype -> esa_q8_format_t


class CacheQ8:
    """An 8-bit key/value cache: codes k, v [B, n_cap, Hkv, D] (torch.float8_e4m3fn or
    torch.int8) and scales k_scale, v_scale [B, ceil(n_cap / block), Hkv] fp32, one for each
    block of tokens and head; a value is code * scale. The tensors are the caller's (see
    cache_q8 for new ones), are checked once, here, and stay the ones of this cache."""

    __slots__ = ("_k", "_k_scale", "_v", "_v_scale", "_c", "_dev", "_shape")

    def __init__(self, k: torch.Tensor, k_scale: torch.Tensor, v: torch.Tensor, v_scale: torch.Tensor, block: int):
        _dev(k, k_scale, v, v_scale)
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in Q8_FORMATS:
            raise ValueError("k and v must be [B, n_cap, Hkv, D] of one dtype, torch.float8_e4m3fn or torch.int8")
        if block not in (16, 32, 64, 128):
            raise ValueError("block must be 16, 32, 64 or 128")
        b, n_cap, hkv, d = k.shape
        want = (b, (n_cap + block - 1) // block, hkv)
        for t in (k_scale, v_scale):
            if t.dtype != torch.float32 or t.shape != want:
                raise ValueError(f"scales must be float32 {list(want)}")
        if len({t.device for t in (k, k_scale, v, v_scale)}) > 1:
            raise ValueError("the cache's tensors must be on one device")
        self._k, self._k_scale, self._v, self._v_scale = k, k_scale, v, v_scale
        self._c = EsaCacheQ8(_ptr(k), _ptr(k_scale), _ptr(v), _ptr(v_scale), n_cap, b, hkv, d, block,
                             Q8_FORMATS[k.dtype])
        self._dev, self._shape = k.get_device(), (b, hkv, d)

    k = property(lambda self: self._k)
    k_scale = property(lambda self: self._k_scale)
    v = property(lambda self: self._v)
    v_scale = property(lambda self: self._v_scale)
    block = property(lambda self: self._c.block)
    device = property(lambda self: self._k.device)


def cache_q8(batch: int, n_cap: int, hkv: int, head_dim: int, dtype: torch.dtype = torch.float8_e4m3fn,
             block: int = 64, device="cuda") -> CacheQ8:
    """A new, empty CacheQ8 (codes and scales zero)."""
    if block not in (16, 32, 64, 128):
        raise ValueError("block must be 16, 32, 64 or 128")

    def codes():
        return torch.zeros((batch, n_cap, hkv, head_dim), dtype=torch.uint8, device=device).view(dtype)

    def scales():
        return torch.zeros((batch, (n_cap + block - 1) // block, hkv), dtype=torch.float32, device=device)
    return CacheQ8(codes(), scales(), codes(), scales(), block)


# (The helpers below are written for few interpreter steps: a call on a small batch takes
# longer here than on the GPU.)
_DTYPE_CODES = {torch.float32: ESA_F32, torch.bfloat16: ESA_BF16}
# (torch's own entries take a third of the public calls' time; a torch without them, one built
# for the CPU among others, has the public calls)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _q8_call(cache: CacheQ8, where: str, *args):
    """Call `where` with args and the current stream of the cache's device, under that
    device. (The raw stream handle: torch.cuda.current_stream() builds a Stream, 3 us.)"""
    dev = cache._dev
    fn = getattr(_lib or load(), where)
    if _current_device() == dev:
        st = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev))
    if st:
        _check(st, where)


def _q8_dtype(t: torch.Tensor) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _q8_tensor(t: torch.Tensor, name: str, cache: CacheQ8, dtype, shape) -> int:
    """t as an argument of a call on the cache: its device, dtype, shape, contiguous. Returns
    its address."""
    if t.get_device() != cache._dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on the cache's device")
    return t.data_ptr()


def _q8_write(where: str, cache: CacheQ8, k: torch.Tensor, v: torch.Tensor, *tail):
    """k, v: new rows [B, T, Hkv, D]: batch and row strides free, each row contiguous."""
    b, h, d = cache._shape
    shape = k.shape
    if len(shape) != 4 or shape[0] != b or shape[2] != h or shape[3] != d or v.shape != shape or v.dtype is not k.dtype:
        raise ValueError(f"k and v must be [B, T, Hkv, D] = [{b}, T, {h}, {d}] of one dtype")
    if k.get_device() != cache._dev or v.get_device() != cache._dev:
        raise ValueError("k and v must be on the cache's device (no CPU path)")
    kb, kr, kh, ke = k.stride()
    vb, vr, vh, ve = v.stride()
    if ke != 1 or ve != 1 or (h > 1 and (kh != d or vh != d)):
        raise ValueError("each row of k and v must be contiguous [Hkv, D]")
    t = shape[1]
    # a stride that no second row or sequence uses may be anything: pass one that is aligned
    if t <= 1:
        kr = vr = h * d
    if b <= 1:
        kb = vb = 0
    _q8_call(cache, where, k.data_ptr(), v.data_ptr(), _q8_dtype(k), t, kb, kr, vb, vr, cache._c, *tail)


def cache_write_q8(cache: CacheQ8, k: torch.Tensor, v: torch.Tensor, start: int) -> None:
    """esa_cache_write_q8: quantise k, v [B, T, Hkv, D] (f32 or bf16; rows may be strided)
    into positions [start, start + T) of every sequence of the cache."""
    _q8_write("esa_cache_write_q8", cache, k, v, start)


def cache_write_q8_varlen(cache: CacheQ8, k: torch.Tensor, v: torch.Tensor, seq_len: torch.Tensor,
                          new_len: Optional[torch.Tensor] = None) -> None:
    """esa_cache_write_q8_varlen: sequence b's rows (the first new_len[b] of its T, or all)
    into positions [seq_len[b] - new_len[b], seq_len[b]). Lengths: int64 [B] on the device."""
    shape = (cache._shape[0],)
    _q8_write("esa_cache_write_q8_varlen", cache, k, v, _q8_tensor(seq_len, "seq_len", cache, torch.int64, shape),
              None if new_len is None else _q8_tensor(new_len, "new_len", cache, torch.int64, shape))


def cache_read_q8(cache: CacheQ8, start: int = 0, rows: Optional[int] = None, idx: Optional[torch.Tensor] = None,
                  dtype: torch.dtype = torch.bfloat16, want_k: bool = True, want_v: bool = True,
                  k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None):
    """esa_cache_read_q8: the values of positions [start, start + rows) (to the end of the
    cache without rows), or of idx [B, n] int32 (outside the cache: zeros).
    Returns (k [B, n, Hkv, D] or None, v or None) of dtype f32 or bf16."""
    b, h, d = cache._shape
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    where = None
    if idx is not None:
        if start != 0 or rows is not None:
            raise ValueError("idx excludes start and rows")
        n = idx.shape[-1] if idx.dim() else 0
        where = _q8_tensor(idx, "idx", cache, torch.int32, (b, n))
    else:
        n = cache._c.n_cap - start if rows is None else rows
        if start < 0 or n < 0 or start + n > cache._c.n_cap:
            raise ValueError("need 0 <= start and start + rows <= n_cap")
    shape = (b, n, h, d)
    kp = vp = None
    if not want_k:
        k_out = None
    elif k_out is None:
        # (empty_strided and empty_like take two thirds of torch.empty's host time)
        k_out = torch.empty_strided(shape, (n * h * d, h * d, d, 1), dtype=dtype, device=cache._k.device)
        kp = k_out.data_ptr()
    else:
        kp = _q8_tensor(k_out, "k_out", cache, dtype, shape)
    if not want_v:
        v_out = None
    elif v_out is None:
        if kp is not None:
            v_out = torch.empty_like(k_out)
        else:
            v_out = torch.empty_strided(shape, (n * h * d, h * d, d, 1), dtype=dtype, device=cache._k.device)
        vp = v_out.data_ptr()
    else:
        vp = _q8_tensor(v_out, "v_out", cache, dtype, shape)
    _q8_call(cache, "esa_cache_read_q8", cache._c, start, n, where, kp, vp, code)
    return k_out, v_out


def _q8_attn(q, cache: CacheQ8, idx, count, p: EsaParams, want_lse, out, lse):
    """Checks and outputs shared by the attention calls. Returns out, lse and the addresses
    of q, idx, count, out, lse, and the number of lists."""
    b, _, d = cache._shape
    shape = q.shape
    if len(shape) != 4 or shape[0] != b or shape[3] != d:
        raise ValueError(f"q must be [B, Lq, Hq, D] = [{b}, Lq, Hq, {d}]")
    if q.get_device() != cache._dev or not q.is_contiguous():
        raise ValueError("q must be contiguous and on the cache's device (no CPU path)")
    if count.dim() == 2:
        lists = count.shape[1]
        cp = _q8_tensor(count, "count", cache, torch.int32, (b, lists))
        ip = _q8_tensor(idx, "idx", cache, torch.int32, (b, lists, p.topk))
    else:
        lists = 1
        cp = _q8_tensor(count, "count", cache, torch.int32, (b,))
        ip = _q8_tensor(idx, "idx", cache, torch.int32, (b, p.topk))
    if out is None:
        out = torch.empty_like(q)
        op = out.data_ptr()
    else:
        op = _q8_tensor(out, "out", cache, q.dtype, shape)
    lp = None
    if not want_lse:
        lse = None
    elif lse is None:
        lse = cache._k_scale.new_empty(b, shape[1], shape[2])
        lp = lse.data_ptr()
    else:
        lp = _q8_tensor(lse, "lse", cache, torch.float32, shape[:3])
    return out, lse, q.data_ptr(), ip, cp, op, lp, lists


def sparse_attn_q8_workspace_size(batch, lq, c0, hq, hkv, d, dtype_code, p: EsaParams) -> int:
    return load().esa_sparse_attn_q8_workspace_size(batch, lq, c0, hq, hkv, d, dtype_code, p)


def sparse_attn_q8(q: torch.Tensor, cache: CacheQ8, c0: int, idx: torch.Tensor, count: torch.Tensor, p: EsaParams,
                   scale: float = 0.0, want_lse: bool = False, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """esa_sparse_attn_q8: q [B, Lq, Hq, D] at positions [c0, c0 + Lq) over the cache's
    initial + idx[:count] + local tokens; idx [B, topk], count [B] int32, or [B, L, topk] and
    [B, L] with L = 1 or Hkv (a list per KV head). Returns (o like q, lse [B, Lq, Hq] or None)."""
    out, lse, qp, ip, cp, op, lp, lists = _q8_attn(q, cache, idx, count, p, want_lse, out, lse)
    b, lq, hq, d = q.shape
    dt = _q8_dtype(q)
    wp, wn = None, 0
    if lq > 1 or hq > 32 * cache._shape[1]:    # a single query of up to 32 heads a KV head needs no workspace
        if workspace is not None and workspace.get_device() != cache._dev:
            raise ValueError("the workspace must be on the cache's device")
        ws = _workspace(sparse_attn_q8_workspace_size(b, lq, c0, hq, cache._shape[1], d, dt, p), q.device, workspace)
        wp, wn = _ws_ptr(ws)
    _q8_call(cache, "esa_sparse_attn_q8", qp, dt, cache._c, lq, c0, hq, ip, cp, lists, p, scale, op, lp, wp, wn)
    return out, lse


def sparse_attn_q8_varlen(q: torch.Tensor, cache: CacheQ8, seq_len: torch.Tensor, idx: torch.Tensor,
                          count: torch.Tensor, p: EsaParams, scale: float = 0.0, want_lse: bool = False,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """esa_sparse_attn_q8_varlen: one query per sequence, q [B, 1, Hq, D], at position
    seq_len[b] - 1 (int64 [B] on the device). Lists and results as sparse_attn_q8."""
    out, lse, qp, ip, cp, op, lp, lists = _q8_attn(q, cache, idx, count, p, want_lse, out, lse)
    if q.shape[1] != 1:
        raise ValueError("one query per sequence")
    _q8_call(cache, "esa_sparse_attn_q8_varlen", qp, _q8_dtype(q), cache._c,
             _q8_tensor(seq_len, "seq_len", cache, torch.int64, (cache._shape[0],)), q.shape[2], ip, cp, lists, p,
             scale, op, lp)
    return out, lse


def gram(x: torch.Tensor, workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """esa_gram: G = X^T X (fp64 [dim, dim]) of bf16 rows x [n, dim] (any leading shape
    flattened to rows)."""
    _dev(x)
    dim = x.shape[-1]
    n = x.numel() // dim
    if out is None:
        out = torch.empty((dim, dim), dtype=torch.float64, device=x.device)
    ws = _workspace(load().esa_gram_workspace_size(n, dim), x.device, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().esa_gram(_ptr(x), _dtype_code(x), n, dim, _ptr(out), wp, wn, _stream()), "esa_gram")
    return out


def fit_workspace_size(n_q, n_k, hq, hkv, d, d_c, oversample) -> int:
    return load().esa_fit_workspace_size(n_q, n_k, hq, hkv, d, d_c, oversample)


def fit_maps(q: torch.Tensor, k: torch.Tensor, d_c: int, omega: torch.Tensor, ridge: float = 0.0,
             power_iters: int = 8, workspace: Optional[torch.Tensor] = None):
    """esa_fit_maps: compression maps fitted to calibration queries q [n_q, hq, d] and keys
    k [n_k, hkv, d] (bf16). omega: [hkv * d, d_c + oversample] float64 standard normal
    start (its width sets the oversampling). Returns (w_q, w_k), fp32 [hq * d, d_c] each,
    in the layout esa_compress takes."""
    _dev(q, k, omega)
    n_q, hq, d = q.shape
    n_k, hkv = k.shape[0], k.shape[1]
    if omega.dtype != torch.float64 or omega.dim() != 2 or omega.shape[0] != hkv * d or omega.shape[1] < d_c:
        raise ValueError("omega must be a contiguous float64 [hkv * d, d_c + oversample] tensor")
    oversample = omega.shape[1] - d_c
    w_q = torch.empty((hq * d, d_c), dtype=torch.float32, device=q.device)
    w_k = torch.empty((hq * d, d_c), dtype=torch.float32, device=q.device)
    ws = _workspace(fit_workspace_size(n_q, n_k, hq, hkv, d, d_c, oversample), q.device, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().esa_fit_maps(_ptr(q), n_q, _ptr(k), n_k, _dtype_code(q), hq, hkv, d, d_c, oversample,
                               float(ridge), int(power_iters), _ptr(omega), _ptr(w_q), _ptr(w_k), wp, wn,
                               _stream()), "esa_fit_maps")
    return w_q, w_k


def cca_workspace_size(batch, seq, hq, d, group) -> int:
    return load().cca_workspace_size(batch, seq, hq, d, group)


def cca_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, group: int, window: int, scale: float = 0.0,
             want_lse: bool = False, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None):
    """cca_attn: CCA-style causal attention. q [B, S, Hq, D], k, v [B, S, Hkv, D] bf16.
    Returns (o [B, S, Hq, D], lse [B, S, Hq] f32 or None)."""
    _dev(q, k, v)
    b, s, hq, d = q.shape
    hkv = k.shape[2]
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((b, s, hq), dtype=torch.float32, device=q.device)
    ws = _workspace(cca_workspace_size(b, s, hq, d, group), q.device, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().cca_attn(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), b, s, hq, hkv, d, group, window, scale,
                           _ptr(out), _ptr(lse) if want_lse else None, wp, wn, _stream()), "cca_attn")
    return out, (lse if want_lse else None)


def moba_block_means(k: torch.Tensor, block: int, blk_begin: int = 0, blk_end: Optional[int] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moba_block_means: means of blocks [blk_begin, blk_end) of k [B, n_cap, H, D] bf16
    into kbar [B, H, ceil(n_cap / block), D] fp32 (allocated when out is None)."""
    _dev(k)
    b, n_cap, h, d = k.shape
    nb = (n_cap + block - 1) // block
    if out is None:
        out = torch.zeros((b, h, nb, d), dtype=torch.float32, device=k.device)
    end = nb if blk_end is None else blk_end
    _check(load().moba_block_means(_ptr(k), _dtype_code(k), b, n_cap, h, d, block, blk_begin, end, _ptr(out),
                                   _stream()), "moba_block_means")
    return out


def moba_decode_workspace_size(batch, n_cap, pos, heads, d, block, topk) -> int:
    return load().moba_decode_workspace_size(batch, n_cap, pos, heads, d, block, topk)


def moba_decode_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: int, kbar: torch.Tensor, block: int,
                     topk: int, scale: float = 0.0, want_lse: bool = False, want_blocks: bool = False,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     blocks: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """moba_decode_attn: one decode step for the query q [B, 1, H, D] at position pos.
    Returns (o [B, 1, H, D], lse [B, 1, H] or None, blocks [B, H, topk+1] int16 or None)."""
    _dev(q, k, v, kbar)
    b, _, h, d = q.shape
    n_cap = k.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((b, 1, h), dtype=torch.float32, device=q.device)
    if want_blocks and blocks is None:
        blocks = torch.empty((b, h, topk + 1), dtype=torch.int16, device=q.device)
    ws = _workspace(moba_decode_workspace_size(b, n_cap, pos, h, d, block, topk), q.device, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().moba_decode_attn(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), b, n_cap, pos, h, d, block, topk,
                                   _ptr(kbar), scale, _ptr(out), _ptr(lse) if want_lse else None,
                                   _ptr(blocks) if want_blocks else None, wp, wn, _stream()), "moba_decode_attn")
    return out, (lse if want_lse else None), (blocks if want_blocks else None)


def moba_workspace_size(which, batch, seq, heads, d, block, topk) -> int:
    return load().moba_workspace_size(which, batch, seq, heads, d, block, topk)


def moba_block_gate(q, k, block: int, topk: int, out=None, workspace=None) -> torch.Tensor:
    """moba_block_gate -> blocks [B, S, H, topk+1] int16."""
    _dev(q, k)
    b, s, h, d = q.shape
    if out is None:
        out = torch.empty((b, s, h, topk + 1), dtype=torch.int16, device=q.device)
    ws = _workspace(moba_workspace_size(0, b, s, h, d, block, topk), q.device, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().moba_block_gate(_ptr(q), _ptr(k), _dtype_code(q), b, s, h, d, block, topk, _ptr(out), wp, wn,
                                  _stream()), "moba_block_gate")
    return out


def moba_block_attn(q, k, v, block: int, topk: int, blocks: torch.Tensor, scale: float = 0.0,
                    want_lse: bool = False, out=None, lse=None, workspace=None):
    """moba_block_attn -> (o [B, S, H, D], lse [B, S, H] or None)."""
    _dev(q, k, v, blocks)
    b, s, h, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((b, s, h), dtype=torch.float32, device=q.device)
    ws = _workspace(moba_workspace_size(1, b, s, h, d, block, topk), q.device, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().moba_block_attn(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), b, s, h, d, block, topk, _ptr(blocks),
                                  scale, _ptr(out), _ptr(lse) if want_lse else None, wp, wn, _stream()),
           "moba_block_attn")
    return out, (lse if want_lse else None)


def moba_block_gate_attn(q, k, v, block: int, topk: int, scale: float = 0.0, want_blocks: bool = False,
                         want_lse: bool = False, out=None, lse=None, blocks=None, workspace=None):
    """moba_block_gate_attn -> (o, lse or None, blocks or None)."""
    _dev(q, k, v)
    b, s, h, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((b, s, h), dtype=torch.float32, device=q.device)
    if want_blocks and blocks is None:
        blocks = torch.empty((b, s, h, topk + 1), dtype=torch.int16, device=q.device)
    ws = _workspace(moba_workspace_size(2, b, s, h, d, block, topk), q.device, workspace)
    wp, wn = _ws_ptr(ws)
    _check(load().moba_block_gate_attn(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), b, s, h, d, block, topk, scale,
                                       _ptr(out), _ptr(lse) if want_lse else None,
                                       _ptr(blocks) if want_blocks else None, wp, wn, _stream()),
           "moba_block_gate_attn")
    return out, (lse if want_lse else None), (blocks if want_blocks else None)


def launch_count() -> int:
    """Kernels libesa has launched in this process."""
    return int(load().esa_launch_count())


def wait_selftest(limit_ns: int) -> None:
    """esa_wait_selftest: a kernel whose bounded wait runs out after limit_ns and
    records a timeout (read back by device_status)."""
    _check(load().esa_wait_selftest(int(limit_ns), _stream()), "esa_wait_selftest")


def device_status() -> None:
    """Raise EsaError if a kernel's bounded wait ran out since the last check."""
    _check(load().esa_device_status(_stream()), "esa_device_status")
