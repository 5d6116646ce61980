"""attention_forward_05_gb300 -- Python binding of libfa (FlashAttention forward for GB300).

This module only marshals arguments: it checks tensors, takes their device
pointers and the current CUDA stream, and calls the C ABI of ``libfa.so``
(declared in ``include/fa.h``).  Every step of the computation runs in the
library's CUDA kernels; there is no fallback.  If the library is missing or
fails to load, importing the binding's entry points raises.  The position and
paged-cache calls (fa_rope and below) marshal in compiled code
(``csrc/fa_binding.cpp``), the others through ctypes.

Entry points (same names as the C ABI):
  fa_fwd(q, k, v, scale=None, o=None, lse=None, with_lse=True, kv_splits=0, causal=False, workspace=None)
      -> (o, lse)      (calls fa_fwd_ex; k/v may have fewer heads than q)
  fa_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d, dtype, causal, kv_splits)
  fa_fwd_host(q, k, v, scale=None, o=None, lse=None, with_lse=True, causal=False, workspace=None)
      -> (o, lse)      (host tensors in and out; copies overlap compute)
  fa_fwd_host_workspace_bytes(B, H, Hkv, Nq, Nk, d, dtype, causal)
  fa_decode_splitkv(q, k, v, splits, o=None) -> o
  fa_decode_splitkv_ex(q, k, v, splits, scale=None, workspace=None, merge_order=None, with_lse=False)
  fa_decode_workspace_bytes(B, H, d, splits)
  fa_decode_splitkv_gqa(q, k, v, splits, scale=None, workspace=None, merge_order=None, with_lse=False)
  fa_bwd(q, k, v, o, dout, lse, scale=None, causal=False, workspace=None) -> (dq, dk, dv)
  fa_bwd_workspace_bytes(B, H, Nq, d)
  fa_rope_freqs(rot, theta=10000.0) -> float64 frequencies
  fa_rope(q, k, positions, freqs, axes=None, interleaved=False) -> (q_out, k_out)
  fa_rope_bwd(dq, dk, positions, freqs, axes=None, interleaved=False) -> (dq_in, dk_in)
  fa_paged_append(k, v, k_cache, v_cache, slots, q=None, positions=None, freqs=None, axes=None,
                  interleaved=False) -> q_out or None
  fa_decode_paged(q, k_cache, v_cache, page_table, seq_lens, scale=None, workspace=None, with_lse=False)
      -> (o, lse)
  fa_decode_paged_prefix(q, k_cache, v_cache, prefix_pages, prefix_len, page_table, seq_lens, scale=None,
                         workspace=None, with_lse=False) -> (o, lse)
  fa_decode_paged_workspace_bytes(B, H, Hkv, d, page_size, prefix_len=0)
  fa_decode_paged_call_bytes(B, H, Hkv, d, page_size, max_pages, prefix_len=0)
  fa_check_device_error()
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import threading

import torch

from . import _build

FA_FP32, FA_BF16 = 0, 1
FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)

_lock = threading.Lock()
_lib = None


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {status_string(status)} ({status})"
        if status == FA_ERR_CUDA:
            L = lib()
            msg += f": {L.fa_last_cuda_error_string().decode()} [{L.fa_last_cuda_error()}]"
        super().__init__(msg)


def lib_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded libfa.so (built first if stale).  Raises if it cannot be built or loaded."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build() if _build.is_stale() else _build.LIB
            L = ctypes.CDLL(path)
            vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
            L.fa_fwd.restype = i
            L.fa_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, i, vp, sz, vp]
            L.fa_fwd_ex.restype = i
            L.fa_fwd_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i, i]
            L.fa_fwd_workspace_bytes.restype = sz
            L.fa_decode_splitkv.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp]
            L.fa_decode_splitkv.restype = i
            L.fa_decode_splitkv_ex.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, vp, sz, vp, vp, vp]
            L.fa_decode_splitkv_ex.restype = i
            L.fa_decode_splitkv_gqa.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, vp, sz, vp, vp, vp]
            L.fa_decode_splitkv_gqa.restype = i
            L.fa_decode_workspace_bytes.argtypes = [i, i, i, i]
            L.fa_decode_workspace_bytes.restype = sz
            L.fa_fwd_host.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp, sz, vp]
            L.fa_fwd_host.restype = i
            L.fa_fwd_host_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
            L.fa_fwd_host_workspace_bytes.restype = sz
            L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp, sz, vp]
            L.fa_bwd.restype = i
            L.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
            L.fa_bwd_workspace_bytes.restype = sz
            ll = ctypes.c_longlong
            L.fa_rope.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, i, vp, vp, i, i, i, i, vp]
            L.fa_rope.restype = i
            L.fa_paged_append.argtypes = [vp] * 9 + [i] * 6 + [vp, vp, vp, i, i, i, vp]
            L.fa_paged_append.restype = i
            L.fa_decode_paged.argtypes = [vp, vp, vp, vp, vp, ll, vp, i, i, i, i, i, i, i, vp, f, vp, sz, vp, vp]
            L.fa_decode_paged.restype = i
            L.fa_decode_paged_prefix.argtypes = [vp, vp, vp, vp, vp, i, vp, ll, vp, i, i, i, i, i, i, i, vp, f, vp, sz,
                                                 vp, vp]
            L.fa_decode_paged_prefix.restype = i
            L.fa_decode_paged_workspace_bytes.argtypes = [i, i, i, i, i, i]
            L.fa_decode_paged_workspace_bytes.restype = sz
            L.fa_decode_paged_call_bytes.argtypes = [i, i, i, i, i, i, i]
            L.fa_decode_paged_call_bytes.restype = sz
            L.fa_check_device_error.argtypes = []
            L.fa_check_device_error.restype = i
            L.fa_status_string.argtypes = [i]
            L.fa_status_string.restype = ctypes.c_char_p
            L.fa_debug_set_fault.argtypes = [i]
            L.fa_debug_set_fault.restype = i
            L.fa_last_cuda_error.argtypes = []
            L.fa_last_cuda_error.restype = i
            L.fa_last_cuda_error_string.argtypes = []
            L.fa_last_cuda_error_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().fa_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != FA_OK:
        raise FAError(status, where)


def _stream_handle(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float32:
        return FA_FP32
    raise TypeError(f"unsupported dtype {t.dtype}: bf16 or fp32")


def _need_cuda_contig(name: str, t: torch.Tensor) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        # the library launches on the current device and encodes its tensor maps there
        raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{torch.cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fa_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
           o: torch.Tensor | None = None, lse: torch.Tensor | None = None, with_lse: bool = True,
           stream=None, kv_splits: int = 0, causal: bool = False, workspace: torch.Tensor | None = None):
    """Exact attention softmax(q k^T * scale) v; returns (o, lse or None).

    q [B, H, Nq, d]; k, v [B, Hkv, Nk, d] with H a multiple of Hkv (grouped-query
    attention when Hkv < H).  kv_splits: 0 automatic, 1 none, n > 1 split keys.
    Calls fa_fwd_ex.
    """
    for n, t in (("q", q), ("k", k), ("v", v)):
        _need_cuda_contig(n, t)
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or q.shape[0] != k.shape[0] or q.shape[3] != k.shape[3]:
        raise ValueError("q [B,H,Nq,d], k/v [B,Hkv,Nk,d] expected")
    if q.shape[1] % k.shape[1] != 0:
        raise ValueError("query heads must be a multiple of key/value heads")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    _need_cuda_contig("o", o)
    if o.shape != q.shape or o.dtype != q.dtype:
        raise ValueError("o must match q")
    if lse is None and with_lse:
        lse = torch.empty((B, H, Nq), device=q.device, dtype=torch.float32)
    if lse is not None:
        _need_cuda_contig("lse", lse)
        if lse.shape != (B, H, Nq) or lse.dtype != torch.float32:
            raise ValueError("lse must be fp32 [B,H,Nq]")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need_cuda_contig("workspace", workspace)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib().fa_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                         lse.data_ptr() if lse is not None else None, B, H, Hkv, Nq, Nk, d, float(scale),
                         _dtype_code(q), int(bool(causal)), int(kv_splits), ws_ptr, ws_bytes,
                         _stream_handle(stream))
    _check(st, "fa_fwd_ex")
    return o, lse


def fa_fwd_workspace_bytes(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int, dtype=torch.bfloat16,
                           causal: bool = False, kv_splits: int = 0) -> int:
    code = FA_BF16 if dtype == torch.bfloat16 else FA_FP32
    return int(lib().fa_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d, code, int(bool(causal)), int(kv_splits)))


def _need_host_contig(name: str, t: torch.Tensor) -> None:
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fa_fwd_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
                o: torch.Tensor | None = None, lse: torch.Tensor | None = None, with_lse: bool = True,
                causal: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """fa_fwd on host (CPU) tensors; returns host (o, lse or None), valid once `stream` (default: the
    current CUDA stream) has finished.  Pinned inputs and outputs let the copies overlap the compute."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _need_host_contig(n, t)
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or q.shape[0] != k.shape[0] or q.shape[3] != k.shape[3]:
        raise ValueError("q [B,H,Nq,d], k/v [B,Hkv,Nk,d] expected")
    if q.shape[1] % k.shape[1] != 0:
        raise ValueError("query heads must be a multiple of key/value heads")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype, pin_memory=q.is_pinned())
    _need_host_contig("o", o)
    if o.shape != q.shape or o.dtype != q.dtype:
        raise ValueError("o must match q")
    if lse is None and with_lse:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, pin_memory=q.is_pinned())
    if lse is not None:
        _need_host_contig("lse", lse)
        if lse.shape != (B, H, Nq) or lse.dtype != torch.float32:
            raise ValueError("lse must be fp32 [B,H,Nq]")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need_cuda_contig("workspace", workspace)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib().fa_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                           lse.data_ptr() if lse is not None else None, B, H, Hkv, Nq, Nk, d, float(scale),
                           _dtype_code(q), int(bool(causal)), ws_ptr, ws_bytes, _stream_handle(stream))
    _check(st, "fa_fwd_host")
    return o, lse


def fa_fwd_host_workspace_bytes(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int, dtype=torch.bfloat16,
                                causal: bool = False) -> int:
    code = FA_BF16 if dtype == torch.bfloat16 else FA_FP32
    return int(lib().fa_fwd_host_workspace_bytes(B, H, Hkv, Nq, Nk, d, code, int(bool(causal))))


def fa_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, dout: torch.Tensor,
           lse: torch.Tensor, scale: float | None = None, causal: bool = False,
           dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
           workspace: torch.Tensor | None = None, stream=None):
    """Gradients (dq, dk, dv) of attention given the forward's o and lse and the output gradient dout.

    q, o, dout [B, H, Nq, d]; k, v [B, Hkv, Nk, d], all bf16 or all fp32; lse [B, H, Nq] fp32 from fa_fwd.
    """
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("lse", lse)):
        _need_cuda_contig(n, t)
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or q.shape[0] != k.shape[0] or q.shape[3] != k.shape[3]:
        raise ValueError("q [B,H,Nq,d], k/v [B,Hkv,Nk,d] expected")
    if o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("o and dout must match q")
    if q.shape[1] % k.shape[1] != 0:
        raise ValueError("query heads must be a multiple of key/value heads")
    if not (q.dtype == k.dtype == v.dtype == o.dtype == dout.dtype):
        raise TypeError("q, k, v, o, dout must share a dtype")
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if lse.shape != (B, H, Nq) or lse.dtype != torch.float32:
        raise ValueError("lse must be fp32 [B,H,Nq]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for n, t, ref in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        _need_cuda_contig(n, t)
        if t.shape != ref.shape or t.dtype != ref.dtype:
            raise ValueError(f"{n} must match its input")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need_cuda_contig("workspace", workspace)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
                      dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Hkv, Nq, Nk, d, float(scale),
                      _dtype_code(q), int(bool(causal)), ws_ptr, ws_bytes, _stream_handle(stream))
    _check(st, "fa_bwd")
    return dq, dk, dv


def fa_bwd_workspace_bytes(B: int, H: int, Nq: int, d: int) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, H, Nq, d))


def _decode_shapes(q, k, v):
    for n, t in (("q", q), ("k", k), ("v", v)):
        _need_cuda_contig(n, t)
    if k.dim() != 4 or k.shape != v.shape:
        raise ValueError("k/v [B,H,Nk,d] expected")
    B, H, Nk, d = k.shape
    if q.numel() != B * H * d:
        raise ValueError("q must hold B*H*d elements ([B,H,d] or [B,H,1,d])")
    if not (q.dtype == k.dtype == v.dtype == torch.bfloat16):
        raise TypeError("decode takes bf16 q, k, v")
    return B, H, Nk, d


def fa_decode_splitkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, splits: int,
                      o: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Split-KV decode with scale 1/sqrt(d); returns o [B, H, d] bf16."""
    B, H, Nk, d = _decode_shapes(q, k, v)
    if o is None:
        o = torch.empty((B, H, d), device=q.device, dtype=torch.bfloat16)
    _need_cuda_contig("o", o)
    st = lib().fa_decode_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, H, Nk, d,
                                 int(splits), _stream_handle(stream))
    _check(st, "fa_decode_splitkv")
    return o


def fa_decode_workspace_bytes(B: int, H: int, d: int, splits: int) -> int:
    return int(lib().fa_decode_workspace_bytes(B, H, d, splits))


def fa_decode_splitkv_ex(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, splits: int,
                         scale: float | None = None, workspace: torch.Tensor | None = None,
                         merge_order: torch.Tensor | None = None, with_lse: bool = False,
                         o: torch.Tensor | None = None, stream=None):
    """Split-KV decode with explicit scale, caller workspace, merge order and LSE; returns (o, lse)."""
    B, H, Nk, d = _decode_shapes(q, k, v)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty((B, H, d), device=q.device, dtype=torch.bfloat16)
    _need_cuda_contig("o", o)
    lse = torch.empty((B, H), device=q.device, dtype=torch.float32) if with_lse else None
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need_cuda_contig("workspace", workspace)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    ord_ptr = None
    if merge_order is not None:
        _need_cuda_contig("merge_order", merge_order)
        if merge_order.dtype != torch.int32 or merge_order.numel() != splits:
            raise ValueError("merge_order must be int32 [splits]")
        ord_ptr = merge_order.data_ptr()
    st = lib().fa_decode_splitkv_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, H, Nk, d,
                                    int(splits), float(scale), ws_ptr, ws_bytes, ord_ptr,
                                    lse.data_ptr() if lse is not None else None, _stream_handle(stream))
    _check(st, "fa_decode_splitkv_ex")
    return o, lse


def fa_decode_splitkv_gqa(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, splits: int,
                          scale: float | None = None, workspace: torch.Tensor | None = None,
                          merge_order: torch.Tensor | None = None, with_lse: bool = False,
                          o: torch.Tensor | None = None, stream=None):
    """Split-KV decode with Hkv = k.shape[1] key/value heads shared by q's H query heads; returns (o, lse).

    q [B, H, d] or [B, H, 1, d]; k, v [B, Hkv, Nk, d]; all bf16.
    """
    for n, t in (("q", q), ("k", k), ("v", v)):
        _need_cuda_contig(n, t)
    if k.dim() != 4 or k.shape != v.shape:
        raise ValueError("k/v [B,Hkv,Nk,d] expected")
    B, Hkv, Nk, d = k.shape
    if q.dim() not in (3, 4) or q.shape[0] != B or q.shape[-1] != d or (q.dim() == 4 and q.shape[2] != 1):
        raise ValueError("q [B,H,d] or [B,H,1,d] expected")
    H = q.shape[1]
    if not (q.dtype == k.dtype == v.dtype == torch.bfloat16):
        raise TypeError("decode takes bf16 q, k, v")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty((B, H, d), device=q.device, dtype=torch.bfloat16)
    _need_cuda_contig("o", o)
    lse = torch.empty((B, H), device=q.device, dtype=torch.float32) if with_lse else None
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need_cuda_contig("workspace", workspace)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    ord_ptr = None
    if merge_order is not None:
        _need_cuda_contig("merge_order", merge_order)
        if merge_order.dtype != torch.int32 or merge_order.numel() != splits:
            raise ValueError("merge_order must be int32 [splits]")
        ord_ptr = merge_order.data_ptr()
    st = lib().fa_decode_splitkv_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, H, Hkv, Nk, d,
                                     int(splits), float(scale), ws_ptr, ws_bytes, ord_ptr,
                                     lse.data_ptr() if lse is not None else None, _stream_handle(stream))
    _check(st, "fa_decode_splitkv_gqa")
    return o, lse


def fa_decode_splitkv_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, splits: int,
                              o: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fa_decode_splitkv whose partial states use the library's fixed device scratch array.

    For callers that may not allocate device memory during a call; the C
    declaration in include/fa.h lists the size limit and the sharing rules
    (calls that overlap on the GPU race on the one array).
    """
    B, H, Nk, d = _decode_shapes(q, k, v)
    if o is None:
        o = torch.empty((B, H, d), device=q.device, dtype=torch.bfloat16)
    _need_cuda_contig("o", o)
    L = lib()
    fn = L.fa_decode_splitkv_noalloc
    vp, i = ctypes.c_void_p, ctypes.c_int
    fn.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp]
    fn.restype = i
    st = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), B, H, Nk, d, int(splits),
            _stream_handle(stream))
    _check(st, "fa_decode_splitkv_noalloc")
    return o


# The entry points below are called once a generated token or layer, on a few kilobytes as on large tensors, so their
# host path counts: it is compiled (csrc/fa_binding.cpp; checks, allocations, the call of the C ABI).

_binding = None


def _load_binding():
    """The compiled part of the binding (built first if stale).  Raises if it cannot be built or loaded."""
    global _binding
    lib()  # the library that the binding links
    with _lock:
        if _binding is None:
            spec = importlib.util.spec_from_file_location("_fa_binding", _build.build_binding())
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            _binding = module
    return _binding


def _on_stream(stream, *tensors):
    """Makes `stream` current, so that outputs and workspaces are allocated for it.  Tensors used on a stream other
    than their own are recorded there, so that the allocator does not hand their memory on while it is read."""
    if stream != torch.cuda.current_stream():
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
    return torch.cuda.stream(stream)


def _result(r, where: str):
    """A binding call's tensors; raises for a status code."""
    if r.__class__ is int:
        _check(r, where)
    return r


def fa_rope_freqs(rot: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """The usual frequencies theta^(-2i/rot), i < rot/2, as the float64 tensor that fa_rope and fa_paged_append take."""
    return theta ** (torch.arange(0, rot, 2, dtype=torch.float64, device=device) / -rot)


def fa_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, freqs: torch.Tensor,
            axes: torch.Tensor | None = None, interleaved: bool = False, q_out: torch.Tensor | None = None,
            k_out: torch.Tensor | None = None, stream=None):
    """Rotary positions on q [B, H, N, d] and k [B, Hkv, N, d] (or None), bf16 or fp32; returns (q_out, k_out).

    positions: int32 [N], [B, N], or with several axes [axes, B, N] / [axes, 1, N].  freqs: float64 [rot/2], radians
    per position (fa_rope_freqs); the first rot elements of a head are rotated.  axes: int32 [rot/2], the position
    axis of each pair.  q and k may be strided views (heads of a projection's output); new outputs are contiguous.
    An output may be its input itself; otherwise it must overlap no input.  B = 0 or N = 0 gives empty outputs.
    """
    if stream is not None:
        with _on_stream(stream, q, k, positions, freqs, axes, q_out, k_out):
            return fa_rope(q, k, positions, freqs, axes, interleaved, q_out, k_out)
    r = (_binding or _load_binding()).rope(q, k, positions, freqs, axes, interleaved, q_out, k_out, False)
    return r if r.__class__ is tuple else _result(r, "fa_rope")


def fa_rope_bwd(dq: torch.Tensor, dk: torch.Tensor | None, positions: torch.Tensor, freqs: torch.Tensor,
                axes: torch.Tensor | None = None, interleaved: bool = False, dq_in: torch.Tensor | None = None,
                dk_in: torch.Tensor | None = None, stream=None):
    """The backward pass of fa_rope: gradients of its outputs in, gradients (dq_in, dk_in) of its q and k out."""
    if stream is not None:
        with _on_stream(stream, dq, dk, positions, freqs, axes, dq_in, dk_in):
            return fa_rope_bwd(dq, dk, positions, freqs, axes, interleaved, dq_in, dk_in)
    r = (_binding or _load_binding()).rope(dq, dk, positions, freqs, axes, interleaved, dq_in, dk_in, True)
    return r if r.__class__ is tuple else _result(r, "fa_rope (backward)")


def fa_paged_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    slots: torch.Tensor, q: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                    freqs: torch.Tensor | None = None, axes: torch.Tensor | None = None, interleaved: bool = False,
                    q_out: torch.Tensor | None = None, stream=None):
    """Writes new tokens' k, v [T, Hkv, d] to their slots of a paged cache; returns the tokens' queries (or None).

    k_cache, v_cache: bf16 [num_pages, Hkv, page_size, d] (strided views with d contiguous allowed, the same strides
    for both).  slots: int64 [T], page * page_size + row; a negative slot stores nothing.  positions (int32 [T] or
    [axes, T]) with freqs rotate k and q as fa_rope does; without them both are copied.  q [T, H, d] may be strided.
    """
    if stream is not None:
        with _on_stream(stream, k, v, k_cache, v_cache, slots, q, positions, freqs, axes, q_out):
            return fa_paged_append(k, v, k_cache, v_cache, slots, q, positions, freqs, axes, interleaved, q_out)
    r = (_binding or _load_binding()).append(k, v, k_cache, v_cache, slots, q, positions, freqs, axes, interleaved,
                                             q_out)
    return _result(r, "fa_paged_append")


def fa_decode_paged_call_bytes(B: int, H: int, Hkv: int, d: int, page_size: int, max_pages: int, prefix_len: int = 0) -> int:
    """What a call with tables of max_pages pages uses of its workspace: all of it, or nothing."""
    return int(lib().fa_decode_paged_call_bytes(B, H, Hkv, d, int(page_size), int(max_pages), int(prefix_len)))


def fa_decode_paged_workspace_bytes(B: int, H: int, Hkv: int, d: int, page_size: int, prefix_len: int = 0) -> int:
    return int(lib().fa_decode_paged_workspace_bytes(B, H, Hkv, d, int(page_size), int(prefix_len)))


def _decode_paged(q, k_cache, v_cache, prefix_pages, prefix_len, page_table, seq_lens, scale, workspace, with_lse, o,
                  stream, where):
    if stream is not None:
        with _on_stream(stream, q, k_cache, v_cache, prefix_pages, page_table, seq_lens, workspace, o):
            return _decode_paged(q, k_cache, v_cache, prefix_pages, prefix_len, page_table, seq_lens, scale, workspace,
                                 with_lse, o, None, where)
    r = (_binding or _load_binding()).decode(q, k_cache, v_cache, prefix_pages, prefix_len, page_table, seq_lens, scale,
                                             workspace, with_lse, o)
    return r if r.__class__ is tuple else _result(r, where)


def fa_decode_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                    seq_lens: torch.Tensor, scale: float | None = None, workspace: torch.Tensor | None = None,
                    with_lse: bool = False, o: torch.Tensor | None = None, stream=None):
    """One query per head over a paged cache; returns (o [B, H, d], lse [B, H] or None).

    q: bf16 [B, H, d].  k_cache, v_cache as in fa_paged_append.  page_table: int32 [B, max_pages]; sequence b sees its
    first seq_lens[b] (int32, on the device) rows.  A sequence without keys gets o = 0, lse = -inf; one with a bad
    page or length gets NaN and makes fa_check_device_error return FA_ERR_INVALID_ARG.  B = 0 gives empty outputs.
    """
    return _decode_paged(q, k_cache, v_cache, None, 0, page_table, seq_lens, scale, workspace, with_lse, o, stream,
                         "fa_decode_paged")


def fa_decode_paged_prefix(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           prefix_pages: torch.Tensor | None, prefix_len: int, page_table: torch.Tensor,
                           seq_lens: torch.Tensor, scale: float | None = None, workspace: torch.Tensor | None = None,
                           with_lse: bool = False, o: torch.Tensor | None = None, stream=None):
    """fa_decode_paged for sequences that all begin with the prefix_len keys in prefix_pages (int32), read once.

    page_table and seq_lens describe each sequence's own rows behind the prefix; a negative length marks an unused
    place of a padded batch, which sees nothing.
    """
    return _decode_paged(q, k_cache, v_cache, prefix_pages, prefix_len, page_table, seq_lens, scale, workspace,
                         with_lse, o, stream, "fa_decode_paged_prefix")


def fa_check_device_error() -> int:
    """Synchronises the current device and returns (and clears) the library's device status."""
    return int(lib().fa_check_device_error())


def fa_debug_set_fault(mode: int) -> int:
    """Test only: arm (1) or disarm (0) the load-warp fault of the next fa_fwd launch."""
    return int(lib().fa_debug_set_fault(int(mode)))
