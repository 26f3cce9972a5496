"""GB300-native exact attention (FlashAttention-style forward and backward) for sm_103a.

The computation lives in ``libfa.so`` (hand-written CUDA: TMA, tcgen05/TMEM, warp-specialised
roles) behind the C ABI of ``include/fa.h``.  This module is the thin Python binding: the
``fa_*`` functions mirror the C entry points one to one and only marshal torch tensors into
pointers and sizes; ``forward``/``backward`` additionally allocate the outputs with torch.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
from typing import NamedTuple

from . import _lib
from ._lib import FA_BF16, FA_F32, FaError, check, load

__all__ = [
    "FA_BF16", "FA_F32", "FaError", "load", "fa_fwd", "fa_bwd", "fa_bwd_stage", "fa_bwd_workspace_bytes",
    "fa_device_status", "fa_set_wait_limit_ns", "fa_causal_block_counts", "forward", "backward",
    "fa_fwd_varlen", "fa_bwd_varlen", "fa_bwd_varlen_workspace_bytes", "forward_varlen",
    "backward_varlen", "fa_fwd_decode", "fa_decode_workspace_bytes", "fa_decode_num_splits",
    "forward_decode", "fa_checked_build", "fa_fwd_fp8", "fa_fwd_fp8_workspace_bytes",
    "forward_fp8", "fa_fwd_fp8_varlen", "fa_fwd_fp8_varlen_workspace_bytes", "forward_fp8_varlen",
    "RopeTable", "rope_table", "fa_rope", "rope", "rope_backward", "PagedCache", "new_cache",
    "fa_cache_append", "cache_append", "fa_cache_read", "cache_read", "fa_fwd_decode_cache",
    "fa_decode_cache_num_ctas", "fa_decode_cache_workspace_bytes", "forward_decode_cache",
    "fa_fwd_decode_shared", "fa_decode_shared_num_ctas", "fa_decode_shared_workspace_bytes",
    "forward_decode_shared",
]


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float32:
        return FA_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")


def _shape(q):
    if q.dim() != 4:
        raise ValueError("tensors must be [B, H, N, d]")
    return tuple(int(x) for x in q.shape)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check_tensors(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")


def _grouped(q, k) -> bool:
    """True when k has fewer heads or another length than q (the fa_*_gqa entry points)."""
    return tuple(k.shape[1:3]) != tuple(q.shape[1:3])


def fa_fwd(q, k, v, o, lse, scale: float, causal: bool, stream=None, impl: int = 0) -> None:
    """C ``fa_fwd`` (``fa_fwd_impl`` when impl != 0): writes o and lse in place.  With k and v
    of shape [B, Hkv, Nk, d] other than q's [B, H, Nq, d] it calls ``fa_fwd_gqa``."""
    _check_tensors(q, k, v, o, lse)
    if _grouped(q, k):
        if impl:
            raise ValueError("grouped heads and Nq != Nk run on the tensor-core path only")
        B, H, Nq, d = _shape(q)
        _, Hkv, Nk, _ = _shape(k)
        check(load().fa_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, Nq, Nk,
                                d, float(scale), int(bool(causal)), _stream(stream)))
        return
    B, H, N, d = _shape(q)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale),
            int(bool(causal)), _dtype_code(q))
    lib = load()
    if impl:
        check(lib.fa_fwd_impl(*args, int(impl), _stream(stream)))
    else:
        check(lib.fa_fwd(*args, _stream(stream)))


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_bytes(B, H, N, d))


def fa_bwd(q, k, v, o, do, lse, dq, dk, dv, scale: float, causal: bool, workspace,
           stream=None, impl: int = 0) -> None:
    """C ``fa_bwd`` (``fa_bwd_impl`` when impl != 0): writes dq, dk, dv in place; grouped or
    non-square shapes call ``fa_bwd_gqa``."""
    _check_tensors(q, k, v, o, do, lse, dq, dk, dv, workspace)
    nbytes = workspace.numel() * workspace.element_size()
    if _grouped(q, k):
        if impl:
            raise ValueError("grouped heads and Nq != Nk run on the tensor-core path only")
        B, H, Nq, d = _shape(q)
        _, Hkv, Nk, _ = _shape(k)
        check(load().fa_bwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                                _ptr(dk), _ptr(dv), B, H, Hkv, Nq, Nk, d, float(scale),
                                int(bool(causal)), _ptr(workspace), nbytes, _stream(stream)))
        return
    B, H, N, d = _shape(q)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
            _ptr(dv), B, H, N, d, float(scale), int(bool(causal)), _dtype_code(q), _ptr(workspace),
            nbytes)
    lib = load()
    if impl:
        check(lib.fa_bwd_impl(*args, int(impl), _stream(stream)))
    else:
        check(lib.fa_bwd(*args, _stream(stream)))


def fa_bwd_stage(q, k, v, o, do, lse, dq, dk, dv, scale: float, causal: bool, workspace,
                 stage: int, stream=None) -> None:
    """C ``fa_bwd_stage``: 0 = preprocess, 1 = dK/dV, 2 = dQ (0, 1, 2 in order = fa_bwd)."""
    _check_tensors(q, k, v, o, do, lse, dq, dk, dv, workspace)
    B, H, N, d = _shape(q)
    nbytes = workspace.numel() * workspace.element_size()
    check(load().fa_bwd_stage(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
        B, H, N, d, float(scale), int(bool(causal)), _dtype_code(q), _ptr(workspace), nbytes,
        int(stage), _stream(stream)))


def fa_device_status(stream=None) -> None:
    """C ``fa_device_status``: synchronises and raises FaError if a device wait timed out."""
    check(load().fa_device_status(_stream(stream)))


def fa_set_wait_limit_ns(ns: int) -> None:
    load().fa_set_wait_limit_ns(int(ns))


def fa_checked_build() -> bool:
    """C ``fa_checked_build``: whether the library in use is the bounds-checked variant."""
    return bool(load().fa_checked_build())


def fa_fwd_fp8_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_fwd_fp8_workspace_bytes(B, H, N, d))


def fa_fwd_fp8(q, k, v, o, lse, scale: float, q_descale: float, k_descale: float,
               v_descale: float, causal: bool, workspace, stream=None) -> None:
    """C ``fa_fwd_fp8``: q, k, v [B, H, N, 128] e4m3 codes (any 1-byte dtype, for example
    torch.float8_e4m3fn or uint8), o [B, H, N, 128] bf16, lse [B, H, N] fp32 or None."""
    _check_tensors(q, k, v, o, lse, workspace)
    for t in (q, k, v):
        if t.element_size() != 1 or tuple(t.shape) != tuple(q.shape):
            raise ValueError("q, k and v must be [B, H, N, d] tensors of 1-byte e4m3 codes")
    B, H, N, d = _shape(q)
    nbytes = workspace.numel() * workspace.element_size()
    check(load().fa_fwd_fp8(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale),
        float(q_descale), float(k_descale), float(v_descale), int(bool(causal)), _ptr(workspace),
        nbytes, _stream(stream)))


def forward_fp8(q, k, v, q_descale: float = 1.0, k_descale: float = 1.0, v_descale: float = 1.0,
                scale: float | None = None, causal: bool = False, stream=None):
    """Allocate O (bf16), LSE and the workspace and run fa_fwd_fp8."""
    import torch

    B, H, N, d = _shape(q)
    if scale is None:
        scale = d ** -0.5
    o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    ws = torch.empty(max(fa_fwd_fp8_workspace_bytes(B, H, N, d), 16), dtype=torch.uint8,
                     device=q.device)
    fa_fwd_fp8(q, k, v, o, lse, scale, q_descale, k_descale, v_descale, causal, ws, stream)
    return o, lse


def fa_fwd_fp8_varlen_workspace_bytes(B: int, max_seqlen_k: int, Hkv: int, d: int) -> int:
    return int(load().fa_fwd_fp8_varlen_workspace_bytes(B, max_seqlen_k, Hkv, d))


def fa_fwd_fp8_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                      max_seqlen_k: int, scale: float, q_descale: float, k_descale: float,
                      v_descale: float, causal: bool, workspace, stream=None) -> None:
    """C ``fa_fwd_fp8_varlen``: q [total_q, H, 128], k, v [total_k, Hkv, 128] e4m3 codes (any
    1-byte dtype), o [total_q, H, 128] bf16, lse [H, total_q] fp32 or None, cu_seqlens_* int32
    [B + 1] on the device."""
    _check_tensors(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, workspace)
    for t in (q, k, v):
        if t.element_size() != 1:
            raise ValueError("q, k and v must hold 1-byte e4m3 codes")
    B, total_q, total_k, H, Hkv, d = _varlen_shapes(q, k, cu_seqlens_q, cu_seqlens_k)
    nbytes = workspace.numel() * workspace.element_size()
    check(load().fa_fwd_fp8_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B,
        int(max_seqlen_q), int(max_seqlen_k), total_q, total_k, H, Hkv, d, float(scale),
        float(q_descale), float(k_descale), float(v_descale), int(bool(causal)), _ptr(workspace),
        nbytes, _stream(stream)))


def forward_fp8_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                       q_descale: float = 1.0, k_descale: float = 1.0, v_descale: float = 1.0,
                       scale: float | None = None, causal: bool = False, stream=None):
    """Allocate O (bf16), LSE and the workspace and run fa_fwd_fp8_varlen."""
    import torch

    total_q, H, d = (int(x) for x in q.shape)
    if scale is None:
        scale = d ** -0.5
    B, Hkv = int(cu_seqlens_q.numel()) - 1, int(k.shape[1])
    o = torch.empty((total_q, H, d), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((H, total_q), dtype=torch.float32, device=q.device)
    ws = torch.empty(max(fa_fwd_fp8_varlen_workspace_bytes(B, max_seqlen_k, Hkv, d), 16),
                     dtype=torch.uint8, device=q.device)
    fa_fwd_fp8_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                      scale, q_descale, k_descale, v_descale, causal, ws, stream)
    return o, lse


def fa_causal_block_counts(q_block: int, Br: int, Bc: int, N: int) -> tuple[int, int]:
    """C ``fa_causal_block_counts``: (unmasked blocks, masked diagonal blocks)."""
    nf, nm = ctypes.c_int(), ctypes.c_int()
    check(load().fa_causal_block_counts(q_block, Br, Bc, N, ctypes.byref(nf), ctypes.byref(nm)))
    return nf.value, nm.value


def forward(q, k, v, scale: float | None = None, causal: bool = False, stream=None,
            impl: int = 0):
    """Allocate O ([B,H,N,d], q's dtype) and LSE ([B,H,N] fp32) and run fa_fwd."""
    import torch

    B, H, N, d = _shape(q)
    if scale is None:
        scale = d ** -0.5
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, o, lse, scale, causal, stream, impl)
    return o, lse


def backward(q, k, v, o, do, lse, scale: float | None = None, causal: bool = False,
             stream=None, impl: int = 0, workspace=None):
    """Allocate dQ, dK, dV (and the workspace unless given) and run fa_bwd."""
    import torch

    B, H, N, d = _shape(q)
    if scale is None:
        scale = d ** -0.5
    if workspace is None:
        workspace = torch.empty(fa_bwd_workspace_bytes(B, H, N, d), dtype=torch.uint8,
                                device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd(q, k, v, o, do, lse, dq, dk, dv, scale, causal, workspace, stream, impl)
    return dq, dk, dv


# --------------------------------------------------------------------------- packed batches

def _varlen_shapes(q, k, cu_q, cu_k):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("packed tensors must be [total, heads, d]")
    if cu_q.dtype != _torch_int32() or cu_k.dtype != _torch_int32():
        raise TypeError("cu_seqlens must be int32")
    if cu_q.dim() != 1 or cu_k.dim() != 1 or cu_q.numel() != cu_k.numel() or cu_q.numel() < 2:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must be 1-D with B + 1 entries each")
    total_q, H, d = (int(x) for x in q.shape)
    total_k, Hkv = int(k.shape[0]), int(k.shape[1])
    return cu_q.numel() - 1, total_q, total_k, H, Hkv, d


def _torch_int32():
    import torch

    return torch.int32


def _strides_or_none(*ts):
    """(row, head) element strides of packed [rows, heads, d] views, or None when every tensor
    is contiguous (the plain entry points apply).  The d elements of a head must be
    contiguous."""
    if all(t.is_contiguous() for t in ts):
        return None
    vals = []
    for t in ts:
        if t.dim() != 3 or t.stride(2) != 1:
            raise ValueError("packed views need contiguous head dimensions (stride 1 in d)")
        vals += [int(t.stride(0)), int(t.stride(1))]
    return (ctypes.c_longlong * len(vals))(*vals)


def _check_views(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors")


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                  max_seqlen_k: int, scale: float, causal: bool, stream=None) -> None:
    """C ``fa_fwd_varlen``: q, o [total_q, H, d]; k, v [total_k, Hkv, d] (bf16); lse
    [H, total_q] fp32 (or None); cu_seqlens_* int32 [B + 1] on the device.  Views with other
    row / head strides go through ``fa_fwd_varlen_strided``."""
    _check_views(q, k, v, o)
    _check_tensors(lse, cu_seqlens_q, cu_seqlens_k)
    B, total_q, total_k, H, Hkv, d = _varlen_shapes(q, k, cu_seqlens_q, cu_seqlens_k)
    tail = (_ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, int(max_seqlen_q), int(max_seqlen_k),
            total_q, total_k, H, Hkv, d, float(scale), int(bool(causal)), _stream(stream))
    st = _strides_or_none(q, k, v, o)
    if st is None:
        check(load().fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), *tail))
    else:
        check(load().fa_fwd_varlen_strided(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), st,
                                           *tail))


def fa_bwd_varlen_workspace_bytes(total_q: int, H: int, d: int) -> int:
    return int(load().fa_bwd_varlen_workspace_bytes(total_q, H, d))


def fa_bwd_varlen(q, k, v, o, do, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k,
                  max_seqlen_q: int, max_seqlen_k: int, scale: float, causal: bool, workspace,
                  stream=None) -> None:
    """C ``fa_bwd_varlen``: writes dq [total_q, H, d], dk, dv [total_k, Hkv, d] in place.
    Views with other row / head strides go through ``fa_bwd_varlen_strided``."""
    _check_views(q, k, v, o, do, dq, dk, dv)
    _check_tensors(lse, workspace, cu_seqlens_q, cu_seqlens_k)
    B, total_q, total_k, H, Hkv, d = _varlen_shapes(q, k, cu_seqlens_q, cu_seqlens_k)
    nbytes = workspace.numel() * workspace.element_size()
    head = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
            _ptr(dv))
    tail = (_ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, int(max_seqlen_q), int(max_seqlen_k),
            total_q, total_k, H, Hkv, d, float(scale), int(bool(causal)), _ptr(workspace), nbytes,
            _stream(stream))
    st = _strides_or_none(q, k, v, o, do, dq, dk, dv)
    if st is None:
        check(load().fa_bwd_varlen(*head, *tail))
    else:
        check(load().fa_bwd_varlen_strided(*head, st, *tail))


def forward_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                   scale: float | None = None, causal: bool = False, stream=None):
    """Allocate O ([total_q, H, d]) and LSE ([H, total_q] fp32) and run fa_fwd_varlen."""
    import torch

    d = int(q.shape[-1])
    if scale is None:
        scale = d ** -0.5
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty((int(q.shape[1]), int(q.shape[0])), dtype=torch.float32, device=q.device)
    fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale,
                  causal, stream)
    return o, lse


def backward_varlen(q, k, v, o, do, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                    max_seqlen_k: int, scale: float | None = None, causal: bool = False,
                    stream=None, workspace=None):
    """Allocate dQ, dK, dV (and the workspace unless given) and run fa_bwd_varlen."""
    import torch

    total_q, H, d = (int(x) for x in q.shape)
    if scale is None:
        scale = d ** -0.5
    if workspace is None:
        workspace = torch.empty(fa_bwd_varlen_workspace_bytes(total_q, H, d), dtype=torch.uint8,
                                device=q.device)
    dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
    fa_bwd_varlen(q, k, v, o, do, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                  max_seqlen_k, scale, causal, workspace, stream)
    return dq, dk, dv


# --------------------------------------------------------------------------- split-KV decode

def fa_decode_num_splits(B: int, Hkv: int, max_seqlen_k: int) -> int:
    """C ``fa_decode_num_splits``: a split count that fills this GPU's SMs."""
    n = int(load().fa_decode_num_splits(B, Hkv, max_seqlen_k))
    check(min(n, 0))
    return n


def fa_decode_workspace_bytes(total_q: int, H: int, d: int, num_splits: int) -> int:
    return int(load().fa_decode_workspace_bytes(total_q, H, d, num_splits))


def fa_fwd_decode(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                  max_seqlen_k: int, scale: float, causal: bool, num_splits: int, workspace,
                  stream=None) -> None:
    """C ``fa_fwd_decode``: packed tensors as fa_fwd_varlen; workspace may be None for
    num_splits = 1."""
    _check_tensors(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, workspace)
    B, total_q, total_k, H, Hkv, d = _varlen_shapes(q, k, cu_seqlens_q, cu_seqlens_k)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(load().fa_fwd_decode(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B,
        int(max_seqlen_q), int(max_seqlen_k), total_q, total_k, H, Hkv, d, float(scale),
        int(bool(causal)), int(num_splits), _ptr(workspace), nbytes, _stream(stream)))


def forward_decode(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                   scale: float | None = None, causal: bool = False, num_splits: int | None = None,
                   stream=None):
    """Allocate O, LSE (and the split workspace) and run fa_fwd_decode."""
    import torch

    total_q, H, d = (int(x) for x in q.shape)
    if scale is None:
        scale = d ** -0.5
    if num_splits is None:
        num_splits = fa_decode_num_splits(int(cu_seqlens_q.numel()) - 1, int(k.shape[1]),
                                          max_seqlen_k)
    nbytes = fa_decode_workspace_bytes(total_q, H, d, num_splits)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
    o = torch.empty_like(q)
    lse = torch.empty((H, total_q), dtype=torch.float32, device=q.device)
    fa_fwd_decode(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale,
                  causal, num_splits, ws, stream)
    return o, lse


# --------------------------------------------------------------------------- serving helpers
# These calls are made once for every token of a decode, so their host side is kept short: plain
# ints for pointers and streams, one check of each property, one device lookup.

@functools.lru_cache(maxsize=None)
def _torch():
    import torch

    return torch


@functools.lru_cache(maxsize=None)
def _raw_stream_of():
    """device index -> cudaStream_t of torch's current stream there."""
    torch = _torch()
    fast = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return fast or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _device(*ts) -> int:
    """The index of the tensors' one CUDA device; raises unless all lie on it."""
    index = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must lie on one device")
    if index < 0 or not ts[0].is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    return index


@contextlib.contextmanager
def _switched(index, stream):
    torch = _torch()
    with torch.cuda.device(index):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _place(index, stream):
    """Context for a call that allocates: the tensors' device, and the stream the call runs on (so
    that torch's allocator ties outputs and workspaces to it).  None where both are current."""
    if stream is None and _torch().cuda.current_device() == index:
        return None
    return _switched(index, stream)


def _call(fn, index, stream, *args):
    """One C call on the tensors' device and on ``stream`` (default: that device's current)."""
    raw = _raw_stream_of()(index) if stream is None else stream.cuda_stream
    torch = _torch()
    if torch.cuda.current_device() == index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc:
        check(rc)


def _at(t):
    return None if t is None else t.data_ptr()


def _view_strides(*ts):
    """(row, head) element strides of [rows, heads, d] views, or None when all are contiguous."""
    for t in ts:
        if t is not None and not t.is_contiguous():
            break
    else:
        return None
    vals = []
    for t in ts:
        if t is None:
            vals += [0, 0]
            continue
        if t.stride(2) != 1:
            raise ValueError("packed views need contiguous head dimensions (stride 1 in d)")
        # a dimension of one row or head is never stepped over: any valid step will do
        rows, heads, d = t.shape
        hs = t.stride(1) if heads > 1 else d
        vals += [t.stride(0) if rows > 1 else heads * hs, hs]
    return (ctypes.c_longlong * len(vals))(*vals)


def _int32(name, t, *shape):
    if t.dtype != _torch().int32:
        raise TypeError(f"{name} must be int32")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {list(shape)}")


def _dtype_of(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float32:
        return FA_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")


# --------------------------------------------------------------------------- rotary positions

class RopeTable:
    """Which angle each rotated pair of a head turns by: pair p by positions[axis[p]] *
    inv_freq[p].  ``interleaved`` pairs are neighbours (2p, 2p + 1), else (p, pairs + p)."""

    def __init__(self, d: int, inv_freq, axis, interleaved: bool = False):
        self.d, self.interleaved = int(d), bool(interleaved)
        self.inv_freq = tuple(float(x) for x in inv_freq)
        self.axis = tuple(int(a) for a in axis)
        self.pairs, self.axes = len(self.inv_freq), max(self.axis, default=-1) + 1
        if len(self.axis) != self.pairs:
            raise ValueError("inv_freq and axis must have one entry for each rotated pair")
        self._freq = (ctypes.c_double * self.pairs)(*self.inv_freq)
        self._axis = (ctypes.c_int * self.pairs)(*self.axis)


@functools.lru_cache(maxsize=64)
def rope_table(d: int, sections, base: float = 10000.0, per_axis: bool = False,
               interleaved: bool = False) -> RopeTable:
    """The table of a head of d elements whose first sum(sections) pairs turn, sections[a] of
    them by axis a.  Frequencies run base^(-i / pairs) over all rotated pairs, or, per_axis,
    base^(-i / sections[a]) afresh for each axis."""
    pairs = sum(sections)
    freq, axis = [], []
    for a, n in enumerate(sections):
        for i in range(n):
            freq.append(math.pow(base, -i / n) if per_axis else math.pow(base, -len(freq) / pairs))
            axis.append(a)
    return RopeTable(d, freq, axis, interleaved)


def fa_rope(q, k, q_out, k_out, positions, table: RopeTable, inverse: bool = False,
            stream=None) -> None:
    """C ``fa_rope``: q, q_out [total, H, d], k, k_out [total, Hkv, d] (or both None), bf16 or
    fp32, contiguous or (row, head)-strided views; positions int32 [axes, total].  Outputs may
    be their inputs."""
    index = _rope_check(q, k, positions, table)
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out come together")
    if q_out.shape != q.shape or q_out.dtype != q.dtype or (
            k is not None and (k_out.shape != k.shape or k_out.dtype != q.dtype)):
        raise ValueError("outputs must have their inputs' shape and dtype")
    _device(q, q_out, k_out)
    _rope_call(index, q, k, q_out, k_out, positions, table, inverse, stream)


def _rope_check(q, k, positions, table):
    total, _, d = q.shape
    if table.d != d:
        raise ValueError(f"the table is made for d = {table.d}")
    if k is not None and (k.dtype != q.dtype or k.dim() != 3 or k.shape[0] != total
                          or k.shape[2] != d):
        raise ValueError("q and k must be [total, heads, d] of one dtype")
    if positions.dim() != 2:
        raise ValueError("positions must be [axes, total]")
    _int32("positions", positions, max(table.axes, positions.shape[0]), total)
    return _device(q, k, positions)


def _rope_call(index, q, k, q_out, k_out, positions, table, inverse, stream):
    total, H, d = q.shape
    _call(load().fa_rope, index, stream, q.data_ptr(), _at(k), q_out.data_ptr(), _at(k_out),
          positions.data_ptr(), table._freq, table._axis, _view_strides(q, k, q_out, k_out), total,
          H, 0 if k is None else k.shape[1], d, positions.shape[0], table.pairs,
          int(table.interleaved), 1 if inverse else 0, _dtype_of(q))


def rope(q, k, positions, table: RopeTable, stream=None):
    """Allocate and return q and k (None: only q) turned by their positions."""
    return _rope(q, k, positions, table, False, stream)


def rope_backward(dq, dk, positions, table: RopeTable, stream=None):
    """The gradients of ``rope``'s inputs from those of its outputs."""
    return _rope(dq, dk, positions, table, True, stream)


def _rope(q, k, positions, table, inverse, stream):
    index = _rope_check(q, k, positions, table)
    place = _place(index, stream)
    if place is not None:
        with place:
            return _rope(q, k, positions, table, inverse, None)
    torch = _torch()
    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    k_out = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
    _rope_call(index, q, k, q_out, k_out, positions, table, inverse, None)
    return q_out, k_out


# --------------------------------------------------------------------------- the paged e4m3 cache

class PagedCache(NamedTuple):
    """The tensors of a paged cache: e4m3 codes [num_pages, Hkv, page_size, d] and one biased
    exponent byte a row [num_pages, Hkv, page_size] (any 1-byte dtypes)."""
    k: object
    v: object
    k_exp: object
    v_exp: object


def new_cache(num_pages: int, page_size: int, Hkv: int, d: int, device="cuda") -> PagedCache:
    """A zeroed cache (code 0 under exponent byte 127, the value 0)."""
    import torch

    shape = (num_pages, Hkv, page_size)
    k, v = (torch.zeros(shape + (d,), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
            for _ in range(2))
    ke, ve = (torch.full(shape, 127, dtype=torch.uint8, device=device) for _ in range(2))
    return PagedCache(k, v, ke, ve)


def _cache_sizes(cache, page_table):
    """(num_pages, Hkv, page_size, d, B, max_pages), the tensors checked against them."""
    k, v, ke, ve = cache
    shape = k.shape
    if len(shape) != 4 or v.shape != shape:
        raise ValueError("the cache's codes must be [num_pages, Hkv, page_size, d]")
    if ke.shape != shape[:3] or ve.shape != shape[:3]:
        raise ValueError("the cache's exponents must be [num_pages, Hkv, page_size]")
    for t in cache:
        if t.element_size() != 1 or not t.is_contiguous():
            raise ValueError("the cache's tensors must be contiguous, of 1-byte elements")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    if page_table.dtype != _torch().int32:
        raise TypeError("page_table must be int32")
    if not page_table.is_contiguous():
        raise ValueError("page_table must be contiguous")
    return (*shape, *page_table.shape)


def fa_cache_append(cache: PagedCache, k, v, cu_seqlens_new, seqlens_k, page_table,
                    max_seqlen_new: int, stream=None) -> None:
    """C ``fa_cache_append``: quantises the new rows k, v [total_new, Hkv, d] (bf16 or fp32,
    contiguous or strided) into the cache's pages; seqlens_k int32 [B] are the lengths after
    the call."""
    pages, Hkv, ps, d, B, max_pages = _cache_sizes(cache, page_table)
    _check_rows(k, v, Hkv, d)
    _int32("cu_seqlens_new", cu_seqlens_new, B + 1)
    _int32("seqlens_k", seqlens_k, B)
    kc, vc, ke, ve = cache
    index = _device(k, v, kc, vc, ke, ve, cu_seqlens_new, seqlens_k, page_table)
    _call(load().fa_cache_append, index, stream, k.data_ptr(), v.data_ptr(), _view_strides(k, v),
          kc.data_ptr(), vc.data_ptr(), ke.data_ptr(), ve.data_ptr(), cu_seqlens_new.data_ptr(),
          seqlens_k.data_ptr(), page_table.data_ptr(), B, int(max_seqlen_new), k.shape[0],
          max_pages, pages, ps, Hkv, d, _dtype_of(k))


def _check_rows(k, v, Hkv, d):
    shape = k.shape
    if len(shape) != 3 or shape[1] != Hkv or shape[2] != d or v.shape != shape or v.dtype != k.dtype:
        raise ValueError("k and v must be [rows, Hkv, d] of one dtype")


cache_append = fa_cache_append


def fa_cache_read(cache: PagedCache, k, v, cu_seqlens_k, page_table, max_seqlen_k: int,
                  stream=None) -> None:
    """C ``fa_cache_read``: writes the cached rows of every sequence back to back into k, v
    [total_k, Hkv, d] (bf16 or fp32, contiguous or strided)."""
    pages, Hkv, ps, d, B, max_pages = _cache_sizes(cache, page_table)
    _check_rows(k, v, Hkv, d)
    _int32("cu_seqlens_k", cu_seqlens_k, B + 1)
    kc, vc, ke, ve = cache
    index = _device(k, v, kc, vc, ke, ve, cu_seqlens_k, page_table)
    _call(load().fa_cache_read, index, stream, kc.data_ptr(), vc.data_ptr(), ke.data_ptr(),
          ve.data_ptr(), k.data_ptr(), v.data_ptr(), _view_strides(k, v), cu_seqlens_k.data_ptr(),
          page_table.data_ptr(), B, int(max_seqlen_k), k.shape[0], max_pages, pages, ps, Hkv, d,
          _dtype_of(k))


def cache_read(cache: PagedCache, cu_seqlens_k, page_table, max_seqlen_k: int, total_k: int,
               dtype=None, stream=None):
    """Allocate K and V ([total_k, Hkv, d], bf16 unless dtype says otherwise) and run
    fa_cache_read."""
    place = _place(_device(cache.k), stream)
    if place is not None:
        with place:
            return cache_read(cache, cu_seqlens_k, page_table, max_seqlen_k, total_k, dtype)
    torch = _torch()
    _, Hkv, _, d = cache.k.shape
    dev, dtype = cache.k.device, dtype or torch.bfloat16
    k = torch.empty((total_k, Hkv, d), dtype=dtype, device=dev)
    v = torch.empty((total_k, Hkv, d), dtype=dtype, device=dev)
    fa_cache_read(cache, k, v, cu_seqlens_k, page_table, max_seqlen_k)
    return k, v


def fa_decode_cache_num_ctas(B: int, H: int, Hkv: int, max_seqlen_q: int,
                             max_seqlen_k: int) -> int:
    """C ``fa_decode_cache_num_ctas``: the number of thread blocks that fills this GPU."""
    n = int(load().fa_decode_cache_num_ctas(B, H, Hkv, max_seqlen_q, max_seqlen_k))
    check(min(n, 0))
    return n


def fa_decode_cache_workspace_bytes(H: int, Hkv: int, d: int, max_seqlen_q: int,
                                    num_ctas: int) -> int:
    return int(load().fa_decode_cache_workspace_bytes(H, Hkv, d, max_seqlen_q, num_ctas))


def fa_fwd_decode_cache(q, cache: PagedCache, o, lse, cu_seqlens_q, seqlens_k, page_table,
                        max_seqlen_q: int, max_seqlen_k: int, scale: float, causal: bool,
                        num_ctas: int, workspace, stream=None) -> None:
    """C ``fa_fwd_decode_cache``: q, o [total_q, H, d] bf16, lse [H, total_q] fp32 or None;
    workspace (fa_decode_cache_workspace_bytes) may be None for num_ctas = 1."""
    pages, Hkv, ps, d, B, max_pages = _cache_sizes(cache, page_table)
    _check_decode_io(q, o, lse, d)
    _int32("cu_seqlens_q", cu_seqlens_q, B + 1)
    _int32("seqlens_k", seqlens_k, B)
    kc, vc, ke, ve = cache
    index = _device(q, kc, vc, ke, ve, o, lse, cu_seqlens_q, seqlens_k, page_table, workspace)
    total_q, H, _ = q.shape
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call(load().fa_fwd_decode_cache, index, stream, q.data_ptr(), kc.data_ptr(), vc.data_ptr(),
          ke.data_ptr(), ve.data_ptr(), o.data_ptr(), _at(lse), cu_seqlens_q.data_ptr(),
          seqlens_k.data_ptr(), page_table.data_ptr(), B, int(max_seqlen_q), int(max_seqlen_k),
          total_q, max_pages, pages, ps, H, Hkv, d, float(scale), 1 if causal else 0,
          int(num_ctas), _at(workspace), nbytes)


def _check_decode_io(q, o, lse, d):
    torch = _torch()
    shape = q.shape
    if len(shape) != 3 or shape[2] != d or o.shape != shape:
        raise ValueError("q and o must be [total_q, H, d]")
    if q.dtype != torch.bfloat16 or o.dtype != torch.bfloat16:
        raise TypeError("q and o must be bfloat16")
    if not q.is_contiguous() or not o.is_contiguous():
        raise ValueError("q and o must be contiguous")
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()
                            or lse.shape != (shape[1], shape[0])):
        raise ValueError("lse must be contiguous fp32 [H, total_q]")


@functools.lru_cache(maxsize=256)
def _decode_cache_plan(index, B, H, Hkv, d, max_q, max_k):
    """(thread blocks, workspace bytes) for these sizes on device `index` (the current one)."""
    n = fa_decode_cache_num_ctas(B, H, Hkv, max_q, max_k)
    return n, fa_decode_cache_workspace_bytes(H, Hkv, d, max_q, n)


def forward_decode_cache(q, cache: PagedCache, cu_seqlens_q, seqlens_k, page_table,
                         max_seqlen_q: int, max_seqlen_k: int, scale: float | None = None,
                         causal: bool = False, num_ctas: int | None = None, stream=None):
    """Allocate O, LSE (and the workspace) and run fa_fwd_decode_cache."""
    index = _device(q)
    place = _place(index, stream)
    if place is not None:
        with place:
            return forward_decode_cache(q, cache, cu_seqlens_q, seqlens_k, page_table,
                                        max_seqlen_q, max_seqlen_k, scale, causal, num_ctas)
    torch = _torch()
    total_q, H, d = q.shape
    Hkv, dev = cache.k.shape[1], q.device
    if num_ctas is None:
        num_ctas, nbytes = _decode_cache_plan(index, page_table.shape[0], H, Hkv, d, max_seqlen_q,
                                              max_seqlen_k)
    else:
        nbytes = fa_decode_cache_workspace_bytes(H, Hkv, d, max_seqlen_q, num_ctas)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    o = torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty((H, total_q), dtype=torch.float32, device=dev)
    fa_fwd_decode_cache(q, cache, o, lse, cu_seqlens_q, seqlens_k, page_table, max_seqlen_q,
                        max_seqlen_k, d ** -0.5 if scale is None else scale, causal, num_ctas, ws)
    return o, lse


# --------------------------------------------------------------------------- shared prefixes

def fa_decode_shared_num_ctas() -> int:
    """C ``fa_decode_shared_num_ctas``: the number of thread blocks that fills this GPU."""
    n = int(load().fa_decode_shared_num_ctas())
    check(min(n, 0))
    return n


def fa_decode_shared_workspace_bytes(total_q: int, H: int, d: int, num_ctas: int) -> int:
    return int(load().fa_decode_shared_workspace_bytes(total_q, H, d, num_ctas))


def fa_fwd_decode_shared(q, k_prefix, v_prefix, k, v, o, lse, cu_seqlens_q, cu_seqlens_k,
                         cu_groups, cu_seqlens_p, max_seqlen_q: int, max_seqlen_k: int,
                         max_group_q: int, max_seqlen_p: int, scale: float, causal: bool,
                         num_ctas: int, workspace, stream=None) -> None:
    """C ``fa_fwd_decode_shared``: q, o [total_q, H, d]; k_prefix, v_prefix [total_p, Hkv, d];
    k, v [total_k, Hkv, d] (bf16); lse [H, total_q] fp32 or None; cu_seqlens_q, cu_seqlens_k
    int32 [B + 1]; cu_groups (first sequence of each group), cu_seqlens_p int32 [groups + 1]."""
    torch = _torch()
    total_q, H, d = q.shape
    _check_decode_io(q, o, lse, d)
    Hkv = k.shape[1]
    _check_rows(k, v, Hkv, d)
    _check_rows(k_prefix, v_prefix, Hkv, d)
    for t in (k, v, k_prefix, v_prefix):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("keys and values must be contiguous bfloat16")
    B, groups = cu_seqlens_q.numel() - 1, cu_groups.numel() - 1
    _int32("cu_seqlens_q", cu_seqlens_q, B + 1)
    _int32("cu_seqlens_k", cu_seqlens_k, B + 1)
    _int32("cu_groups", cu_groups, groups + 1)
    _int32("cu_seqlens_p", cu_seqlens_p, groups + 1)
    index = _device(q, k_prefix, v_prefix, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, cu_groups,
                    cu_seqlens_p, workspace)
    _call(load().fa_fwd_decode_shared, index, stream, q.data_ptr(), k_prefix.data_ptr(),
          v_prefix.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _at(lse),
          cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), cu_groups.data_ptr(),
          cu_seqlens_p.data_ptr(), B, groups, int(max_seqlen_q), int(max_seqlen_k),
          int(max_group_q), int(max_seqlen_p), total_q, k.shape[0], k_prefix.shape[0], H, Hkv, d,
          float(scale), 1 if causal else 0, int(num_ctas), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())


@functools.lru_cache(maxsize=None)
def _decode_shared_ctas(index):
    """fa_decode_shared_num_ctas of device `index` (the current one)."""
    return fa_decode_shared_num_ctas()


def forward_decode_shared(q, k_prefix, v_prefix, k, v, cu_seqlens_q, cu_seqlens_k, cu_groups,
                          cu_seqlens_p, max_seqlen_q: int, max_seqlen_k: int, max_group_q: int,
                          max_seqlen_p: int, scale: float | None = None, causal: bool = False,
                          num_ctas: int | None = None, stream=None):
    """Allocate O, LSE and the workspace and run fa_fwd_decode_shared."""
    index = _device(q)
    place = _place(index, stream)
    if place is not None:
        with place:
            return forward_decode_shared(q, k_prefix, v_prefix, k, v, cu_seqlens_q, cu_seqlens_k,
                                         cu_groups, cu_seqlens_p, max_seqlen_q, max_seqlen_k,
                                         max_group_q, max_seqlen_p, scale, causal, num_ctas)
    torch = _torch()
    total_q, H, d = q.shape
    dev = q.device
    if num_ctas is None:
        num_ctas = _decode_shared_ctas(index)
    ws = torch.empty(fa_decode_shared_workspace_bytes(total_q, H, d, num_ctas), dtype=torch.uint8,
                     device=dev)
    o = torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty((H, total_q), dtype=torch.float32, device=dev)
    fa_fwd_decode_shared(q, k_prefix, v_prefix, k, v, o, lse, cu_seqlens_q, cu_seqlens_k,
                         cu_groups, cu_seqlens_p, max_seqlen_q, max_seqlen_k, max_group_q,
                         max_seqlen_p, d ** -0.5 if scale is None else scale, causal, num_ctas, ws)
    return o, lse
