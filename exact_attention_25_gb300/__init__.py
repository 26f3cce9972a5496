"""GB300-native exact attention (FlashAttention-style forward and backward) for sm_103a.

The computation lives in ``libfa.so`` (hand-written CUDA: TMA, tcgen05/TMEM, warp-specialised
roles) behind the C ABI of ``include/fa.h``.  This module is the thin Python binding: the
``fa_*`` functions mirror the C entry points one to one and only marshal torch tensors into
pointers and sizes; ``forward``/``backward`` additionally allocate the outputs with torch.  The
serving calls (rotary positions, the paged cache and its pages, the decodes over it and over shared
prefixes) do the same through a small native module.
"""
from __future__ import annotations

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
    "forward_decode_shared", "fa_tree_mask", "tree_mask", "fa_fwd_decode_tree",
    "fa_decode_tree_num_ctas", "fa_decode_tree_workspace_bytes", "forward_decode_tree",
    "fa_cache_copy_pages", "cache_copy_pages", "fa_cache_compact", "cache_compact",
    "fa_pages_update", "fa_pages_workspace_bytes", "pages_update",
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


# --------------------------------------------------------------------------- serving calls
# Made once for every token and layer of a decode, so their host side is native (the _serve module,
# csrc/serve_binding.cpp): it checks the tensors, allocates what is to be returned, and makes the C
# call on the tensors' device and its current stream.  A call on another stream makes that the
# current one first, so torch's allocator ties outputs and workspaces to it.  A step in which no sequence has
# a row (a total, or the longest sequence's number, of 0) does nothing and returns what it was given, or
# tensors that nothing is written to.

@functools.lru_cache(maxsize=None)
def _native():
    import torch  # noqa: F401  (the module links against torch's libraries)

    try:
        from . import _serve
    except ImportError as e:
        raise ImportError(f"the native binding is missing or was built for another torch or Python ({e}): "
                          "build it with exact_attention_25_gb300.build.build_all() (there is no "
                          "fallback implementation)") from e
    return _serve


def _entry(*names):
    """Addresses of C entry points of the library in use."""
    lib = _lib._lib or load()
    try:
        return lib.entry_addresses[names]
    except AttributeError:
        lib.entry_addresses = {}
    except KeyError:
        pass
    at = tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names)
    lib.entry_addresses[names] = at
    return at


def _on(stream, t):
    """Context that makes ``stream``, a stream of t's device, the current one."""
    import torch

    if stream.device_index != t.get_device():
        raise ValueError("the stream belongs to another device than the tensors")
    return torch.cuda.stream(stream)


def _done(result):
    if result.__class__ is int:
        check(result)
    return result


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
        # what every call passes after the tensors
        self._args = (ctypes.addressof(self._freq), ctypes.addressof(self._axis), self.axes,
                      self.d, self.pairs, self.interleaved)

    def __reduce__(self):  # copies and pickles make arrays, and addresses, of their own
        return RopeTable, (self.d, self.inv_freq, self.axis, self.interleaved)


def rope_table(d: int, sections, base: float = 10000.0, per_axis: bool = False,
               interleaved: bool = False) -> RopeTable:
    """The table of a head of d elements whose first sum(sections) pairs turn, sections[a] of
    them by axis a.  Frequencies run base^(-i / pairs) over all rotated pairs, or, per_axis,
    base^(-i / sections[a]) afresh for each axis."""
    return _rope_table(int(d), tuple(int(n) for n in sections), float(base), bool(per_axis),
                       bool(interleaved))


@functools.lru_cache(maxsize=64)
def _rope_table(d, sections, base, per_axis, interleaved):
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
    if q_out is None or (k is None) != (k_out is None):
        raise ValueError("every input has its output")
    if stream is not None:
        with _on(stream, q):
            return fa_rope(q, k, q_out, k_out, positions, table, inverse)
    _done(_native().rope(*_entry("fa_rope"), q, k, q_out, k_out, positions, *table._args, inverse))


def rope(q, k, positions, table: RopeTable, stream=None):
    """Allocate and return q and k (None: only q) turned by their positions."""
    if stream is not None:
        with _on(stream, q):
            return rope(q, k, positions, table)
    return _done(_native().rope(*_entry("fa_rope"), q, k, None, None, positions, *table._args,
                                False))


def rope_backward(dq, dk, positions, table: RopeTable, stream=None):
    """The gradients of ``rope``'s inputs from those of its outputs."""
    if stream is not None:
        with _on(stream, dq):
            return rope_backward(dq, dk, positions, table)
    return _done(_native().rope(*_entry("fa_rope"), dq, dk, None, None, positions, *table._args,
                                True))


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


def fa_cache_append(cache: PagedCache, k, v, cu_seqlens_new, seqlens_k, page_table,
                    max_seqlen_new: int, stream=None) -> None:
    """C ``fa_cache_append``: quantises the new rows k, v [total_new, Hkv, d] (bf16 or fp32,
    contiguous or strided) into the cache's pages; seqlens_k int32 [B] are the lengths after
    the call, page_table int32 [B, max_pages]."""
    if stream is not None:
        with _on(stream, k):
            return fa_cache_append(cache, k, v, cu_seqlens_new, seqlens_k, page_table,
                                   max_seqlen_new)
    _done(_native().cache_append(*_entry("fa_cache_append"), *cache, k, v, cu_seqlens_new,
                                 seqlens_k, page_table, max_seqlen_new))


cache_append = fa_cache_append


def fa_cache_read(cache: PagedCache, k, v, cu_seqlens_k, page_table, max_seqlen_k: int,
                  stream=None) -> None:
    """C ``fa_cache_read``: writes the cached rows of every sequence back to back into k, v
    [total_k, Hkv, d] (bf16 or fp32, contiguous or strided)."""
    if k is None or v is None:
        raise ValueError("k and v must be given")
    if stream is not None:
        with _on(stream, k):
            return fa_cache_read(cache, k, v, cu_seqlens_k, page_table, max_seqlen_k)
    _done(_native().cache_read(*_entry("fa_cache_read"), *cache, k, v, cu_seqlens_k, page_table,
                               max_seqlen_k, 0, False))


def cache_read(cache: PagedCache, cu_seqlens_k, page_table, max_seqlen_k: int, total_k: int,
               dtype=None, stream=None):
    """Allocate K and V ([total_k, Hkv, d], bf16 unless dtype is torch.float32) and run
    fa_cache_read."""
    import torch

    if dtype not in (None, torch.bfloat16, torch.float32):
        raise TypeError(f"unsupported dtype {dtype}; use bfloat16 or float32")
    if stream is not None:
        with _on(stream, cache.k):
            return cache_read(cache, cu_seqlens_k, page_table, max_seqlen_k, total_k, dtype)
    return _done(_native().cache_read(*_entry("fa_cache_read"), *cache, None, None, cu_seqlens_k,
                                      page_table, max_seqlen_k, total_k, dtype is torch.float32))


def fa_decode_cache_num_ctas(B: int, H: int, Hkv: int, max_seqlen_q: int,
                             max_seqlen_k: int) -> int:
    """C ``fa_decode_cache_num_ctas``: the number of thread blocks that fills this GPU."""
    n = int(load().fa_decode_cache_num_ctas(B, H, Hkv, max_seqlen_q, max_seqlen_k))
    check(min(n, 0))
    return n


def fa_decode_cache_workspace_bytes(H: int, Hkv: int, d: int, max_seqlen_q: int,
                                    num_ctas: int) -> int:
    return int(load().fa_decode_cache_workspace_bytes(H, Hkv, d, max_seqlen_q, num_ctas))


_DECODE_CACHE = ("fa_fwd_decode_cache", "fa_decode_cache_num_ctas",
                 "fa_decode_cache_workspace_bytes")


def fa_fwd_decode_cache(q, cache: PagedCache, o, lse, cu_seqlens_q, seqlens_k, page_table,
                        max_seqlen_q: int, max_seqlen_k: int, scale: float, causal: bool,
                        num_ctas: int, workspace, stream=None) -> None:
    """C ``fa_fwd_decode_cache``: q, o [total_q, H, d] bf16, lse [H, total_q] fp32 or None;
    cu_seqlens_q int32 [B + 1], seqlens_k int32 [B], page_table int32 [B, max_pages]; workspace
    (fa_decode_cache_workspace_bytes) may be None for num_ctas = 1."""
    if o is None:
        raise ValueError("o must be given")
    if num_ctas < 1:
        raise ValueError("num_ctas must be >= 1")
    if stream is not None:
        with _on(stream, q):
            return fa_fwd_decode_cache(q, cache, o, lse, cu_seqlens_q, seqlens_k, page_table,
                                       max_seqlen_q, max_seqlen_k, scale, causal, num_ctas,
                                       workspace)
    _done(_native().decode_cache(*_entry(*_DECODE_CACHE), q, *cache, o, lse, workspace,
                                 cu_seqlens_q, seqlens_k, page_table, max_seqlen_q, max_seqlen_k,
                                 scale, causal, num_ctas))


def forward_decode_cache(q, cache: PagedCache, cu_seqlens_q, seqlens_k, page_table,
                         max_seqlen_q: int, max_seqlen_k: int, scale: float | None = None,
                         causal: bool = False, num_ctas: int | None = None, stream=None):
    """Allocate O, LSE (and the workspace) and run fa_fwd_decode_cache."""
    if stream is not None:
        with _on(stream, q):
            return forward_decode_cache(q, cache, cu_seqlens_q, seqlens_k, page_table,
                                        max_seqlen_q, max_seqlen_k, scale, causal, num_ctas)
    return _done(_native().decode_cache(
        *_entry(*_DECODE_CACHE), q, *cache, None, None, None, cu_seqlens_q, seqlens_k, page_table,
        max_seqlen_q, max_seqlen_k, q.shape[-1] ** -0.5 if scale is None else scale, causal,
        num_ctas or 0))


# --------------------------------------------------------------------------- trees of drafted tokens

def fa_tree_mask(parents, mask, cu_seqlens_q, max_seqlen_q: int, stream=None) -> None:
    """C ``fa_tree_mask``: parents int32 [total_q], each token's parent as an index within its
    sequence (-1 for a root); mask int32 [total_q, words], 32 * words >= max_seqlen_q."""
    if mask is None:
        raise ValueError("mask must be given")
    if stream is not None:
        with _on(stream, parents):
            return fa_tree_mask(parents, mask, cu_seqlens_q, max_seqlen_q)
    _done(_native().tree_mask(*_entry("fa_tree_mask"), parents, mask, cu_seqlens_q, max_seqlen_q))


def tree_mask(parents, cu_seqlens_q, max_seqlen_q: int, stream=None):
    """Allocate and return the mask rows of trees given by their tokens' parents: bit j of a
    token's row is set for the token itself and its ancestors.  Rows that belong to no sequence are
    not written and hold anything, as in the decodes' outputs."""
    if stream is not None:
        with _on(stream, parents):
            return tree_mask(parents, cu_seqlens_q, max_seqlen_q)
    return _done(_native().tree_mask(*_entry("fa_tree_mask"), parents, None, cu_seqlens_q,
                                     max_seqlen_q))


def fa_decode_tree_num_ctas(B: int, H: int, Hkv: int, max_seqlen_q: int, max_seqlen_k: int) -> int:
    """C ``fa_decode_tree_num_ctas``: the number of thread blocks that fills this GPU."""
    n = int(load().fa_decode_tree_num_ctas(B, H, Hkv, max_seqlen_q, max_seqlen_k))
    check(min(n, 0))
    return n


def fa_decode_tree_workspace_bytes(H: int, Hkv: int, d: int, max_seqlen_q: int,
                                   num_ctas: int) -> int:
    return int(load().fa_decode_tree_workspace_bytes(H, Hkv, d, max_seqlen_q, num_ctas))


_DECODE_TREE = ("fa_fwd_decode_tree", "fa_decode_tree_num_ctas", "fa_decode_tree_workspace_bytes")


def fa_fwd_decode_tree(q, cache: PagedCache, o, lse, mask, cu_seqlens_q, seqlens_k, page_table,
                       max_seqlen_q: int, max_seqlen_k: int, scale: float, tree_start,
                       num_ctas: int, workspace, stream=None) -> None:
    """C ``fa_fwd_decode_tree``: q, o [total_q, H, d] bf16, lse [H, total_q] fp32 or None; mask
    int32 [total_q, words]; cu_seqlens_q int32 [B + 1], seqlens_k int32 [B], page_table int32 [B,
    max_pages], tree_start int32 [B] or None; workspace (fa_decode_tree_workspace_bytes) may be
    None for num_ctas = 1."""
    if o is None:
        raise ValueError("o must be given")
    if num_ctas < 1:
        raise ValueError("num_ctas must be >= 1")
    if stream is not None:
        with _on(stream, q):
            return fa_fwd_decode_tree(q, cache, o, lse, mask, cu_seqlens_q, seqlens_k, page_table,
                                      max_seqlen_q, max_seqlen_k, scale, tree_start, num_ctas,
                                      workspace)
    _done(_native().decode_tree(*_entry(*_DECODE_TREE), q, *cache, o, lse, workspace, mask,
                                cu_seqlens_q, seqlens_k, page_table, tree_start, max_seqlen_q,
                                max_seqlen_k, scale, num_ctas))


def forward_decode_tree(q, cache: PagedCache, mask, cu_seqlens_q, seqlens_k, page_table,
                        max_seqlen_q: int, max_seqlen_k: int, scale: float | None = None,
                        tree_start=None, num_ctas: int | None = None, stream=None):
    """Allocate O, LSE (and the workspace) and run fa_fwd_decode_tree: every token sees its
    sequence's keys before tree_start (None: before the sequence's own queries' keys, the last ones) and
    the drafted keys that its mask row names."""
    if stream is not None:
        with _on(stream, q):
            return forward_decode_tree(q, cache, mask, cu_seqlens_q, seqlens_k, page_table,
                                       max_seqlen_q, max_seqlen_k, scale, tree_start, num_ctas)
    return _done(_native().decode_tree(
        *_entry(*_DECODE_TREE), q, *cache, None, None, None, mask, cu_seqlens_q, seqlens_k,
        page_table, tree_start, max_seqlen_q, max_seqlen_k,
        q.shape[-1] ** -0.5 if scale is None else scale, num_ctas or 0))


# --------------------------------------------------------------------------- pages

def fa_cache_copy_pages(src: PagedCache, dst: PagedCache, copies, stream=None) -> None:
    """C ``fa_cache_copy_pages``: copies int32 [n, 3], rows of (source page, destination page,
    rows); src and dst may be one cache."""
    if stream is not None:
        with _on(stream, dst.k):
            return fa_cache_copy_pages(src, dst, copies)
    _done(_native().cache_copy_pages(*_entry("fa_cache_copy_pages"), *src, *dst, copies))


cache_copy_pages = fa_cache_copy_pages


def fa_cache_compact(cache: PagedCache, keep, cu_keep, start, page_table, max_keep: int,
                     stream=None) -> None:
    """C ``fa_cache_compact``: position start[b] + i of sequence b becomes what position start[b]
    + keep[cu_keep[b] + i] was; keep int32 [total_keep], rising within a sequence, cu_keep int32
    [B + 1], start int32 [B]."""
    if stream is not None:
        with _on(stream, cache.k):
            return fa_cache_compact(cache, keep, cu_keep, start, page_table, max_keep)
    _done(_native().cache_compact(*_entry("fa_cache_compact"), *cache, keep, cu_keep, start,
                                  page_table, max_keep))


cache_compact = fa_cache_compact


def fa_pages_workspace_bytes(slots: int, max_pages: int, num_pages: int) -> int:
    return int(load().fa_pages_workspace_bytes(slots, max_pages, num_pages))


_PAGES = ("fa_pages_update", "fa_pages_workspace_bytes")


def fa_pages_update(refs, page_table, seqlens, source, kept, new_lens, page_size: int, copies,
                    counts, workspace, stream=None) -> None:
    """C ``fa_pages_update``: refs int32 [num_pages] and page_table int32 [slots, max_pages] in
    place; seqlens, source, kept, new_lens int32 [slots]; copies int32 [slots, 3], counts int32
    [2], workspace of fa_pages_workspace_bytes."""
    if copies is None or counts is None or workspace is None:
        raise ValueError("copies, counts and the workspace must be given")
    if stream is not None:
        with _on(stream, refs):
            return fa_pages_update(refs, page_table, seqlens, source, kept, new_lens, page_size,
                                   copies, counts, workspace)
    _done(_native().pages_update(*_entry(*_PAGES), refs, page_table, seqlens, source, kept,
                                 new_lens, page_size, copies, counts, workspace))


def pages_update(refs, page_table, seqlens, source, kept, new_lens, page_size: int, stream=None):
    """One step of the bookkeeping of a cache's pages: slot b goes on from the first kept[b] rows
    of slot source[b] (itself, another that it forks, -1 for none) with room for new_lens[b] rows.
    refs (entries that name each page, 0: free) and page_table are updated in place.  Returns copies
    (int32 [slots, 3], for ``cache_copy_pages`` on every layer's cache) and counts (int32 [2]: pages
    missing, in which case nothing was changed, and pages free).  Without slots only the free pages are counted."""
    if stream is not None:
        with _on(stream, refs):
            return pages_update(refs, page_table, seqlens, source, kept, new_lens, page_size)
    return _done(_native().pages_update(*_entry(*_PAGES), refs, page_table, seqlens, source, kept,
                                        new_lens, page_size, None, None, None))


# --------------------------------------------------------------------------- shared prefixes

def fa_decode_shared_num_ctas() -> int:
    """C ``fa_decode_shared_num_ctas``: the number of thread blocks that fills this GPU."""
    n = int(load().fa_decode_shared_num_ctas())
    check(min(n, 0))
    return n


def fa_decode_shared_workspace_bytes(total_q: int, H: int, d: int, num_ctas: int) -> int:
    return int(load().fa_decode_shared_workspace_bytes(total_q, H, d, num_ctas))


_DECODE_SHARED = ("fa_fwd_decode_shared", "fa_decode_shared_num_ctas",
                  "fa_decode_shared_workspace_bytes")


def fa_fwd_decode_shared(q, k_prefix, v_prefix, k, v, o, lse, cu_seqlens_q, cu_seqlens_k,
                         cu_groups, cu_seqlens_p, max_seqlen_q: int, max_seqlen_k: int,
                         max_group_q: int, max_seqlen_p: int, scale: float, causal: bool,
                         num_ctas: int, workspace, stream=None) -> None:
    """C ``fa_fwd_decode_shared``: q, o [total_q, H, d]; k_prefix, v_prefix [total_p, Hkv, d];
    k, v [total_k, Hkv, d] (bf16); lse [H, total_q] fp32 or None; cu_seqlens_q, cu_seqlens_k
    int32 [B + 1]; cu_groups (first sequence of each group), cu_seqlens_p int32 [groups + 1].  A batch
    without own keys, or without prefixes, has tensors of no rows there."""
    if o is None:
        raise ValueError("o must be given")
    if num_ctas < 1:
        raise ValueError("num_ctas must be >= 1")
    if stream is not None:
        with _on(stream, q):
            return fa_fwd_decode_shared(q, k_prefix, v_prefix, k, v, o, lse, cu_seqlens_q,
                                        cu_seqlens_k, cu_groups, cu_seqlens_p, max_seqlen_q,
                                        max_seqlen_k, max_group_q, max_seqlen_p, scale, causal,
                                        num_ctas, workspace)
    _done(_native().decode_shared(*_entry(*_DECODE_SHARED), q, k_prefix, v_prefix, k, v, o, lse,
                                  workspace, cu_seqlens_q, cu_seqlens_k, cu_groups, cu_seqlens_p,
                                  max_seqlen_q, max_seqlen_k, max_group_q, max_seqlen_p, scale,
                                  causal, num_ctas))


def forward_decode_shared(q, k_prefix, v_prefix, k, v, cu_seqlens_q, cu_seqlens_k, cu_groups,
                          cu_seqlens_p, max_seqlen_q: int, max_seqlen_k: int, max_group_q: int,
                          max_seqlen_p: int, scale: float | None = None, causal: bool = False,
                          num_ctas: int | None = None, stream=None):
    """Allocate O, LSE and the workspace and run fa_fwd_decode_shared."""
    if stream is not None:
        with _on(stream, q):
            return forward_decode_shared(q, k_prefix, v_prefix, k, v, cu_seqlens_q, cu_seqlens_k,
                                         cu_groups, cu_seqlens_p, max_seqlen_q, max_seqlen_k,
                                         max_group_q, max_seqlen_p, scale, causal, num_ctas)
    return _done(_native().decode_shared(
        *_entry(*_DECODE_SHARED), q, k_prefix, v_prefix, k, v, None, None, None, cu_seqlens_q,
        cu_seqlens_k, cu_groups, cu_seqlens_p, max_seqlen_q, max_seqlen_k, max_group_q,
        max_seqlen_p, q.shape[-1] ** -0.5 if scale is None else scale, causal, num_ctas or 0))
