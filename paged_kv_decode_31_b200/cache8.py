"""Binding of the calls over an 8-bit paged cache (include/pagedkv.h): the
append that quantises into it and the attention that reads it.

The cache is a pair of torch.float8_e4m3fn tensors [num_blocks, block_size,
Hkv, D] with a power-of-two scale for each block and KV head: torch.
float8_e8m0fnu tensors [num_blocks, Hkv] (uint8 with the same bytes is taken
too).  Argument marshalling only, as in binding.py.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import torch

from .binding import (_I, _I64, _P, _check, _need_cache_and_table, _need_cuda_bf16, _need_cuda_i32,
                      _need_err, _need_lse, _need_one_device, _need_packed_bf16, _need_rows, _ptr,
                      _st2, lib, varlen_workspace_size, workspace_size)
from .rotary import _need_freq, _new_tokens, _on, _params, _strides

DEVERR_SCALE = 32


def _need_cache8(k_cache, v_cache, k_scale, v_scale) -> None:
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not t.is_cuda or t.dtype != torch.float8_e4m3fn:
            raise TypeError(f"{name} must be a float8_e4m3fn CUDA tensor (got {t.dtype} on {t.device})")
        if t.dim() != 4 or t.stride(-1) != 1:
            raise ValueError(f"{name} must be 4-D with a unit stride on the last axis")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if not t.is_cuda or t.dtype not in (torch.float8_e8m0fnu, torch.uint8):
            raise TypeError(f"{name} must be a float8_e8m0fnu (or uint8) CUDA tensor")
        if t.dim() != 2 or tuple(t.shape) != (k_cache.shape[0], k_cache.shape[2]):
            raise ValueError(f"{name} must be [num_blocks, Hkv] = "
                             f"[{k_cache.shape[0]}, {k_cache.shape[2]}] (got {list(t.shape)})")


@functools.lru_cache(maxsize=4096)
def _scale_strides(strides: tuple, shape: tuple) -> ctypes.Array:
    return (ctypes.c_int64 * 2)(*[s if n > 1 else max(s, 1) for s, n in zip(strides, shape)])


def _sst(t: torch.Tensor) -> ctypes.Array:
    """(block, head) strides; an axis of size 1 is never stepped over."""
    return _scale_strides(t.stride(), t.shape)


def kv_append_q8(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 block_table: torch.Tensor, seqlens: torch.Tensor, *,
                 q: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
                 cu_seqlens_new: Optional[torch.Tensor] = None, interleaved: bool = False,
                 mscale: float = 1.0, q_out: Optional[torch.Tensor] = None,
                 err: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Append bf16 k_new / v_new ([B, n, Hkv, D], or packed [total, Hkv, D] with
    cu_seqlens_new) to an 8-bit cache at positions seqlens[b] + t, with the keys
    (and q, returned) rotated on the way when inv_freq is given.  The scales of
    the blocks touched are updated, earlier tokens of a block requantised when
    its scale rises.  seqlens is not advanced."""
    B, n, total = _new_tokens(k_new, v_new, q, q_out, block_table, seqlens, cu_seqlens_new, err)
    Hkv, D = int(k_new.shape[-2]), int(k_new.shape[-1])
    _need_cache8(k_cache, v_cache, k_scale, v_scale)
    _need_cache_and_table(B, Hkv, D, k_cache, v_cache, block_table, seqlens)
    par = None
    if inv_freq is not None:
        _need_freq(inv_freq, D)
        par = _params(inv_freq, interleaved, mscale)
    elif q is not None:
        raise ValueError("q is rotated: it needs inv_freq")
    _need_one_device(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, q,
                     inv_freq, cu_seqlens_new, q_out, err)
    fn = lib().pkv_kv_append_q8
    if not fn.argtypes:
        fn.argtypes = [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P,
                       _I64, _P, _I64, _I, _P, _I, _I, _I, _I, _I, _P, _P, _P]
        fn.restype = _I
    with _on(k_new.device, stream) as s:
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k_new.numel():
            rc = fn(_ptr(q), _strides(q), _ptr(q_out), _strides(q_out),
                    0 if q is None else int(q.shape[-2]), k_new.data_ptr(), _strides(k_new),
                    v_new.data_ptr(), _strides(v_new), _ptr(cu_seqlens_new), total,
                    k_cache.data_ptr(), _strides(k_cache), v_cache.data_ptr(), _strides(v_cache),
                    k_scale.data_ptr(), _sst(k_scale), v_scale.data_ptr(), _sst(v_scale),
                    int(k_cache.shape[0]), block_table.data_ptr(), int(block_table.stride(0)),
                    int(block_table.shape[1]), seqlens.data_ptr(), B, n, Hkv, D,
                    int(k_cache.shape[1]), None if par is None else ctypes.addressof(par),
                    _ptr(err), s)
            _check("pkv_kv_append_q8", rc)
    return q_out


def _attn_q8(name, q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, max_seqlen_k, scale,
             causal, out, lse, workspace, err, stream):
    _need_cuda_bf16("q", q)
    _need_cache8(k_cache, v_cache, k_scale, v_scale)
    _need_cuda_i32("block_table", block_table)
    _need_cuda_i32("seqlens", seqlens)
    _need_err(err)
    B, sq, Hq, D = (int(x) for x in q.shape)
    num_blocks, bs, Hkv, _ = (int(x) for x in k_cache.shape)
    _need_cache_and_table(B, None, D, k_cache, v_cache, block_table, seqlens)
    fn = getattr(lib(), name)
    if not fn.argtypes:
        fn.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _I64, _I, _P, _I, _I, _I,
                       _I, _I, _I, _I, ctypes.c_float, _I, _P, _P, _P, _P, ctypes.c_size_t, _P, _P]
        fn.restype = _I
    with _on(q.device, stream) as s:
        if max_seqlen_k is None:
            max_seqlen_k = int(seqlens.max().item()) if seqlens.numel() else 0
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        if out is None:
            out = torch.empty(B, sq, Hq, D, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty(B, Hq, sq, dtype=torch.float32, device=q.device)
        _need_lse("lse", lse, (B, Hq, sq))
        _need_rows("out", out, (B, sq, Hq, D))
        if workspace is None:
            workspace = torch.empty(workspace_size(B, sq, Hq, D, max_seqlen_k), dtype=torch.uint8,
                                    device=q.device)
        _need_one_device(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, out, lse,
                         workspace, err)
        rc = fn(q.data_ptr(), _strides(q), k_cache.data_ptr(), _strides(k_cache), v_cache.data_ptr(),
                _strides(v_cache), k_scale.data_ptr(), _sst(k_scale), v_scale.data_ptr(),
                _sst(v_scale), num_blocks, block_table.data_ptr(), int(block_table.stride(0)),
                int(block_table.shape[1]), seqlens.data_ptr(), int(max_seqlen_k), B, sq, Hq, Hkv,
                D, bs, float(scale), int(bool(causal)), out.data_ptr(), _strides(out), lse.data_ptr(),
                workspace.data_ptr(), workspace.numel() * workspace.element_size(), _ptr(err), s)
        _check(name, rc)
    return out, lse


def paged_decode_attn_q8(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, *,
                         max_seqlen_k=None, scale=None, causal=False, out=None, lse=None,
                         workspace=None, err=None, stream=None):
    """paged_decode_attn over an 8-bit cache: attention of q [B, sq, Hq, D] bf16;
    returns (out [B, sq, Hq, D] bf16, lse [B, Hq, sq] fp32)."""
    return _attn_q8("pkv_paged_decode_attn_q8", q, k_cache, v_cache, k_scale, v_scale, block_table,
                    seqlens, max_seqlen_k, scale, causal, out, lse, workspace, err, stream)


def paged_prefill_attn_q8(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, *,
                          max_seqlen_k=None, scale=None, causal=True, out=None, lse=None,
                          workspace=None, err=None, stream=None):
    """paged_prefill_attn over an 8-bit cache (causal or chunked prefill)."""
    return _attn_q8("pkv_paged_prefill_attn_q8", q, k_cache, v_cache, k_scale, v_scale, block_table,
                    seqlens, max_seqlen_k, scale, causal, out, lse, workspace, err, stream)


def paged_varlen_attn_q8(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, cu_seqlens_q,
                         max_seqlen_q, *, max_seqlen_k=None, scale=None, causal=True, out=None,
                         lse=None, final=False, final_out=None, final_lse=None, workspace=None,
                         err=None, stream=None):
    """paged_varlen_attn over an 8-bit cache: packed q [total_q, Hq, D]; returns
    (out [total_q, Hq, D], lse [Hq, total_q]), with final=True also each
    request's last row (final_out [B, Hq, D], final_lse [B, Hq])."""
    _need_packed_bf16("q", q)
    _need_cache8(k_cache, v_cache, k_scale, v_scale)
    for n, t in (("block_table", block_table), ("seqlens", seqlens), ("cu_seqlens_q", cu_seqlens_q)):
        _need_cuda_i32(n, t)
    _need_err(err)
    total_q, Hq, D = (int(x) for x in q.shape)
    B = int(seqlens.shape[0])
    if tuple(cu_seqlens_q.shape) != (B + 1,) or not cu_seqlens_q.is_contiguous():
        raise ValueError("cu_seqlens_q must be a contiguous tensor of batch + 1 entries")
    num_blocks, bs, Hkv, _ = (int(x) for x in k_cache.shape)
    _need_cache_and_table(B, None, D, k_cache, v_cache, block_table, seqlens)
    fn = lib().pkv_paged_varlen_attn_q8
    if not fn.argtypes:
        fn.argtypes = [_P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _I64, _I, _P,
                       _I, _I, _I, _I, _I, _I, ctypes.c_float, _I, _P, _P, _P, _P, _P, _P, _P,
                       ctypes.c_size_t, _P, _P]
        fn.restype = _I
    with _on(q.device, stream) as s:
        if max_seqlen_k is None:
            max_seqlen_k = int(seqlens.max().item()) if seqlens.numel() else 0
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        new = dict(device=q.device)
        if out is None:
            out = torch.empty(total_q, Hq, D, dtype=torch.bfloat16, **new)
        if lse is None:
            lse = torch.empty(Hq, total_q, dtype=torch.float32, **new)
        _need_rows("out", out, (total_q, Hq, D))
        _need_lse("lse", lse, (Hq, total_q))
        if final or final_out is not None:
            if final_out is None:
                final_out = torch.empty(B, Hq, D, dtype=torch.bfloat16, **new)
            if final_lse is None:
                final_lse = torch.empty(B, Hq, dtype=torch.float32, **new)
            _need_rows("final_out", final_out, (B, Hq, D))
            _need_lse("final_lse", final_lse, (B, Hq))
        if workspace is None:
            workspace = torch.empty(varlen_workspace_size(total_q, Hq, D, max_seqlen_k),
                                    dtype=torch.uint8, **new)
        _need_one_device(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, cu_seqlens_q,
                         out, lse, final_out, final_lse, workspace, err)
        rc = fn(q.data_ptr(), _st2(q), cu_seqlens_q.data_ptr(), total_q, int(max_seqlen_q),
                k_cache.data_ptr(), _strides(k_cache), v_cache.data_ptr(), _strides(v_cache),
                k_scale.data_ptr(), _sst(k_scale), v_scale.data_ptr(), _sst(v_scale), num_blocks,
                block_table.data_ptr(), int(block_table.stride(0)), int(block_table.shape[1]),
                seqlens.data_ptr(), int(max_seqlen_k), B, Hq, Hkv, D, bs, float(scale),
                int(bool(causal)), out.data_ptr(), _st2(out), lse.data_ptr(), _ptr(final_out),
                None if final_out is None else _st2(final_out),
                None if final_out is None else _ptr(final_lse), workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), _ptr(err), s)
        _check("pkv_paged_varlen_attn_q8", rc)
    if final_out is not None:
        return out, lse, final_out, final_lse
    return out, lse
