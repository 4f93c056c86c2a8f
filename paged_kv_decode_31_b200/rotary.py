"""Binding of the rotary calls (include/pagedkv.h): rotation of queries and
keys, the rotating append into a paged cache and its backward.

Argument marshalling only, as in binding.py; `rope_frequencies` computes the
table of inverse frequencies on the host.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple, Union

import torch

from .binding import (_I, _I64, _P, _check, _need_cache_and_table, _need_cuda_bf16, _need_cuda_i32,
                      _need_err, _need_one_device, _ptr, _stream_handle, lib)


class _RopeParams(ctypes.Structure):
    _fields_ = [("inv_freq", _P), ("rotary_dim", _I), ("interleaved", _I),
                ("mscale", ctypes.c_float)]


def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: Optional[str] = None,
                     factor: float = 1.0, original_max: Optional[int] = None,
                     fast: float = 32.0, slow: float = 1.0,
                     device=None) -> Tuple[torch.Tensor, float]:
    """Inverse frequencies (fp32 [rotary_dim / 2], computed in fp64 and rounded
    once) and the magnitude factor for rope().  f_i = base ** (-2 i / rotary_dim),
    stretched for contexts `factor` times the trained length by

      None      not at all;
      "linear"  f_i / factor (positions interpolated);
      "base"    a larger base, base * factor ** (r / (r - 2)): the fastest pair
                keeps its frequency, the slowest is divided by factor;
      "blend"   pairs that turn at least `fast` times within original_max keep
                f_i, those that turn at most `slow` times get f_i / factor, with
                a ramp linear in the pair index between, and the magnitude factor
                0.1 ln(factor) + 1;
      "bands"   the same borders with a ramp linear in the number of turns, and
                magnitude 1."""
    if rotary_dim <= 0 or rotary_dim % 16:
        raise ValueError(f"rotary_dim must be a positive multiple of 16 (got {rotary_dim})")
    if not base > 1 or not factor >= 1:
        raise ValueError("base must be above 1 and factor at least 1")
    half = rotary_dim // 2
    i = torch.arange(half, dtype=torch.float64)
    m = 1.0
    if scaling == "base":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = float(base) ** (-i / half)
    if scaling == "linear":
        f = f / factor
    elif scaling in ("blend", "bands"):
        if original_max is None or original_max <= 0 or not fast > slow > 0:
            raise ValueError(f"scaling {scaling!r} needs original_max > 0 and fast > slow > 0")
        turns = original_max * f / (2 * math.pi)
        if scaling == "bands":
            keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        else:
            # pair index at which f_i turns n times within original_max
            at = [half * math.log(original_max / (2 * math.pi * n)) / math.log(base)
                  for n in (fast, slow)]
            # whole indexes, held to [0, rotary_dim - 1]: the upper border may lie
            # past the last pair, which then keeps a part of its frequency
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rotary_dim - 1)
            # (hi <= 0: not even the fastest pair turns more than `slow` times)
            keep = 1 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1) if hi > 0 else torch.zeros_like(i)
            m = 0.1 * math.log(factor) + 1.0
        f = f * keep + f / factor * (1 - keep)
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(torch.float32).to(device), m


class _on:
    """The tensors' device and the call's stream made current: outputs and
    workspaces are allocated for the stream that uses them.  Entering gives the
    stream's handle.  (A class, and nothing switched when both are current
    already: the host's share of a small call is most of its time.)"""

    __slots__ = ("device", "stream", "inside")

    def __init__(self, device: torch.device, stream):
        self.device, self.stream, self.inside = device, stream, None

    def __enter__(self) -> int:
        index = self.device.index
        if self.stream is None and index == torch.cuda.current_device():
            return _stream_handle(None) if _raw_stream is None else _raw_stream(index)
        guard = torch.cuda.device(self.device)
        guard.__enter__()
        self.inside = [guard]
        stream = self.stream
        if stream is None:
            return _stream_handle(None)
        try:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=self.device) if int(stream) else \
                    torch.cuda.default_stream(self.device)
            switch = torch.cuda.stream(stream)
            switch.__enter__()
        except BaseException:
            guard.__exit__(None, None, None)
            raise
        self.inside.append(switch)
        return _stream_handle(stream)

    def __exit__(self, *exc) -> None:
        for ctx in reversed(self.inside or ()):
            ctx.__exit__(*exc)


# the current stream's handle without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _need_freq(inv_freq: torch.Tensor, D: int) -> None:
    if not inv_freq.is_cuda or inv_freq.dtype != torch.float32:
        raise TypeError("inv_freq must be a float32 CUDA tensor")
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be 1-D and contiguous")
    r = 2 * int(inv_freq.shape[0])
    if r == 0 or r % 16 or r > D:
        raise ValueError(f"inv_freq holds {r // 2} pairs: the rotated part must be a multiple of 16 "
                         f"elements, at most head_dim {D}")


def _params(inv_freq: torch.Tensor, interleaved: bool, mscale: float):
    if not 0 < float(mscale) < 3.0e38:
        raise ValueError(f"mscale must be positive and finite (got {mscale})")
    return _RopeParams(inv_freq.data_ptr(), 2 * int(inv_freq.shape[0]), int(bool(interleaved)),
                       float(mscale))


def _need_tokens(name: str, t: torch.Tensor, packed: bool, lead=None, tail=None) -> None:
    """bf16 rows [tokens, heads, D] (packed) or [B, n, heads, D], unit last
    stride; `lead` / `tail`: the leading / trailing sizes they must have."""
    if not t.is_cuda or t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be a bf16 CUDA tensor (got {t.dtype} on {t.device})")
    want = 3 if packed else 4
    if t.dim() != want or t.stride(-1) != 1:
        raise ValueError(f"{name} must be {want}-D with a unit stride on the last axis")
    if (lead is not None and tuple(t.shape[:-2]) != tuple(lead)) or \
            (tail is not None and tuple(t.shape[-len(tail):]) != tuple(tail)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}: it disagrees with the other tensors")


@functools.lru_cache(maxsize=4096)
def _stride_array(strides: tuple, shape: tuple) -> ctypes.Array:
    st = [s if n > 1 else max(s, 1) * 16 for s, n in zip(strides, shape)][:-1]
    return (ctypes.c_int64 * 3)(*([st[0]] + st if len(st) == 2 else st))


def _strides(t: Optional[torch.Tensor]):
    """(batch, token, head) strides; a packed tensor repeats its token stride.
    Axes of size 1 are never stepped over and get a stride that passes.  (The
    arrays are shared between calls: nothing writes to them.)"""
    return None if t is None else _stride_array(t.stride(), t.shape)


def rope(q: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, *,
         k: Optional[torch.Tensor] = None, interleaved: bool = False, mscale: float = 1.0,
         inverse: bool = False, out: Optional[torch.Tensor] = None,
         k_out: Optional[torch.Tensor] = None,
         stream=None) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """Rotate q [B, n, Hq, D] (or packed [tokens, Hq, D]) at `positions` (int32,
    one per token), and k beside it; returns q's rows, or both.  The first
    2 * len(inv_freq) elements of a head turn, the rest is copied.  out / k_out
    may be q / k.  inverse=True is the transpose: the gradient of the forward
    call.  See include/pagedkv.h."""
    packed = q.dim() == 3
    _need_tokens("q", q, packed)
    lead, D = q.shape[:-2], int(q.shape[-1])
    if k is not None:
        _need_tokens("k", k, packed, lead, (D,))
    elif k_out is not None:
        raise ValueError("k_out needs k")
    _need_cuda_i32("positions", positions)
    if positions.shape != lead or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous {tuple(lead)} tensor")
    _need_freq(inv_freq, D)
    par = _params(inv_freq, interleaved, mscale)
    fn = lib().pkv_rope
    if not fn.argtypes:
        fn.argtypes = [_P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P, _I, _P]
        fn.restype = _I
    with _on(q.device, stream) as s:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        _need_tokens("out", out, packed, lead, q.shape[-2:])
        if k is not None:
            _need_tokens("k_out", k_out, packed, lead, k.shape[-2:])
        _need_one_device(q, k, positions, inv_freq, out, k_out)
        B, n = (1, int(lead[0])) if packed else (int(lead[0]), int(lead[1]))
        if q.numel() or (k is not None and k.numel()):
            rc = fn(q.data_ptr(), _strides(q), out.data_ptr(), _strides(out), int(q.shape[-2]),
                    _ptr(k), _strides(k), _ptr(k_out), _strides(k_out),
                    0 if k is None else int(k.shape[-2]), positions.data_ptr(), B, n, D,
                    ctypes.addressof(par), int(bool(inverse)), s)
            _check("pkv_rope", rc)
    return out if k is None else (out, k_out)


def _need_cu(cu: Optional[torch.Tensor], seqlens: torch.Tensor) -> int:
    """The batch of a packed call; cu_seqlens_new must be [batch + 1]."""
    B = int(seqlens.shape[0])
    _need_cuda_i32("cu_seqlens_new", cu)
    if tuple(cu.shape) != (B + 1,) or not cu.is_contiguous():
        raise ValueError("cu_seqlens_new must be a contiguous tensor of batch + 1 entries")
    return B


def _new_tokens(k_new, v_new, q, q_out, block_table, seqlens, cu, err):
    """Checks of an append's new tokens; returns (batch, n_new, total_new)."""
    packed = cu is not None
    _need_tokens("k_new", k_new, packed)
    lead, D = k_new.shape[:-2], int(k_new.shape[-1])
    _need_tokens("v_new", v_new, packed, lead, k_new.shape[-2:])
    if q is not None:
        _need_tokens("q", q, packed, lead, (D,))
        if q_out is not None:
            _need_tokens("q_out", q_out, packed, lead, q.shape[-2:])
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _need_cuda_i32("block_table", block_table)
    _need_cuda_i32("seqlens", seqlens)
    _need_err(err)
    if packed:
        return _need_cu(cu, seqlens), 0, int(lead[0])
    return int(lead[0]), int(lead[1]), 0


def kv_append_rope(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, block_table: torch.Tensor, seqlens: torch.Tensor,
                   inv_freq: torch.Tensor, *, q: Optional[torch.Tensor] = None,
                   cu_seqlens_new: Optional[torch.Tensor] = None, interleaved: bool = False,
                   mscale: float = 1.0, q_out: Optional[torch.Tensor] = None,
                   err: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """kv_append with the rotation on the way: k_new [B, n, Hkv, D] (or packed
    [total, Hkv, D] with cu_seqlens_new) is rotated at seqlens[b] + t and stored,
    v_new stored as it is; q [.., Hq, D], if given, is rotated at the same
    positions and returned (into q_out, which may be q).  seqlens is not
    advanced."""
    B, n, total = _new_tokens(k_new, v_new, q, q_out, block_table, seqlens, cu_seqlens_new, err)
    Hkv, D = int(k_new.shape[-2]), int(k_new.shape[-1])
    _need_cuda_bf16("k_cache", k_cache)
    _need_cuda_bf16("v_cache", v_cache)
    _need_cache_and_table(B, Hkv, D, k_cache, v_cache, block_table, seqlens)
    _need_freq(inv_freq, D)
    par = _params(inv_freq, interleaved, mscale)
    _need_one_device(k_new, v_new, k_cache, v_cache, block_table, seqlens, inv_freq, q,
                     cu_seqlens_new, q_out, err)
    fn = lib().pkv_kv_append_rope
    if not fn.argtypes:
        fn.argtypes = [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _I64, _P, _I64,
                       _I, _P, _I, _I, _I, _I, _I, _P, _P, _P]
        fn.restype = _I
    with _on(k_new.device, stream) as s:
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k_new.numel():
            rc = fn(_ptr(q), _strides(q), _ptr(q_out), _strides(q_out),
                    0 if q is None else int(q.shape[-2]), k_new.data_ptr(), _strides(k_new),
                    v_new.data_ptr(), _strides(v_new), _ptr(cu_seqlens_new), total,
                    k_cache.data_ptr(), _strides(k_cache), v_cache.data_ptr(), _strides(v_cache),
                    int(k_cache.shape[0]), block_table.data_ptr(), int(block_table.stride(0)),
                    int(block_table.shape[1]), seqlens.data_ptr(), B, n, Hkv, D,
                    int(k_cache.shape[1]), ctypes.addressof(par), _ptr(err), s)
            _check("pkv_kv_append_rope", rc)
    return q_out


def kv_append_rope_bwd(dq_rot: Optional[torch.Tensor], dk_cache: torch.Tensor,
                       dv_cache: torch.Tensor, block_table: torch.Tensor, seqlens: torch.Tensor,
                       inv_freq: torch.Tensor, *, n_new: Optional[int] = None,
                       cu_seqlens_new: Optional[torch.Tensor] = None,
                       total_new: Optional[int] = None, interleaved: bool = False,
                       mscale: float = 1.0, dq: Optional[torch.Tensor] = None,
                       dk_new: Optional[torch.Tensor] = None,
                       dv_new: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                       stream=None):
    """Backward of kv_append_rope: (dq, dk_new, dv_new) from the gradient of the
    rotated queries (or None, then dq is None) and the cache-row gradients of
    paged_prefill_attn_bwd.  The tokens are those of the forward call (seqlens
    before it): dense with n_new (dq_rot's second size when that is given), or
    packed with cu_seqlens_new and total_new (dq_rot's first size)."""
    packed = cu_seqlens_new is not None
    _need_cuda_bf16("dk_cache", dk_cache)
    _need_cuda_bf16("dv_cache", dv_cache)
    _need_cuda_i32("block_table", block_table)
    _need_cuda_i32("seqlens", seqlens)
    _need_err(err)
    _, bs, Hkv, D = (int(x) for x in dk_cache.shape)
    if dq_rot is not None:
        _need_tokens("dq_rot", dq_rot, packed, None, (D,))
    elif dq is not None:
        raise ValueError("dq needs dq_rot")
    if packed:
        B = _need_cu(cu_seqlens_new, seqlens)
        if total_new is None and dq_rot is None:
            raise ValueError("a packed call without dq_rot needs total_new")
        lead = (int(dq_rot.shape[0] if total_new is None else total_new),)
    else:
        B = int(seqlens.shape[0]) if dq_rot is None else int(dq_rot.shape[0])
        if n_new is None and dq_rot is None:
            raise ValueError("a dense call without dq_rot needs n_new")
        lead = (B, int(dq_rot.shape[1] if n_new is None else n_new))
    if min(lead) < 0:
        raise ValueError("n_new and total_new must not be negative")
    if dq_rot is not None:
        _need_tokens("dq_rot", dq_rot, packed, lead, (D,))
        if dq is not None:
            _need_tokens("dq", dq, packed, lead, dq_rot.shape[-2:])
    for name, t in (("dk_new", dk_new), ("dv_new", dv_new)):
        if t is not None:
            _need_tokens(name, t, packed, lead, (Hkv, D))
    _need_cache_and_table(B, Hkv, D, dk_cache, dv_cache, block_table, seqlens)
    _need_freq(inv_freq, D)
    par = _params(inv_freq, interleaved, mscale)
    _need_one_device(dk_cache, dv_cache, block_table, seqlens, inv_freq, dq_rot, cu_seqlens_new,
                     dq, dk_new, dv_new, err)
    fn = lib().pkv_kv_append_rope_bwd
    if not fn.argtypes:
        fn.argtypes = [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I64, _P, _I64,
                       _I, _P, _I, _I, _I, _I, _I, _P, _P, _P]
        fn.restype = _I
    with _on(dk_cache.device, stream) as s:
        new = dict(dtype=torch.bfloat16, device=dk_cache.device)
        if dq_rot is not None and dq is None:
            dq = torch.empty(dq_rot.shape, **new)
        dk_new = torch.empty(*lead, Hkv, D, **new) if dk_new is None else dk_new
        dv_new = torch.empty(*lead, Hkv, D, **new) if dv_new is None else dv_new
        if dk_new.numel():
            rc = fn(_ptr(dq_rot), _strides(dq_rot), _ptr(dq), _strides(dq),
                    0 if dq is None else int(dq.shape[-2]), dk_cache.data_ptr(),
                    _strides(dk_cache), dv_cache.data_ptr(), _strides(dv_cache),
                    dk_new.data_ptr(), _strides(dk_new), dv_new.data_ptr(), _strides(dv_new),
                    _ptr(cu_seqlens_new), lead[0] if packed else 0, int(dk_cache.shape[0]),
                    block_table.data_ptr(), int(block_table.stride(0)), int(block_table.shape[1]),
                    seqlens.data_ptr(), B, 0 if packed else lead[1], Hkv, D, bs,
                    ctypes.addressof(par), _ptr(err), s)
            _check("pkv_kv_append_rope_bwd", rc)
    return dq, dk_new, dv_new
