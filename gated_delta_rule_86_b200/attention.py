"""Python binding of the softmax-attention calls of the C ABI (include/kda.h).

As in ``ops``: argument marshalling only.  Shapes are checked, outputs and
workspaces are allocated with torch, pointers and the stream are passed to
libkda_b200.so, and a non-OK status becomes a :class:`KdaError`.  All tensors
of a call live on one CUDA device; the call runs on that device's current
stream, whichever device is current.  A token tensor whose last two dimensions
are dense and whose tokens lie an even distance apart (a slice of a fused
projection, say) is read where it is; any other layout is copied first.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from .ops import _DTYPES


def _check_device(dev, tensors):
    if dev.type != "cuda":
        raise ValueError("softmax attention takes CUDA tensors")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"all tensors of a call must be on one device: got {t.device} beside {dev}")


def _code(*ts):
    dt = ts[0].dtype
    if dt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dt}; use torch.float32 or torch.bfloat16")
    for t in ts:
        if t is not None and t.dtype != dt:
            raise TypeError("all token tensors and the cache must share one dtype")
    return _DTYPES[dt]


def _int32(t, name, n=None):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.dim() != 1:
        raise TypeError(f"{name} must be a one-dimensional int32 tensor")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} entries")
    return t.contiguous()


def _p(t):
    return None if t is None else t.data_ptr()


def _tokens(t):
    """(tensor, elements from one token to the next) of [B, T, H, d] as the kernels can read it."""
    B, T, H, d = t.shape
    if t.is_contiguous():
        step = H * d
    else:
        sb, step, sh, sd = t.stride()
        if T == 1:
            step = sb   # one token per row: the rows are the tokens
        elif B > 1 and sb != T * step:
            step = 0
        if sd != 1 or (sh != d and H > 1) or step < H * d or step * t.element_size() % 16 or B * T < 2:
            t, step = t.contiguous(), H * d
    if t.data_ptr() % 16:
        t, step = t.clone(memory_format=torch.contiguous_format), H * d
    return t, step


class _on:
    """Makes a tensor's device current for the call; nothing to do where it is already."""

    __slots__ = ("dev", "guard")

    def __init__(self, dev):
        self.dev = dev

    def __enter__(self):
        self.guard = None
        if torch.cuda.current_device() != self.dev.index:
            self.guard = torch.cuda.device(self.dev)
            self.guard.__enter__()
        return torch.cuda.current_stream(self.dev).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


# ---- prompts ------------------------------------------------------------------------------------


def _prompt_args(q, k, v, cu, cu_k, causal, scale):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B, Tq, Hq, d] and k, v [B, Tk, Hkv, d]")
    B, Tq, Hq, d = q.shape
    Tk, Hkv = k.shape[1], k.shape[2]
    if k.shape != (B, Tk, Hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, Tk, Hkv, d] with q's B and d")
    if Hkv == 0 or Hq % Hkv:
        raise ValueError(f"the {Hq} query heads must be a multiple of the {Hkv} heads of k and v")
    if cu is None and cu_k is not None:
        raise ValueError("cu_seqlens_k needs cu_seqlens")
    cu, cu_k = _int32(cu, "cu_seqlens"), _int32(cu_k, "cu_seqlens_k", None if cu is None else cu.numel())
    n = 0
    if cu is not None:
        n = cu.numel() - 1
        if B != 1 or n < 1:
            raise ValueError("cu_seqlens requires B == 1 and at least two offsets")
        if cu_k is None and Tk != Tq:
            raise ValueError("packed k and v of another length than q need cu_seqlens_k")
    dt = _code(q, k, v)
    _check_device(q.device, (k, v, cu, cu_k))
    (q, qs), (k, ks), (v, vs) = _tokens(q), _tokens(k), _tokens(v)
    args = [_p(q), _p(k), _p(v), qs, ks, vs, _p(cu), _p(cu_k), n, B, Tq, Tk, Hq, Hkv, d, int(bool(causal)),
            _scale(scale, d), dt]
    return args, (q, k, v, cu, cu_k), (B, Tq, Tk, Hq, Hkv, d)


def _out_tensor(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.shape != tuple(shape) or out.dtype != dtype or out.device != device or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {list(shape)} on {device}")
    return out


def kda_attn_fwd(q, k, v, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None, out=None, return_lse=False):
    """Attention over whole prompts: ``softmax(scale q k^T + mask) v``.

    q: [B, Tq, Hq, d]; k, v: [B, Tk, Hkv, d] (bf16 or fp32, d 64 or 128); query head h reads head
    ``h // (Hq // Hkv)``.  cu_seqlens: int32 [N+1] offsets of packed sequences (B == 1), cu_seqlens_k
    those of k and v where they differ.  Causal: query i of a sequence sees keys j <= i + nk - nq; a
    query that sees none gets zeros.  scale: 1 / sqrt(d) by default.  Returns out [B, Tq, Hq, d] in the
    inputs' dtype, with ``return_lse`` also the fp32 [B, Hq, Tq] logarithms of the softmax sums.  Rows
    behind the last packed sequence are not written.
    """
    args, (q, *_keep), (B, Tq, _, Hq, _, d) = _prompt_args(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale)
    o = _out_tensor(out, (B, Tq, Hq, d), q.dtype, q.device)
    lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device) if return_lse else None
    with _on(q.device) as stream:
        _lib.check(_lib.load().kda_attn_fwd(*args, _p(o), _p(lse), stream), "kda_attn_fwd")
    return (o, lse) if return_lse else o


def kda_attn_bwd(q, k, v, out, lse, d_out, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None):
    """Gradient of :func:`kda_attn_fwd`: ``(dq, dk, dv)`` in the inputs' dtype, from the forward's inputs,
    its ``out`` and ``lse``, and ``d_out``.  dk and dv are summed over the query heads that share them.
    Rows behind the last packed sequence get zeros.  The same call gives the same bits."""
    args, (q, *_keep), (B, Tq, Tk, Hq, Hkv, d) = _prompt_args(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale)
    dev = q.device
    if out.shape != (B, Tq, Hq, d) or d_out.shape != out.shape or lse.shape != (B, Hq, Tq):
        raise ValueError("out and d_out must have q's shape, and lse [B, Hq, Tq]")
    if lse.dtype != torch.float32:
        raise TypeError("lse must be float32")
    _check_device(dev, (out, lse, d_out))
    _code(q, out, d_out)
    out, lse, d_out = _tokens(out.contiguous())[0], lse.contiguous(), _tokens(d_out.contiguous())[0]
    like = dict(dtype=q.dtype, device=dev)
    dq, dk, dv = torch.empty((B, Tq, Hq, d), **like), torch.empty((B, Tk, Hkv, d), **like), torch.empty((B, Tk, Hkv, d), **like)
    lib, size = _lib.load(), ctypes.c_size_t(0)
    with _on(dev) as stream:
        _lib.check(lib.kda_attn_bwd_workspace_size(B, Tq, Hq, ctypes.byref(size)), "kda_attn_bwd_workspace_size")
        ws = torch.empty(max(size.value, 16), dtype=torch.uint8, device=dev)
        _lib.check(lib.kda_attn_bwd(*args, _p(out), _p(lse), _p(d_out), _p(dq), _p(dk), _p(dv), _p(ws), ws.numel(),
                                    stream), "kda_attn_bwd")
    return dq, dk, dv


class _KdaAttn(torch.autograd.Function):
    """Autograd wrapper: forward = kda_attn_fwd, backward = kda_attn_bwd (both in the library)."""

    @staticmethod
    def forward(ctx, q, k, v, cu, cu_k, causal, scale):
        out, lse = kda_attn_fwd(q, k, v, cu, cu_k, causal, scale, return_lse=True)
        ctx.save_for_backward(q, k, v, out, lse, cu, cu_k)
        ctx.causal, ctx.scale = causal, scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out):
        q, k, v, out, lse, cu, cu_k = ctx.saved_tensors
        grads = kda_attn_bwd(q, k, v, out, lse, d_out, cu, cu_k, ctx.causal, ctx.scale)
        return (*(g if need else None for g, need in zip(grads, ctx.needs_input_grad)), None, None, None, None)


def kda_attn(q, k, v, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None):
    """Differentiable attention over whole prompts: :func:`kda_attn_fwd` with gradients for q, k and v
    (through :func:`kda_attn_bwd`).  Rows of the output behind the last packed sequence are not written
    and must not reach the loss."""
    return _KdaAttn.apply(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale)


# ---- the paged cache ----------------------------------------------------------------------------


def _cache_args(k_cache, v_cache, page_table, n):
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [num_pages, Hkv, page_size, d]")
    pages, H, size, d = k_cache.shape
    dense = (size * d, d, 1)
    for c in (k_cache, v_cache):   # the cache is used in place: no copy can stand in for it
        if c.stride()[1:] != dense and not c.is_contiguous():
            raise ValueError("a page of the cache must be dense; pages may lie apart")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != n:
        raise ValueError(f"page_table must be an int32 tensor [{n}, pages of a sequence]")
    if page_table.stride(1) != 1 and page_table.shape[1] > 1:
        page_table = page_table.contiguous()
    row = page_table.stride(0) if n > 1 else page_table.shape[1]
    step = [c.stride(0) if pages > 1 else H * size * d for c in (k_cache, v_cache)]
    return page_table, row, step, (pages, H, size, d)


def kda_kv_append(k, v, k_cache, v_cache, page_table, cache_lens, inv_freq=None, q=None, cu_seqlens=None,
                  interleaved=False, return_k=False, q_out=None):
    """Appends k and v to a paged cache, rotating k (and q) by position; returns ``(q_rotated, k_rotated)``.

    k, v: [B, T, Hkv, d]; q: [B, T, Hq, d] or None.  k_cache, v_cache: [num_pages, Hkv, page_size, d],
    written in place (page_size a power of two; pages may lie apart).  page_table: int32 [N, width]; token
    p of sequence n lies in page ``page_table[n, p // page_size]``.  cache_lens: int32 [N], the tokens of
    each sequence before the call (negative: an unused row); new token j gets position
    ``cache_lens[n] + j``.  inv_freq: fp32 [r / 2]: the first r channels turn in pairs (i, i + r/2), or
    (2i, 2i+1) when ``interleaved``, by position * inv_freq[i]; None: no rotation.  q_rotated is None
    without q and is written to ``q_out`` where given (it may be a contiguous q itself); k_rotated is None unless
    ``return_k``.  Tokens without a valid page are left out and :func:`device_error` reports it.
    """
    if k.dim() != 4 or v.shape != k.shape:
        raise ValueError("k and v must be [B, T, Hkv, d]")
    B, T, Hkv, d = k.shape
    if q is not None and (q.dim() != 4 or q.shape[:2] != k.shape[:2] or q.shape[3] != d or q.shape[2] % Hkv):
        raise ValueError("q must be [B, T, Hq, d] with Hq a multiple of Hkv")
    cu = _int32(cu_seqlens, "cu_seqlens")
    n = B if cu is None else cu.numel() - 1
    if cu is not None and (B != 1 or n < 1):
        raise ValueError("cu_seqlens requires B == 1 and at least two offsets")
    cache_lens = _int32(cache_lens, "cache_lens", n)
    table, row, steps, (pages, H, size, cd) = _cache_args(k_cache, v_cache, page_table, n)
    if (H, cd) != (Hkv, d):
        raise ValueError(f"the cache holds {H} heads of {cd} channels, k and v {Hkv} of {d}")
    dt = _code(k, v, q, k_cache, v_cache)
    dev = k.device
    _check_device(dev, (v, q, k_cache, v_cache, table, cache_lens, inv_freq, cu, q_out))
    if inv_freq is not None and (inv_freq.dtype != torch.float32 or inv_freq.dim() != 1):
        raise TypeError("inv_freq must be a one-dimensional float32 tensor")
    freq = None if inv_freq is None else inv_freq.contiguous()
    Hq, qs, qo = 0, 0, None
    (k, ks), (v, vs) = _tokens(k), _tokens(v)
    if q is not None:
        Hq = q.shape[2]
        qo = _out_tensor(q_out, q.shape, q.dtype, dev)
        q, qs = _tokens(q)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    ko = torch.empty((B, T, Hkv, d), dtype=k.dtype, device=dev) if return_k else None
    with _on(dev) as stream:
        _lib.check(_lib.load().kda_kv_append(
            _p(q), _p(k), _p(v), qs, ks, vs, _p(freq), 0 if freq is None else 2 * freq.numel(),
            int(bool(interleaved)), _p(cu), n, B, T, Hq, Hkv, d, dt, _p(cache_lens), _p(table), row, table.shape[1],
            _p(k_cache), _p(v_cache), steps[0], steps[1], pages, size, _p(qo), _p(ko), stream), "kda_kv_append")
    return qo, ko


def kda_attn_decode_step(q, k_cache, v_cache, page_table, seq_lens, scale=None, out=None, return_lse=False):
    """Attention of one new token per sequence over a paged cache (see :func:`kda_kv_append` for its layout).

    q: [B, Hq, d]; seq_lens: int32 [B], the tokens of each sequence in the cache, the new one among them
    (0 or less: the row's output is zero).  Returns out [B, Hq, d] in q's dtype (``out``, if given,
    receives it), with ``return_lse`` also the fp32 [B, Hq] logarithms of the softmax sums.
    """
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, d]")
    B, Hq, d = q.shape
    table, row, steps, (pages, Hkv, size, cd) = _cache_args(k_cache, v_cache, page_table, B)
    if cd != d or Hkv == 0 or Hq % Hkv:
        raise ValueError(f"q of {Hq} heads of {d} channels does not go with a cache of {Hkv} of {cd}")
    seq_lens = _int32(seq_lens, "seq_lens", B)
    dt = _code(q, k_cache, v_cache)
    dev = q.device
    _check_device(dev, (k_cache, v_cache, table, seq_lens))
    qt, qs = _tokens(q.unsqueeze(1))
    o = _out_tensor(out, (B, Hq, d), q.dtype, dev)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev) if return_lse else None
    lib, need = _lib.load(), ctypes.c_size_t(0)
    with _on(dev) as stream:
        _lib.check(lib.kda_attn_decode_workspace_size(B, Hq, Hkv, d, dt, ctypes.byref(need)),
                   "kda_attn_decode_workspace_size")
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
        _lib.check(lib.kda_attn_decode_step(
            _p(qt), qs, _p(k_cache), _p(v_cache), steps[0], steps[1], pages, size, _p(table), row, table.shape[1],
            _p(seq_lens), B, Hq, Hkv, d, _scale(scale, d), dt, _p(o), _p(lse), _p(ws), need.value, stream),
            "kda_attn_decode_step")
    return (o, lse) if return_lse else o
