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
import functools

import torch

from . import _lib
from .ops import _DTYPES, KdaError


_raw_stream = torch._C._cuda_getCurrentRawStream   # a device's current stream as an integer


def _same(t, tensors):
    """The (library's code of the) dtype that these tensors share with t, and the device that they lie on."""
    dt, dev = t.dtype, t.get_device()
    for x in tensors:
        if x.dtype != dt:
            raise TypeError(f"all token tensors and the cache must share one dtype: got {x.dtype} beside {dt}")
        if x.get_device() != dev:
            raise ValueError(f"all tensors of a call must be on one device: got {x.device} beside {t.device}")
    if dt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dt}; use torch.float32 or torch.bfloat16")
    if dev < 0:
        raise ValueError("softmax attention takes CUDA tensors")
    return _DTYPES[dt], dev


def _ints(t, name, n, dev):
    """A one-dimensional int32 tensor of n entries (any number: None) on the call's device, dense."""
    if t.dtype != torch.int32 or t.dim() != 1:
        raise TypeError(f"{name} must be a one-dimensional int32 tensor")
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors")
    return t if t.is_contiguous() else t.contiguous()


def _call(name, dev, *args):
    """Runs a library call with its device current, on that device's current stream."""
    fn = getattr(_lib.load(), name)
    if torch.cuda.current_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        raise KdaError(status, name)


def _p(t):
    return None if t is None else t.data_ptr()


def _tokens(t):
    """(tensor, elements from one token to the next) of [B, T, H, d] as the kernels can read it."""
    B, T, H, d = t.shape
    step = H * d
    if not t.is_contiguous():
        sb, st, sh, sd = t.stride()
        if T == 1:
            st = sb   # one token per row: the rows are the tokens
        elif B > 1 and sb != T * st:
            st = 0
        if sd != 1 or (sh != d and H > 1) or st < step or st * t.element_size() % 16 or B * T < 2:
            t = t.contiguous()
        else:
            step = st
    if t.data_ptr() % 16:
        t, step = t.clone(memory_format=torch.contiguous_format), H * d
    return t, step


def _out_tensor(out, like):
    """A dense tensor for a result of `like`'s shape, type and device, or the caller's."""
    if out is None:
        return torch.empty_like(like) if like.is_contiguous() else torch.empty(like.shape, dtype=like.dtype, device=like.device)
    if out.shape != like.shape or out.dtype != like.dtype or out.device != like.device or not out.is_contiguous() \
            or out.data_ptr() % 16:
        raise ValueError(f"out must be a contiguous {like.dtype} tensor of shape {list(like.shape)} on {like.device}")
    return out


# ---- prompts ------------------------------------------------------------------------------------


def _prompt_args(q, k, v, cu, cu_k, causal, scale):
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape:
        raise ValueError("q must be [B, Tq, Hq, d] and k, v [B, Tk, Hkv, d]")
    B, Tq, Hq, d = q.shape
    Bk, Tk, Hkv, dk = k.shape
    if Bk != B or dk != d:
        raise ValueError("k and v must be [B, Tk, Hkv, d] with q's B and d")
    if Hkv == 0 or Hq % Hkv:
        raise ValueError(f"the {Hq} query heads must be a multiple of the {Hkv} heads of k and v")
    if cu is None and cu_k is not None:
        raise ValueError("cu_seqlens_k needs cu_seqlens")
    if cu is not None and cu_k is None and Tk != Tq:
        raise ValueError("packed k and v of another length than q need cu_seqlens_k")
    n = 0
    if cu is not None:
        n = cu.numel() - 1
        cu = _ints(cu, "cu_seqlens", None, q.get_device())
        if cu_k is not None:
            cu_k = _ints(cu_k, "cu_seqlens_k", n + 1, q.get_device())
        if B != 1 or n < 1:
            raise ValueError("cu_seqlens requires B == 1 and at least two offsets")
    dt, dev = _same(q, (k, v))
    (q, qs), (k, ks), (v, vs) = _tokens(q), _tokens(k), _tokens(v)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, _p(cu), _p(cu_k), n, B, Tq, Tk, Hq, Hkv, d,
            1 if causal else 0, d ** -0.5 if scale is None else scale, dt)
    return args, dev, (q, k, v, cu, cu_k)


def kda_attn_fwd(q, k, v, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None, out=None, return_lse=False):
    """Attention over whole prompts: ``softmax(scale q k^T + mask) v``.

    q: [B, Tq, Hq, d]; k, v: [B, Tk, Hkv, d] (bf16 or fp32, d 64 or 128); query head h reads head
    ``h // (Hq // Hkv)``.  cu_seqlens: int32 [N+1] offsets of packed sequences (B == 1), cu_seqlens_k
    those of k and v where they differ.  Causal: query i of a sequence sees keys j <= i + nk - nq; a
    query that sees none gets zeros.  scale: 1 / sqrt(d) by default.  Returns out [B, Tq, Hq, d] in the
    inputs' dtype, with ``return_lse`` also the fp32 [B, Hq, Tq] logarithms of the softmax sums.  Rows
    behind the last packed sequence are not written.
    """
    args, dev, keep = _prompt_args(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale)
    out, lse = _out_tensor(out, q), None
    if return_lse:
        lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=q.device)
    _call("kda_attn_fwd", dev, *args, out.data_ptr(), _p(lse))
    return (out, lse) if return_lse else out


def kda_attn_bwd(q, k, v, out, lse, d_out, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None):
    """Gradient of :func:`kda_attn_fwd`: ``(dq, dk, dv)`` in the inputs' dtype, from the forward's inputs,
    its ``out`` and ``lse``, and ``d_out``.  dk and dv are summed over the query heads that share them.
    Rows behind the last packed sequence get zeros.  The same call gives the same bits."""
    args, dev, keep = _prompt_args(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale)
    B, Tq, Hq, _ = q.shape
    if out.shape != q.shape or d_out.shape != q.shape or lse.shape != (B, Hq, Tq):
        raise ValueError("out and d_out must have q's shape, and lse [B, Hq, Tq]")
    if lse.dtype != torch.float32:
        raise TypeError("lse must be float32")
    if lse.get_device() != dev:
        raise ValueError("lse must be on the device of the other tensors")
    _same(q, (out, d_out))
    out, lse, d_out = _tokens(out.contiguous())[0], lse.contiguous(), _tokens(d_out.contiguous())[0]
    dq, dk, dv = _out_tensor(None, q), _out_tensor(None, k), _out_tensor(None, k)
    ws = torch.empty_like(lse)   # kda_attn_bwd_workspace_size: a float for each row of a head
    _call("kda_attn_bwd", dev, *args, out.data_ptr(), lse.data_ptr(), d_out.data_ptr(), dq.data_ptr(), dk.data_ptr(),
          dv.data_ptr(), ws.data_ptr(), 4 * ws.numel())
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
    """The cache's sizes, the elements between pages and between rows of the page table."""
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [num_pages, Hkv, page_size, d]")
    pages, H, size, d = k_cache.shape
    steps = []
    for c in (k_cache, v_cache):   # the cache is used in place: no copy can stand in for it
        if c.is_contiguous():
            steps.append(H * size * d)
            continue
        sp, sh, ss, sd = c.stride()
        if sd != 1 or (ss != d and size > 1) or (sh != size * d and H > 1):
            raise ValueError("a page of the cache must be dense; pages may lie apart")
        steps.append(sp if pages > 1 else H * size * d)
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != n:
        raise ValueError(f"page_table must be an int32 tensor [{n}, pages of a sequence]")
    if page_table.get_device() != k_cache.get_device():
        raise ValueError("page_table must be on the device of the cache")
    width = page_table.shape[1]
    if not page_table.is_contiguous():
        sr, sc = page_table.stride()
        if sc != 1 or sr < width:
            page_table = page_table.contiguous()
        elif n > 1:
            return pages, H, size, d, steps, page_table, sr, width
    return pages, H, size, d, steps, page_table, width, width


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
    n, cu = B, cu_seqlens
    if cu is not None:
        n = cu.numel() - 1
        if B != 1 or n < 1:
            raise ValueError("cu_seqlens requires B == 1 and at least two offsets")
    pages, H, size, cd, steps, table, row, width = _cache_args(k_cache, v_cache, page_table, n)
    if H != Hkv or cd != d:
        raise ValueError(f"the cache holds {H} heads of {cd} channels, k and v {Hkv} of {d}")
    dt, dev = _same(k, (v, k_cache, v_cache))
    cache_lens = _ints(cache_lens, "cache_lens", n, dev)
    if cu is not None:
        cu = _ints(cu, "cu_seqlens", None, dev)
    rotary = 0
    if inv_freq is not None:
        if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1:
            raise TypeError("inv_freq must be a one-dimensional float32 tensor")
        if inv_freq.get_device() != dev:
            raise ValueError("inv_freq must be on the device of the other tensors")
        inv_freq = inv_freq.contiguous()
        rotary = 2 * inv_freq.shape[0]
    Hq = qs = 0
    qt = qo = ko = None
    (k, ks), (v, vs) = _tokens(k), _tokens(v)
    if q is not None:
        if q.dim() != 4 or q.shape[0] != B or q.shape[1] != T or q.shape[3] != d or Hkv == 0 or q.shape[2] % Hkv:
            raise ValueError("q must be [B, T, Hq, d] with Hq a multiple of Hkv")
        _same(k, (q,))
        Hq = q.shape[2]
        qo = _out_tensor(q_out, q)
        qt, qs = _tokens(q)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if return_k:
        ko = _out_tensor(None, k)
    _call("kda_kv_append", dev, _p(qt), k.data_ptr(), v.data_ptr(), qs, ks, vs, _p(inv_freq), rotary,
          1 if interleaved else 0, _p(cu), n, B, T, Hq, Hkv, d, dt, cache_lens.data_ptr(), table.data_ptr(), row, width,
          k_cache.data_ptr(), v_cache.data_ptr(), steps[0], steps[1], pages, size, _p(qo), _p(ko))
    return qo, ko


@functools.lru_cache(maxsize=None)
def _decode_workspace(dev, B, Hq, Hkv, d, tokens, dt):
    """Bytes that the decode step needs; a function of the sizes and the device's number of SMs."""
    size = ctypes.c_size_t(0)
    with torch.cuda.device(dev):
        _lib.check(_lib.load().kda_attn_decode_workspace_size(B, Hq, Hkv, d, tokens, dt, ctypes.byref(size)),
                   "kda_attn_decode_workspace_size")
    return size.value


def kda_attn_decode_step(q, k_cache, v_cache, page_table, seq_lens, scale=None, out=None, return_lse=False):
    """Attention of one new token per sequence over a paged cache (see :func:`kda_kv_append` for its layout).

    q: [B, Hq, d]; seq_lens: int32 [B], the tokens of each sequence in the cache, the new one among them
    (0 or less: the row's output is zero).  Returns out [B, Hq, d] in q's dtype (``out``, if given,
    receives it), with ``return_lse`` also the fp32 [B, Hq] logarithms of the softmax sums.
    """
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, d]")
    B, Hq, d = q.shape
    pages, Hkv, size, cd, steps, table, row, width = _cache_args(k_cache, v_cache, page_table, B)
    if cd != d or Hkv == 0 or Hq % Hkv:
        raise ValueError(f"q of {Hq} heads of {d} channels does not go with a cache of {Hkv} of {cd}")
    seq_lens = _ints(seq_lens, "seq_lens", B, q.get_device())
    dt, dev = _same(q, (k_cache, v_cache))
    qt, qs = _tokens(q.unsqueeze(1))
    out, lse, ws = _out_tensor(out, q), None, None
    if return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    need = _decode_workspace(dev, B, Hq, Hkv, d, max(width * size, 1), dt)
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    _call("kda_attn_decode_step", dev, qt.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(), steps[0], steps[1],
          pages, size, table.data_ptr(), row, width, seq_lens.data_ptr(), B, Hq, Hkv, d,
          d ** -0.5 if scale is None else scale, dt, out.data_ptr(), _p(lse), _p(ws), need)
    return (out, lse) if return_lse else out
