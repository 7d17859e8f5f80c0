"""Python binding of the softmax-attention calls of the C ABI (include/kda.h).

As in ``ops``: argument marshalling only.  It lives in the native module
``_attention`` (csrc/attn_binding.cpp), since a decode step takes less time on
the GPU than the same marshalling takes in Python; here are the entry points'
contracts.  All tensors of a call live on one CUDA device; the call runs on that
device's current stream, whichever device is current.  A token tensor whose last
two dimensions are dense and whose tokens lie an even distance apart (a slice
of a fused projection, say) is read where it is; any other layout is copied
first.  Wrong shapes raise ValueError, wrong types TypeError, and a non-OK
status of the library :class:`KdaError`.  Gradients flow through
:func:`kda_attn` alone; the results of the other calls are detached.
"""
from __future__ import annotations

import importlib

_module = None


def _native():
    """The native module.  Raises if it has not been built: there is no fallback."""
    global _module
    if _module is None:
        try:
            import torch  # noqa: F401  (the module links to torch's libraries)
            _module = importlib.import_module("._attention", __package__)
        except ImportError as e:
            raise ImportError(f"{e}; build it with gated_delta_rule_86_b200.build.build_binding()"
                              " (or __graft_entry__.build())") from e
    return _module


# ---- prompts ------------------------------------------------------------------------------------


def kda_attn_fwd(q, k, v, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None, out=None, return_lse=False,
                 return_rest=False):
    """Attention over whole prompts: ``softmax(scale q k^T + mask) v``.

    q: [B, Tq, Hq, d]; k, v: [B, Tk, Hkv, d] (bf16 or fp32, d 64 or 128); query head h reads head
    ``h // (Hq // Hkv)``.  cu_seqlens: int32 [N+1] offsets of packed sequences (B == 1), cu_seqlens_k
    those of k and v where they differ.  Causal: query i of a sequence sees keys j <= i + nk - nq; a
    query that sees none gets zeros.  scale: 1 / sqrt(d) by default.  Returns out [B, Tq, Hq, d] in the
    inputs' dtype, with ``return_lse`` also the fp32 [B, Hq, Tq] logarithms of the softmax sums, with
    ``return_rest`` also what rounding took from a bf16 out (None for fp32), for :func:`kda_attn_bwd`.  Rows
    behind the last packed sequence are not written.  Sequences never mix, whatever they hold; inside one,
    keys and values that the causal mask hides must be finite (a hidden row counts with weight zero, which a
    NaN survives).
    """
    return _native().fwd(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale, out, return_lse, return_rest)


def kda_attn_bwd(q, k, v, out, lse, d_out, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None, out_rest=None):
    """Gradient of :func:`kda_attn_fwd`: ``(dq, dk, dv)`` in the inputs' dtype, from the forward's inputs,
    its ``out`` and ``lse`` (and ``out_rest``: without it bf16 dq errs by up to a fifth more), and ``d_out``.
    dk and dv are summed over the query heads that share them.  Rows behind the last packed sequence get zeros.  The same call gives the same bits."""
    return _native().bwd(q, k, v, out, lse, d_out, cu_seqlens, cu_seqlens_k, causal, scale, out_rest)


def kda_attn(q, k, v, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None):
    """Differentiable attention over whole prompts: :func:`kda_attn_fwd` with gradients for q, k and v
    (through :func:`kda_attn_bwd`).  Rows of the output behind the last packed sequence are not written
    and must not reach the loss.  Differentiable once: a backward pass with ``create_graph=True`` raises, and
    so do inputs with tangents of forward-mode differentiation.
    Under CUDA graph capture it raises while an autograd graph of the same leaves lives on another stream."""
    return _native().attn(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale)


# ---- the paged cache ----------------------------------------------------------------------------


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
    The call has no gradient, and warns where an input requires one.
    """
    return _native().kv_append(k, v, k_cache, v_cache, page_table, cache_lens, inv_freq, q, cu_seqlens, interleaved,
                               return_k, q_out)


def kda_attn_decode_step(q, k_cache, v_cache, page_table, seq_lens, scale=None, out=None, return_lse=False):
    """Attention of one new token per sequence over a paged cache (see :func:`kda_kv_append` for its layout).

    q: [B, Hq, d]; seq_lens: int32 [B], the tokens of each sequence in the cache, the new one among them
    (0 or less: the row's output is zero).  Returns out [B, Hq, d] in q's dtype (``out``, if given,
    receives it), with ``return_lse`` also the fp32 [B, Hq] logarithms of the softmax sums.
    """
    return _native().decode_step(q, k_cache, v_cache, page_table, seq_lens, scale, out, return_lse)
