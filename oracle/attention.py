"""Softmax attention, its gradient, and the paged cache in 64 bits, from the definitions.

Plain torch in float64 on the device of the inputs, one sequence and head at a
time, dense scores, no running maximum.  Beside each result stands a bound on
how far a kernel may be from it that computes in fp32 and rounds the weights
(and the score gradients) once to the inputs' type for the second product, as
the tensor cores need; it counts each rounding at its worst:

  u     half a step of the inputs' type (2^-8 for bf16, 2^-24 for fp32);
  e     2^-24, a rounding of fp32; the tensor cores' sums may truncate, so a
        d-term sum counts 4 d e.
  eta   relative error of a weight P_ij = exp(S_ij - lse_i): the scores' error
        enters twice (once in S_ij, once in lse_i), exp2 and the log cost a few e
        (2^-22 for the SFU's exp2, in the weight and in the sum), the sum over
        n keys n e; the exponent's own rounding is e times its size.
"""
from __future__ import annotations

import math

import torch

E32 = 2.0 ** -24


def _unit(dtype):
    return torch.finfo(dtype).eps / 2


def sequences(q, k, cu, cu_k):
    """(batch row, queries' slice, keys' slice) of every sequence."""
    if cu is None:
        return [(b, slice(0, q.shape[1]), slice(0, k.shape[1])) for b in range(q.shape[0])]
    a = cu.tolist()
    c = a if cu_k is None else cu_k.tolist()
    return [(0, slice(a[i], a[i + 1]), slice(c[i], c[i + 1])) for i in range(len(a) - 1)]


def _weights(q, k, scale, causal):
    """Weights [nq, nk], their relative error bound eta [nq, 1] and lse [nq], of one head in float64."""
    nq, nk, d = q.shape[0], k.shape[0], q.shape[1]
    s = scale * (q @ k.T)
    size = scale * (q.abs() @ k.abs().T)
    if causal:
        i = torch.arange(nq, device=q.device)[:, None]
        j = torch.arange(nk, device=q.device)[None]
        hidden = j > i + nk - nq
        s, size = s.masked_fill(hidden, -math.inf), size.masked_fill(hidden, 0)
    if nk == 0:
        return s, torch.zeros(nq, 1, dtype=q.dtype, device=q.device), torch.full((nq,), -math.inf, dtype=q.dtype,
                                                                                   device=q.device)
    lse = torch.logsumexp(s, 1)
    p = torch.where(torch.isinf(lse)[:, None], torch.zeros_like(s), torch.exp(s - lse[:, None]))
    top = size.amax(1, keepdim=True)
    eta = E32 * (2 * (4 * (d + 4) * top) + 8 * top + 2 * nk + 32)
    return p, eta, lse


def attention(q, k, v, cu=None, cu_k=None, causal=True, scale=None):
    """(out, lse, bound of out, bound of lse); rows behind the last sequence are zero."""
    u = _unit(q.dtype)
    B, Tq, Hq, d = q.shape
    group = Hq // k.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64, device=q.device)
    ltol = torch.zeros_like(lse)
    for b, r, c in sequences(q, k, cu, cu_k):
        for h in range(Hq):
            x, y, z = q[b, r, h].double(), k[b, c, h // group].double(), v[b, c, h // group].double()
            p, eta, ls = _weights(x, y, scale, causal)
            o = p @ z
            mass = p @ z.abs()
            out[b, r, h] = o
            tol[b, r, h] = 1.01 * (u * mass + u * o.abs() + eta * mass) + 1e-30
            lse[b, h, r] = ls
            ltol[b, h, r] = eta[:, 0] + 4 * E32 * ls.abs().nan_to_num(posinf=0.0, neginf=0.0)
    return out, lse, tol, ltol


def attention_grad(q, k, v, d_out, cu=None, cu_k=None, causal=True, scale=None):
    """((dq, dk, dv), their bounds).  The bounds add to eta: out is read as rounded (u of each product in
    delta), dP and delta are sums over d, P and dS are rounded once, and so is each result."""
    u = _unit(q.dtype)
    d, group = q.shape[3], q.shape[2] // k.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    vals = [torch.zeros(t.shape, dtype=torch.float64, device=q.device) for t in (q, k, v)]
    tols = [torch.zeros_like(t) for t in vals]
    for b, r, c in sequences(q, k, cu, cu_k):
        nq, nk = r.stop - r.start, c.stop - c.start
        for h in range(q.shape[2]):
            hk = h // group
            x, y, z, g = q[b, r, h].double(), k[b, c, hk].double(), v[b, c, hk].double(), d_out[b, r, h].double()
            p, eta, _ = _weights(x, y, scale, causal)
            o = p @ z
            delta = (g * o).sum(1, keepdim=True)
            dp = g @ z.T
            ds = p * (dp - delta)
            mass = p @ z.abs()
            # error of dP - delta: sums over d, out's own error times dO
            slack = 4 * (d + 4) * E32 * (g.abs() @ z.abs().T + (g.abs() * o.abs()).sum(1, keepdim=True)) + \
                (g.abs() * (2 * u * mass + eta * mass)).sum(1, keepdim=True)
            ds_tol = (u + 4 * E32) * ds.abs() + eta * ds.abs() + p * slack
            p_tol = (u + eta) * p
            n = 4 * E32
            parts = [(ds @ y * scale, (ds_tol @ y.abs() + n * nk * (ds.abs() @ y.abs())) * scale),
                     (ds.T @ x * scale, (ds_tol.T @ x.abs() + n * nq * group * (ds.abs().T @ x.abs())) * scale),
                     (p.T @ g, p_tol.T @ g.abs() + n * nq * group * (p.T @ g.abs()))]
            for i, (val, tol) in enumerate(parts):
                rows, head = (r, h) if i == 0 else (c, hk)
                vals[i][b, rows, head] += val
                tols[i][b, rows, head] += tol
    tols = [1.01 * (t + u * x.abs()) + 1e-30 for t, x in zip(tols, vals)]
    return vals, tols


def rotate(x, pos, inv_freq, interleaved):
    """x [tokens, heads, d] rotated by its positions, in float64."""
    x = x.double().clone()
    r = 2 * inv_freq.numel()
    angle = pos.double()[:, None, None] * inv_freq.double()
    i = torch.arange(r // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    a, b = x[..., first].clone(), x[..., second].clone()
    x[..., first] = a * angle.cos() - b * angle.sin()
    x[..., second] = b * angle.cos() + a * angle.sin()
    return x


def gather_cache(cache, table, length):
    """The first `length` rows [length, heads, d] of one sequence (its row `table` of the page table)."""
    size = cache.shape[2]
    p = torch.arange(length, device=cache.device)
    return cache[table[p // size].long(), :, p % size]
