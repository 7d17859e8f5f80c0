"""Softmax attention beside the linear-attention layers, in plain form and through the package's entry points.

Hybrid models put full-attention layers between KDA layers.  Three operators serve those: appending rotated keys and
values to a paged cache, attention of one new token over that cache, and attention over whole prompts with its gradient.

The cache is ``[pages, heads, page_size, d]``; sequence n's token at position p lives in page
``page_table[n, p // page_size]``, slot ``p % page_size``.  Token tensors are ``[B, T, heads, d]``; packed sequences
have B = 1 and offsets ``cu_seqlens``.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one user's next token: the cost of a call
        dict(name="append-one-token", op="append", dtype="bf16", n=1, lo=1, hi=1, past_lo=700, past_hi=700, lens_seed=1,
             hq=16, hkv=4, d=64, page=16, rotary=64, interleaved=False, return_k=False),
        # a decode step of a full serving batch, sequences of all ages
        dict(name="append-step-256", op="append", dtype="bf16", n=256, lo=1, hi=1, past_lo=16, past_hi=16384, lens_seed=2,
             hq=32, hkv=8, d=128, page=64, rotary=128, interleaved=False, return_k=False),
        # a packed batch of new prompts, long ones among them; the rotated keys also go to the prompt attention
        dict(name="append-prompts", op="append", dtype="bf16", n=8, lo=1024, hi=16384, past_lo=0, past_hi=0, lens_seed=3,
             hq=32, hkv=8, d=128, page=64, rotary=128, interleaved=False, return_k=True),
        # one user, short context: latency
        dict(name="decode-one-short", op="decode", dtype="bf16", n=1, lo=333, hi=333, lens_seed=4, hq=16, hkv=4, d=128, page=16),
        # a serving batch of ragged contexts
        dict(name="decode-64-ragged", op="decode", dtype="bf16", n=64, lo=64, hi=16384, lens_seed=5, hq=32, hkv=8, d=128, page=64),
        # one user, very long context: the split over the length
        dict(name="decode-one-long", op="decode", dtype="bf16", n=1, lo=131071, hi=131071, lens_seed=6, hq=32, hkv=8, d=128, page=64),
        # a short question
        dict(name="prompt-short", op="prompt", dtype="bf16", n=1, lo=200, hi=200, past_lo=0, past_hi=0, lens_seed=7, hq=16, hkv=4, d=128, causal=True),
        # a packed batch of ragged prompts, narrow heads
        dict(name="prompt-packed", op="prompt", dtype="bf16", n=8, lo=64, hi=4096, past_lo=0, past_hi=0, lens_seed=8, hq=32, hkv=8, d=64, causal=True),
        # one long document
        dict(name="prompt-long", op="prompt", dtype="bf16", n=1, lo=16384, hi=16384, past_lo=0, past_hi=0, lens_seed=9, hq=32, hkv=8, d=128, causal=True),
        # a small single-precision training step, as in gradient checks
        dict(name="train-tiny-fp32", op="train", dtype="fp32", n=1, lo=256, hi=256, past_lo=0, past_hi=0, lens_seed=10, hq=2, hkv=2, d=64, causal=True),
        # a packed training batch of ragged documents with shared heads
        dict(name="train-packed", op="train", dtype="bf16", n=6, lo=200, hi=4096, past_lo=0, past_hi=0, lens_seed=11, hq=16, hkv=4, d=64, causal=True),
        # an ordinary training batch
        dict(name="train-4096", op="train", dtype="bf16", n=2, lo=4096, hi=4096, past_lo=0, past_hi=0, lens_seed=12, hq=16, hkv=16, d=128, causal=True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prompt", "train"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 6, 8, 16) if hkv * g <= 32])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]), lens_seed=rng.randrange(1 << 30), hq=hq, hkv=hkv, d=d)
    wide = case["dtype"] == "fp32"
    if op == "append":
        n = _log_uniform(rng, 1, 256)
        steps = rng.random() < 0.5
        most = 1 if steps else max(2, min(8192, 32768 // n))
        past = rng.choice([0, _log_uniform(rng, 1, 16384)])
        case.update(n=n, lo=1, hi=most, past_lo=0, past_hi=past, page=rng.choice([16, 32, 64, 128]),
                    rotary=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3, return_k=not steps)
    elif op == "decode":
        n = _log_uniform(rng, 1, 256)
        most = _log_uniform(rng, 32, max(64, min(131072, (131072 if wide else 262144) // n)))
        case.update(n=n, lo=_log_uniform(rng, 1, most), hi=most, page=rng.choice([16, 32, 64, 128]))
    else:
        most = _log_uniform(rng, 8, 1024 if wide else 8192 if op == "prompt" else 4096)
        n = _log_uniform(rng, 1, max(1, min(16, (2048 if wide else 16384) // most)))
        past = rng.choice([0, 0, rng.randint(0, most)])
        case.update(n=n, lo=_log_uniform(rng, 1, most), hi=most, past_lo=0, past_hi=past, causal=rng.random() < 0.8)
        while work(case)["flops"] > 1e12:
            case.update(lo=min(case["lo"], case["hi"] // 2), hi=case["hi"] // 2)
    return case


def _lens(case, lo, hi, salt):
    """The sequences' lengths: log-uniform over [lo, hi], by the case alone."""
    rng = random.Random(case["lens_seed"] * 7 + salt)
    return [lo if hi <= lo else max(lo, _log_uniform(rng, max(lo, 1), hi) if lo else rng.randint(lo, hi)) for _ in range(case["n"])]


def _sizes(case):
    new = _lens(case, case["lo"], case["hi"], 0)
    past = _lens(case, case["past_lo"], case["past_hi"], 1) if "past_lo" in case else [0] * case["n"]
    return new, past


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _pages(lens, page, rng, device):
    """A page table for these lengths whose pages lie in any order in a pool with some to spare; -1 where there is none."""
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(need) + 3, generator=rng, device=device)[: sum(need)].to(torch.int32)
    width = max(max(need), 1)
    col = torch.arange(width, device=device)
    counts = torch.tensor(need, device=device)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=device)
    table[col[None] < counts[:, None]] = ids
    return table, sum(need) + 3


def prepare(case, seed):
    dev = torch.device("cuda")
    rng = torch.Generator(device=dev).manual_seed(int(seed) * 1000003 + case["lens_seed"] % 1000)
    dtype, hq, hkv, d = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["d"]
    new, past = _sizes(case)

    def normal(*shape):
        return torch.randn(shape, generator=rng, device=dev, dtype=torch.float32).to(dtype) if math.prod(shape) < 1 << 28 \
            else torch.randn(shape, generator=rng, device=dev, dtype=dtype)

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    state = dict(case=case, new=new, past=past)
    if case["op"] in ("append", "decode"):
        lens = [a + b for a, b in zip(new, past)]
        state["table"], pages = _pages(lens, case["page"], rng, dev)
        state["kc"], state["vc"] = normal(pages, hkv, case["page"], d), normal(pages, hkv, case["page"], d)
    if case["op"] == "decode":
        state.update(q=normal(case["n"], hq, d), lens=whole(new))
        return state
    step = case["op"] == "append" and max(new) == 1
    packed = case["n"] > 1 and not step and (min(new) != max(new) or min(past) != max(past))
    lead = (case["n"], 1) if step else (1, sum(new)) if packed else (case["n"], new[0])
    keys = lead if case["op"] == "append" else (1, sum(new) + sum(past)) if packed else (case["n"], new[0] + past[0])
    state.update(q=normal(*lead, hq, d), k=normal(*keys, hkv, d), v=normal(*keys, hkv, d))
    state["cu"] = whole(_offsets(new)) if packed else None
    if case["op"] == "append":
        state["cache_lens"] = whole(past)
        r = case["rotary"]
        state["inv_freq"] = (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().to(dev)
    else:
        state["cu_k"] = whole(_offsets([a + b for a, b in zip(new, past)])) if packed and max(past) else None
        if case["op"] == "train":
            state["dout"] = normal(*lead, hq, d)
            for name in ("q", "k", "v"):
                state[name].requires_grad_()
    return state


# ---- plain forms --------------------------------------------------------------------------------


def _rotate(x, angle, interleaved):
    """x [tokens, heads, d] with its first 2 * angle.shape[1] channels rotated in pairs by angle [tokens, pairs]."""
    r = 2 * angle.shape[1]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., : r // 2], x[..., r // 2: r])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _append_plain(s):
    c = s["case"]
    q, k, v = (s[n].flatten(0, 1) for n in ("q", "k", "v"))
    tokens = torch.arange(k.shape[0], device=k.device)
    if s["cu"] is None:
        seq, j = tokens // s["k"].shape[1], tokens % s["k"].shape[1]
    else:
        seq = torch.searchsorted(s["cu"], tokens, right=True) - 1
        j = tokens - s["cu"][seq]
    pos = s["cache_lens"][seq] + j
    angle = pos.double()[:, None] * s["inv_freq"].double()   # far positions need the bits
    qr = _rotate(q, angle, c["interleaved"]).to(q.dtype).view_as(s["q"])
    kr = _rotate(k, angle, c["interleaved"]).to(k.dtype)
    page, slot = s["table"][seq, pos // c["page"]], pos % c["page"]
    s["kc"][page, :, slot] = kr
    s["vc"][page, :, slot] = v
    return [qr, s["kc"], s["vc"]] + ([kr.view_as(s["k"])] if c["return_k"] else [])


def _softmax_rows(x, seen):
    """Softmax over the last axis of the entries that are seen; zeros where a row sees none."""
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(x.dtype).min)
    p = (x - m).exp()
    total = p.sum(-1, keepdim=True)
    return p / total.clamp(min=torch.finfo(x.dtype).tiny)


def _decode_plain(s):
    c, q, table = s["case"], s["q"], s["table"]
    pos = torch.arange(table.shape[1] * c["page"], device=q.device)
    seen = pos < s["lens"][:, None]
    page = table[:, pos // c["page"]].clamp(min=0)
    k, v = (x[page, :, pos % c["page"]].float() for x in (s["kc"], s["vc"]))      # [n, tokens, hkv, d]
    qg = q.float().view(q.shape[0], c["hkv"], -1, c["d"])
    p = _softmax_rows(torch.einsum("bhgd,bnhd->bhgn", qg, k) / math.sqrt(c["d"]), seen[:, None, None])
    return torch.einsum("bhgn,bnhd->bhgd", p, v).reshape(q.shape).to(q.dtype)


def _sequences(s):
    """(row of the batch, queries' slice, keys' slice) of every sequence."""
    new, past = s["new"], s["past"]
    both = [a + b for a, b in zip(new, past)]
    if s["cu"] is None:
        return [(i, slice(0, a), slice(0, b)) for i, (a, b) in enumerate(zip(new, both))]
    at, kat = _offsets(new), _offsets(both)
    return [(0, slice(at[i], at[i + 1]), slice(kat[i], kat[i + 1])) for i in range(len(new))]


def _seen(nq, nk, causal, device):
    rows, cols = torch.arange(nq, device=device)[:, None], torch.arange(nk, device=device)
    return cols <= rows + (nk - nq) if causal else cols >= 0 * rows


def _prompt_plain(s, dout=None):
    c = s["case"]
    q, k, v = (s[n].detach() for n in ("q", "k", "v"))
    out = torch.empty_like(q)
    grads = [torch.empty_like(x) for x in (q, k, v)] if dout is not None else []
    group, scale = c["hq"] // c["hkv"], 1 / math.sqrt(c["d"])
    for b, rows, cols in _sequences(s):
        seen = _seen(rows.stop - rows.start, cols.stop - cols.start, c["causal"], q.device)
        for h in range(c["hkv"]):   # one head's scores at a time: a long prompt's do not fit together
            heads = slice(h * group, (h + 1) * group)
            qh = q[b, rows, heads].float().transpose(0, 1)
            kh, vh = k[b, cols, h].float(), v[b, cols, h].float()
            p = _softmax_rows(qh @ kh.T * scale, seen)
            oh = p @ vh
            out[b, rows, heads] = oh.transpose(0, 1).to(out.dtype)
            if dout is not None:
                gh = dout[b, rows, heads].float().transpose(0, 1)
                ds = p * (gh @ vh.T - (gh * oh).sum(-1, keepdim=True)) * scale
                grads[0][b, rows, heads] = (ds @ kh).transpose(0, 1).to(q.dtype)
                grads[1][b, cols, h] = (ds.transpose(1, 2) @ qh).sum(0).to(k.dtype)
                grads[2][b, cols, h] = (p.transpose(1, 2) @ gh).sum(0).to(v.dtype)
    return [out] + grads if dout is not None else out


def run(state):
    c, op = state["case"], state["case"]["op"]
    if own:
        import gated_delta_rule_86_b200 as kda
        if op == "append":
            qr, kr = kda.kda_kv_append(state["k"], state["v"], state["kc"], state["vc"], state["table"], state["cache_lens"],
                                       inv_freq=state["inv_freq"], q=state["q"], cu_seqlens=state["cu"],
                                       interleaved=c["interleaved"], return_k=c["return_k"])
            return [qr, state["kc"], state["vc"]] + ([kr] if c["return_k"] else [])
        if op == "decode":
            return kda.kda_attn_decode_step(state["q"], state["kc"], state["vc"], state["table"], state["lens"])
        if op == "prompt":
            return kda.kda_attn_fwd(state["q"], state["k"], state["v"], cu_seqlens=state["cu"], cu_seqlens_k=state["cu_k"],
                                    causal=c["causal"])
        leaves = (state["q"], state["k"], state["v"])
        out = kda.kda_attn(*leaves, cu_seqlens=state["cu"], cu_seqlens_k=state["cu_k"], causal=c["causal"])
        return [out, *torch.autograd.grad(out, leaves, state["dout"])]
    if op == "append":
        return _append_plain(state)
    if op == "decode":
        return _decode_plain(state)
    return _prompt_plain(state, state.get("dout"))


def _visible(case):
    """Pairs of a query and a key that it sees, over all sequences."""
    new, past = _sizes(case)
    return sum(n * (n + 1) // 2 + n * p if case["causal"] else n * (n + p) for n, p in zip(new, past))


def work(case):
    new, past = _sizes(case)
    size = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    tokens, keys = sum(new), sum(new) + sum(past)
    if case["op"] == "append":   # q, k, v in; q, the cache's k and v, and k again where it is asked for, out
        moved = tokens * d * size * (2 * hq + (5 if case["return_k"] else 4) * hkv)
        return {"bytes": moved, "flops": 3 * tokens * case["rotary"] * (hq + hkv)}
    if case["op"] == "decode":
        return {"bytes": size * d * (2 * tokens * hkv + 2 * case["n"] * hq), "flops": 4 * tokens * hq * d}
    forward = size * d * (2 * tokens * hq + 2 * keys * hkv), 4 * _visible(case) * hq * d
    if case["op"] == "prompt":
        return {"bytes": forward[0], "flops": forward[1]}
    # the gradient adds: its own five products with the scores computed again; dout in, dq, dk and dv out
    return {"bytes": forward[0] + size * d * (2 * tokens * hq + 2 * keys * hkv), "flops": forward[1] * 3.5}


# ---- the definition in 64 bits ------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    wide = {n: s[n].detach().double() for n in ("q", "k", "v", "kc", "vc", "dout") if n in s}
    new, past = s["new"], s["past"]
    if case["op"] == "append":
        freq = s["inv_freq"].double()
        pos = torch.cat([torch.arange(p, p + n, device="cuda", dtype=torch.float64) for n, p in zip(new, past)])
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, None] * freq)[:, None]

        def rotated(x):   # pairs as complex numbers times e^(i angle)
            x, r = x.flatten(0, 1).clone(), case["rotary"]
            pairs = x[..., :r].unflatten(-1, (-1, 2)) if case["interleaved"] else x[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)
            turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            x[..., :r] = (turned if case["interleaved"] else turned.transpose(-1, -2)).flatten(-2)
            return x

        qr, kr, v = rotated(wide["q"]), rotated(wide["k"]), wide["v"].flatten(0, 1)
        table, at = s["table"].tolist(), 0
        for n, (a, p) in enumerate(zip(new, past)):
            while a:   # up to the end of a page at a time
                page, slot = table[n][p // case["page"]], p % case["page"]
                m = min(a, case["page"] - slot)
                wide["kc"][page, :, slot: slot + m] = kr[at: at + m].transpose(0, 1)
                wide["vc"][page, :, slot: slot + m] = v[at: at + m].transpose(0, 1)
                at, p, a = at + m, p + m, a - m
        return [qr.view(s["q"].shape), wide["kc"], wide["vc"]] + ([kr.view(s["k"].shape)] if case["return_k"] else [])
    if case["op"] == "decode":
        out = torch.zeros_like(wide["q"])
        for n, length in enumerate(new):
            pages = s["table"][n, : -(-length // case["page"])].long()
            k, v = (wide[x][pages].transpose(0, 1).reshape(hkv, -1, d)[:, :length] for x in ("kc", "vc"))
            w = torch.softmax(wide["q"][n].view(hkv, hq // hkv, d) @ k.transpose(1, 2) * d ** -0.5, -1)
            out[n] = (w @ v).view(hq, d)
        return out
    training = case["op"] == "train"
    results = [torch.zeros_like(wide[n]) for n in ("q", "q", "k", "v")][: 4 if training else 1]
    for b, rows, cols in _sequences(s):
        nq, nk = rows.stop - rows.start, cols.stop - cols.start
        hidden = torch.ones(nq, nk, dtype=torch.bool, device="cuda").triu(nk - nq + 1) if case["causal"] else None
        for h in range(hq):
            g = h // (hq // hkv)
            q, k, v = wide["q"][b, rows, h], wide["k"][b, cols, g], wide["v"][b, cols, g]
            if training:
                q, k, v = (x.detach().requires_grad_() for x in (q, k, v))
            x = q @ k.T * d ** -0.5
            if hidden is not None:
                x = x.masked_fill(hidden, -math.inf)
            o = torch.softmax(x, -1) @ v
            results[0][b, rows, h] = o.detach()
            if training:
                dq, dk, dv = torch.autograd.grad(o, (q, k, v), wide["dout"][b, rows, h])
                results[1][b, rows, h] = dq
                results[2][b, cols, g] += dk
                results[3][b, cols, g] += dv
    return results if training else results[0]
