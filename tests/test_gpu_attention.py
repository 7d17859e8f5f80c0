"""Softmax attention on the GPU: prompts and their gradient, the paged cache's append and decode step,
each against the definitions in 64 bits (oracle/attention.py) within bounds that count every rounding."""
import math
import threading

import pytest
import torch

import gated_delta_rule_86_b200 as kda
from oracle import attention as ref

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _library(cuda_lib):
    yield
    torch.cuda.synchronize()
    kda.device_error()   # one test's report does not reach the next


def make(shape, seed, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def inside(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - want).abs() / tol).max().item() if got.numel() else 0.0
    assert over <= 1, f"{what}: {over:.3g} times its bound"


def check_lse(got, want, tol):
    dead = torch.isinf(want)
    assert torch.equal(torch.isinf(got), dead) and not torch.isnan(got).any()
    inside(torch.where(dead, 0, got.double()), torch.where(dead, 0, want), tol + 1e-30, "lse")


# ---- prompts ------------------------------------------------------------------------------------

# (lengths of the queries, of the keys or None, packed); tiles are 64 to 256 rows high
LENGTHS = {
    "one": ([1], None, False),
    "two-rows": ([65, 65], None, False),
    "tile-edge": ([128], None, False),
    "past-tile": ([257], None, False),
    "odd": ([333], None, False),
    "packed": ([1, 0, 130, 7, 256, 61], None, True),
    "longer-keys": ([5, 130], [200, 130], True),
    "fewer-keys": ([140, 9, 3], [100, 0, 300], True),
    "dense-longer-keys": ([70], [200], False),
    "dense-fewer-keys": ([200], [70], False),
    "long": ([700], None, False),
}


def prompt(name, hq, hkv, d, dtype, seed=0, std=1.0):
    nq, nk, packed = LENGTHS[name]
    nk = nq if nk is None else nk
    if packed:
        lead_q, lead_k = (1, sum(nq)), (1, sum(nk))
        cu, cu_k = offsets(nq), (None if nk is nq else offsets(nk))
    else:
        lead_q, lead_k, cu, cu_k = (len(nq), nq[0]), (len(nk), nk[0]), None, None
    q = make((*lead_q, hq, d), seed + 1, dtype, std)
    k, v = (make((*lead_k, hkv, d), seed + i, dtype, std) for i in (2, 3))
    return q, k, v, cu, cu_k


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", sorted(LENGTHS))
def test_prompt(name, causal, d, dtype):
    q, k, v, cu, cu_k = prompt(name, 4, 2, d, dtype)
    out, lse = kda.kda_attn_fwd(q, k, v, cu, cu_k, causal, return_lse=True)
    o, l, tol, ltol = ref.attention(q, k, v, cu, cu_k, causal)
    inside(out, o, tol, "out")
    check_lse(lse, l, ltol)
    assert out.dtype == dtype and kda.device_error() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (6, 2), (16, 1), (5, 5)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prompt_groups_and_scale(hq, hkv, dtype):
    q, k, v, _, _ = prompt("odd", hq, hkv, 64, dtype, seed=9)
    out = kda.kda_attn_fwd(q, k, v, scale=0.3)
    o, _, tol, _ = ref.attention(q, k, v, scale=0.3)
    inside(out, o, tol, "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", sorted(LENGTHS))
def test_prompt_gradient(name, causal, d, dtype):
    q, k, v, cu, cu_k = prompt(name, 4, 2, d, dtype, seed=20)
    g = make(q.shape, 25, dtype)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    out = kda.kda_attn(*leaves, cu, cu_k, causal)
    got = torch.autograd.grad(out, leaves, g)
    want, tols = ref.attention_grad(q.detach(), k.detach(), v.detach(), g, cu, cu_k, causal)
    for x, y, t, n in zip(got, want, tols, ("dq", "dk", "dv")):
        assert x.dtype == dtype
        inside(x, y, t, n)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 2), (12, 1)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prompt_gradient_groups(hq, hkv, dtype):
    q, k, v, cu, cu_k = prompt("packed", hq, hkv, 128, dtype, seed=40)
    g = make(q.shape, 45, dtype)
    out, lse = kda.kda_attn_fwd(q, k, v, cu, return_lse=True, scale=0.2)
    got = kda.kda_attn_bwd(q, k, v, out, lse, g, cu, scale=0.2)
    want, tols = ref.attention_grad(q, k, v, g, cu, scale=0.2)
    for x, y, t, n in zip(got, want, tols, ("dq", "dk", "dv")):
        inside(x, y, t, n)


@pytest.mark.parametrize("tq,tk,hq,hkv", [(640, 640, 16, 2), (70, 9500, 1, 1), (300, 40, 3, 1), (40, 300, 2, 2)])
def test_prompt_gradient_fp32_blocks(tq, tk, hq, hkv):
    """Queries and keys that differ in the rows of a block, and both small in one launch."""
    q, k, v, g = (make((1, t, h, 64), 130 + i, FP32) for i, (t, h) in enumerate(((tq, hq), (tk, hkv), (tk, hkv), (tq, hq))))
    for causal in (True, False):
        out, lse = kda.kda_attn_fwd(q, k, v, causal=causal, return_lse=True)
        got = kda.kda_attn_bwd(q, k, v, out, lse, g, causal=causal)
        want, tols = ref.attention_grad(q, k, v, g, causal=causal)
        for x, y, t, n in zip(got, want, tols, ("dq", "dk", "dv")):
            inside(x, y, t, n)
        assert all(torch.equal(a, b) for a, b in zip(got, kda.kda_attn_bwd(q, k, v, out, lse, g, causal=causal)))


def test_prompt_gradient_against_differences():
    """The derivative of a weighted sum of the library's own fp32 outputs along a random direction, by
    central differences: the truncation is of order h^2, the outputs' rounding e / h."""
    q, k, v, cu, _ = prompt("packed", 4, 2, 64, FP32, seed=60, std=0.5)
    g = make(q.shape, 65, FP32)
    dirs = [make(t.shape, 66 + i, FP32) for i, t in enumerate((q, k, v))]
    leaves = [t.requires_grad_() for t in (q, k, v)]
    grads = torch.autograd.grad(kda.kda_attn(*leaves, cu), leaves, g)
    h = 2.0 ** -8
    with torch.no_grad():
        ends = [(kda.kda_attn_fwd(*(t + s * h * x for t, x in zip(leaves, dirs)), cu).double() * g.double()).sum()
                for s in (1, -1)]
    slope = ((ends[0] - ends[1]) / (2 * h)).item()
    want = sum((a.double() * b.double()).sum().item() for a, b in zip(grads, dirs))
    size = math.sqrt(sum((a.double() * b.double()).square().sum().item() for a, b in zip(grads, dirs)))
    # h^2 times the third derivative (of order 1 along a unit-variance direction) and e / h per output
    assert abs(slope - want) <= size * (64 * h * h + 2.0 ** -24 / h * 64)


def test_gradient_with_the_rest_of_out():
    """What rounding took from out: together they are the output to 2^-17 beside the weights' rounding, and
    the gradient through autograd, which passes it on, is nearer to the formula's."""
    q, k, v, cu, _ = prompt("packed", 4, 2, 128, BF16, seed=68)
    g = make(q.shape, 69, BF16)
    out, lse, rest = kda.kda_attn_fwd(q, k, v, cu, return_lse=True, return_rest=True)
    o, _, tol, _ = ref.attention(q, k, v, cu)
    inside(out.double() + rest.double(), o, tol, "out and rest")
    assert (rest.double().abs() <= 2.0 ** -8 * out.double().abs() + 1e-38).all()
    plain = kda.kda_attn_bwd(q, k, v, out, lse, g, cu)
    better = kda.kda_attn_bwd(q, k, v, out, lse, g, cu, out_rest=rest)
    leaves = [t.detach().requires_grad_() for t in (q, k, v)]
    auto = torch.autograd.grad(kda.kda_attn(*leaves, cu), leaves, g)
    want, _ = ref.attention_grad(q, k, v, g, cu)
    for a, b, c, w in zip(plain, better, auto, want):
        assert torch.equal(b, c)
        assert (b.double() - w).norm() <= (a.double() - w).norm()
    assert kda.kda_attn_fwd(q.float(), k.float(), v.float(), cu, return_rest=True)[1] is None


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prompt_reads_slices_of_a_projection(dtype):
    B, T, hq, hkv, d = 2, 150, 4, 2, 64
    qkv = make((B, T, (hq + 2 * hkv) * d), 70, dtype)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split((hq * d, hkv * d, hkv * d), -1))
    assert not q.is_contiguous()
    out = kda.kda_attn_fwd(q, k, v)
    assert torch.equal(out, kda.kda_attn_fwd(q.contiguous(), k.contiguous(), v.contiguous()))
    # heads before tokens: no stride of the kernels', so it is copied
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(out, kda.kda_attn_fwd(qt, k, v))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_neighbours_never_mix(dtype, d):
    """Sequences whose neighbours hold NaN and infinities, and rows behind the last one."""
    lens = [70, 130, 33]
    tail = 40
    q, k, v = (make((1, sum(lens) + tail, h, d), 80 + i, dtype) for i, h in enumerate((4, 2, 2)))
    g = make(q.shape, 84, dtype)
    for t in (q, k, v, g):
        t[:, 70:200] = float("nan")
        t[:, 233:] = float("inf")
    cu = offsets(lens)
    out = torch.full_like(q, 7.0)
    out_, lse = kda.kda_attn_fwd(q, k, v, cu, out=out, return_lse=True)
    assert out_ is out and (out[:, 233:] == 7.0).all()
    dq, dk, dv = kda.kda_attn_bwd(q, k, v, out, lse, g, cu)
    for a, b in ((0, 70), (200, 233)):
        x = [t[:, a:b].contiguous() for t in (q, k, v, g)]
        o, l = kda.kda_attn_fwd(*x[:3], return_lse=True)
        inside(o, *(ref.attention(*x[:3])[i] for i in (0, 2)), "alone")
        assert torch.equal(o, out[:, a:b])
        for full, part in zip((dq, dk, dv), kda.kda_attn_bwd(*x[:3], o, l, x[3])):
            assert torch.equal(full[:, a:b], part)
    for t in (dq, dk, dv):
        assert (t[:, 233:] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_outputs_on_sixteen_bytes(dtype):
    """Outputs and inputs that lie on 16 bytes and no more."""
    off = 128 // torch.finfo(dtype).bits
    q, k, v, _, _ = prompt("two-rows", 4, 4, 64, dtype, seed=87)
    want = kda.kda_attn_fwd(q, k, v)
    shifted = []
    for t in (q, k, v):
        b = torch.empty(t.numel() + off, dtype=dtype, device="cuda")[off:].view(t.shape)
        shifted.append(b.copy_(t))
    out = torch.empty(q.numel() + off, dtype=dtype, device="cuda")[off:].view(q.shape)
    assert out.data_ptr() % 32 == 16
    assert torch.equal(kda.kda_attn_fwd(*shifted, out=out), want)
    kc, vc, table = cache_of([30, 41], 4, 64, 16, dtype, 88)
    seq = torch.tensor([30, 41], dtype=torch.int32, device="cuda")
    step = kda.kda_attn_decode_step(q[:, 0], kc, vc, table, seq)
    o = torch.empty(step.numel() + off, dtype=dtype, device="cuda")[off:].view(step.shape)
    assert torch.equal(kda.kda_attn_decode_step(shifted[0][:, 0], kc, vc, table, seq, out=o), step)


def test_prompt_large_scores():
    """Scores of hundreds: a running maximum that grows tile by tile, and weights that all but vanish."""
    q, k, v, _, _ = prompt("long", 2, 1, 128, BF16, seed=90)
    k = k * torch.linspace(1, 30, k.shape[1], device="cuda").to(BF16)[None, :, None, None]
    out = kda.kda_attn_fwd(q, k, v)
    o, _, tol, _ = ref.attention(q, k, v)
    inside(out, o, tol, "out")


def test_prompt_same_call_same_bits():
    q, k, v, cu, _ = prompt("packed", 6, 2, 128, BF16, seed=95)
    g = make(q.shape, 99, BF16)
    runs = []
    for _ in range(3):
        out, lse = kda.kda_attn_fwd(q, k, v, cu, return_lse=True)
        runs.append((out, lse, *kda.kda_attn_bwd(q, k, v, out, lse, g, cu)))
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_prompt_many_sequences():
    lens = [(7 * i) % 23 for i in range(700)]
    q, k, v = (make((1, sum(lens), 2, 64), 100 + i, BF16) for i in range(3))
    cu = offsets(lens)
    out = kda.kda_attn_fwd(q, k, v, cu)
    o, _, tol, _ = ref.attention(q, k, v, cu)
    inside(out, o, tol, "out")


def test_prompt_without_tokens():
    q = torch.empty(1, 0, 2, 64, dtype=BF16, device="cuda")
    assert kda.kda_attn_fwd(q, q, q).shape == q.shape
    k = make((1, 5, 2, 64), 1, BF16)
    out, lse = kda.kda_attn_fwd(q, k, k, return_lse=True)
    dq, dk, dv = kda.kda_attn_bwd(q, k, k, out, lse, q)
    assert dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()
    out, lse = kda.kda_attn_fwd(k, q, q, return_lse=True)
    assert (out == 0).all() and torch.isinf(lse).all()
    assert (kda.kda_attn_bwd(k, q, q, out, lse, k)[0] == 0).all()


# ---- the paged cache ----------------------------------------------------------------------------


def cache_of(lens, hkv, d, size, dtype, seed, spare=2, fill=None):
    """A pool whose pages are handed out in a random order; unused entries of the table are -1."""
    need = [-(-max(n, 0) // size) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    for n, c in enumerate(need):
        for j in range(c):
            table[n, j] = order.pop()
    kc, vc = (make((pages, hkv, size, d), seed + i, dtype) for i in (1, 2))
    if fill is not None:
        for n, length in enumerate(lens):   # what lies behind a sequence's end on its last page
            for p in range(max(length, 0), need[n] * size):
                kc[table[n, p // size], :, p % size] = fill
                vc[table[n, p // size], :, p % size] = fill
        kc[order] = fill
        vc[order] = fill
    return kc, vc, table.cuda()


def decode_ref(q, kc, vc, table, lens, scale=None):
    outs = [ref.attention(q[n:n + 1, None], *(ref.gather_cache(c, table[n], max(length, 0))[None] for c in (kc, vc)),
                          causal=False, scale=scale) for n, length in enumerate(lens)]
    return [torch.cat([x[i] for x in outs]) for i in range(4)]


def check_decode(q, kc, vc, table, lens, scale=None):
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = kda.kda_attn_decode_step(q, kc, vc, table, seq, scale=scale, return_lse=True)
    o, l, tol, ltol = decode_ref(q, kc, vc, table, lens, scale)
    inside(out, o[:, 0], tol[:, 0], "out")
    check_lse(lse, l[..., 0], ltol[..., 0])
    return out


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1, 16, 64, 128])
def test_decode(size, d, dtype):
    lens = [1, 0, 17, 64, 65, 700, 63, -3, 128]
    kc, vc, table = cache_of(lens, 2, d, size, dtype, 200, fill=float("nan"))
    check_decode(make((len(lens), 8, d), 210, dtype), kc, vc, table, lens)
    assert kda.device_error() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (5, 1), (8, 1), (12, 2), (16, 1), (20, 1), (32, 8)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_groups(hq, hkv, dtype):
    lens = [300, 41]
    kc, vc, table = cache_of(lens, hkv, 128, 32, dtype, 220)
    check_decode(make((2, hq, 128), 221, dtype), kc, vc, table, lens, scale=0.11)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_one_long_sequence(dtype):
    lens = [40001]
    kc, vc, table = cache_of(lens, 2, 64, 64, dtype, 230)
    check_decode(make((1, 4, 64), 231, dtype), kc, vc, table, lens)


@pytest.mark.parametrize("n", [300, 1100])
def test_decode_many_sequences(n):
    lens = [(37 * i) % 211 for i in range(n)]
    kc, vc, table = cache_of(lens, 1, 64, 16, BF16, 240)
    q = make((n, 3, 64), 241, BF16)
    out = check_decode(q, kc, vc, table, lens)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert torch.equal(out, kda.kda_attn_decode_step(q, kc, vc, table, seq))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_shared_pages(dtype):
    """Sequences with a prefix in common name its pages twice."""
    lens = [200, 170, 129, 128, 64]
    kc, vc, table = cache_of(lens, 2, 64, 64, dtype, 250, fill=float("nan"))
    for n, shared in ((1, 2), (2, 2), (3, 2), (4, 1)):
        table[n, :shared] = table[0, :shared]
    check_decode(make((len(lens), 4, 64), 251, dtype), kc, vc, table, lens)


def test_decode_reads_one_pool_and_strided_queries():
    """Keys and values interleaved page by page in one tensor, queries a slice of a projection."""
    lens = [90, 200]
    kc, vc, table = cache_of(lens, 2, 128, 32, BF16, 250)
    pool = torch.stack((kc, vc), 1)
    q = make((2, 12, 128), 251, BF16)[:, 3:11]
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = kda.kda_attn_decode_step(q.contiguous(), kc, vc, table, seq)
    assert torch.equal(kda.kda_attn_decode_step(q, pool[:, 0], pool[:, 1], table, seq), want)
    wide = torch.cat((table, table), 1)[:, : table.shape[1]]
    assert torch.equal(kda.kda_attn_decode_step(q, pool[:, 0], pool[:, 1], wide, seq), want)


def test_decode_bad_pages_are_left_out():
    lens = [100, 70]
    kc, vc, table = cache_of(lens, 1, 64, 16, BF16, 260)
    q = make((2, 4, 64), 261, BF16)
    broken = table.clone()
    broken[0, 2], broken[0, 4], broken[1, 0] = -1, kc.shape[0], 2 ** 31 - 1
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = kda.kda_attn_decode_step(q, kc, vc, broken, seq)
    assert kda.device_error() == 5
    for n, gone in enumerate(([2, 4], [0])):
        keep = [p for p in range(lens[n]) if p // 16 not in gone]
        k, v = (ref.gather_cache(c, table[n], lens[n])[keep][None] for c in (kc, vc))
        o, _, tol, _ = ref.attention(q[n:n + 1, None], k, v, causal=False)
        inside(out[n], o[0, 0], tol[0, 0], "out")
    # a length beyond the table's row is cut there
    kda.kda_attn_decode_step(q, kc, vc, table, torch.tensor([100, 10000], dtype=torch.int32, device="cuda"))
    assert kda.device_error() == 5


def test_decode_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: the last pages are read where they are."""
    pages, size, d = 70000, 256, 128
    kc = torch.zeros((pages, 1, size, d), dtype=BF16, device="cuda")
    vc = kc.clone()
    table = torch.tensor([[pages - 1, pages // 2 + 3]], dtype=torch.int32, device="cuda")
    for p in table[0].tolist():
        kc[p], vc[p] = make((1, size, d), p, BF16), make((1, size, d), p + 1, BF16)
    q = make((1, 4, d), 5, BF16)
    new = make((1, 1, 1, d), 6, BF16)
    kda.kda_kv_append(new, new, kc, vc, table, torch.tensor([299], dtype=torch.int32, device="cuda"))
    assert torch.equal(kc[pages // 2 + 3, 0, 43], new[0, 0, 0])
    check_decode(q, kc, vc, table, [300])


# ---- append -------------------------------------------------------------------------------------


def freqs(r):
    return (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()


def check_append(new, past, hq, hkv, d, size, dtype, rotary, interleaved=False, packed=None, seed=300):
    lens = [a + max(p, 0) for a, p in zip(new, past)]
    kc, vc, table = cache_of(lens, hkv, d, size, dtype, seed)
    packed = len(set(new)) > 1 if packed is None else packed
    lead = (1, sum(new)) if packed else (len(new), new[0])
    q, k, v = (make((*lead, h, d), seed + 5 + i, dtype) for i, h in enumerate((hq, hkv, hkv)))
    cu = offsets(new) if packed else None
    inv = freqs(rotary) if rotary else None
    want = [kc.double(), vc.double()]
    before = [kc.clone(), vc.clone()]
    qr, kr = kda.kda_kv_append(k, v, kc, vc, table, torch.tensor(past, dtype=torch.int32, device="cuda"), inv, q, cu,
                               interleaved, return_k=True)
    u = torch.finfo(dtype).eps / 2

    def rotated(x, pos):
        return ref.rotate(x, pos, inv, interleaved) if rotary else x.double()

    flat = [t.flatten(0, 1) for t in (q, k, v, qr, kr)]
    touched = torch.zeros(kc.shape, dtype=torch.bool, device="cuda")
    at = 0
    for n, (a, p) in enumerate(zip(new, past)):
        r = slice(at, at + a)
        at += a
        if p < 0 or a == 0:
            continue
        pos = torch.arange(p, p + a, device="cuda")
        page, slot = table[n][pos // size].long(), pos % size
        for src, got in ((flat[0], flat[3]), (flat[1], flat[4])):
            x = src[r]
            y = rotated(x, pos)
            # sine and cosine to 2^-21 of the pair's size, one rounding of the result
            pair = x.double().abs().amax(-1, keepdim=True) * 2
            inside(got[r], y, u * y.abs() + 2.0 ** -21 * pair + 1e-30, "rotated")
        assert torch.equal(kc[page, :, slot], flat[4][r]) and torch.equal(vc[page, :, slot], flat[2][r])
        touched[page, :, slot] = True
    for c, b in zip((kc, vc), before):
        assert torch.equal(c[~touched], b[~touched])
    assert len(want) == 2
    return kc, vc, table


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d,rotary,interleaved", [(64, 64, False), (128, 128, False), (128, 64, False), (64, 16, False),
                                                  (128, 128, True), (64, 48, True), (64, 0, False), (128, 112, False)])
def test_append(d, rotary, interleaved, dtype):
    check_append([1] * 5, [0, 15, 16, 300, -1], 4, 2, d, 16, dtype, rotary, interleaved)
    check_append([33, 0, 1, 100], [0, 7, 500, 28], 6, 2, d, 32, dtype, rotary, interleaved)
    assert kda.device_error() == 0


def test_append_many_tokens():
    check_append([700, 1, 901], [3, 0, 64], 2, 1, 64, 64, BF16, 64)
    check_append([400] * 4, [0, 1, 2, 3], 2, 2, 128, 1, BF16, 128, packed=False)


def test_append_far_positions():
    """Angles of positions near 2^20 and 2^24, where fp32 products have lost whole radians."""
    size, d = 64, 128
    for pos in (1 << 20, (1 << 24) - 3):
        k = make((1, 3, 1, d), 310, FP32)
        pages = 2
        kc, vc = (torch.zeros((pages, 1, size, d), device="cuda") for _ in range(2))
        width = pos // size + 2
        table = torch.zeros((1, width), dtype=torch.int32, device="cuda")
        table[0, (pos + 2) // size] = 1
        _, kr = kda.kda_kv_append(k, k, kc, vc, table, torch.tensor([pos], dtype=torch.int32, device="cuda"), freqs(d),
                                  return_k=True)
        want = ref.rotate(k[0], torch.arange(pos, pos + 3, device="cuda"), freqs(d), False)
        inside(kr[0], want, 2.0 ** -21 * 2 * k[0].double().abs().amax(-1, keepdim=True) + 2.0 ** -24 * want.abs(), "rotated")


def test_append_strides_in_place_and_rows_behind():
    lens, d = [20, 13], 64
    tokens = sum(lens) + 4   # four rows behind the last sequence
    qkv = make((1, tokens, 8 * d), 320, BF16)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split((4 * d, 2 * d, 2 * d), -1))
    kc, vc, table = cache_of(lens, 2, d, 16, BF16, 321)
    past = torch.zeros(2, dtype=torch.int32, device="cuda")
    cu = offsets(lens)
    k2, v2 = kc.clone(), vc.clone()
    q_out = torch.full((1, tokens, 4, d), 3.0, dtype=BF16, device="cuda")
    a, _ = kda.kda_kv_append(k, v, kc, vc, table, past, freqs(d), q, cu, q_out=q_out)
    assert a is q_out and (a[:, sum(lens):] == 3.0).all()
    dense = q.contiguous()
    b, _ = kda.kda_kv_append(k.contiguous(), v.contiguous(), k2, v2, table, past, freqs(d), dense, cu, q_out=dense)
    assert b is dense and torch.equal(a[:, : sum(lens)], b[:, : sum(lens)])
    assert torch.equal(b[:, sum(lens):], q[:, sum(lens):])
    assert torch.equal(kc, k2) and torch.equal(vc, v2)


def test_append_bad_pages_write_nothing():
    kc, vc = (torch.zeros((4, 1, 16, 64), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.tensor([[-1, 7], [2, 1]], dtype=torch.int32, device="cuda")
    k = make((2, 3, 1, 64), 330, BF16)
    past = torch.tensor([14, 30], dtype=torch.int32, device="cuda")   # row 0: pages -1 and 7; row 1: page 1, then past the row
    kda.kda_kv_append(k, k, kc, vc, table, past)
    assert kda.device_error() == 5
    assert torch.equal(kc[1, 0, 14:], k[1, :2, 0]) and torch.equal(vc[1, 0, 14:], k[1, :2, 0])
    kc[1, 0, 14:] = 0
    vc[1, 0, 14:] = 0
    assert (kc == 0).all() and (vc == 0).all()


# ---- together -----------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prompt_then_tokens(dtype):
    """A hybrid model's attention layer as it serves: packed prompts go into the cache and through the
    prompt attention, then tokens come one by one; every output equals the attention over all tokens."""
    lens, steps, hq, hkv, d, size = [50, 7, 129], 5, 8, 2, 128, 16
    kc, vc, table = cache_of([n + steps for n in lens], hkv, d, size, dtype, 400)
    q, k, v = (make((1, sum(lens), h, d), 410 + i, dtype) for i, h in enumerate((hq, hkv, hkv)))
    tok = [make((steps, 3, h, d), 420 + i, dtype) for i, h in enumerate((hq, hkv, hkv))]
    cu, inv = offsets(lens), freqs(d)
    have = torch.zeros(3, dtype=torch.int32, device="cuda")
    qr, kr = kda.kda_kv_append(k, v, kc, vc, table, have, inv, q, cu, return_k=True)
    out = kda.kda_attn_fwd(qr, kr, v, cu)
    o, _, tol, _ = ref.attention(qr, kr, v, cu)
    inside(out, o, tol, "prompt")
    have = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for i in range(steps):
        qi, ki, vi = (t[i][:, None] for t in tok)
        qn, _ = kda.kda_kv_append(ki, vi, kc, vc, table, have, inv, qi)
        have = have + 1
        out = kda.kda_attn_decode_step(qn[:, 0], kc, vc, table, have)
        o, _, tol, _ = decode_ref(qn[:, 0], kc, vc, table, have.tolist())
        inside(out, o[:, 0], tol[:, 0], "token")
    assert kda.device_error() == 0


def test_decode_step_in_a_graph():
    """Append and decode captured once and replayed with the lengths moving on, beside eager calls; two
    graphs hold workspaces of their own."""
    B, hq, hkv, d, size, steps = 3, 4, 2, 64, 16, 6
    start = [10, 31, 100]
    inv = freqs(d)

    def state():
        kc, vc, table = cache_of([n + steps for n in start], hkv, d, size, BF16, 500)
        return kc, vc, table, torch.tensor(start, dtype=torch.int32, device="cuda")

    tok = [make((steps, B, 1, h, d), 510 + i, BF16) for i, h in enumerate((hq, hkv, hkv))]

    def step(q, k, v, kc, vc, table, have):
        qn, _ = kda.kda_kv_append(k, v, kc, vc, table, have, inv, q)
        return kda.kda_attn_decode_step(qn[:, 0], kc, vc, table, have + 1)

    kc, vc, table, have = state()
    want = []
    for i in range(steps):
        want.append(step(*(t[i] for t in tok), kc, vc, table, have).clone())
        have += 1
    graphs = []
    for _ in range(2):
        s = state()
        buf = [t[0].clone() for t in tok]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(*buf, *s)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*buf, *s)
        graphs.append((g, s, buf, out))
    for i in range(steps):
        for g, s, buf, out in graphs:
            for b, t in zip(buf, tok):
                b.copy_(t[i])
            g.replay()
            s[3].add_(1)
        for g, s, buf, out in graphs:
            assert torch.equal(out, want[i])
    torch.cuda.synchronize()


def test_prompt_in_a_graph():
    """Forward and gradient captured through the direct calls and replayed on new inputs."""
    lens = [100, 28, 200]
    cu = offsets(lens)

    def fresh(seed):
        return [make((1, sum(lens), h, 128), seed + i, BF16) for i, h in enumerate((4, 2, 2, 4))]

    def both(q, k, v, g):
        out, lse = kda.kda_attn_fwd(q, k, v, cu, return_lse=True)
        return (out, *kda.kda_attn_bwd(q, k, v, out, lse, g, cu))

    buf = fresh(600)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(*buf)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both(*buf)
    for seed in (610, 620):
        x = fresh(seed)
        for b, t in zip(buf, x):
            b.copy_(t)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, both(*x)))
    torch.cuda.synchronize()


def test_other_streams():
    q, k, v, cu, _ = prompt("packed", 4, 2, 64, BF16, seed=700)
    want = kda.kda_attn_fwd(q, k, v, cu)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(kda.kda_attn_fwd(q, k, v, cu))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


def test_fresh_threads():
    """Every call as the first of its thread, where no CUDA context is bound yet."""
    q, k, v, cu, _ = prompt("packed", 4, 2, 128, BF16, seed=710)
    g = make(q.shape, 715, BF16)
    out, lse = kda.kda_attn_fwd(q, k, v, cu, return_lse=True)
    want = kda.kda_attn_bwd(q, k, v, out, lse, g, cu)
    kc, vc, table = cache_of([40], 2, 128, 16, BF16, 720)
    seq = torch.tensor([40], dtype=torch.int32, device="cuda")
    dec = kda.kda_attn_decode_step(q[:, 0], kc, vc, table, seq)
    torch.cuda.synchronize()
    got, calls = {}, dict(
        fwd=lambda: kda.kda_attn_fwd(q, k, v, cu), bwd=lambda: kda.kda_attn_bwd(q, k, v, out, lse, g, cu),
        dec=lambda: kda.kda_attn_decode_step(q[:, 0], kc, vc, table, seq))
    for name, call in calls.items():
        t = threading.Thread(target=lambda: got.__setitem__(name, call()))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert torch.equal(got["fwd"], out) and torch.equal(got["dec"], dec)
    assert all(torch.equal(a, b) for a, b in zip(got["bwd"], want))


def test_refusals_name_their_status():
    q = make((1, 8, 2, 96), 800, BF16)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_attn_fwd(q, q, q)
    assert e.value.status == 2
    q = make((1, 8, 2, 64), 801, BF16)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_attn_fwd(q, q, q, scale=0.0)
    assert e.value.status == 1
    kc = make((4, 2, 24, 64), 802, BF16)
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(kda.KdaError) as e:
        kda.kda_attn_decode_step(q[:, 0], kc, kc, table, table[0, :1])
    assert e.value.status == 2


def test_gradient_is_taken_once():
    q = make((1, 40, 2, 64), 810, BF16).requires_grad_()
    k = make((1, 40, 1, 64), 811, BF16)
    out = kda.kda_attn(q, k, k)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(out.float().sum(), q, create_graph=True)
    # only what needs a gradient gets one, and through several uses they add up
    out = kda.kda_attn(q, k, k)
    (out.float().sum() + out.float().sum()).backward()
    once = torch.autograd.grad(kda.kda_attn(q, k, k).float().sum(), q)[0]
    assert k.grad is None
    # twice the upstream gradient is exact in bf16
    assert torch.equal(q.grad, 2 * once)


def test_gradient_in_a_graph_beside_an_eager_one():
    """A gradient captured through the direct calls while an eager graph of the same leaves lives."""
    q, k, v = (make((1, 130, h, 64), 820 + i, BF16).requires_grad_() for i, h in enumerate((4, 2, 2)))
    g = make(q.shape, 825, BF16)
    alive = kda.kda_attn(q, k, v)
    qd, kd, vd = (t.detach() for t in (q, k, v))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = kda.kda_attn_fwd(qd, kd, vd, return_lse=True)
        kda.kda_attn_bwd(qd, kd, vd, out, lse, g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, rest = kda.kda_attn_fwd(qd, kd, vd, return_lse=True, return_rest=True)
        got = kda.kda_attn_bwd(qd, kd, vd, out, lse, g, out_rest=rest)
    graph.replay()
    want = torch.autograd.grad(alive, (q, k, v), g)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()


def test_captured_gradient_of_live_leaves_is_refused():
    """Capture of the differentiable call: refused while an eager graph of its leaves lives, sound without one."""
    q, k, v = (make((1, 70, h, 64), 840 + i, BF16).requires_grad_() for i, h in enumerate((4, 2, 2)))
    g = make(q.shape, 845, BF16)
    alive = kda.kda_attn(q, k, v)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="another stream"), torch.cuda.graph(graph):
        kda.kda_attn(q, k, v)
    want = torch.autograd.grad(alive, (q, k, v), g)
    del alive
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kda.kda_attn(q, k, v)
        got = torch.autograd.grad(out, (q, k, v), g)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    del out, got
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_differentiable_call_without_a_graph(dtype):
    q, k, v = (make((2, 50, h, 64), 850 + i, dtype).requires_grad_() for i, h in enumerate((4, 2, 2)))
    with torch.no_grad():
        out = kda.kda_attn(q, k, v)
    assert not out.requires_grad and torch.equal(out, kda.kda_attn(q, k, v))
    assert torch.equal(out, kda.kda_attn(q.detach(), k.detach(), v.detach()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(16, 4), (6, 6)])
def test_prompt_more_items_than_sms(hq, hkv, d):
    """Batches whose tiles outnumber the SMs several times, so that every block works through many."""
    lens = [700, 33, 1, 0, 390, 128, 517, 256, 64, 900, 300, 129]
    cu = offsets(lens)
    q, k, v, g = (make((1, sum(lens), h, d), 830 + i, BF16) for i, h in enumerate((hq, hkv, hkv, hq)))
    out, lse = kda.kda_attn_fwd(q, k, v, cu, return_lse=True)
    o, l, tol, ltol = ref.attention(q, k, v, cu)
    inside(out, o, tol, "out")
    check_lse(lse, l, ltol)
    want, tols = ref.attention_grad(q, k, v, g, cu)
    first = None
    for _ in range(5):
        got = kda.kda_attn_bwd(q, k, v, out, lse, g, cu)
        assert kda.device_error() == 0
        if first is None:
            first = got
            for x, y, t, n in zip(got, want, tols, ("dq", "dk", "dv")):
                inside(x, y, t, n)
        assert all(torch.equal(a, b) for a, b in zip(first, got))
