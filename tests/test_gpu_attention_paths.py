"""Softmax attention on the GPU, on the paths that a call takes by its sizes: shares and join of the decode step, the
large fp32 blocks, more than 128 packed sequences, appends of many tokens.  Bounds as in test_gpu_attention."""
import math

import pytest
import torch

import gated_delta_rule_86_b200 as kda
from oracle import attention as ref
from test_gpu_attention import (BF16, FP32, cache_of, check_append, check_decode, check_lse, decode_ref, inside, make,
                                offsets)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _library(cuda_lib):
    yield
    torch.cuda.synchronize()
    kda.device_error()


# ---- decode: tables that hold more than a block takes by itself -----------------------------------

LENS = [1500, 1, 0, 129, 3001, 2048, -2, 700]


@pytest.mark.parametrize("hq,hkv", [(2, 2), (2, 1), (4, 1), (6, 2), (8, 1), (16, 1), (20, 1), (24, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_shares(hq, hkv, d, dtype):
    kc, vc, table = cache_of(LENS, hkv, d, 64, dtype, 900, fill=float("nan"))
    check_decode(make((len(LENS), hq, d), 910, dtype), kc, vc, table, LENS)
    assert kda.device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1, 8, 16, 128])
def test_decode_shares_pages(size, d, dtype):
    lens = [1100, 77, 2049]
    kc, vc, table = cache_of(lens, 2, d, size, dtype, 920)
    check_decode(make((3, 8, d), 921, dtype), kc, vc, table, lens, scale=0.13)


@pytest.mark.parametrize("d,hq", [(64, 4), (128, 4), (128, 16)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_decode_shares_with_bad_pages_and_cut_lengths(dtype, d, hq):
    lens = [1300, 2100]
    kc, vc, table = cache_of(lens, 1, d, 32, dtype, 930)
    q = make((2, hq, d), 931, dtype)
    broken = table.clone()
    gone = [[0, 7, 40], [3, 64, 65]]
    for n, pages in enumerate(gone):
        for page, bad in zip(pages, (-1, kc.shape[0], -2 ** 31)):
            broken[n, page] = bad
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = kda.kda_attn_decode_step(q, kc, vc, broken, seq)
    assert kda.device_error() == 5
    for n in range(2):
        keep = [p for p in range(lens[n]) if p // 32 not in gone[n]]
        k, v = (ref.gather_cache(c, table[n], lens[n])[keep][None] for c in (kc, vc))
        o, _, tol, _ = ref.attention(q[n:n + 1, None], k, v, causal=False)
        inside(out[n], o[0, 0], tol[0, 0], "out")
    # a length beyond the table's row counts as the row's
    narrow = table[:, :40].contiguous()
    out = kda.kda_attn_decode_step(q, kc, vc, narrow, seq)
    assert kda.device_error() == 5
    o, _, tol, _ = decode_ref(q, kc, vc, narrow, [1280, 1280])
    inside(out, o[:, 0], tol[:, 0], "cut")


def test_decode_shares_in_a_graph_with_lengths_that_it_moves():
    """The lengths are changed by a kernel of the graph just before the step, whose second kernel reads them early."""
    B, hq, hkv, d, size, steps = 5, 16, 2, 128, 16, 24
    start = [1000, 120, 1270, 3, 2040]
    kc, vc, table = cache_of([n + steps + 1 for n in start], hkv, d, size, BF16, 940)
    q = make((B, hq, d), 941, BF16)
    have = torch.tensor(start, dtype=torch.int32, device="cuda")
    want = [kda.kda_attn_decode_step(q, kc, vc, table, have + i) for i in range(1, steps + 1)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kda.kda_attn_decode_step(q, kc, vc, table, have)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        have.add_(1)
        out = kda.kda_attn_decode_step(q, kc, vc, table, have)
    got = []
    for _ in range(steps):
        graph.replay()
        got.append(out.clone())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,wide", [(4, False), (16, False), (4, True), (16, True)])
def test_decode_weights_keep_their_bits(hq, wide, d):
    """bf16 outputs off by their own rounding alone.  Queries and keys with one channel each that is not zero make the
    scores exact, so a weight's error is that of its exponent (the scale's product and the subtraction of the maximum
    round, 2 e each for |x| < 8 in log2 units: 32 e), of the power (2^-22 = 4 e, in the weight and in the sum), of the
    sum (n e) and of its rounding to two bf16 numbers, 2^-16; the sum of n products may truncate, 2 n e."""
    n, size = 40, 16
    lens = [n, 7, n - 1] + ([2000] if wide else [])
    kc, vc, table = cache_of(lens, 1, d, size, BF16, 950)
    kc[..., 1:] = 0
    q = torch.zeros((len(lens), hq, d), dtype=BF16, device="cuda")
    q[..., 0] = make((len(lens), hq), 951, BF16)
    kc[..., 0].clamp_(-2, 2)
    q.clamp_(-2, 2)
    out = kda.kda_attn_decode_step(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for b, length in enumerate(lens[:3]):
        k, v = (ref.gather_cache(c, table[b], length)[:, 0].double() for c in (kc, vc))
        p = torch.softmax(q[b].double() @ k.T / math.sqrt(d), 1)
        want, mass = p @ v, p @ v.abs()
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -16 + (2 * (32 + 4) + 3 * length) * 2.0 ** -24) * mass
        inside(out[b], want, 1.01 * tol, "out")


# ---- prompts ------------------------------------------------------------------------------------


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_fp32_large_blocks(causal, d):
    """As many blocks of 64 rows as there are SMs and more, dense and packed."""
    for lens, B in ((None, 2), ([300, 0, 129, 571], 1)):
        T = sum(lens) if lens else 500
        q, k, v, g = (make((B, T, h, d), 960 + i, FP32) for i, h in enumerate((12, 12, 12, 12)))
        cu = offsets(lens) if lens else None
        out, lse = kda.kda_attn_fwd(q, k, v, cu, causal=causal, return_lse=True)
        o, l, tol, ltol = ref.attention(q, k, v, cu, causal=causal)
        inside(out, o, tol, "out")
        check_lse(lse, l, ltol)
        got = kda.kda_attn_bwd(q, k, v, out, lse, g, cu, causal=causal)
        want, tols = ref.attention_grad(q, k, v, g, cu, causal=causal)
        for x, y, t, name in zip(got, want, tols, ("dq", "dk", "dv")):
            inside(x, y, t, name)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (FP32, 64)])
@pytest.mark.parametrize("own_keys", [False, True])
def test_prompt_more_than_128_sequences(own_keys, dtype, d):
    """Sequences of several tiles among many short and empty ones, with keys of their own lengths or not."""
    nq = [(11 * i) % 40 for i in range(150)]
    for i, n in ((3, 300), (40, 129), (77, 513), (128, 256), (149, 400)):
        nq[i] = n
    nk = [(n + 17 * i) % 150 if i % 3 else n for i, n in enumerate(nq)] if own_keys else nq
    if own_keys:
        nk[77], nk[128] = 700, 100
    q, k, v, g = (make((1, sum(n), h, d), 970 + i, dtype) for i, (n, h) in enumerate(((nq, 4), (nk, 2), (nk, 2), (nq, 4))))
    cu, cu_k = offsets(nq), offsets(nk) if own_keys else None
    out, lse = kda.kda_attn_fwd(q, k, v, cu, cu_k, return_lse=True)
    o, l, tol, ltol = ref.attention(q, k, v, cu, cu_k)
    inside(out, o, tol, "out")
    check_lse(lse, l, ltol)
    got = kda.kda_attn_bwd(q, k, v, out, lse, g, cu, cu_k)
    want, tols = ref.attention_grad(q, k, v, g, cu, cu_k)
    for x, y, t, name in zip(got, want, tols, ("dq", "dk", "dv")):
        inside(x, y, t, name)


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (3, 1, 64), (2, 2, 128), (8, 2, 128)])
@pytest.mark.parametrize("T,past,limit", [(9, 0, 1.25), (20, 0, 1.25), (64, 0, 1.25), (128, 0, 1.25), (128, 1, 1.25), (70, 90, 1.25),
                                          (1024, 0, math.sqrt(2)), (900, 7, math.sqrt(2))])
def test_gradient_of_few_keys_keeps_its_bits(T, past, limit, hq, hkv, d):
    """The error of bf16 gradients, against that of the formula's gradient rounded to bf16, which is the least.  Where the
    first query of each tile sees a tile of keys at most, what is left comes through delta: the forward's weights are
    rounded, in an output that averages over the keys, so at most half of a rounding's energy: sqrt(1 + 1/2).  Beyond,
    the rounding of the weights and of dS adds one rounding's energy at most, sqrt(1 + 1)."""
    B = 1 if T > 128 else 16
    q, k, v, g = (make((B, t, h, d), 975 + i, BF16) for i, (t, h) in enumerate(((T, hq), (T + past, hkv), (T + past, hkv), (T, hq))))
    leaves = [t.requires_grad_() for t in (q, k, v)]
    got = torch.autograd.grad(kda.kda_attn(*leaves), leaves, g)
    want, _ = ref.attention_grad(*(t.detach() for t in (q, k, v)), g)
    for x, w, name in zip(got, want, ("dq", "dk", "dv")):
        least = (w.bfloat16().double() - w).norm().item()
        assert (x.double() - w).norm().item() <= limit * least, name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_gradient_fp32_of_many_terms(causal, d):
    """dK and dV over 16 heads of 1024 queries.  A sum of n terms one after another errs by some sqrt(n) / 2 half steps
    of 2^-24 of a random sum's size: sqrt(16384) / 2 = 64 of them in one go, (sqrt(64) + sqrt(256)) / 2 = 12 by tiles of 64;
    8 more for scores, powers and dP."""
    q, k, v, g = (make((1, 1024, h, d), 990 + i, FP32) for i, h in enumerate((16, 1, 1, 16)))
    out, lse = kda.kda_attn_fwd(q, k, v, causal=causal, return_lse=True)
    got = kda.kda_attn_bwd(q, k, v, out, lse, g, causal=causal)
    want, _ = ref.attention_grad(q, k, v, g, causal=causal)
    for x, w, name in zip(got, want, ("dq", "dk", "dv")):
        assert (x.double() - w).norm() <= 20 * 2.0 ** -24 * w.norm(), name


# ---- append -------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d,rotary,interleaved", [(64, 64, False), (128, 128, True), (128, 48, False), (64, 0, False)])
def test_append_thousands_of_tokens(d, rotary, interleaved, dtype):
    check_append([1300, 0, 5, 2200], [3, 9, 70, 0], 4, 2, d, 16, dtype, rotary, interleaved, seed=980)
    check_append([650] * 3, [0, 31, 32], 3, 1, d, 32, dtype, rotary, interleaved, packed=False, seed=985)
    assert kda.device_error() == 0
