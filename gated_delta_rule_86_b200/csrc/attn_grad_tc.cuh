// attn_grad_tc.cuh -- gradient of attention over whole prompts on the tensor cores (bf16 inputs).
//
//     P = 2^(c S - lse log2 e),  S = Q K^T,  c = scale log2 e,     dP = dO V^T,   dS = P o (dP - delta),
//     dV = P^T dO,   dK = scale dS^T Q,   dQ = scale dS K,         delta = rowsum(dO o O)
// in two kernels, so that every sum has one owner and one order (no atomics, the same bits each call):
//
//   keys:     a block owns 128 keys of one head of the cache and walks the query tiles of all heads of
//             the group; dK and dV stay in Tensor Memory from the first tile to the last.  Scores are
//             formed transposed (rows = keys), so P^T and dS^T are written by the threads that computed
//             them straight into Tensor Memory as the second products' A operands.
//   queries:  a block owns 128 queries of one head and walks the key tiles; dQ stays in Tensor Memory.
//
// S and dP are computed in both: seven products of 128 x 128 x d in place of five.  The price of the
// second pair is less than that of adding dQ tiles to memory from every key block, and buys the fixed order.
//
// Warp roles: 0-15 compute (thread = row, four groups of 32 columns), 16 issues the products, 17 loads
// (TMA, and the queries' lse and delta), 18 waits for the loads on 16's behalf, zeroes rows that must not
// count, and joins its word to the compute warps' (a wait behind products in flight returns only with
// them).  P and dS are rounded once, to bf16, as operands.
//
// Rows past the end of a sequence in its last tile belong to others.  Where they are rows of a result
// they are not stored; where they are summed over (queries in the keys' kernel, keys in the other) they
// are zeroed in shared memory, since a weight of zero does not hide a NaN.
#pragma once

#include "attn_prompt_tc.cuh"

namespace kda {
namespace attn {

template <int D> struct GradCfg {
    static constexpr int kTileBytes = kTile * D * 2;
    // Stages of one tile each, released one by one: of a turn's two tiles (Q and dO, or K and V) the first
    // is read again at the turn's end, so more of it are held.  (One ring for both: 262 us for dQ at B2
    // T4096 H16, its loads of V waiting for dQ's products.)
    static constexpr int kFirst = D == 128 ? 3 : 4, kSecond = D == 128 ? 2 : 4, kStages = kFirst + kSecond;
    static constexpr int kOwn = 0;                        // the block's own two tiles
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kOut = kRing + (kFirst - 1) * kTileBytes;    // queries' kernel: O, in a stage filled late
    static constexpr int kStats = kRing + kStages * kTileBytes;       // keys' kernel: -lse and -delta of two turns' queries
    static constexpr int kBars = kStats + 2 * 2 * kTile * 4;
    static constexpr int kSmem = kBars + 512;
    static_assert(kSmem <= 232448, "shared memory");
    static constexpr int kThreads = 640;
};

struct GradBars {
    uint64_t own_full, out_full, out_read, first, full[8], empty[8], stats[2], stats_read[2], s_full, dp_full[2], q_word,
        a_ready, b_ready, done, drain;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(GradBars) <= 512, "barriers");

// Barriers and Tensor Memory; every thread.  Returns the Tensor Memory's base.
template <int D> __device__ __forceinline__ uint32_t grad_setup(GradBars &bars, int a_count, int b_count) {
    using C = GradCfg<D>;
    if (threadIdx.x == 0) {
        bars.abort = 0;
        tc::mbar_init(&bars.own_full, 1);
        tc::mbar_init(&bars.first, 1);
        tc::mbar_init(&bars.out_full, 1);
        tc::mbar_init(&bars.out_read, 16);
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(&bars.full[i], 1);
            tc::mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars.stats[i], 1);
            tc::mbar_init(&bars.stats_read[i], 16);
        }
        tc::mbar_init(&bars.s_full, 1);
        tc::mbar_init(&bars.dp_full[0], 1);
        tc::mbar_init(&bars.dp_full[1], 1);
        tc::mbar_init(&bars.q_word, 1);
        tc::mbar_init(&bars.a_ready, a_count);   // sixteen compute warps, and the next loads' word where it goes with them
        tc::mbar_init(&bars.b_ready, b_count);
        tc::mbar_init(&bars.done, 1);
        tc::mbar_init(&bars.drain, 1);
        tc::fence_mbar_init();
    }
    if (threadIdx.x >> 5 == 16) {
        tc::tmem_alloc(&bars.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    return bars.tmem;
}

// Load k is tile k & 1 of turn k >> 1: its stage, the parity of that stage's filling, and its place.
template <int D> __device__ __forceinline__ int stage_no(int k) {
    using C = GradCfg<D>;
    return k & 1 ? C::kFirst + (k >> 1) % C::kSecond : (k >> 1) % C::kFirst;
}
template <int D> __device__ __forceinline__ uint32_t filling(int k) {
    using C = GradCfg<D>;
    return (k >> 1) / (k & 1 ? C::kSecond : C::kFirst);
}
template <int D> __device__ __forceinline__ uint32_t stage_of(int k) {
    return GradCfg<D>::kRing + stage_no<D>(k) * GradCfg<D>::kTileBytes;
}

// Warp 17's lane: loads both tiles of `total` turns, issue(k, place, barrier) starting load k.  The stage
// that holds O at first waits for `hold`, if given.
template <int D, typename F>
__device__ __forceinline__ void load_ring(GradBars &bars, int total, uint64_t *hold, F issue) {
    using C = GradCfg<D>;
    volatile int *abort = &bars.abort;
    bool ok = true;
    int k = 0;
    for (; k < 2 * total; ++k) {
        const int st = stage_no<D>(k);
        const uint32_t n = filling<D>(k);
        if (n > 0) ok = tc::mbar_wait(&bars.empty[st], (n - 1) & 1, abort);
        else if (hold && stage_of<D>(k) == C::kOut) ok = tc::mbar_wait(hold, 0, abort);
        if (!ok) break;
        tc::mbar_arrive_expect_tx(&bars.full[st], C::kTileBytes);
        issue(k, stage_of<D>(k), &bars.full[st]);
    }
    if (!ok) {   // a wait ran out: leave no copy in flight
        int quit = 0;
        tc::mbar_wait(&bars.own_full, 0, &quit);
        for (int i = k > 2 * C::kFirst ? k - 2 * C::kFirst : 0; i < k; ++i) {
            quit = 0;
            tc::mbar_wait(&bars.full[stage_no<D>(i)], filling<D>(i) & 1, &quit);
        }
    }
}

// Warp 18: waits for load k and zeroes its rows from `rows` on, where that is below 128.
template <int D> __device__ __forceinline__ bool watch_load(GradBars &bars, uint8_t *smem, int k, int rows, int lane) {
    if (!warp_wait(&bars.full[stage_no<D>(k)], filling<D>(k) & 1, &bars.abort)) return false;
    if (rows < kTile) {
        zero_rows<D>(smem + stage_of<D>(k), rows, lane);
        __syncwarp();
    }
    return true;
}

// 32 numbers of a thread's row, rounded, into Tensor Memory as an operand, over the first 16 columns of
// the 32 that they were read from.
__device__ __forceinline__ void put_operand(uint32_t taddr, const float2 (&x)[16]) {
    uint32_t u[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) u[e] = pack_bf16(x[e].x, x[e].y);
    tc::tmem_st16(taddr, u);
}
// d (+)= x y with x such an operand of 128 columns, y an MN-major tile.
__device__ __forceinline__ void chain_ts32(uint32_t d, uint32_t x, uint64_t y, uint32_t idesc, bool accumulate,
                                           uint32_t leader) {
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk)
        mma_ts(d, x + (kk >> 1) * 32 + (kk & 1) * 8, y + kk * 128, idesc, accumulate || kk > 0, leader);
}

__device__ __forceinline__ void arrive_operand(uint64_t *bar, int lane) {
    tc::tmem_st_wait();
    tc::tc_fence_before();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

// Gradients of rows behind the last packed sequence: zero.  Normally there are none; every block takes its share.
template <int D> __device__ __forceinline__ void zero_behind(__nv_bfloat16 *g, const int32_t *cu, int n, int T, int heads) {
    if (cu == nullptr) return;
    const int from = min(max(__ldg(cu + n), 0), T);
    const int64_t pieces = (int64_t)(T - from) * heads * (D / 8);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * blockDim.x)
        reinterpret_cast<uint4 *>(g + (int64_t)from * heads * D)[i] = make_uint4(0, 0, 0, 0);
}

// A warp's 32 rows of an accumulator to global memory.
template <int D>
__device__ __forceinline__ void store_rows(uint32_t taddr, uint8_t *stage, int lane, __nv_bfloat16 *dst, int64_t stride,
                                           int rows, float mul, bool zero) {
    RowWriter<D> out{stage};
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        float x[32];
        if (zero) {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = 0.f;
        } else {
            tc::tmem_ld32(taddr + c * 32, x);
            tc::tmem_ld_wait();
        }
        out.put(lane, c, x, mul);
    }
    out.flush(lane, dst, stride, rows);
}

// ---- dK and dV ----------------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(GradCfg<D>::kThreads, 1)
attn_grad_kv_tc_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ PromptMaps maps) {
    using C = GradCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    GradBars &bars = *reinterpret_cast<GradBars *>(smem + C::kBars);
    const uint32_t sbase = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    next_may_start();
    const uint32_t tmem = grad_setup<D>(bars, D == 64 ? 16 : 17, 17);
    if (tid == 32) prefetch_map(&maps.q), prefetch_map(&maps.k), prefetch_map(&maps.v), prefetch_map(&maps.g);
    wait_for_previous();
    zero_behind<D>(static_cast<__nv_bfloat16 *>(a.dk), a.bt.cu_k, a.bt.n, a.bt.Tk, a.bt.Hkv);
    zero_behind<D>(static_cast<__nv_bfloat16 *>(a.dv), a.bt.cu_k, a.bt.n, a.bt.Tk, a.bt.Hkv);
    // the first keys of a sequence are seen by the most queries: they go first
    int n;
    int count, level;
    if (!place_of(a.bt.cu_k, a.bt.n, a.bt.Tk, kTile, blockIdx.x / a.bt.Hkv, lane, n, count, level)) {
        if (warp == 16) tc::tmem_dealloc(tmem, 512);
        return;
    }
    const Seq s = seq_of(a.bt, n);
    const int hk = blockIdx.x % a.bt.Hkv, c0 = (count - level) * kTile, group = a.bt.Hq / a.bt.Hkv;
    const int ahead = s.nk - s.nq;   // causal: query i sees keys j <= i + ahead
    const int start = a.causal ? max(0, c0 - ahead) / kTile : 0;
    const int per_head = max(0, (s.nq + kTile - 1) / kTile - start), total = per_head * group;

    volatile int *abort = &bars.abort;
    const uint32_t tP = tmem + kTile, tV = tmem + 2 * kTile, tK = tV + D;
    // With d = 64 there is Tensor Memory for the next turn's scores beside this one's: they are formed ahead,
    // and the powers of a turn follow the dS of the one before without a product in between.
    constexpr bool kAhead = D == 64;
    auto tS = [&](int it) { return kAhead && (it & 1) ? tK + D : tmem; };
    float *stats = reinterpret_cast<float *>(smem + C::kStats);
    // turn `it` is query tile r0 of head h; its Q is load 2 it, its dO load 2 it + 1
    auto head_of = [&](int it) { return hk * group + it / per_head; };
    auto row_of = [&](int it) { return (start + it % per_head) * kTile; };

    if (warp == 17) {
        if (lane == 0 && total > 0) {
            tc::mbar_arrive_expect_tx(&bars.own_full, 2 * C::kTileBytes);
            tma_tile<D>(C::kOwn, smem, &maps.k, hk, s.k0 + c0, &bars.own_full);
            tma_tile<D>(C::kOwn + C::kTileBytes, smem, &maps.v, hk, s.k0 + c0, &bars.own_full);
            load_ring<D>(bars, total, nullptr, [&](int k, uint32_t at, uint64_t *bar) {
                tma_tile<D>(at, smem, k & 1 ? &maps.g : &maps.q, head_of(k >> 1), s.q0 + row_of(k >> 1), bar);
            });
        }
    } else if (warp == 19) {
        // -lse in log2 units, -inf (weight zero) where there is no query or it sees nothing; -delta.  Read a
        // turn before they are needed: the loads wait long behind the tiles' traffic.
        const int64_t at0 = stat_at(a.bt, s.q0, 0);   // a head's rows of a sequence lie side by side
        float ls[4], de[4];
        int h = hk * group, r0 = start * kTile;
        auto fetch = [&]() {
            const int64_t at = at0 + (int64_t)h * a.bt.Tq + r0 + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool there = r0 + e * 32 + lane < s.nq;
                ls[e] = there ? __ldg(a.lse + at + e * 32) : -CUDART_INF_F;
                de[e] = there ? __ldg(a.delta + at + e * 32) : 0.f;
            }
            if ((r0 += kTile) >= s.nq) r0 = start * kTile, ++h;
        };
        if (total > 0) fetch();
        for (int it = 0; it < total; ++it) {
            float l[4], d[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                l[e] = ls[e] == -CUDART_INF_F ? ls[e] : -ls[e] * kLog2e;
                d[e] = -de[e];
            }
            if (it + 1 < total) fetch();
            if (it >= 2 && !warp_wait(&bars.stats_read[it & 1], (it / 2 - 1) & 1, abort)) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                stats[(it & 1) * 2 * kTile + e * 32 + lane] = l[e];
                stats[(it & 1) * 2 * kTile + kTile + e * 32 + lane] = d[e];
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars.stats[it & 1]);
        }
    } else if (warp == 18) {
        // Queries that are not there are summed over with weight zero.  The word on the next Q goes with the
        // weights of this turn, that on the next dO with its dS; each word belongs to one turn.
        bool ok = total > 0;
        for (int it = 0; it <= total && ok; ++it) {
            const int left = it < total ? s.nq - row_of(it) : kTile;
            for (int x = 0; x < 2 && ok; ++x) {
                if (it < total && !(ok = watch_load<D>(bars, smem, 2 * it + x, left, lane))) break;
                if (it == 0) {
                    if (x == 1 && lane == 0) tc::mbar_arrive(&bars.first);
                    continue;
                }
                if (kAhead && x == 0) {   // a word of its own, not before the one before it has been heard
                    if (it == total) continue;
                    if (it > 1 && !(ok = warp_wait(&bars.s_full, (it - 1) & 1, abort))) break;
                }
                uint64_t *word = x ? &bars.b_ready : kAhead ? &bars.q_word : &bars.a_ready;
                if (lane == 0) tc::mbar_arrive(word);
                if (x == 1) ok = warp_wait(&bars.b_ready, (it - 1) & 1, abort);   // a_ready's turn is over, too
            }
        }
    } else if (warp == 16) {
        constexpr uint32_t idS = tc::make_idesc_bf16(kTile, kTile, false, false);
        constexpr uint32_t idG = tc::make_idesc_bf16(kTile, D, false, true);
        const uint32_t leader = elect_lane();
        const uint32_t sK = sbase + C::kOwn, sV = sK + C::kTileBytes;
        bool ok = true;
        if (total > 0) {
            ok = warp_wait(&bars.own_full, 0, abort) && warp_wait(&bars.first, 0, abort);
            if (ok) {
                chain_ss<D>(tS(0), desc_k(sK, 0), desc_k(sbase + stage_of<D>(0), 0), idS, leader);
                commit_by(&bars.s_full, leader);
                chain_ss<D>(tP, desc_k(sV, 0), desc_k(sbase + stage_of<D>(1), 0), idS, leader);
                commit_by(&bars.dp_full[0], leader);
            }
        }
        for (int it = 0; it < total && ok; ++it) {
            const bool more = it + 1 < total;
            auto next_scores = [&]() {
                chain_ss<D>(tS(it + 1), desc_k(sK, 0), desc_k(sbase + stage_of<D>(2 * it + 2), 0), idS, leader);
                commit_by(&bars.s_full, leader);
            };
            if (kAhead && more) {
                if (!(ok = warp_wait(&bars.q_word, it & 1, abort))) break;
                next_scores();
            }
            if (!(ok = warp_wait(&bars.a_ready, it & 1, abort))) break;
            tc::tc_fence_after();
            chain_ts32(tV, tS(it), desc_mn(sbase + stage_of<D>(2 * it + 1), 0), idG, it > 0, leader);
            if (!kAhead && more) next_scores();
            commit_by(&bars.empty[stage_no<D>(2 * it + 1)], leader);
            if (!(ok = warp_wait(&bars.b_ready, it & 1, abort))) break;
            tc::tc_fence_after();
            chain_ts32(tK, tP, desc_mn(sbase + stage_of<D>(2 * it), 0), idG, it > 0, leader);
            if (more) {
                chain_ss<D>(tP, desc_k(sV, 0), desc_k(sbase + stage_of<D>(2 * it + 3), 0), idS, leader);
                commit_by(&bars.dp_full[0], leader);
            }
            commit_by(more ? &bars.empty[stage_no<D>(2 * it)] : &bars.done, leader);
        }
        if (!ok) {   // no product in flight when the memory is given back
            int quit = 0;
            commit_by(&bars.drain, leader);
            warp_wait(&bars.drain, 0, &quit);
        }
    } else if (warp < 16) {
        const int part = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tc::tmem_lane_base(warp) + part * 32;
        const float sc = a.scale * kLog2e;
        const float2 sc2 = make_float2(sc, sc);
        bool ok = true;
        for (int it = 0; it < total; ++it) {
            const int r0 = row_of(it) + part * 32;
            const float *ls = stats + (it & 1) * 2 * kTile + part * 32, *de = ls + kTile;
            // this row's key is seen by the tile's queries from column `from` on
            const int from = c0 + row - ahead - r0;
            const bool partly = a.causal && c0 + (warp & 3) * 32 + 31 - ahead - r0 > 0;
            ok = warp_wait(&bars.stats[it & 1], (it >> 1) & 1, abort) && warp_wait(&bars.s_full, it & 1, abort);
            if (!ok) break;
            tc::tc_fence_after();
            float2 p[16];
            {
                float x[32];
                tc::tmem_ld32(tS(it) + lanes, x);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 l4 = *reinterpret_cast<const float4 *>(ls + 2 * e);
                    p[e] = fma2(make_float2(x[2 * e], x[2 * e + 1]), sc2, make_float2(l4.x, l4.y));
                    p[e + 1] = fma2(make_float2(x[2 * e + 2], x[2 * e + 3]), sc2, make_float2(l4.z, l4.w));
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = make_float2(ex2_approx(p[e].x), ex2_approx(p[e].y));
            if (partly) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (2 * e < from) p[e].x = 0.f;
                    if (2 * e + 1 < from) p[e].y = 0.f;
                }
            }
            put_operand(tS(it) + lanes, p);
            arrive_operand(&bars.a_ready, lane);
            ok = warp_wait(&bars.dp_full[0], it & 1, abort);
            if (!ok) break;
            tc::tc_fence_after();
            {
                float x[32];
                tc::tmem_ld32(tP + lanes, x);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 d4 = *reinterpret_cast<const float4 *>(de + 2 * e);
                    p[e] = mul2(p[e], add2(make_float2(x[2 * e], x[2 * e + 1]), make_float2(d4.x, d4.y)));
                    p[e + 1] = mul2(p[e + 1], add2(make_float2(x[2 * e + 2], x[2 * e + 3]), make_float2(d4.z, d4.w)));
                }
            }
            if (partly) {   // a hidden query's dP may be anything
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (2 * e < from) p[e].x = 0.f;
                    if (2 * e + 1 < from) p[e].y = 0.f;
                }
            }
            put_operand(tP + lanes, p);
            arrive_operand(&bars.b_ready, lane);
            if (lane == 0) tc::mbar_arrive(&bars.stats_read[it & 1]);
        }
        if (ok && total > 0) ok = warp_wait(&bars.done, 0, abort);
        if (ok && part < 2) {
            tc::tc_fence_after();
            // one warpgroup writes dV, another dK, through the tiles of K and V, which are done with
            const int k0 = c0 + (warp & 3) * 32;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(part ? a.dk : a.dv) + ((s.k0 + k0) * a.bt.Hkv + hk) * D;
            store_rows<D>((part ? tK : tV) + tc::tmem_lane_base(warp),
                          smem + C::kOwn + part * C::kTileBytes + (warp & 3) * 32 * D * 2, lane, dst,
                          (int64_t)a.bt.Hkv * D, s.nk - k0, part ? a.scale : 1.f, total == 0);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ---- dQ, and delta for the keys' kernel ---------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(GradCfg<D>::kThreads, 1)
attn_grad_q_tc_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ PromptMaps maps) {
    using C = GradCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    GradBars &bars = *reinterpret_cast<GradBars *>(smem + C::kBars);
    const uint32_t sbase = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    next_may_start();
    const uint32_t tmem = grad_setup<D>(bars, 17, 16);
    if (tid == 32) prefetch_map(&maps.q), prefetch_map(&maps.k), prefetch_map(&maps.v), prefetch_map(&maps.g), prefetch_map(&maps.o);
    wait_for_previous();
    zero_behind<D>(static_cast<__nv_bfloat16 *>(a.dq), a.bt.cu_q, a.bt.n, a.bt.Tq, a.bt.Hq);
    int n, count, level;
    if (!place_of(a.bt.cu_q, a.bt.n, a.bt.Tq, kTile, blockIdx.x / a.bt.Hq, lane, n, count, level)) {
        if (warp == 16) tc::tmem_dealloc(tmem, 512);
        return;
    }
    const Seq s = seq_of(a.bt, n);
    const int h = blockIdx.x % a.bt.Hq, hk = h / (a.bt.Hq / a.bt.Hkv), r0 = (level - 1) * kTile;
    const int total = (keys_seen(s, min(r0 + kTile, s.nq) - 1, a.causal) + kTile - 1) / kTile;

    volatile int *abort = &bars.abort;
    const uint32_t tS = tmem, tP = tmem + kTile, tQ = tmem + 3 * kTile;

    // turn j is key tile j: K is load 2 j, V load 2 j + 1
    if (warp == 17) {
        if (lane == 0) {
            tc::mbar_arrive_expect_tx(&bars.own_full, 2 * C::kTileBytes);
            tma_tile<D>(C::kOwn, smem, &maps.q, h, s.q0 + r0, &bars.own_full);
            tma_tile<D>(C::kOwn + C::kTileBytes, smem, &maps.g, h, s.q0 + r0, &bars.own_full);
            tc::mbar_arrive_expect_tx(&bars.out_full, C::kTileBytes);
            tma_tile<D>(C::kOut, smem, &maps.o, h, s.q0 + r0, &bars.out_full);
            load_ring<D>(bars, total, &bars.out_read, [&](int k, uint32_t at, uint64_t *bar) {
                tma_tile<D>(at, smem, k & 1 ? &maps.v : &maps.k, hk, s.k0 + (int64_t)(k >> 1) * kTile, bar);
            });
        }
    } else if (warp == 18) {
        // keys that are not there are summed over with weight zero (their values only masked); the word on
        // the next K and V goes with the reading of this turn's scores
        bool ok = total > 0;
        for (int j = 0; j < total && ok; ++j) {
            ok = watch_load<D>(bars, smem, 2 * j, s.nk - j * kTile, lane) && watch_load<D>(bars, smem, 2 * j + 1, kTile, lane);
            if (!ok) break;
            if (lane == 0) tc::mbar_arrive(j == 0 ? &bars.first : &bars.a_ready);
            if (j > 0) ok = warp_wait(&bars.a_ready, (j - 1) & 1, abort);
        }
    } else if (warp == 16) {
        constexpr uint32_t idS = tc::make_idesc_bf16(kTile, kTile, false, false);
        constexpr uint32_t idG = tc::make_idesc_bf16(kTile, D, false, true);
        const uint32_t leader = elect_lane();
        const uint32_t sQ = sbase + C::kOwn, sG = sQ + C::kTileBytes;
        bool ok = true;
        auto scores = [&](int j) {
            chain_ss<D>(tS, desc_k(sQ, 0), desc_k(sbase + stage_of<D>(2 * j), 0), idS, leader);
            commit_by(&bars.s_full, leader);
            chain_ss<D>(tP + (j & 1) * kTile, desc_k(sG, 0), desc_k(sbase + stage_of<D>(2 * j + 1), 0), idS, leader);
            commit_by(&bars.dp_full[j & 1], leader);
            commit_by(&bars.empty[stage_no<D>(2 * j + 1)], leader);
        };
        if (total > 0) {
            ok = warp_wait(&bars.own_full, 0, abort) && warp_wait(&bars.first, 0, abort);
            if (ok) scores(0);
        }
        for (int j = 0; j < total && ok; ++j) {
            const bool more = j + 1 < total;
            if (more) {   // the next scores as soon as these have been read; dP alternates between two places
                if (!(ok = warp_wait(&bars.a_ready, j & 1, abort))) break;
                tc::tc_fence_after();
                scores(j + 1);
            }
            if (!(ok = warp_wait(&bars.b_ready, j & 1, abort))) break;
            tc::tc_fence_after();
            chain_ts32(tQ, tP + (j & 1) * kTile, desc_mn(sbase + stage_of<D>(2 * j), 0), idG, j > 0, leader);
            commit_by(more ? &bars.empty[stage_no<D>(2 * j)] : &bars.done, leader);
        }
        if (!ok) {   // no product in flight when the memory is given back
            int quit = 0;
            commit_by(&bars.drain, leader);
            warp_wait(&bars.drain, 0, &quit);
        }
    } else if (warp < 16) {
        const int part = warp >> 2, row = (warp & 3) * 32 + lane, r = r0 + row;
        const uint32_t lanes = tc::tmem_lane_base(warp) + part * 32;
        const float sc = a.scale * kLog2e;
        const int seen = r < s.nq ? keys_seen(s, r, a.causal) : 0;
        const int first_row = r0 + (warp & 3) * 32;
        const int seen_all = first_row + 31 < s.nq ? keys_seen(s, first_row, a.causal) : 0;   // by every row of the warp
        float ls = -CUDART_INF_F;
        const int64_t at = r < s.nq ? stat_at(a.bt, s.q0 + r, h) : 0;
        if (r < s.nq) {
            ls = a.lse[at] * kLog2e;
            if (ls != -CUDART_INF_F) ls = -ls;
        }
        bool ok = warp_wait(&bars.own_full, 0, abort) && warp_wait(&bars.out_full, 0, abort);
        float de = 0.f;
        if (ok) {   // delta = dO . O of this row, the same in all four groups
            const uint8_t *g = smem + C::kOwn + C::kTileBytes, *o = smem + C::kOut;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint32_t off = (c >> 3) * (kTile * 128) + tc::sw128(row, c & 7);
                const uint4 x = *reinterpret_cast<const uint4 *>(g + off), y = *reinterpret_cast<const uint4 *>(o + off);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    de = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), de);
                    de = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), de);
                }
            }
            if (part == 0 && r < s.nq) a.delta[at] = de;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars.out_read);
        }
        const float2 sc2 = make_float2(sc, sc), ls2 = make_float2(ls, ls), de2 = make_float2(-de, -de);
        for (int j = 0; j < total && ok; ++j) {
            const uint32_t dp = tP + (j & 1) * kTile + lanes;
            const int limit = seen - j * kTile - part * 32;   // columns at or past it are hidden
            const bool partly = j * kTile + (part + 1) * 32 > seen_all;
            if (!(ok = warp_wait(&bars.s_full, j & 1, abort))) break;
            tc::tc_fence_after();
            float2 p[16];
            {
                float x[32];
                tc::tmem_ld32(tS + lanes, x);
                tc::tmem_ld_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars.a_ready);
#pragma unroll
                for (int e = 0; e < 16; ++e) p[e] = fma2(make_float2(x[2 * e], x[2 * e + 1]), sc2, ls2);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = make_float2(ex2_approx(p[e].x), ex2_approx(p[e].y));
            if (!(ok = warp_wait(&bars.dp_full[j & 1], (j >> 1) & 1, abort))) break;
            tc::tc_fence_after();
            {
                float x[32];
                tc::tmem_ld32(dp, x);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) p[e] = mul2(p[e], add2(make_float2(x[2 * e], x[2 * e + 1]), de2));
            }
            if (partly) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (2 * e >= limit) p[e].x = 0.f;
                    if (2 * e + 1 >= limit) p[e].y = 0.f;
                }
            }
            put_operand(dp, p);
            arrive_operand(&bars.b_ready, lane);
        }
        if (ok && total > 0) ok = warp_wait(&bars.done, 0, abort);
        if (ok && part == 0) {
            tc::tc_fence_after();
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.dq) + ((s.q0 + first_row) * a.bt.Hq + h) * D;
            store_rows<D>(tQ + lanes, smem + C::kOwn + (warp & 3) * 32 * D * 2, lane, dst, (int64_t)a.bt.Hq * D,
                          s.nq - first_row, a.scale, total == 0);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D> cudaError_t launch_prompt_grad_tc(const PromptArgs &a, cudaStream_t st) {
    using C = GradCfg<D>;
    cudaError_t e;
    const int64_t gk = a.bt.Tk == 0 ? 0 : max_tiles(a.bt.cu_k, a.bt.n, a.bt.Tk, kTile) * a.bt.Hkv;
    const int64_t gq = a.bt.Tq == 0 ? 0 : max_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq, kTile) * a.bt.Hq;
    if (gk > 0x7fffffff || gq > 0x7fffffff) return cudaErrorInvalidValue;
    // before the maps: it binds the device's context to this thread (autograd's may have none yet), which
    // their encoding needs
    if ((e = allow_smem(attn_grad_q_tc_kernel<D>, C::kSmem)) != cudaSuccess) return e;
    PromptMaps maps = {};
    if (a.bt.Tq > 0 && !encode_prompt_maps(maps, a, D)) return cudaErrorInvalidValue;
    if (gq > 0) {   // first: it forms the delta that the other reads
        if ((e = launch_behind(attn_grad_q_tc_kernel<D>, (unsigned)gq, C::kThreads, C::kSmem, st, a, maps)) != cudaSuccess)
            return e;
    }
    if (gk > 0) {
        if ((e = allow_smem(attn_grad_kv_tc_kernel<D>, C::kSmem)) != cudaSuccess) return e;
        return launch_behind(attn_grad_kv_tc_kernel<D>, (unsigned)gk, C::kThreads, C::kSmem, st, a, maps);
    }
    return cudaSuccess;
}

}  // namespace attn
}  // namespace kda
