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
// Warp roles: 0-7 compute (thread = row, the warpgroups take 64 columns each), 8 issues the products, 9
// loads (TMA, and the queries' lse and delta).  P and dS are rounded once, to bf16, as operands.
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
    static constexpr int kStages = D == 128 ? 2 : 4;      // of two tiles each
    static constexpr int kOwn = 0;                        // the block's own two tiles
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kStats = kRing + kStages * 2 * kTileBytes;   // lse and delta of a stage's queries
    static constexpr int kBars = kStats + kStages * 2 * kTile * 4;
    static constexpr int kSmem = kBars + 512 + 1024;
    static constexpr int kThreads = 320;
};

struct GradBars {
    uint64_t own_full, full[4], empty[4], stats[4], s_full, dp_full[2], a_ready, b_ready, done, drain;
    uint32_t tmem;
    int abort;
    int scratch[34];
};

// Barriers and Tensor Memory; every thread.  Returns the Tensor Memory's base.
template <int D> __device__ __forceinline__ uint32_t grad_setup(GradBars &bars) {
    using C = GradCfg<D>;
    if (threadIdx.x == 0) {
        bars.abort = 0;
        tc::mbar_init(&bars.own_full, 1);
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(&bars.full[i], 1);
            tc::mbar_init(&bars.empty[i], 1);
            tc::mbar_init(&bars.stats[i], 1);
        }
        tc::mbar_init(&bars.s_full, 1);
        tc::mbar_init(&bars.dp_full[0], 1);
        tc::mbar_init(&bars.dp_full[1], 1);
        tc::mbar_init(&bars.a_ready, 8);
        tc::mbar_init(&bars.b_ready, 8);
        tc::mbar_init(&bars.done, 1);
        tc::mbar_init(&bars.drain, 1);
        tc::fence_mbar_init();
    }
    if (threadIdx.x >> 5 == 8) {
        tc::tmem_alloc(&bars.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    return bars.tmem;
}

// After a wait that ran out: waits for the loads of the last `stages` puts, so that none is in flight.
template <int D> __device__ __forceinline__ void drain_loads(GradBars &bars, int put) {
    using C = GradCfg<D>;
    int quit = 0;
    tc::mbar_wait(&bars.own_full, 0, &quit);
    for (int k = put > C::kStages ? put - C::kStages : 0; k < put; ++k) {
        quit = 0;
        tc::mbar_wait(&bars.full[k % C::kStages], (k / C::kStages) & 1, &quit);
    }
}

__device__ __forceinline__ void drain_products(GradBars &bars) {
    int quit = 0;
    tc::mma_commit(&bars.drain);
    tc::mbar_wait(&bars.drain, 0, &quit);
}

// 32 weights or score gradients of a thread's row, rounded, into Tensor Memory.
__device__ __forceinline__ void put_operand(uint32_t taddr, const float (&x)[32]) {
    uint32_t u[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) u[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
    tc::tmem_st16(taddr, u);
}

__device__ __forceinline__ void arrive_operand(uint64_t *bar, int lane) {
    tc::tmem_st_wait();
    tc::tc_fence_before();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
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
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
    GradBars &bars = *reinterpret_cast<GradBars *>(smem + C::kBars);
    const uint32_t sbase = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // the first keys of a sequence are seen by the most queries: they go first
    int n, t;
    if (!find_tile(a.bt.cu_k, a.bt.n, a.bt.Tk, kTile, blockIdx.x / a.bt.Hkv, bars.scratch, n, t)) return;
    const Seq s = seq_of(a.bt, n);
    const int hk = blockIdx.x % a.bt.Hkv, c0 = t * kTile, group = a.bt.Hq / a.bt.Hkv;
    const int ahead = s.nk - s.nq;   // causal: query i sees keys j <= i + ahead
    const int start = a.causal ? max(0, c0 - ahead) / kTile : 0;
    const int per_head = max(0, (s.nq + kTile - 1) / kTile - start), total = per_head * group;

    const uint32_t tmem = grad_setup<D>(bars);
    volatile int *abort = &bars.abort;
    const uint32_t tS = tmem, tP = tmem + kTile, tV = tmem + 2 * kTile, tK = tV + D;
    float *stats = reinterpret_cast<float *>(smem + C::kStats);

    if (warp == 9) {
        if (total > 0) {
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&bars.own_full, 2 * C::kTileBytes);
                tma_tile<D>(C::kOwn, smem, &maps.k, hk, s.k0 + c0, &bars.own_full);
                tma_tile<D>(C::kOwn + C::kTileBytes, smem, &maps.v, hk, s.k0 + c0, &bars.own_full);
            }
            bool ok = true;
            int put = 0;
            for (int it = 0; it < total; ++it) {
                const int st = it % C::kStages, h = hk * group + it / per_head, r0 = (start + it % per_head) * kTile;
                // lse in log2 units, +inf (weight zero) where there is no query or it sees nothing
                float ls[4], de[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = r0 + e * 32 + lane;
                    ls[e] = CUDART_INF_F;
                    de[e] = 0.f;
                    if (r < s.nq) {
                        const int64_t at = stat_at(a.bt, s.q0 + r, h);
                        const float x = a.lse[at] * kLog2e;
                        ls[e] = x == -CUDART_INF_F ? CUDART_INF_F : x;
                        de[e] = a.delta[at];
                    }
                }
                if (it >= C::kStages) ok = warp_wait(&bars.empty[st], (it / C::kStages - 1) & 1, abort);
                if (!ok) break;
                if (lane == 0) {
                    const uint32_t at = C::kRing + st * 2 * C::kTileBytes;
                    tc::mbar_arrive_expect_tx(&bars.full[st], 2 * C::kTileBytes);
                    tma_tile<D>(at, smem, &maps.q, h, s.q0 + r0, &bars.full[st]);
                    tma_tile<D>(at + C::kTileBytes, smem, &maps.g, h, s.q0 + r0, &bars.full[st]);
                }
                ++put;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    stats[st * 2 * kTile + e * 32 + lane] = ls[e];
                    stats[st * 2 * kTile + kTile + e * 32 + lane] = de[e];
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars.stats[st]);
            }
            if (!ok && lane == 0) drain_loads<D>(bars, put);
        }
    } else if (warp == 8) {
        constexpr uint32_t idS = tc::make_idesc_bf16(kTile, kTile, false, false);
        constexpr uint32_t idG = tc::make_idesc_bf16(kTile, D, false, true);
        bool ok = true;
        auto load_ready = [&](int it) {
            const int st = it % C::kStages;
            if (!warp_wait(&bars.full[st], (it / C::kStages) & 1, abort)) return false;
            const int left = s.nq - (start + it % per_head) * kTile;
            if (left < kTile) {   // queries that are not there are summed over with weight zero
                zero_rows<D>(smem + C::kRing + st * 2 * C::kTileBytes, left, lane);
                zero_rows<D>(smem + C::kRing + st * 2 * C::kTileBytes + C::kTileBytes, left, lane);
                __syncwarp();
            }
            return true;
        };
        auto product = [&](uint32_t d, uint32_t x, uint32_t y, uint64_t *bar) {   // d = x y^T
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) tc::mma_f16(d, desc_k(x, kk), desc_k(y, kk), idS, kk > 0);
            tc::mma_commit(bar);
        };
        const uint32_t sK = sbase + C::kOwn, sV = sK + C::kTileBytes;
        if (total > 0) {
            ok = warp_wait(&bars.own_full, 0, abort) && load_ready(0);
            if (ok && lane == 0) {
                product(tS, sK, sbase + C::kRing, &bars.s_full);
                product(tP, sV, sbase + C::kRing + C::kTileBytes, &bars.dp_full[0]);
            }
        }
        for (int it = 0; it < total && ok; ++it) {
            const uint32_t q = sbase + C::kRing + (it % C::kStages) * 2 * C::kTileBytes, g = q + C::kTileBytes;
            const uint32_t qn = sbase + C::kRing + ((it + 1) % C::kStages) * 2 * C::kTileBytes;
            const bool more = it + 1 < total;
            if (more && !(ok = load_ready(it + 1))) break;
            if (!(ok = warp_wait(&bars.a_ready, it & 1, abort))) break;
            tc::tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    tc::mma_f16_ta(tV, tS + operand_col(kk), desc_mn(g, kk), idG, it > 0 || kk > 0);
                if (more) product(tS, sK, qn, &bars.s_full);
            }
            if (!(ok = warp_wait(&bars.b_ready, it & 1, abort))) break;
            tc::tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    tc::mma_f16_ta(tK, tP + operand_col(kk), desc_mn(q, kk), idG, it > 0 || kk > 0);
                tc::mma_commit(more ? &bars.empty[it % C::kStages] : &bars.done);
                if (more) product(tP, sV, qn + C::kTileBytes, &bars.dp_full[0]);
            }
        }
        if (!ok && lane == 0) drain_products(bars);
        __syncwarp();
    } else {
        const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tc::tmem_lane_base(warp);
        const float sc = a.scale * kLog2e;
        bool ok = true;
        for (int it = 0; it < total; ++it) {
            const int st = it % C::kStages, r0 = (start + it % per_head) * kTile;
            const float *ls = stats + st * 2 * kTile + wg * 64, *de = ls + kTile;
            // this row's key is seen by the tile's queries from column `from` on
            const int from = a.causal ? c0 + row - ahead - r0 - wg * 64 : 0;
            const bool partly = a.causal && c0 + (warp & 3) * 32 + 31 - ahead - r0 - wg * 64 > 0;
            ok = warp_wait(&bars.stats[st], (it / C::kStages) & 1, abort) && warp_wait(&bars.s_full, it & 1, abort);
            if (!ok) break;
            tc::tc_fence_after();
            float p[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::tmem_ld32(tS + lanes + wg * 64 + c * 32, p[c]);
            tc::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 l4 = *reinterpret_cast<const float4 *>(ls + c * 32 + e);
                    p[c][e] = ex2_approx(fmaf(p[c][e], sc, -l4.x));
                    p[c][e + 1] = ex2_approx(fmaf(p[c][e + 1], sc, -l4.y));
                    p[c][e + 2] = ex2_approx(fmaf(p[c][e + 2], sc, -l4.z));
                    p[c][e + 3] = ex2_approx(fmaf(p[c][e + 3], sc, -l4.w));
                }
                if (partly) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e < from) p[c][e] = 0.f;
                }
                put_operand(tS + lanes + wg * 64 + c * 16, p[c]);
            }
            arrive_operand(&bars.a_ready, lane);
            ok = warp_wait(&bars.dp_full[0], it & 1, abort);
            if (!ok) break;
            tc::tc_fence_after();
            float x[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::tmem_ld32(tP + lanes + wg * 64 + c * 32, x[c]);
            tc::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 d4 = *reinterpret_cast<const float4 *>(de + c * 32 + e);
                    x[c][e] = p[c][e] * (x[c][e] - d4.x);
                    x[c][e + 1] = p[c][e + 1] * (x[c][e + 1] - d4.y);
                    x[c][e + 2] = p[c][e + 2] * (x[c][e + 2] - d4.z);
                    x[c][e + 3] = p[c][e + 3] * (x[c][e + 3] - d4.w);
                }
                if (partly) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e < from) x[c][e] = 0.f;
                }
                put_operand(tP + lanes + wg * 64 + c * 16, x[c]);
            }
            arrive_operand(&bars.b_ready, lane);
        }
        if (ok && total > 0) ok = warp_wait(&bars.done, 0, abort);
        if (ok) {
            tc::tc_fence_after();
            // one warpgroup writes dV, the other dK, through the tiles of K and V, which are done with
            const int r0 = c0 + (warp & 3) * 32;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(wg ? a.dk : a.dv) + ((s.k0 + r0) * a.bt.Hkv + hk) * D;
            store_rows<D>((wg ? tK : tV) + lanes, smem + C::kOwn + wg * C::kTileBytes + (warp & 3) * 32 * D * 2, lane,
                          dst, (int64_t)a.bt.Hkv * D, s.nk - r0, wg ? a.scale : 1.f, total == 0);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ---- dQ -----------------------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(GradCfg<D>::kThreads, 1)
attn_grad_q_tc_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ PromptMaps maps) {
    using C = GradCfg<D>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
    GradBars &bars = *reinterpret_cast<GradBars *>(smem + C::kBars);
    const uint32_t sbase = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int64_t tiles = gridDim.x / a.bt.Hq;
    int n, t;
    if (!find_tile(a.bt.cu_q, a.bt.n, a.bt.Tq, kTile, tiles - 1 - blockIdx.x / a.bt.Hq, bars.scratch, n, t)) return;
    const Seq s = seq_of(a.bt, n);
    const int h = blockIdx.x % a.bt.Hq, hk = h / (a.bt.Hq / a.bt.Hkv), r0 = t * kTile;
    const int total = (keys_seen(s, min(r0 + kTile, s.nq) - 1, a.causal) + kTile - 1) / kTile;

    const uint32_t tmem = grad_setup<D>(bars);
    volatile int *abort = &bars.abort;
    const uint32_t tS = tmem, tP = tmem + kTile, tQ = tmem + 3 * kTile;

    if (warp == 9) {
        if (lane == 0 && total > 0) {
            tc::mbar_arrive_expect_tx(&bars.own_full, 2 * C::kTileBytes);
            tma_tile<D>(C::kOwn, smem, &maps.q, h, s.q0 + r0, &bars.own_full);
            tma_tile<D>(C::kOwn + C::kTileBytes, smem, &maps.g, h, s.q0 + r0, &bars.own_full);
            bool ok = true;
            int put = 0;
            for (int j = 0; j < total; ++j) {
                const int st = j % C::kStages;
                if (j >= C::kStages) ok = tc::mbar_wait(&bars.empty[st], (j / C::kStages - 1) & 1, abort);
                if (!ok) break;
                const uint32_t at = C::kRing + st * 2 * C::kTileBytes;
                tc::mbar_arrive_expect_tx(&bars.full[st], 2 * C::kTileBytes);
                tma_tile<D>(at, smem, &maps.k, hk, s.k0 + (int64_t)j * kTile, &bars.full[st]);
                tma_tile<D>(at + C::kTileBytes, smem, &maps.v, hk, s.k0 + (int64_t)j * kTile, &bars.full[st]);
                ++put;
            }
            if (!ok) drain_loads<D>(bars, put);
        }
    } else if (warp == 8) {
        constexpr uint32_t idS = tc::make_idesc_bf16(kTile, kTile, false, false);
        constexpr uint32_t idG = tc::make_idesc_bf16(kTile, D, false, true);
        bool ok = true;
        auto load_ready = [&](int j) {
            const int st = j % C::kStages;
            if (!warp_wait(&bars.full[st], (j / C::kStages) & 1, abort)) return false;
            const int left = s.nk - j * kTile;
            if (left < kTile) {   // keys that are not there are summed over with weight zero
                zero_rows<D>(smem + C::kRing + st * 2 * C::kTileBytes, left, lane);
                __syncwarp();
            }
            return true;
        };
        auto product = [&](uint32_t d, uint32_t x, uint32_t y, uint64_t *bar) {   // d = x y^T
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) tc::mma_f16(d, desc_k(x, kk), desc_k(y, kk), idS, kk > 0);
            tc::mma_commit(bar);
        };
        const uint32_t sQ = sbase + C::kOwn, sG = sQ + C::kTileBytes;
        if (total > 0) {
            ok = warp_wait(&bars.own_full, 0, abort) && load_ready(0);
            if (ok && lane == 0) {
                product(tS, sQ, sbase + C::kRing, &bars.s_full);
                product(tP, sG, sbase + C::kRing + C::kTileBytes, &bars.dp_full[0]);
            }
        }
        for (int j = 0; j < total && ok; ++j) {
            const uint32_t k = sbase + C::kRing + (j % C::kStages) * 2 * C::kTileBytes;
            const uint32_t kn = sbase + C::kRing + ((j + 1) % C::kStages) * 2 * C::kTileBytes;
            const bool more = j + 1 < total;
            if (more) {
                // the next scores as soon as these have been read; dP alternates between two places
                if (!(ok = load_ready(j + 1))) break;
                if (!(ok = warp_wait(&bars.a_ready, j & 1, abort))) break;
                tc::tc_fence_after();
                if (lane == 0) {
                    product(tS, sQ, kn, &bars.s_full);
                    product(tP + ((j + 1) & 1) * kTile, sG, kn + C::kTileBytes, &bars.dp_full[(j + 1) & 1]);
                }
            }
            if (!(ok = warp_wait(&bars.b_ready, j & 1, abort))) break;
            tc::tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    tc::mma_f16_ta(tQ, tP + (j & 1) * kTile + operand_col(kk), desc_mn(k, kk), idG, j > 0 || kk > 0);
                tc::mma_commit(more ? &bars.empty[j % C::kStages] : &bars.done);
            }
        }
        if (!ok && lane == 0) drain_products(bars);
        __syncwarp();
    } else {
        const int wg = warp >> 2, row = (warp & 3) * 32 + lane, r = r0 + row;
        const uint32_t lanes = tc::tmem_lane_base(warp);
        const float sc = a.scale * kLog2e;
        const int seen = r < s.nq ? keys_seen(s, r, a.causal) : 0;
        const int first_row = r0 + (warp & 3) * 32;
        const int seen_all = first_row + 31 < s.nq ? keys_seen(s, first_row, a.causal) : 0;   // by every row of the warp
        float ls = CUDART_INF_F, de = 0.f;
        if (r < s.nq) {
            const int64_t at = stat_at(a.bt, s.q0 + r, h);
            ls = a.lse[at] * kLog2e;
            if (ls == -CUDART_INF_F) ls = CUDART_INF_F;
            de = a.delta[at];
        }
        bool ok = true;
        for (int j = 0; j < total; ++j) {
            const uint32_t dp = tP + (j & 1) * kTile + lanes + wg * 64;
            const int limit = seen - j * kTile - wg * 64;   // columns at or past it are hidden
            const bool partly = j * kTile + kTile > seen_all;
            ok = warp_wait(&bars.s_full, j & 1, abort);
            if (!ok) break;
            tc::tc_fence_after();
            float p[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::tmem_ld32(tS + lanes + wg * 64 + c * 32, p[c]);
            tc::tmem_ld_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars.a_ready);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e) p[c][e] = ex2_approx(fmaf(p[c][e], sc, -ls));
            ok = warp_wait(&bars.dp_full[j & 1], (j >> 1) & 1, abort);
            if (!ok) break;
            tc::tc_fence_after();
            float x[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::tmem_ld32(dp + c * 32, x[c]);
            tc::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[c][e] = p[c][e] * (x[c][e] - de);
                if (partly) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e >= limit) x[c][e] = 0.f;
                }
                put_operand(dp + c * 16, x[c]);
            }
            arrive_operand(&bars.b_ready, lane);
        }
        if (ok && total > 0) ok = warp_wait(&bars.done, 0, abort);
        if (ok && wg == 0) {
            tc::tc_fence_after();
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.dq) + ((s.q0 + first_row) * a.bt.Hq + h) * D;
            store_rows<D>(tQ + lanes, smem + C::kOwn + (warp & 3) * 32 * D * 2, lane, dst, (int64_t)a.bt.Hq * D,
                          s.nq - first_row, a.scale, total == 0);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D> cudaError_t launch_prompt_grad_tc(const PromptArgs &a, cudaStream_t st) {
    using C = GradCfg<D>;
    cudaError_t e = launch_delta<__nv_bfloat16, D>(a, st);
    if (e != cudaSuccess) return e;
    const int64_t gk = a.bt.Tk == 0 ? 0 : max_tiles(a.bt.cu_k, a.bt.n, a.bt.Tk, kTile) * a.bt.Hkv;
    const int64_t gq = a.bt.Tq == 0 ? 0 : max_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq, kTile) * a.bt.Hq;
    if (gk > 0x7fffffff || gq > 0x7fffffff) return cudaErrorInvalidValue;
    PromptMaps maps = {};
    if (a.bt.Tq > 0 && !encode_prompt_maps(maps, a, D)) return cudaErrorInvalidValue;
    if (gk > 0) {
        if ((e = allow_smem(attn_grad_kv_tc_kernel<D>, C::kSmem)) != cudaSuccess) return e;
        attn_grad_kv_tc_kernel<D><<<(unsigned)gk, C::kThreads, C::kSmem, st>>>(a, maps);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (gq > 0) {
        if ((e = allow_smem(attn_grad_q_tc_kernel<D>, C::kSmem)) != cudaSuccess) return e;
        attn_grad_q_tc_kernel<D><<<(unsigned)gq, C::kThreads, C::kSmem, st>>>(a, maps);
    }
    return cudaGetLastError();
}

}  // namespace attn
}  // namespace kda
