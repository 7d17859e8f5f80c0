// attn_prompt_tc.cuh -- attention over whole prompts on the tensor cores (bf16 inputs).
//
//     S = Q K^T,   P = 2^(c S - c m),   O = P V / rowsum(P),   c = scale log2(e),
// one pass over the keys in tiles of 128 with a running row maximum m and sum.
//
// A block works on two tiles of 128 queries that share their keys and values: two heads of a group
// (the same rows) where the group is even, two neighbouring row tiles of one head otherwise.  Both
// products run on tcgen05 with fp32 accumulators in Tensor Memory: S (128 x 128) per tile, O (128 x d)
// per tile.  Warp roles:
//   warps 0-3, 4-7  softmax of tile 0 and 1: thread = row.  They read S, write P (bf16) over it as the
//                   second product's A operand, and hold m and the sum in registers.
//   warp 8          issues the products:  O_i += P_i V_j, then S_i = Q_i K_{j+1}, for i = 0, 1 in turn,
//                   so one tile's softmax runs under the other tile's products.
//   warp 9          TMA loads: Q once, then K_j, V_j through a ring of stages.
// m is allowed to lag: while a row's new maximum exceeds the m in use by less than 2^8 the weights are
// only scaled differently (up to 2^8, exact in fp32 and no less precise in bf16), so O is rescaled
// rarely, by the softmax warps themselves: S_i of a tile is issued after the previous O_i, and the
// tensor pipe works in order, so a complete S_i means a complete O_i.  P is rounded once, to bf16, the
// operand type of V; the sum takes the unrounded weights.
//
// Rows past the end of a sequence in its last tile are another sequence's (or whatever lies behind):
// their scores are masked, and their values are zeroed in shared memory before the product, since a
// weight of zero does not hide a NaN.
#pragma once

#include <cuda.h>

#include "attn_prompt.cuh"
#include "kda_chunk_tc.cuh"
#include "tc_utils.cuh"

namespace kda {
namespace attn {

constexpr int kTile = 128;   // queries of a tile, keys of a tile

// ---- helpers shared with the gradient -----------------------------------------------------------

// K-major operand: [rows x 64-column SW128 blocks]; k-step kk of 16 columns.
__device__ __forceinline__ uint64_t desc_k(uint32_t base, int kk) {
    return tc::make_sdesc(base + (kk >> 2) * (kTile * 128) + (kk & 3) * 32, 16, 1024, tc::kSwz128);
}
// The same bytes as an MN-major operand: K runs over the 128 rows, MN over the columns.
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, int kk) {
    return tc::make_sdesc(base + kk * 2048, kTile * 128, 1024, tc::kSwz128);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
          "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

// A whole warp's wait: one answer for all lanes, so that they leave loops together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort));
}

// A head's tile of 128 tokens in 64-column blocks.
template <int D>
__device__ __forceinline__ void tma_tile(uint32_t dst, uint8_t *smem, const CUtensorMap *map, int head, int64_t row,
                                         uint64_t *bar) {
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
        tc::tma_load_3d(smem + dst + b * (kTile * 128), map, b * 64, head, (int)row, bar);
}

// Zeroes rows [from, 128) of a staged tile; a whole warp.
template <int D> __device__ __forceinline__ void zero_rows(uint8_t *tile, int from, int lane) {
    for (int i = from * 8 + lane; i < kTile * 8; i += 32)
#pragma unroll
        for (int b = 0; b < D / 64; ++b) reinterpret_cast<uint4 *>(tile + b * (kTile * 128))[i] = make_uint4(0, 0, 0, 0);
    tc::fence_async_smem();
}

// A warp's 32 rows of D values (thread = row, columns [32 c, 32 c + 32) at a time) to global memory
// through its own shared memory, so that a row is written in whole 16-byte pieces side by side.
template <int D> struct RowWriter {
    static constexpr int CH = D * 2 / 16;
    uint8_t *smem;
    __device__ __forceinline__ void put(int lane, int c, const float (&x)[32], float mul) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint4 u;
            u.x = pack_bf16(x[8 * e] * mul, x[8 * e + 1] * mul);
            u.y = pack_bf16(x[8 * e + 2] * mul, x[8 * e + 3] * mul);
            u.z = pack_bf16(x[8 * e + 4] * mul, x[8 * e + 5] * mul);
            u.w = pack_bf16(x[8 * e + 6] * mul, x[8 * e + 7] * mul);
            const int ch = c * 4 + e;
            *reinterpret_cast<uint4 *>(smem + lane * (CH * 16) + ((ch ^ (lane & 7)) << 4)) = u;
        }
    }
    // row r of the warp to dst + r * stride, for r < rows
    __device__ __forceinline__ void flush(int lane, __nv_bfloat16 *dst, int64_t stride, int rows) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int r = (i * 32 + lane) / CH, ch = (i * 32 + lane) % CH;
            const uint4 u = *reinterpret_cast<const uint4 *>(smem + r * (CH * 16) + ((ch ^ (r & 7)) << 4));
            if (r < rows) *reinterpret_cast<uint4 *>(dst + r * stride + ch * 8) = u;
        }
        __syncwarp();
    }
};

// ---- forward ------------------------------------------------------------------------------------

struct PromptMaps {
    CUtensorMap q, k, v, g;   // g: d_out (gradient only)
};

template <int D> struct FwdCfg {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kQ = 0;                          // two query tiles
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kBars = kRing + kStages * kTileBytes;
    static constexpr int kSmem = kBars + 512 + 1024;      // + alignment of the base
    static constexpr int kThreads = 320;
};

struct FwdBars {
    uint64_t q_full[2], full[8], empty[8], s_full[2], p_ready[2], o_full[2], drain;
    uint32_t tmem;
    int abort;
    int scratch[34];
};

// Which two tiles of queries a block has.
struct TwoTiles {
    Seq s;
    int head[2], r0[2], blocks[2];   // head, first row, tiles of keys that it sees
    int hk;
};

template <int D>
__global__ void __launch_bounds__(FwdCfg<D>::kThreads, 1)
attn_prompt_tc_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ PromptMaps maps, int pair_heads) {
    using C = FwdCfg<D>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
    FwdBars &bars = *reinterpret_cast<FwdBars *>(smem + C::kBars);
    const uint32_t sbase = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // the last tiles of a sequence have the most keys: they go first
    const int units = pair_heads ? a.bt.Hq / 2 : a.bt.Hq;
    const int rows = pair_heads ? kTile : 2 * kTile;
    const int64_t tiles = gridDim.x / units;
    int n, t;
    if (!find_tile(a.bt.cu_q, a.bt.n, a.bt.Tq, rows, tiles - 1 - blockIdx.x / units, bars.scratch, n, t)) return;
    TwoTiles w;
    w.s = seq_of(a.bt, n);
    {
        const int u = blockIdx.x % units;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            w.head[i] = pair_heads ? 2 * u + i : u;
            w.r0[i] = t * rows + (pair_heads ? 0 : i * kTile);
            const int last = min(w.r0[i] + kTile, w.s.nq) - 1;
            w.blocks[i] = w.r0[i] < w.s.nq ? (keys_seen(w.s, last, a.causal) + kTile - 1) / kTile : 0;
        }
        w.hk = w.head[0] / (a.bt.Hq / a.bt.Hkv);
    }
    const int blocks = max(w.blocks[0], w.blocks[1]);

    if (tid == 0) {
        bars.abort = 0;
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars.q_full[i], 1);
            tc::mbar_init(&bars.s_full[i], 1);
            tc::mbar_init(&bars.p_ready[i], 4);
            tc::mbar_init(&bars.o_full[i], 1);
        }
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(&bars.full[i], 1);
            tc::mbar_init(&bars.empty[i], 1);
        }
        tc::mbar_init(&bars.drain, 1);
        tc::fence_mbar_init();
    }
    if (warp == 8) {
        tc::tmem_alloc(&bars.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = bars.tmem;
    volatile int *abort = &bars.abort;
    constexpr uint32_t kO = 256;

    if (warp == 9) {
        if (lane == 0 && blocks > 0) {
            for (int i = 0; i < 2; ++i) {
                if (w.blocks[i] == 0) continue;
                tc::mbar_arrive_expect_tx(&bars.q_full[i], C::kTileBytes);
                tma_tile<D>(C::kQ + i * C::kTileBytes, smem, &maps.q, w.head[i], w.s.q0 + w.r0[i], &bars.q_full[i]);
            }
            int st = 0, put = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int j = 0; j < 2 * blocks && ok; ++j) {   // K_0, V_0, K_1, ...
                if (put >= C::kStages) ok = tc::mbar_wait(&bars.empty[st], ph ^ 1, abort);
                if (!ok) break;
                tc::mbar_arrive_expect_tx(&bars.full[st], C::kTileBytes);
                tma_tile<D>(C::kRing + st * C::kTileBytes, smem, j & 1 ? &maps.v : &maps.k, w.hk,
                            w.s.k0 + (int64_t)(j >> 1) * kTile, &bars.full[st]);
                ++put;
                if (++st == C::kStages) st = 0, ph ^= 1;
            }
            if (!ok) {   // a wait ran out: leave no copy in flight
                int quit = 0;
                for (int i = 0; i < 2; ++i)
                    if (w.blocks[i]) tc::mbar_wait(&bars.q_full[i], 0, &quit);
                const int from = put > C::kStages ? put - C::kStages : 0;
                for (int k = from; k < put; ++k) {
                    quit = 0;
                    tc::mbar_wait(&bars.full[k % C::kStages], (k / C::kStages) & 1, &quit);
                }
            }
        }
    } else if (warp == 8) {
        constexpr uint32_t idS = tc::make_idesc_bf16(kTile, kTile, false, false);
        constexpr uint32_t idO = tc::make_idesc_bf16(kTile, D, false, true);
        bool ok = true;
        int st = 0;
        uint32_t ph = 0;
        auto scores = [&](int i, uint32_t ks) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                tc::mma_f16(tmem + i * kTile, desc_k(sbase + C::kQ + i * C::kTileBytes, kk), desc_k(ks, kk), idS, kk > 0);
            tc::mma_commit(&bars.s_full[i]);
        };
        if (blocks > 0) {
            ok = warp_wait(&bars.full[0], 0, abort);
            for (int i = 0; i < 2 && ok; ++i) {
                if (w.blocks[i] == 0) continue;
                ok = warp_wait(&bars.q_full[i], 0, abort);
                if (ok && lane == 0) scores(i, sbase + C::kRing);
            }
            if (ok && lane == 0) tc::mma_commit(&bars.empty[0]);
            st = 1;
        }
        for (int j = 0; j < blocks && ok; ++j) {
            const int vst = st;
            ok = warp_wait(&bars.full[vst], ph, abort);
            if (!ok) break;
            if (++st == C::kStages) st = 0, ph ^= 1;
            const int left = w.s.nk - j * kTile;
            if (left < kTile) {
                zero_rows<D>(smem + C::kRing + vst * C::kTileBytes, left, lane);
                __syncwarp();
            }
            const int kst = st;
            bool have_k = false;
            for (int i = 0; i < 2 && ok; ++i) {
                if (j >= w.blocks[i]) continue;
                ok = warp_wait(&bars.p_ready[i], j & 1, abort);
                if (!ok) break;
                tc::tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        tc::mma_f16_ta(tmem + kO + i * D, tmem + i * kTile + kk * 8,
                                       desc_mn(sbase + C::kRing + vst * C::kTileBytes, kk), idO, j > 0 || kk > 0);
                }
                if (j + 1 < w.blocks[i]) {
                    if (!have_k) {
                        ok = warp_wait(&bars.full[kst], ph, abort);
                        if (!ok) break;
                        have_k = true;
                    }
                    if (lane == 0) scores(i, sbase + C::kRing + kst * C::kTileBytes);
                } else if (lane == 0) {
                    tc::mma_commit(&bars.o_full[i]);
                }
            }
            if (!ok) break;
            if (lane == 0) {
                tc::mma_commit(&bars.empty[vst]);
                if (have_k) tc::mma_commit(&bars.empty[kst]);
            }
            if (j + 1 < blocks && ++st == C::kStages) st = 0, ph ^= 1;
        }
        if (!ok && lane == 0) {   // no product in flight when the memory is given back
            int quit = 0;
            tc::mma_commit(&bars.drain);
            tc::mbar_wait(&bars.drain, 0, &quit);
        }
        __syncwarp();
    } else {
        const int i = warp >> 2, row = (warp & 3) * 32 + lane, r = w.r0[i] + row;
        const uint32_t lanes = tc::tmem_lane_base(warp), tS = tmem + i * kTile + lanes, tO = tmem + kO + i * D + lanes;
        const int seen = r < w.s.nq ? keys_seen(w.s, r, a.causal) : w.s.nk;
        const int seen_all = keys_seen(w.s, min(w.r0[i] + (warp & 3) * 32, w.s.nq - 1), a.causal);   // by every row of the warp
        const float sc = a.scale * kLog2e;
        float m = -CUDART_INF_F, l = 0.f;
        bool ok = true;
        for (int j = 0; j < w.blocks[i]; ++j) {
            ok = warp_wait(&bars.s_full[i], j & 1, abort);
            if (!ok) break;
            tc::tc_fence_after();
            float x[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tc::tmem_ld32(tS + c * 32, x[c]);
            tc::tmem_ld_wait();
            const int c0 = j * kTile;
            if (c0 + kTile > seen_all) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c0 + c * 32 + e >= seen) x[c][e] = -CUDART_INF_F;
            }
            float top[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                top[c] = x[c][0];
#pragma unroll
                for (int e = 1; e < 32; ++e) top[c] = fmaxf(top[c], x[c][e]);
            }
            const float mt = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), m);
            // the maximum in use follows the true one when it is 2^8 behind
            const bool grow = (mt - m) * sc > 8.f;
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? ex2_approx((m - mt) * sc) : 1.f;
                if (grow) m = mt;
                l *= f;
                if (j > 0) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tc::tmem_ld32(tO + c * 32, o);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            uint32_t u[16];
#pragma unroll
                            for (int y = 0; y < 16; ++y) u[y] = __float_as_uint(o[e + y] * f);
                            tc::tmem_st16(tO + c * 32 + e, u);
                        }
                    }
                }
            }
            const float base = m == -CUDART_INF_F ? 0.f : -m * sc;
            const float2 sc2 = make_float2(sc, sc), base2 = make_float2(base, base);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t u[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float2 y = fma2(make_float2(x[c][2 * e], x[c][2 * e + 1]), sc2, base2);
                    y.x = ex2_approx(y.x);
                    y.y = ex2_approx(y.y);
                    sum = add2(sum, y);
                    u[e] = pack_bf16(y.x, y.y);
                }
                tc::tmem_st16(tS + c * 16, u);
            }
            l += sum.x + sum.y;
            tc::tmem_st_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars.p_ready[i]);
        }
        const int rows_left = w.s.nq - (w.r0[i] + (warp & 3) * 32);
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) +
                             ((w.s.q0 + w.r0[i] + (warp & 3) * 32) * a.bt.Hq + w.head[i]) * (int64_t)D;
        // Q_i's shared memory is free once O_i is complete
        RowWriter<D> out{smem + C::kQ + i * C::kTileBytes + (warp & 3) * 32 * D * 2};
        if (ok && w.blocks[i] > 0) {
            ok = warp_wait(&bars.o_full[i], 0, abort);
        }
        if (ok && rows_left > 0) {
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            tc::tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                if (w.blocks[i] > 0) {
                    tc::tmem_ld32(tO + c * 32, o);
                    tc::tmem_ld_wait();
                }
                if (w.blocks[i] == 0 || inv == 0.f) {   // nothing seen: zero, whatever the accumulator holds
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                out.put(lane, c, o, inv);
            }
            out.flush(lane, dst, (int64_t)a.bt.Hq * D, rows_left);
            if (a.lse && r < w.s.nq)
                a.lse[stat_at(a.bt, w.s.q0 + r, w.head[i])] =
                    l == 0.f ? -CUDART_INF_F : m * a.scale + logf(l);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// Map of a [tokens][heads][d] bf16 tensor (tokens `stride` elements apart) with boxes of 128 tokens x 64
// channels of one head, swizzled as the tensor cores read them.
inline bool encode_tile_map(CUtensorMap *m, const void *base, int64_t stride, int d, int heads, int64_t tokens) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kTile};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool encode_prompt_maps(PromptMaps &m, const PromptArgs &a, int d) {
    const int64_t rows = a.bt.cu_q ? 1 : a.bt.n, tq = rows * a.bt.Tq, tk = rows * a.bt.Tk;
    return encode_tile_map(&m.q, a.q, a.q_stride, d, a.bt.Hq, tq) &&
           (tk == 0 || (encode_tile_map(&m.k, a.k, a.k_stride, d, a.bt.Hkv, tk) &&
                        encode_tile_map(&m.v, a.v, a.v_stride, d, a.bt.Hkv, tk))) &&
           (!a.d_out || encode_tile_map(&m.g, a.d_out, (int64_t)a.bt.Hq * d, d, a.bt.Hq, tq));
}

template <int D> cudaError_t launch_prompt_tc(const PromptArgs &a, cudaStream_t st) {
    using C = FwdCfg<D>;
    // two heads of a group share rows, keys and the number of key tiles; an odd group takes two row tiles
    const int pair = a.bt.Hq / a.bt.Hkv % 2 == 0;
    const int64_t tiles = max_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq, pair ? kTile : 2 * kTile);
    const int64_t grid = tiles * (pair ? a.bt.Hq / 2 : a.bt.Hq);
    if (a.bt.Tq == 0 || grid == 0) return cudaSuccess;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    PromptMaps maps = {};
    if (!encode_prompt_maps(maps, a, D)) return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem(attn_prompt_tc_kernel<D>, C::kSmem);
    if (e != cudaSuccess) return e;
    attn_prompt_tc_kernel<D><<<(unsigned)grid, C::kThreads, C::kSmem, st>>>(a, maps, pair);
    return cudaGetLastError();
}

}  // namespace attn
}  // namespace kda
