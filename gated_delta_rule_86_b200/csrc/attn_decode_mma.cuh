// attn_decode_mma.cuh -- the decode step's block for bf16, with the products on warp-level matrix
// instructions, and the launch of both types.
//
// The schedule is that of attn_decode.cuh; here a block has 8 warps and a tile 128 tokens.  A head's
// cache is read once for all query heads of its group, which at 8 heads asks for 8 multiplications per
// loaded value and product: more than the FMA units give at the memory's pace, and little for m16n8k16
// instructions.  Rows are the group's heads (up to 16), columns the warp's 16 tokens:
//     S (16 x 16) = Q K^T      K straight from the staged rows
//     O (16 x d) += P V        P from S's own registers, as the sum of two bf16 numbers, the operand type of V:
//                              the weight rounded, and what that took from it: good to 2^-16 of the weight, so only
//                              the result's own rounding shows.  For up to 8 heads the second number takes the rows
//                              that would be empty and costs nothing, for 16 a product of its own (heads of 128:
//                              64 sequences of 4096 tokens 56.7 us, 56.6 without; 16 of 700 13.4 and 12.8).
// tcgen05 would want 64 or 128 rows and its operands through Tensor Memory for the same few products;
// the kernel is bound by the cache's bytes, not by these.
// Measured, heads of 128, 4 query heads to one of the cache: 64 sequences of 64 to 16384 tokens 135 us, 6.2 TB/s;
// one of 131071 tokens 94 us, 5.7 TB/s (some 8 us of it are the start of a share, the last join and its launch).
#pragma once

#include "attn_decode.cuh"

namespace kda {
namespace attn {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two bf16 numbers in a word, and each of them as fp32.
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float low_half(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high_half(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// The page of a warp's first token of a tile, -1 where it has none; its lookup runs a tile ahead of its use.
template <int TILE>
__host__ __device__ __forceinline__ int first_page(const DecodeArgs &a, const Walk<TILE> &w, int warp) {
    const int tok = w.tile * TILE + warp * kWarpTokens;
    return tok < w.len ? a.cache.table[w.b * a.cache.row + (tok >> a.cache.page_log2)] : -1;
}
// Moves to the next tile and looks up its page.  Behind the share's end the walk may stand behind the last
// sequence, where the table has no row.
template <int TILE> __host__ __device__ __forceinline__ int next_page(const DecodeArgs &a, Walk<TILE> &w, int warp) {
    w.next(a);
    return w.more() ? first_page(a, w, warp) : -1;
}

// load_tokens where the 16 tokens all exist and lie on one good page (`page`): 16 rows side by side in
// memory, so that a lane's addresses are one base and constants.
template <int D, int TILE>
__device__ __forceinline__ void load_whole(const DecodeArgs &a, const Walk<TILE> &w, int warp, int lane, int hkv,
                                           uint32_t stage, int page) {
    constexpr int CH = D * 2 / 16, ROWS = 32 / CH, N = kWarpTokens / ROWS;   // rows of one instruction, instructions
    const int t0 = w.tile * TILE + warp * kWarpTokens;
    const int64_t slot = ((int64_t)hkv << a.cache.page_log2) + (t0 & ((1 << a.cache.page_log2) - 1));
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.cache.k) + page * a.cache.k_stride + slot * D + lane * 8;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.cache.v) + page * a.cache.v_stride + slot * D + lane * 8;
    // chunk c of row r lies at chunk (c ^ r) & 7 of its half row; r = i ROWS + r_lane, the two apart in their bits
    const int rl = lane / CH, c = lane % CH;
    const uint32_t at = rl * (CH * 16) + (((c & ~7) | ((c ^ rl) & 7)) << 4);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t dst = stage + i * (ROWS * CH * 16) + (at ^ ((i * ROWS & 7) << 4));
        cp_async16(dst, k + i * ROWS * D, true);
        cp_async16(dst + kWarpTokens * CH * 16, v + i * ROWS * D, true);
    }
}

template <int D, int GC> struct DecodeMmaCfg {
    static constexpr int kWarps = 8;
    static constexpr int kTile = kWarps * kWarpTokens;
    static constexpr int kRowBytes = D * 2;
    static constexpr int kStageBytes = 2 * kWarpTokens * kRowBytes;
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kJoinRows = 64;   // (warp, head) results that the join buffer holds at once
    static constexpr int kPitch = D + 4;   // of a result: o, then m and the sum
    static constexpr int kJoin = kJoinRows * kPitch * 4;
    static constexpr int kSmem = kRing + kJoin + 160;
    static_assert(kSmem <= 232448, "shared memory");
};

template <int D, int GC>
__global__ void __launch_bounds__(DecodeMmaCfg<D, GC>::kWarps * 32, 1) attn_decode_mma_kernel(const DecodeArgs a) {
    using C = DecodeMmaCfg<D, GC>;
    constexpr int CH = C::kRowBytes / 16;
    constexpr int kShare = (GC * D + 255) / 256;   // of a pair's results, per thread, in the join
    constexpr bool kBoth = GC > 8;   // rows 8-15 hold heads too
    extern __shared__ __align__(1024) uint8_t smem[];
    float *s_join = reinterpret_cast<float *>(smem + C::kRing);
    int64_t *scratch = reinterpret_cast<int64_t *>(smem + C::kRing + C::kJoin);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, gc = lane & 3;   // a fragment's row and column pair
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * C::kStages * C::kStageBytes;

    if (a.per_pair) next_may_start();
    wait_for_previous();
    if (!a.per_pair) next_may_start();   // only now: the join reads the lengths before its own wait
    Walk<C::kTile> w;
    const bool work = w.start(a, scratch);
    if (a.per_pair && tid == 0) check_len(a, w.b);
    if (!work) {
        if (a.per_pair) write_empty<__nv_bfloat16, D, GC>(a, w.b, w.vh);
        return;
    }
    Walk<C::kTile> ahead = w;
    int page = first_page(a, ahead, warp);
    // loads the tile at `ahead` into a stage and moves on
    auto load = [&](uint32_t stage, int hkv) {
        uint32_t got = 0xffffu;
        const int tok = ahead.tile * C::kTile + warp * kWarpTokens;
        if (a.cache.page_log2 >= 4 && tok + kWarpTokens <= ahead.len && page >= 0 && page < a.cache.num_pages)
            load_whole<D, C::kTile>(a, ahead, warp, lane, hkv, stage, page);
        else
            got = tok < ahead.len ? load_tokens<__nv_bfloat16, D, C::kTile>(a, ahead, warp, lane, hkv, stage) : 0;
        page = next_page(a, ahead, warp);
        return got;
    };
    const int group = a.Hq / a.Hkv, chunks = a.vheads / a.Hkv;
    uint32_t held[C::kStages];   // which of a stage's tokens there are
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) held[s] = 0;
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) {
        if (ahead.more()) held[s] = load(ring + s * C::kStageBytes, ahead.vh / chunks);
        cp_async_commit();
    }

    // this lane's addresses inside a stage: ldmatrix rows
    const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;   // K: tokens 0-7 | 8-15, chunk 0 | 1
    const int vrow = lane & 15, vch = lane >> 4;                               // V: tokens 0-15, chunk 0 | 1
    const uint32_t kat = krow * (CH * 16) + (((kch ^ krow) & 7) << 4);
    const uint32_t vat = kWarpTokens * C::kRowBytes + vrow * (CH * 16) + (((vch ^ vrow) & 7) << 4);
    uint32_t qf[D / 16][4];
    float o[D / 8][4];
    float m[2], l[2];
    const float sc = a.scale * kLog2e;
    bool starts_inside = w.tile != 0, fresh = true;
    int st = 0;
    // the queries of the pair at w as the A operand
    auto load_q = [&]() {
        const int hkv = w.vh / chunks, h0 = hkv * group + (w.vh % chunks) * GC;
        const int nh = min(GC, hkv * group + group - h0);
        const uint32_t *q = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                               w.b * a.q_stride + (int64_t)h0 * D);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c = kk * 8 + gc;
            qf[kk][0] = gr < nh ? q[gr * (D / 2) + c] : 0u;
            qf[kk][2] = gr < nh ? q[gr * (D / 2) + c + 4] : 0u;
            qf[kk][1] = kBoth && gr + 8 < nh ? q[(gr + 8) * (D / 2) + c] : 0u;
            qf[kk][3] = kBoth && gr + 8 < nh ? q[(gr + 8) * (D / 2) + c + 4] : 0u;
        }
    };
    load_q();
    while (w.more()) {
        const int hkv = w.vh / chunks, h0 = hkv * group + (w.vh % chunks) * GC;
        const int nh = min(GC, hkv * group + group - h0);
        if (fresh) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
            m[0] = m[1] = -CUDART_INF_F;
            l[0] = l[1] = 0.f;
            fresh = false;
        }
        {
            uint32_t got = 0;
            const int into = st == 0 ? C::kStages - 1 : st - 1;
            if (ahead.more()) got = load(ring + into * C::kStageBytes, ahead.vh / chunks);
            cp_async_commit();
#pragma unroll
            for (int s = 0; s < C::kStages; ++s)
                if (s == into) held[s] = got;
        }
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        uint32_t ok = 0;
#pragma unroll
        for (int s = 0; s < C::kStages; ++s)
            if (s == st) ok = held[s];
        if (ok) {   // a warp's share of the tile may be empty
            const uint32_t ks = ring + st * C::kStageBytes;
            float s0[4] = {}, s1[4] = {};   // tokens 0-7, 8-15
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t b[4];
                ldsm4(b, ks + (kat ^ ((2 * kk & 7) << 4)) + (kk >> 2) * 128);
                mma_bf16(s0, qf[kk], b[0], b[1]);
                mma_bf16(s1, qf[kk], b[2], b[3]);
            }
            // scores in log2 units, row 8 y + gr, this lane's four tokens
            constexpr int kRows = kBoth ? 2 : 1;
            float x[kRows][4];
            bool grow = false;
#pragma unroll
            for (int y = 0; y < kRows; ++y) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[y][e] = (e < 2 ? s0 : s1)[2 * y + (e & 1)] * sc;
                if (ok != 0xffffu) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((ok >> (2 * gc + (e & 1) + (e >> 1) * 8)) & 1)) x[y][e] = -CUDART_INF_F;
                }
                grow |= fmaxf(fmaxf(x[y][0], x[y][1]), fmaxf(x[y][2], x[y][3])) - m[y] > 8.f;
            }
            // the maximum in use follows the true one when it is 2^8 behind: weights up to 2^8 are as exact, and
            // the lanes of a row exchange their maxima, and the accumulators are rescaled, rarely
            if (__any_sync(0xffffffffu, grow)) {
                float f[kRows];
#pragma unroll
                for (int y = 0; y < kRows; ++y) {
                    float top = fmaxf(fmaxf(x[y][0], x[y][1]), fmaxf(x[y][2], x[y][3]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    f[y] = 1.f;
                    if (top - m[y] > 8.f) {
                        f[y] = ex2_approx(m[y] - top);
                        m[y] = top;
                    }
                    l[y] *= f[y];
                }
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    o[c][0] *= f[0];
                    o[c][1] *= f[0];
                    o[c][2] *= f[kRows - 1];
                    o[c][3] *= f[kRows - 1];
                }
            }
            uint32_t p[4], pr[4];   // weights, and what rounding took from them
#pragma unroll
            for (int y = 0; y < kRows; ++y) {
                const float base = m[y] == -CUDART_INF_F ? 0.f : m[y];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[y][e] = ex2_approx(x[y][e] - base);
                l[y] += (x[y][0] + x[y][1]) + (x[y][2] + x[y][3]);
                p[y] = pack_pair(x[y][0], x[y][1]);
                p[2 + y] = pack_pair(x[y][2], x[y][3]);
                pr[y] = pack_pair(x[y][0] - low_half(p[y]), x[y][1] - high_half(p[y]));
                pr[2 + y] = pack_pair(x[y][2] - low_half(p[2 + y]), x[y][3] - high_half(p[2 + y]));
            }
            if (!kBoth) p[1] = pr[0], p[3] = pr[2];
#pragma unroll
            for (int c2 = 0; c2 < D / 16; ++c2) {
                uint32_t b[4];
                ldsm4_t(b, ks + (vat ^ ((2 * c2 & 7) << 4)) + (c2 >> 2) * 128);
                mma_bf16(o[2 * c2], p, b[0], b[1]);
                mma_bf16(o[2 * c2 + 1], p, b[2], b[3]);
                if (kBoth) {
                    mma_bf16(o[2 * c2], pr, b[0], b[1]);
                    mma_bf16(o[2 * c2 + 1], pr, b[2], b[3]);
                }
            }
        }
        __syncwarp();   // the stage is read before it is filled again
        st = st + 1 == C::kStages ? 0 : st + 1;

        const Walk<C::kTile> cur = w;
        w.next(a);
        const bool end = !w.more();
        if (end || w.b != cur.b || w.vh != cur.vh) {
            if (!end) load_q();   // of the next pair: on their way during the join
            const bool whole = !starts_inside && cur.tile + 1 == cur.tiles;
            // the warps' results meet in shared memory: all at once for up to 8 heads, in two rounds for 16
            constexpr int kRounds = kBoth ? 2 : 1, kPerRound = C::kWarps / kRounds;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
                l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
            }
            float acc[kShare], top_all[kShare], sum_all[kShare];
#pragma unroll
            for (int x = 0; x < kShare; ++x) acc[x] = 0.f, sum_all[x] = 0.f, top_all[x] = -CUDART_INF_F;
#pragma unroll
            for (int round = 0; round < kRounds; ++round) {
                if (round) __syncthreads();
                if (warp / kPerRound == round) {
#pragma unroll
                    for (int y = 0; y < (kBoth ? 2 : 1); ++y) {
                        float *j = s_join + ((warp % kPerRound) * GC + gr + 8 * y) * C::kPitch;
#pragma unroll
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<float2 *>(j + c * 8 + gc * 2) =
                                kBoth ? make_float2(o[c][2 * y], o[c][2 * y + 1])
                                      : make_float2(o[c][0] + o[c][2], o[c][1] + o[c][3]);
                        if (gc == 0) j[D] = m[y], j[D + 1] = l[y];
                    }
                }
                __syncthreads();
#pragma unroll
                for (int x = 0; x < kShare; ++x) {
                    const int e = x * 256 + tid, g = e / D, c = e % D;
                    if (g >= nh) continue;
                    float top = top_all[x];
#pragma unroll
                    for (int k = 0; k < kPerRound; ++k) top = fmaxf(top, s_join[(k * GC + g) * C::kPitch + D]);
                    const float base = top == -CUDART_INF_F ? 0.f : top, f0 = ex2_approx(top_all[x] - base);
                    acc[x] *= f0;
                    sum_all[x] *= f0;
#pragma unroll
                    for (int k = 0; k < kPerRound; ++k) {
                        const float *j = s_join + (k * GC + g) * C::kPitch;
                        const float f = ex2_approx(j[D] - base);
                        sum_all[x] += f * j[D + 1];
                        acc[x] += f * j[c];
                    }
                    top_all[x] = top;
                }
            }
            float *part = a.part + ((int64_t)blockIdx.x * 2 + (starts_inside || !end ? 0 : 1)) * GC * (D + 2);
#pragma unroll
            for (int x = 0; x < kShare; ++x) {
                const int e = x * 256 + tid, g = e / D, c = e % D;
                if (g >= nh) continue;
                const float sum = sum_all[x];
                if (whole) {
                    const int64_t h = (int64_t)cur.b * a.Hq + h0 + g;
                    static_cast<__nv_bfloat16 *>(a.out)[h * D + c] =
                        __float2bfloat16_rn(sum > 0.f || sum != sum ? acc[x] / sum : 0.f);
                    if (c == 0 && a.lse)
                        a.lse[h] = sum == 0.f ? -CUDART_INF_F : top_all[x] * 0.69314718055994531f + logf(sum);
                } else {
                    part[g * (D + 2) + 2 + c] = acc[x];
                    if (c == 0) {
                        part[g * (D + 2)] = top_all[x];
                        part[g * (D + 2) + 1] = sum;
                    }
                }
            }
            __syncthreads();   // the buffer is read before the next pair's results
            starts_inside = false;
            fresh = true;
        }
    }
    cp_async_wait<0>();
}

// Query heads that a block takes together.  fp32: the whole group up to 8 (their sums are registers of
// every lane); bf16: 8 or 16, half or all rows of a fragment.  A larger group reads its cache again.
inline int decode_group_chunk(int group, bool bf16) {
    if (bf16) return group <= 8 ? 8 : 16;
    return group <= 1 ? 1 : group <= 2 ? 2 : group <= 4 ? 4 : 8;
}

inline int64_t decode_pairs(int64_t n, int Hq, int Hkv, bool bf16) {
    const int group = Hq / Hkv, gc = decode_group_chunk(group, bf16);
    return n * Hkv * ((group + gc - 1) / gc);
}

// Short contexts of few pairs: a block takes a whole pair, which saves the join and its launch.  `tokens`:
// what a row of the page table can hold.
// Whole pairs and shares, us, full rows of the table, 4 query heads to one of the cache:
//   bf16, heads of 128 (64):  1 pair, 768 tokens 8.9 and 9.3 (7.8 and 8.4), 1024 10.8 and 9.6 (9.4 and 8.7);
//                             32 pairs, 1024 11.1 and 11.0 (9.7 and 9.8); 128 pairs, 1024 14.8 and 19.6 (10.6 and 15.0)
//   fp32 (its block walks 64 tokens at a time, in 3.5 us for 128 tokens, so its shares pay sooner):
//                             1 pair, 256 10.7 and 10.2 (8.6 and 9.3), 512 17.8 and 11.4 (14.1 and 10.0);
//                             64 pairs, 256 11.6 and 13.7 (9.3 and 12.7), 512 19.0 and 17.9 (14.9 and 14.7);
//                             128 pairs, 512 20.1 and 24.4 (20.3 and 20.1), 1024 34.3 and 38.4 (35.8 and 31.5)
// Pairs that almost fill the SMs gain beyond these limits as well, but only while their lengths are alike.
inline bool decode_per_pair(int64_t pairs, int64_t tokens, int d, bool bf16, int sms) {
    if (pairs > sms) return false;
    if (bf16) return tokens <= (8 * pairs <= sms ? 768 : 1024);
    return tokens <= (4 * pairs <= 3 * sms ? 256 : d == 128 ? 1024 : 512);
}

inline size_t decode_workspace_bytes(int64_t n, int Hq, int Hkv, int d, int64_t tokens, bool bf16, int sms) {
    if (decode_per_pair(decode_pairs(n, Hq, Hkv, bf16), tokens, d, bf16, sms)) return 0;
    return (size_t)kMaxDecodeBlocks * 2 * decode_group_chunk(Hq / Hkv, bf16) * (d + 2) * 4;
}

template <typename T, int D, int GC, typename C> cudaError_t launch_decode_g(void (*kern)(DecodeArgs), int threads,
                                                                             DecodeArgs a, int sms, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    a.vheads = a.Hkv * ((a.Hq / a.Hkv + GC - 1) / GC);
    const int64_t pairs = (int64_t)a.n * a.vheads, tokens = (int64_t)a.cache.width << a.cache.page_log2;
    a.per_pair = decode_per_pair(pairs, tokens, D, sizeof(T) == 2, sms);
    a.blocks = a.per_pair ? (int)pairs : decode_blocks(a, C::kTile, sms);
    e = launch_behind(kern, (unsigned)a.blocks, threads, C::kSmem, st, a);
    if (e != cudaSuccess || a.per_pair) return e;
    return launch_behind(attn_decode_join_kernel<T, D, GC, C::kTile>, (unsigned)pairs, kJoinThreads, 0, st, a);
}

template <int D> cudaError_t launch_attn_decode_bf16(const DecodeArgs &a, int sms, cudaStream_t st) {
    using T = __nv_bfloat16;
    if (decode_group_chunk(a.Hq / a.Hkv, true) == 8)
        return launch_decode_g<T, D, 8, DecodeMmaCfg<D, 8>>(attn_decode_mma_kernel<D, 8>, 256, a, sms, st);
    return launch_decode_g<T, D, 16, DecodeMmaCfg<D, 16>>(attn_decode_mma_kernel<D, 16>, 256, a, sms, st);
}

template <int D> cudaError_t launch_attn_decode_f32(const DecodeArgs &a, int sms, cudaStream_t st) {
    switch (decode_group_chunk(a.Hq / a.Hkv, false)) {
        case 1: return launch_decode_g<float, D, 1, DecodeCfg<D, 1>>(attn_decode_kernel<D, 1>, 128, a, sms, st);
        case 2: return launch_decode_g<float, D, 2, DecodeCfg<D, 2>>(attn_decode_kernel<D, 2>, 128, a, sms, st);
        case 4: return launch_decode_g<float, D, 4, DecodeCfg<D, 4>>(attn_decode_kernel<D, 4>, 128, a, sms, st);
        default: return launch_decode_g<float, D, 8, DecodeCfg<D, 8>>(attn_decode_kernel<D, 8>, 128, a, sms, st);
    }
}

}  // namespace attn
}  // namespace kda
