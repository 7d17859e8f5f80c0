// attn_prompt_tc.cuh -- attention over whole prompts on the tensor cores (bf16 inputs).
//
//     S = Q K^T,   P = 2^(c S - c m),   O = P V / rowsum(P),   c = scale log2(e),
// one pass over the keys in tiles of 128 with a running row maximum m and sum.
//
// One block per SM takes items in turn, the ones with the most keys first; an item is two tiles of 128
// queries that share their keys and values: two heads of a group
// (the same rows) where the group is even, two neighbouring row tiles of one head otherwise.  Both
// products run on tcgen05 with fp32 accumulators in Tensor Memory: S (128 x 128) per tile, O (128 x d)
// per tile.  Warp roles:
//   warps 0-7, 8-15  softmax of tile 0 and 1: two threads per row, 64 columns each, which exchange their
//                    maxima through shared memory.  They read S and write P (bf16) over what they read,
//                    as the second product's A operand; m and the sum stay in registers.  (One thread per
//                    row leaves one warp of a tile per scheduler, whose 128 powers in a row take longer
//                    than both products: 905 TFLOP/s at 16384 tokens.)
//   warp 16          issues the products:  O_i += P_i V_j, then S_i = Q_i K_{j+1}, for i = 0, 1 in turn, so
//                    one tile's softmax runs under the other tile's products.
//   warp 17          TMA loads: Q once, then K_j, V_j through a ring of stages.
//   warp 18          waits for the loads on warp 16's behalf and joins its word to the softmax warps': a
//                    wait behind products in flight returns only when they are done, so each one costs the
//                    tensor pipe some 200 cycles.  It also zeroes the rows of the last V tile that lie
//                    past the sequence's end.
// m is allowed to lag: while a row's new maximum exceeds the m in use by less than 2^8 the weights are
// only scaled differently (up to 2^8, exact in fp32 and no less precise in bf16), so O is rescaled
// rarely, by the softmax warps themselves: S_i of a tile is issued after the previous O_i, and the
// tensor pipe works in order, so a complete S_i means a complete O_i.  P is rounded once, to bf16, the
// operand type of V; the sum takes the unrounded weights.
//
// The ring of loads runs on from item to item, and an item's first products start under the end of the one
// before: a block per item cost 7.5 us (d = 64) to 9 us (128) of coming up and running dry, as much as 5 turns.
//
// No unit is full (tensor pipe 56%, SFU 42%, issue slots 52% of the cycles at d = 128): a tile's softmax is a chain of
// waits, and its products and powers, which take about the same time at d = 128 and the powers longer at 64, take turns
// two tiles deep.  One prompt of 16384 tokens, 32 heads of 128: 2.1 ms, 1.05 PFLOP/s of visible pairs (three
// quarters of what a library product sustains under the power limit); 8 packed prompts of 64 to 4096, heads of
// 64: 243 us; 200 tokens: 11 us, of which a launch, one TMA round trip and two turns in a row.
//
// Rows past the end of a sequence in its last tile are another sequence's (or whatever lies behind):
// their scores are masked, and their values are zeroed in shared memory before the product, since a
// weight of zero does not hide a NaN.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "attn_prompt.cuh"
#include "kda_chunk_tc.cuh"
#include "tc_utils.cuh"

namespace kda {
namespace attn {

constexpr int kTile = 128;   // queries of a tile, keys of a tile
// One pair of weights in this many takes its powers on the FMA units.  16384 tokens, 32 heads of 128: none
// 2.07 ms, 1 in 8 2.10, 1 in 4 2.04, 1 in 3 2.11; packed prompts, heads of 64: 272, 267, 265, 270 us.
constexpr int kEmulate = 4;

// ---- helpers shared with the gradient -----------------------------------------------------------

// K-major operand: [rows x 64-column SW128 blocks]; k-step kk of 16 columns.
__device__ __forceinline__ uint64_t desc_k(uint32_t base, int kk) {
    return tc::make_sdesc(base + (kk >> 2) * (kTile * 128) + (kk & 3) * 32, 16, 1024, tc::kSwz128);
}
// The same bytes as an MN-major operand: K runs over the 128 rows, MN over the columns.
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, int kk) {
    return tc::make_sdesc(base + kk * 2048, kTile * 128, 1024, tc::kSwz128);
}

// An A operand in Tensor Memory that takes the place of fp32 columns: the threads that read 64 columns
// write theirs as bf16 pairs over the first 32.  Column of k-step kk.
__device__ __forceinline__ uint32_t operand_col(int kk) { return (kk >> 2) * 64 + (kk & 3) * 8; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void st_shared(uint32_t addr, float x) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}
__device__ __forceinline__ float ld_shared(uint32_t addr) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
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

// The larger of three, NaN where one is: a score that is no number makes its row's maximum, and by it the whole row, NaN.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 2^x of two numbers on the FMA units, for x <= 127: x = n + f with |f| <= 1/2, 2^f by the
// polynomial of degree 5 with the least largest relative error (found by exchange; 1.5e-7 with the coefficients
// rounded to fp32, 2.1e-7 as evaluated, no more than the SFU's), n added to the exponent.  Below -126 it stays at 2^-126;
// NaN gives the largest number, infinite once rounded to bf16.
// The SFU gives 16 powers a clock and SM, so a tile of 128 x 128 weights takes as long as its two
// products of depth 128; taking a part of the powers here shortens the longer of the two.
__device__ __forceinline__ float2 ex2_fma(float2 x) {
    x.x = max3_nan(x.x, -126.f, -126.f);
    x.y = max3_nan(x.y, -126.f, -126.f);
    constexpr float kRound = 12582912.f;   // 1.5 * 2^23: adding it rounds to a whole number
    const float2 y = add2(x, make_float2(kRound, kRound));
    const float2 n = add2(y, make_float2(-kRound, -kRound));
    const float2 f = fma2(n, make_float2(-1.f, -1.f), x);
    float2 p = make_float2(1.3276472454890609e-3f, 1.3276472454890609e-3f);
    p = fma2(p, f, make_float2(9.675540961325169e-3f, 9.675540961325169e-3f));
    p = fma2(p, f, make_float2(5.550713092088699e-2f, 5.550713092088699e-2f));
    p = fma2(p, f, make_float2(2.4022120237350464e-1f, 2.4022120237350464e-1f));
    p = fma2(p, f, make_float2(6.931469440460205e-1f, 6.931469440460205e-1f));
    p = fma2(p, f, make_float2(1.0000001192092896f, 1.0000001192092896f));
    p.x = __int_as_float(__float_as_int(p.x) + (__float_as_int(y.x) << 23));
    p.y = __int_as_float(__float_as_int(p.y) + (__float_as_int(y.y) << 23));
    return p;
}

// Registers of a thread, moved between the warpgroups of a block after its launch: what one gives up
// (kDown) others take (kUp each): four warpgroups of softmax take, the fifth gives, and 128 (4 kUp + kDown) may not
// exceed what the launch gave all five.
template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Waits for a turn of a barrier to complete, at most kWaitLimit polls (some tenths of a second to a few
// seconds, where a healthy wait takes microseconds); then records the error, tells the block (*abort) and
// returns false, as it does once the block has been told.
constexpr uint32_t kWaitLimit = 1u << 22;
__device__ __forceinline__ bool bounded_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
    }
    record_device_error(kDevErrTimeout);
    *abort = 1;
    return false;
}

// A whole warp's wait: one answer for all lanes, so that they leave loops together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort));
}

// ---- products issued by a whole warp ----
// The products' operands live in uniform registers.  In a branch of one lane the compiler moves every
// descriptor there anew, some 60 cycles for each product; so the issuing warp stays together, one lane
// elected once and for all issues, and the descriptors of a chain are the first one plus constants.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit_by(uint64_t *bar, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar)),
        "r"(leader)
        : "memory");
}
// d = x y^T over D columns of two K-major tiles (descriptors of their first k-step).
template <int D> __device__ __forceinline__ void chain_ss(uint32_t d, uint64_t x, uint64_t y, uint32_t idesc, uint32_t leader) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t step = (kk >> 2) * (kTile * 128 / 16) + (kk & 3) * 2;
        mma_ss(d, x + step, y + step, idesc, kk > 0, leader);
    }
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
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

// 16 bf16 numbers to global memory: a whole sector at once where the tensor lies on one.
__device__ __forceinline__ void store_sector(__nv_bfloat16 *dst, const uint32_t (&u)[8]) {
    if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                     "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
}

// ---- forward ------------------------------------------------------------------------------------

struct PromptMaps {
    CUtensorMap q, k, v, g, o;   // g, o: d_out and out (gradient only)
};

template <int D> struct FwdCfg {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kQ = 0;                          // two query tiles
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kTop = kRing + kStages * kTileBytes;   // row maxima: [2 tiles][2 halves][128]
    static constexpr int kBars = kTop + 2 * 2 * kTile * 4;
    static constexpr int kSmem = kBars + 512;
    static constexpr int kThreads = 640;
    static constexpr int kUp = 104, kDown = 64;           // launched with 96 each: 128 (4 * 104 + 64) = 640 * 96
    static_assert(4 * kUp + kDown <= 5 * 96, "registers");
    static_assert(kSmem <= 232448, "shared memory");
};

// An item: two tiles of queries.
struct TwoTiles {
    int64_t q0, k0;                  // the sequence's first query and key
    int nq, nk, both;                // both: the larger of blocks; -1: no more items
    int head[2], r0[2], blocks[2];   // head, first row, tiles of keys that it sees
    int hk;                          // head of the cache
};

struct FwdBars {
    uint64_t q_full[2], q_empty[2], full[8], empty[8], s_full[2], p_ready[2][2], o_full[2], item_full[2], item_empty[2],
        drain;
    uint32_t tmem;
    int abort;
    TwoTiles item[2];
};
static_assert(sizeof(FwdBars) <= 512, "barriers");

// A block's r-th item; a whole warp.  Blocks take items there and back, so that none has the largest of
// every round.
__device__ __forceinline__ TwoTiles item_of(const PromptArgs &a, int pair_heads, int r, int lane, PlaceFrom &from) {
    const int units = pair_heads ? a.bt.Hq / 2 : a.bt.Hq, rows = pair_heads ? kTile : 2 * kTile;
    const int64_t index = (int64_t)r * gridDim.x + (r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    int n, count, level;
    TwoTiles w;
    w.both = -1;
    if (!place_of(a.bt.cu_q, a.bt.n, a.bt.Tq, rows, index / units, lane, n, count, level, from)) return w;
    const Seq s = seq_of(a.bt, n);
    w.q0 = s.q0, w.k0 = s.k0, w.nq = s.nq, w.nk = s.nk;
    const int u = (int)(index % units), t = level - 1;
    w.both = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w.head[i] = pair_heads ? 2 * u + i : u;
        w.r0[i] = t * rows + (pair_heads ? 0 : i * kTile);
        const int last = min(w.r0[i] + kTile, s.nq) - 1;
        w.blocks[i] = w.r0[i] < s.nq ? (keys_seen(s, last, a.causal) + kTile - 1) / kTile : 0;
        w.both = max(w.both, w.blocks[i]);
    }
    w.hk = w.head[0] / (a.bt.Hq / a.bt.Hkv);
    return w;
}

// 32 numbers of a thread's row, rounded, to 64 bytes of global memory, and what the rounding took from them,
// rounded in its turn (together they are good to 2^-17), where that is asked for.
__device__ __forceinline__ void store32(__nv_bfloat16 *dst, __nv_bfloat16 *rest, const float (&x)[32], float mul) {
#pragma unroll
    for (int e = 0; e < 32; e += 16) {
        uint32_t u[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) u[y] = pack_bf16(x[e + 2 * y] * mul, x[e + 2 * y + 1] * mul);
        store_sector(dst + e, u);
        if (rest) {
#pragma unroll
            for (int y = 0; y < 8; ++y)
                u[y] = pack_bf16(x[e + 2 * y] * mul - __uint_as_float(u[y] << 16),
                                 x[e + 2 * y + 1] * mul - __uint_as_float(u[y] & 0xffff0000u));
            store_sector(rest + e, u);
        }
    }
}

// Where a test makes one softmax warp give up, as if a wait had run out (place 0: for an item, 1: for scores,
// 2: for the output); here nothing does.
struct NoFault {
    static __device__ __forceinline__ bool gives_up(int, int, volatile int *) { return false; }
};

template <int D, typename Fault = NoFault>
__global__ void __launch_bounds__(FwdCfg<D>::kThreads, 1)
attn_prompt_tc_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ PromptMaps maps, int pair_heads) {
    using C = FwdCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    FwdBars &bars = *reinterpret_cast<FwdBars *>(smem + C::kBars);
    const uint32_t sbase = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    next_may_start();
    if (tid == 32 && a.bt.Tk > 0) prefetch_map(&maps.q), prefetch_map(&maps.k), prefetch_map(&maps.v);
    if (warp == 16) {
        tc::tmem_alloc(&bars.tmem, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        bars.abort = 0;
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars.q_full[i], 1);
            tc::mbar_init(&bars.q_empty[i], 1);
            tc::mbar_init(&bars.s_full[i], 1);
            tc::mbar_init(&bars.p_ready[i][0], 9);   // eight softmax warps and the loads'
            tc::mbar_init(&bars.p_ready[i][1], 8);
            tc::mbar_init(&bars.o_full[i], 1);
        }
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(&bars.full[i], 1);
            tc::mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars.item_full[i], 1);
            tc::mbar_init(&bars.item_empty[i], 19);   // sixteen softmax warps, products, loads, words
        }
        tc::mbar_init(&bars.drain, 1);
        tc::fence_mbar_init();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = bars.tmem;
    volatile int *abort = &bars.abort;
    constexpr uint32_t kO = 256;
    wait_for_previous();
    // the block's r-th item, and the word that a warp is done with it
    auto get_item = [&](int r) { return warp_wait(&bars.item_full[r & 1], (r >> 1) & 1, abort); };
    auto done_item = [&](int r) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars.item_empty[r & 1]);
    };

    // Counts that run on from item to item give the barriers' turns: `base` of the loads (K_0, V_0, K_1, ...
    // of an item; load k lies in stage k mod kStages), `turn[i]` of tile i's key tiles, `had[i]` of the
    // items in which tile i has any.
    if (warp >= 16) {
        regs_down<C::kDown>();
        int base = 0, turn[2] = {0, 0}, had[2] = {0, 0};
        bool ok = true;
        auto advance = [&](int r) {
            const TwoTiles &w = bars.item[r & 1];
            base += 2 * w.both;
#pragma unroll
            for (int i = 0; i < 2; ++i) turn[i] += w.blocks[i], had[i] += w.blocks[i] > 0;
            done_item(r);
        };
        auto loaded = [&](int k) { return warp_wait(&bars.full[k % C::kStages], (k / C::kStages) & 1, abort); };
        if (warp == 19) {
            PlaceFrom from;
            for (int r = 0;; ++r) {
                const TwoTiles w = item_of(a, pair_heads, r, lane, from);
                if (r >= 2 && !warp_wait(&bars.item_empty[r & 1], ((r >> 1) - 1) & 1, abort)) break;
                if (lane == 0) {
                    bars.item[r & 1] = w;
                    tc::mbar_arrive(&bars.item_full[r & 1]);
                }
                if (w.both < 0) break;
            }
        } else if (warp == 17) {
            int put = 0, put_q[2] = {0, 0};   // loads under way
            for (int r = 0; ok && (ok = get_item(r)) && bars.item[r & 1].both >= 0; ++r) {
                const TwoTiles w = bars.item[r & 1];
                for (int j = 0; j < 2 * w.both && ok; ++j) {
                    const int k = base + j, st = k % C::kStages;
                    if (j == min(2, 2 * w.both - 1)) {   // Q, once its place is free; the first keys need not wait for that
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (!ok || w.blocks[i] == 0) continue;
                            if (had[i] > 0 && !(ok = warp_wait(&bars.q_empty[i], (had[i] - 1) & 1, abort))) continue;
                            if (lane == 0) {
                                tc::mbar_arrive_expect_tx(&bars.q_full[i], C::kTileBytes);
                                tma_tile<D>(C::kQ + i * C::kTileBytes, smem, &maps.q, w.head[i], w.q0 + w.r0[i],
                                            &bars.q_full[i]);
                            }
                            ++put_q[i];
                        }
                        if (!ok) break;
                    }
                    if (k >= C::kStages && !(ok = warp_wait(&bars.empty[st], (k / C::kStages - 1) & 1, abort))) break;
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(&bars.full[st], C::kTileBytes);
                        tma_tile<D>(C::kRing + st * C::kTileBytes, smem, j & 1 ? &maps.v : &maps.k, w.hk,
                                    w.k0 + (int64_t)(j >> 1) * kTile, &bars.full[st]);
                    }
                    put = k + 1;
                }
                advance(r);
            }
            if (!ok && lane == 0) {   // a wait ran out: leave no copy in flight (each wait is bounded)
                int quit = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    quit = 0;
                    if (put_q[i] > 0) bounded_wait(&bars.q_full[i], (put_q[i] - 1) & 1, &quit);
                }
                for (int k = max(0, put - C::kStages); k < put; ++k) {
                    quit = 0;
                    bounded_wait(&bars.full[k % C::kStages], (k / C::kStages) & 1, &quit);
                }
            }
        } else if (warp == 18) {
            for (int r = 0; ok && (ok = get_item(r)) && bars.item[r & 1].both >= 0; ++r) {
                const TwoTiles w = bars.item[r & 1];
                const int past = w.both * kTile - w.nk;   // rows of the last V tile behind the sequence's end
                for (int j = 0; j < w.both && ok; ++j) {
                    const int kv = base + 2 * j + 1;
                    const bool more = j + 1 < w.both;
                    if (!(ok = loaded(kv))) break;
                    if (past > 0 && !more) {
                        zero_rows<D>(smem + C::kRing + (kv % C::kStages) * C::kTileBytes, kTile - past, lane);
                        __syncwarp();
                    }
                    if (more && !(ok = loaded(kv + 1))) break;
                    if (lane == 0) {
                        if (j < w.blocks[0]) tc::mbar_arrive(&bars.p_ready[0][0]);
                        if (j < w.blocks[1]) tc::mbar_arrive(&bars.p_ready[1][0]);
                    }
                    // not ahead of the softmax: the next word belongs to the next turn
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (ok && j < w.blocks[i]) ok = warp_wait(&bars.p_ready[i][0], (turn[i] + j) & 1, abort);
                }
                advance(r);
            }
        } else if (warp == 16) {
            constexpr uint32_t idS = tc::make_idesc_bf16(kTile, kTile, false, false);
            constexpr uint32_t idO = tc::make_idesc_bf16(kTile, D, false, true);
            const uint32_t leader = elect_lane();
            // S_i of key tile j, which is load k
            auto scores = [&](int i, bool last, int k) {
                chain_ss<D>(tmem + i * kTile, desc_k(sbase + C::kQ + i * C::kTileBytes, 0),
                            desc_k(sbase + C::kRing + (k % C::kStages) * C::kTileBytes, 0), idS, leader);
                commit_by(&bars.s_full[i], leader);
                if (last) commit_by(&bars.q_empty[i], leader);
            };
            for (int r = 0; ok && (ok = get_item(r)) && bars.item[r & 1].both >= 0; ++r) {
                const int both = bars.item[r & 1].both, blocks[2] = {bars.item[r & 1].blocks[0], bars.item[r & 1].blocks[1]};
                if (both > 0) ok = loaded(base);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!ok || blocks[i] == 0) continue;
                    ok = warp_wait(&bars.q_full[i], had[i] & 1, abort);
                    if (ok) scores(i, blocks[i] == 1, base);
                }
                if (ok && both > 0) commit_by(&bars.empty[base % C::kStages], leader);
                for (int j = 0; j < both && ok; ++j) {
                    const int kv = base + 2 * j + 1;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (!ok || j >= blocks[i]) continue;
                        const uint64_t v = desc_mn(sbase + C::kRing + (kv % C::kStages) * C::kTileBytes, 0);
#pragma unroll
                        for (int part = 0; part < 2 && ok; ++part) {   // the first 32 columns of either half, then the rest
                            if (!(ok = warp_wait(&bars.p_ready[i][part], (turn[i] + j) & 1, abort))) break;
                            tc::tc_fence_after();
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const int kk = (x >> 1) * 4 + part * 2 + (x & 1);
                                mma_ts(tmem + kO + i * D, tmem + i * kTile + operand_col(kk), v + kk * 128, idO,
                                       j > 0 || part + x > 0, leader);
                            }
                        }
                        if (!ok) continue;
                        if (j + 1 < blocks[i]) scores(i, j + 2 == blocks[i], kv + 1);
                        else commit_by(&bars.o_full[i], leader);
                    }
                    if (!ok) break;
                    commit_by(&bars.empty[kv % C::kStages], leader);
                    if (j + 1 < both) commit_by(&bars.empty[(kv + 1) % C::kStages], leader);
                }
                advance(r);
            }
            if (!ok || *abort) {   // no product in flight when the memory is given back
                int quit = 0;
                commit_by(&bars.drain, leader);
                warp_wait(&bars.drain, 0, &quit);
            }
        }
        __syncwarp();
    } else {
        regs_up<C::kUp>();
        const int i = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lanes = tc::tmem_lane_base(warp), tS = tmem + i * kTile + half * 64 + lanes,
                       tO = tmem + kO + i * D + half * (D / 2) + lanes;
        const float sc = a.scale * kLog2e;
        const uint32_t tops = sbase + C::kTop + (i * 2 * kTile + row) * 4 + half * kTile * 4;   // this thread's place
        // The two warps that share rows meet at a barrier of their own, which has no limit; so each meeting tells both
        // whether either gives up, and they leave together: who gives up comes to one more meeting, and who is
        // told there comes to no other.  (The vote costs up to 0.5%: 16384 tokens 2041 us, 2037 without; packed prompts
        // 240.3 and 239.3.  A word in shared memory that both look at: 2062 and 246.)
        const uint32_t pair = 1 + i * 4 + quarter;
        auto meet = [&](bool gone) { return tc::named_sync_or(pair, 64, gone); };
        uint32_t turn = 0, had = 0;   // parities
        bool ok = true, told = false;
        for (int round = 0; ok && (ok = get_item(round) && !Fault::gives_up(warp, 0, abort)) && bars.item[round & 1].both >= 0;
             ++round) {
        const volatile TwoTiles &w = bars.item[round & 1];   // read where it is needed, not kept
        const int blocks = w.blocks[i];
        int seen, seen_all;   // keys that this row sees, less its half's begin; that every row of the warp sees
        {
            const int r0 = w.r0[i], nq = w.nq, nk = w.nk;
            const Seq s{0, 0, nq, nk};
            seen = (r0 + row < nq ? keys_seen(s, r0 + row, a.causal) : nk) - half * 64;
            seen_all = keys_seen(s, min(r0 + quarter * 32, nq - 1), a.causal);
        }
        float m = -CUDART_INF_F, l = 0.f;
        for (int j = 0; j < blocks; ++j) {
            ok = warp_wait(&bars.s_full[i], turn, abort) && !Fault::gives_up(warp, 1, abort);
            turn ^= 1;
            if (!ok) break;
            tc::tc_fence_after();
            const int hidden = seen - j * kTile;   // columns from here on are
            const bool masked = j * kTile + kTile > seen_all;
            // the scores are read twice, for the maximum and for the powers: there are no registers to hold
            // them in between
            float mt = m;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x[32], top[4];
                tc::tmem_ld32(tS + c * 32, x);
                tc::tmem_ld_wait();
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e >= hidden) x[e] = -CUDART_INF_F;
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float *z = x + y * 8;
                    top[y] = max3_nan(max3_nan(max3_nan(z[0], z[1], z[2]), z[3], z[4]), max3_nan(z[5], z[6], z[7]), z[7]);
                }
                mt = max3_nan(max3_nan(top[0], top[1], mt), top[2], top[3]);
            }
            float x[2][16];
            tc::tmem_ld16(tS, x[0]);
            // the row's other half.  It has read this one's by the next turn: the next scores wait for both's weights
            st_shared(tops, mt);
            if ((told = meet(false))) break;
            mt = max3_nan(mt, ld_shared(tops ^ (kTile * 4)), m);
            // the maximum in use follows the true one when it is 2^8 behind (or is NaN)
            const bool grow = !(mt * sc <= m * sc + 8.f);
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? ex2_approx((m - mt) * sc) : 1.f;
                if (grow) m = mt;
                l *= f;
                if (j > 0) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {   // this half of the accumulator's columns
                        float o[16];
                        uint32_t u[16];
                        tc::tmem_ld16(tO + c * 16, o);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int y = 0; y < 16; ++y) u[y] = __float_as_uint(o[y] * f);
                        tc::tmem_st16(tO + c * 16, u);
                    }
                }
            }
            // an infinite maximum: no score at all (weights of zero), or one of +inf (NaN)
            const float base = m == -CUDART_INF_F ? 0.f : m == CUDART_INF_F ? CUDART_NAN_F : -m * sc;
            const float2 sc2 = make_float2(sc, sc), base2 = make_float2(base, base);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {   // 16 columns at a time, the next ones on their way
                tc::tmem_ld_wait();
                if (c < 3) tc::tmem_ld16(tS + (c + 1) * 16, x[(c + 1) & 1]);
                float (&z)[16] = x[c & 1];
                uint32_t u[8];
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float lo = c * 16 + 2 * e < hidden ? ex2_approx(fmaf(z[2 * e], sc, base)) : 0.f;
                        const float hi = c * 16 + 2 * e + 1 < hidden ? ex2_approx(fmaf(z[2 * e + 1], sc, base)) : 0.f;
                        sum = add2(sum, make_float2(lo, hi));
                        u[e] = pack_bf16(lo, hi);
                    }
                } else {   // nothing hidden: a part of the powers goes to the FMA units
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float2 y = fma2(make_float2(z[2 * e], z[2 * e + 1]), sc2, base2);
                        if (e % kEmulate == kEmulate - 1) {
                            y = ex2_fma(y);
                        } else {
                            y.x = ex2_approx(y.x);
                            y.y = ex2_approx(y.y);
                        }
                        sum = add2(sum, y);
                        u[e] = pack_bf16(y.x, y.y);
                    }
                }
                tc::tmem_st8(tS + c * 8, u);
                if (c & 1) {   // half of the weights
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bars.p_ready[i][c >> 1]);
                }
            }
            l += sum.x + sum.y;
        }
        if (ok && !told && blocks > 0) ok = warp_wait(&bars.o_full[i], had, abort) && !Fault::gives_up(warp, 2, abort);
        if (!ok || told) break;
        // the sum of the row's two halves (both scaled by the same m)
        st_shared(tops, l);
        if ((told = meet(false))) break;
        l += ld_shared(tops ^ (kTile * 4));
        tc::named_sync(pair, 64);   // read, before the next item's maxima come; neither gives up in between
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        const int r = w.r0[i] + row, head = w.head[i];
        const bool there = r < w.nq;
        const int64_t at = w.q0 + r;
        done_item(round);
        tc::tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {   // this half's columns
            float o[32];
            if (blocks > 0) {
                tc::tmem_ld32(tO + c * 32, o);
                tc::tmem_ld_wait();
            }
            if (blocks == 0 || inv == 0.f) {   // nothing seen: zero, whatever the accumulator holds
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
            }
            if (there) {
                const int64_t to = (at * a.bt.Hq + head) * (int64_t)D + half * (D / 2) + c * 32;
                store32(static_cast<__nv_bfloat16 *>(a.out) + to,
                        a.rest ? static_cast<__nv_bfloat16 *>(a.rest) + to : nullptr, o, inv);
            }
        }
        if (a.lse && half == 0 && there) a.lse[stat_at(a.bt, at, head)] = l == 0.f ? -CUDART_INF_F : m * a.scale + logf(l);
        had ^= blocks > 0;
        }
        if (!told) meet(!ok);   // the last meeting
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 16) {
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
           (!a.d_out || (encode_tile_map(&m.g, a.d_out, (int64_t)a.bt.Hq * d, d, a.bt.Hq, tq) &&
                         encode_tile_map(&m.o, a.out, (int64_t)a.bt.Hq * d, d, a.bt.Hq, tq)));
}

template <int D, typename Fault = NoFault> cudaError_t launch_prompt_tc(const PromptArgs &a, int sms, cudaStream_t st) {
    using C = FwdCfg<D>;
    // two heads of a group share rows, keys and the number of key tiles; an odd group takes two row tiles
    const int pair = a.bt.Hq / a.bt.Hkv % 2 == 0;
    const int64_t tiles = max_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq, pair ? kTile : 2 * kTile);
    const int64_t grid = tiles * (pair ? a.bt.Hq / 2 : a.bt.Hq);   // items
    if (a.bt.Tq == 0 || grid == 0) return cudaSuccess;
    // before the maps: it binds the device's context to this thread, which their encoding needs
    const cudaError_t e = allow_smem(attn_prompt_tc_kernel<D, Fault>, C::kSmem);
    if (e != cudaSuccess) return e;
    PromptMaps maps = {};
    if (!encode_prompt_maps(maps, a, D)) return cudaErrorInvalidValue;
    return launch_behind(attn_prompt_tc_kernel<D, Fault>, (unsigned)(grid < sms ? grid : sms), C::kThreads, C::kSmem, st, a,
                         maps, pair);
}

}  // namespace attn
}  // namespace kda
