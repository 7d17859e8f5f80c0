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
// One block per SM takes items in turn, the longest first; rings, products and loads run on from one to the
// next (a block per item cost some 7 us each of coming up and running dry).  Warp roles: 0-15 compute
// (thread = row, four groups of 32 columns), 16 issues the products, 17 finds the items and loads their tiles
// (TMA), 18 waits for the loads on 16's behalf, zeroes rows that must not count, and joins its word to the
// compute warps' (a wait behind products in flight returns only with them), 19 brings the queries' lse and
// delta to the keys' kernel.  P and dS become operands in bf16 (see kFineKeys).
//
// Bound by the turns that weights and products of one tile take (tensor pipe 55 to 59% of the cycles): B2 T4096, 16 heads of
// 128, 427 us, its seven products at 1.13 PFLOP/s (0.8 of what a library product sustains); 6 packed documents,
// 16 + 4 heads of 64, 190 us, where P and dS take as long as the products.  Powers on the FMA units, as the forward has
// them, change nothing here.
//
// delta is taken from O as it was before its rounding where the caller kept what the rounding took (`rest`):
// delta is subtracted from every dP of its row, so the rounding's error in it (2^-9 |dO| |O|) does not cancel
// in the sum.  dQ's error against 64 bits is 1.74e-3 of its size with it, 2.04e-3 without, for 64 tokens, 2.06 and
// 2.20e-3 for 1024; 1 us.
//
// Rows past the end of a sequence in its last tile belong to others.  Where they are rows of a result
// they are not stored; where they are summed over (queries in the keys' kernel, keys in the other) they
// are zeroed in shared memory, since a weight of zero does not hide a NaN.
#pragma once

#include <limits.h>

#include "attn_prompt_tc.cuh"

namespace kda {
namespace attn {

template <int D> struct GradCfg {
    static constexpr int kTileBytes = kTile * D * 2;
    // Stages of one tile each, released one by one: of a turn's two tiles (Q and dO, or K and V) the first
    // is read again at the turn's end, so more of it are held.  (One ring for both: 262 us for dQ at B2
    // T4096 H16, its loads of V waiting for dQ's products; 201 with two.)
    static constexpr int kFirst = D == 128 ? 3 : 4, kSecond = D == 128 ? 2 : 4, kStages = kFirst + kSecond;
    static constexpr int kOwn = 0;                               // an item's own two tiles
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kStats = kRing + kStages * kTileBytes;  // -lse and -delta of two turns' queries, or parts of delta
    static constexpr int kBars = kStats + 2 * 2 * kTile * 4;
    static constexpr int kSmem = kBars + 512;
    static_assert(kSmem <= 232448, "shared memory");
    static constexpr int kThreads = 640;
};

// An item of a block: 128 keys of one head of the cache, or 128 queries of one head.
struct GradItem {
    int64_t q0, k0;                            // the sequence's first query and key
    int nq, nk, total;                         // total: turns; -1: no more items
    int head, row0, start, per_head;           // keys' kernel: first query tile, turns per query head
    int fine;                                  // operands as two numbers: keys' kernel: in so many turns at a head's begin
};

// P and dS enter their products rounded to bf16, or, where the first of a tile of queries sees kFineKeys or less, as two
// bf16 numbers, the second what rounding took from the first.  Among many keys the roundings' errors average out: they
// add as much to the result's error as its own rounding does, 1.41 times that in all.  Queries that see a few have few
// weights and the largest dS of their sequence: rounded, they make it 2.2 times for 2 tokens, 1.6 for 64, and still 1.5
// for a causal sequence of 2048; as two numbers 1.3, 1.1 and 1.3.  Costs: 64 sequences of 64 tokens 72 us from 63, 16 of
// 1024 240 from 237 (16 + 4 heads of 64), B2 T4096 H16 433 from 427; everywhere it would be 505.
constexpr int kFineKeys = kTile;

struct GradBars {
    uint64_t own_full, own_empty, out_read, first, full[8], empty[8], stats[2], stats_read[2], s_full[2], dp_full[2], q_word,
        a_ready[2], b_ready[2], done, drain, item_full[2], item_empty[2];
    uint32_t tmem;
    int abort;
    GradItem item[2];
};
static_assert(sizeof(GradBars) <= 512, "barriers");

// Scores, dP and the operands made of them pass through two barriers each, taken in turn: turn n + 1 may be
// complete before a late warp has looked for turn n, and a single barrier's parity would then have come
// round.  (Turn n + 2 needs what the waiter of turn n does next, in either kernel.)
__device__ __forceinline__ bool wait_turn(uint64_t (&bar)[2], int n, volatile int *abort) {
    return warp_wait(&bar[n & 1], (n >> 1) & 1, abort);
}

// Arrivals that complete a turn of the barriers whose number differs between the kernels.
struct GradCounts {
    int own_empty, a_ready, b_ready, item_empty;
};

// Barriers and Tensor Memory; every thread.  Returns the Tensor Memory's base.
template <int D> __device__ __forceinline__ uint32_t grad_setup(GradBars &bars, const GradCounts &n) {
    using C = GradCfg<D>;
    if (threadIdx.x == 0) {
        bars.abort = 0;
        tc::mbar_init(&bars.own_full, 1);
        tc::mbar_init(&bars.own_empty, n.own_empty);
        tc::mbar_init(&bars.out_read, 16);
        tc::mbar_init(&bars.first, 1);
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(&bars.full[i], 1);
            tc::mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars.stats[i], 1);
            tc::mbar_init(&bars.stats_read[i], 16);
            tc::mbar_init(&bars.s_full[i], 1);
            tc::mbar_init(&bars.dp_full[i], 1);
            tc::mbar_init(&bars.a_ready[i], n.a_ready);
            tc::mbar_init(&bars.b_ready[i], n.b_ready);
            tc::mbar_init(&bars.item_full[i], 1);
            tc::mbar_init(&bars.item_empty[i], n.item_empty);
        }
        tc::mbar_init(&bars.q_word, 1);
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

// Load n of a turn's first tiles, or of its second ones, counted over all items: its stage, the parity of
// that stage's filling, and its place in shared memory.
template <int D, int WHICH> struct Ring {
    using C = GradCfg<D>;
    static constexpr int N = WHICH ? C::kSecond : C::kFirst;
    static __device__ __forceinline__ int stage(int n) { return bar(n % N); }
    // the same by the stage's own number, for those who count it along
    static __device__ __forceinline__ int bar(int st) { return (WHICH ? C::kFirst : 0) + st; }
    static __device__ __forceinline__ uint32_t at(int st) { return C::kRing + bar(st) * C::kTileBytes; }
    static __device__ __forceinline__ int after(int st) { return st + 1 == N ? 0 : st + 1; }
    static __device__ __forceinline__ uint32_t place(int n) { return C::kRing + stage(n) * C::kTileBytes; }
    static __device__ __forceinline__ uint32_t parity(int n) { return (n / N) & 1; }
    // until the stage is free for load n
    static __device__ __forceinline__ bool wait_free(GradBars &bars, int n) {
        return n < N || warp_wait(&bars.empty[stage(n)], (n / N - 1) & 1, &bars.abort);
    }
    static __device__ __forceinline__ bool wait_full(GradBars &bars, int n) {
        return warp_wait(&bars.full[stage(n)], parity(n), &bars.abort);
    }
    // waits for load n and zeroes its rows from `rows` on, where that is below 128; a whole warp
    static __device__ __forceinline__ bool watch(GradBars &bars, uint8_t *smem, int n, int rows, int lane) {
        if (!wait_full(bars, n)) return false;
        if (rows < kTile) {
            zero_rows<D>(smem + place(n), rows, lane);
            __syncwarp();
        }
        return true;
    }
    // after a wait that ran out: until the last loads before n are there
    static __device__ __forceinline__ void drain(GradBars &bars, int n) {
        for (int k = max(0, n - N); k < n; ++k) {
            int quit = 0;
            bounded_wait(&bars.full[stage(k)], parity(k), &quit);
        }
    }
};

// The block's r-th item, handed out by warp 17 (`give`) and taken by the others (`take`; false after a
// wait that ran out).
__device__ __forceinline__ bool give_item(GradBars &bars, const GradItem &w, int r, int lane) {
    if (r >= 2 && !warp_wait(&bars.item_empty[r & 1], ((r >> 1) - 1) & 1, &bars.abort)) return false;
    if (lane == 0) {
        bars.item[r & 1] = w;
        tc::mbar_arrive(&bars.item_full[r & 1]);
    }
    return true;
}
__device__ __forceinline__ bool take_item(GradBars &bars, GradItem &w, int r, int lane) {
    if (!warp_wait(&bars.item_full[r & 1], (r >> 1) & 1, &bars.abort)) return false;
    w = bars.item[r & 1];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bars.item_empty[r & 1]);
    return true;
}
// The same for warps that read the item again when its turns are over: it stays until leave_item.
__device__ __forceinline__ bool see_item(GradBars &bars, int r) {
    return warp_wait(&bars.item_full[r & 1], (r >> 1) & 1, &bars.abort);
}
__device__ __forceinline__ void leave_item(GradBars &bars, int r, int lane) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bars.item_empty[r & 1]);
}
// Blocks take items there and back, so that none has the longest of every round.
__device__ __forceinline__ int64_t item_index(int r) {
    return (int64_t)r * gridDim.x + (r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// 32 numbers of a thread's row, rounded, into Tensor Memory as an operand, over the first 16 columns of
// the 32 that they were read from; FINE: and what rounding took from them over the other 16.
template <bool FINE> __device__ __forceinline__ void put_operand(uint32_t taddr, const float2 (&x)[16]) {
    uint32_t u[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) u[e] = pack_bf16(x[e].x, x[e].y);
    tc::tmem_st16(taddr, u);
    if constexpr (FINE) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            u[e] = pack_bf16(x[e].x - __uint_as_float(u[e] << 16), x[e].y - __uint_as_float(u[e] & 0xffff0000u));
        tc::tmem_st16(taddr + 16, u);
    }
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

// N columns of a thread's row of an accumulator to global memory.
template <int N> __device__ __forceinline__ void store_columns(uint32_t taddr, __nv_bfloat16 *dst, float mul, bool zero, bool there) {
#pragma unroll
    for (int c = 0; c < N; c += 16) {
        float x[16];
        if (!zero) {
            tc::tmem_ld16(taddr + c, x);
            tc::tmem_ld_wait();
        }
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = zero ? 0u : pack_bf16(x[2 * e] * mul, x[2 * e + 1] * mul);
        if (there) store_sector(dst + c, u);
    }
}

// ---- dK and dV ----------------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(GradCfg<D>::kThreads, 1)
attn_grad_kv_tc_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ PromptMaps maps) {
    using C = GradCfg<D>;
    using R1 = Ring<D, 0>;   // Q
    using R2 = Ring<D, 1>;   // dO
    extern __shared__ __align__(1024) uint8_t smem[];
    GradBars &bars = *reinterpret_cast<GradBars *>(smem + C::kBars);
    const uint32_t sbase = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // With d = 64 there is Tensor Memory for the next turn's scores beside this one's: they are formed ahead,
    // and the powers of a turn follow the dS of the one before without a product in between.
    constexpr bool kAhead = D == 64;

    next_may_start();
    const uint32_t tmem = grad_setup<D>(bars, {1, kAhead ? 16 : 17, 17, 19});
    if (tid == 32 && a.bt.Tq > 0) prefetch_map(&maps.q), prefetch_map(&maps.k), prefetch_map(&maps.v), prefetch_map(&maps.g);
    wait_for_previous();
    zero_behind(static_cast<__nv_bfloat16 *>(a.dk), a.bt.cu_k, a.bt.n, a.bt.Tk, a.bt.Hkv * D);
    zero_behind(static_cast<__nv_bfloat16 *>(a.dv), a.bt.cu_k, a.bt.n, a.bt.Tk, a.bt.Hkv * D);

    volatile int *abort = &bars.abort;
    const int group = a.bt.Hq / a.bt.Hkv;
    const uint32_t tP = tmem + kTile, tV = tmem + 2 * kTile, tK = tV + D;
    auto tS = [&](int n) { return kAhead && (n & 1) ? tK + D : tmem; };
    float *stats = reinterpret_cast<float *>(smem + C::kStats);
    // Over all items: `base` turns and `own` items with turns before this one.  Turn `it` of an item is a tile
    // of queries of one of the group's heads; its Q and dO are loads base + it.
    int base = 0, own = 0;
    bool ok = true;
    GradItem w;

    if (warp == 17) {
        int put1 = 0, put2 = 0;   // loads under way
        PlaceFrom from;
        for (int r = 0;; ++r) {
            // the first keys of a sequence are seen by the most queries: they go first
            int n, count, level;
            const int64_t index = item_index(r);
            w.total = -1;
            if (place_of(a.bt.cu_k, a.bt.n, a.bt.Tk, kTile, index / a.bt.Hkv, lane, n, count, level, from)) {
                const Seq s = seq_of(a.bt, n);
                w.q0 = s.q0, w.k0 = s.k0, w.nq = s.nq, w.nk = s.nk;
                w.head = (int)(index % a.bt.Hkv);
                w.row0 = (count - level) * kTile;
                w.start = a.causal ? max(0, w.row0 - (s.nk - s.nq)) / kTile : 0;   // query i sees keys j <= i + nk - nq
                w.per_head = max(0, (s.nq + kTile - 1) / kTile - w.start);
                w.total = w.per_head * group;
                // the first query of tile t sees t kTile + 1 + nk - nq keys
                w.fine = s.nk <= kFineKeys ? w.per_head
                         : a.causal ? min(w.per_head, max(0, (kFineKeys - (s.nk - s.nq) + kTile - 1) / kTile - w.start)) : 0;
            }
            if (!(ok = give_item(bars, w, r, lane)) || w.total < 0) break;
            if (w.total == 0) continue;
            if (own > 0 && !(ok = warp_wait(&bars.own_empty, (own - 1) & 1, abort))) break;
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&bars.own_full, 2 * C::kTileBytes);
                tma_tile<D>(C::kOwn, smem, &maps.k, w.head, w.k0 + w.row0, &bars.own_full);
                tma_tile<D>(C::kOwn + C::kTileBytes, smem, &maps.v, w.head, w.k0 + w.row0, &bars.own_full);
            }
            ++own;
            for (int it = 0; it < w.total && ok; ++it, ++base) {
                const int h = w.head * group + it / w.per_head, r0 = (w.start + it % w.per_head) * kTile;
                if (!(ok = R1::wait_free(bars, base))) break;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&bars.full[R1::stage(base)], C::kTileBytes);
                    tma_tile<D>(R1::place(base), smem, &maps.q, h, w.q0 + r0, &bars.full[R1::stage(base)]);
                }
                put1 = base + 1;
                if (!(ok = R2::wait_free(bars, base))) break;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&bars.full[R2::stage(base)], C::kTileBytes);
                    tma_tile<D>(R2::place(base), smem, &maps.g, h, w.q0 + r0, &bars.full[R2::stage(base)]);
                }
                put2 = base + 1;
            }
            if (!ok) break;
        }
        if (!ok && lane == 0) {   // leave no copy in flight
            int quit = 0;
            if (own > 0) bounded_wait(&bars.own_full, (own - 1) & 1, &quit);
            R1::drain(bars, put1);
            R2::drain(bars, put2);
        }
    } else if (warp == 19) {
        // -lse in log2 units, -inf (weight zero) where there is no query or it sees nothing; -delta.  Read a
        // turn before they are needed: the loads wait long behind the tiles' traffic.
        for (int r = 0; ok && (ok = take_item(bars, w, r, lane)) && w.total >= 0; ++r) {
            if (w.total == 0) continue;
            const int64_t at0 = stat_at(a.bt, w.q0, 0);   // a head's rows of a sequence lie side by side
            float ls[4], de[4];
            int h = w.head * group, r0 = w.start * kTile;
            auto fetch = [&]() {
                const int64_t at = at0 + (int64_t)h * a.bt.Tq + r0 + lane;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool there = r0 + e * 32 + lane < w.nq;
                    ls[e] = there ? a.lse[at + e * 32] : -CUDART_INF_F;
                    de[e] = there ? a.delta[at + e * 32] : 0.f;
                }
                if ((r0 += kTile) >= w.nq) r0 = w.start * kTile, ++h;
            };
            fetch();
            for (int it = 0; it < w.total; ++it, ++base) {
                float l[4], d[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l[e] = ls[e] == -CUDART_INF_F ? ls[e] : -ls[e] * kLog2e;
                    d[e] = -de[e];
                }
                if (it + 1 < w.total) fetch();
                if (base >= 2 && !(ok = warp_wait(&bars.stats_read[base & 1], (base / 2 - 1) & 1, abort))) break;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    stats[(base & 1) * 2 * kTile + e * 32 + lane] = l[e];
                    stats[(base & 1) * 2 * kTile + kTile + e * 32 + lane] = d[e];
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars.stats[base & 1]);
            }
        }
    } else if (warp == 18) {
        // Queries that are not there are summed over with weight zero.  The word on the next Q goes with the
        // weights of this turn (or by itself), that on the next dO with its dS; each word belongs to one turn.
        for (int r = 0; ok && (ok = take_item(bars, w, r, lane)) && w.total >= 0; ++r) {
            for (int it = 0; it <= w.total && w.total > 0 && ok; ++it) {
                const bool load = it < w.total;   // the last turn has no next one
                const int n = base + it, left = load ? w.nq - (w.start + it % w.per_head) * kTile : kTile;
                if (load && !(ok = R1::watch(bars, smem, n, left, lane))) break;
                if (it > 0 && !kAhead && lane == 0) tc::mbar_arrive(&bars.a_ready[(n - 1) & 1]);
                if (it > 0 && kAhead && load) {   // not before the last word has been heard
                    if (it > 1 && !(ok = wait_turn(bars.s_full, n - 1, abort))) break;
                    if (lane == 0) tc::mbar_arrive(&bars.q_word);
                }
                if (load && !(ok = R2::watch(bars, smem, n, left, lane))) break;
                if (lane == 0) tc::mbar_arrive(it == 0 ? &bars.first : &bars.b_ready[(n - 1) & 1]);
                if (it > 0) ok = wait_turn(bars.b_ready, n - 1, abort);   // a_ready's turn is over, too
            }
            base += w.total;
        }
    } else if (warp == 16) {
        constexpr uint32_t idS = tc::make_idesc_bf16(kTile, kTile, false, false);
        constexpr uint32_t idG = tc::make_idesc_bf16(kTile, D, false, true);
        const uint32_t leader = elect_lane();
        const uint64_t dK = desc_k(sbase + C::kOwn, 0), dV = desc_k(sbase + C::kOwn + C::kTileBytes, 0);
        int words = 0, st1 = 0, st2 = 0;   // this turn's stages
        auto scores = [&](int n, int st) {
            chain_ss<D>(tS(n), dK, desc_k(sbase + R1::at(st), 0), idS, leader);
            commit_by(&bars.s_full[n & 1], leader);
        };
        auto products = [&](int n, int st, bool last) {   // dP; the item's own tiles are done with after its last
            chain_ss<D>(tP, dV, desc_k(sbase + R2::at(st), 0), idS, leader);
            commit_by(&bars.dp_full[n & 1], leader);
            if (last) commit_by(&bars.own_empty, leader);
        };
        for (int r = 0; ok && (ok = take_item(bars, w, r, lane)) && w.total >= 0; ++r) {
            const int total = w.total;
            if (total == 0) continue;
            ok = warp_wait(&bars.own_full, own & 1, abort) && warp_wait(&bars.first, own & 1, abort);
            if (!ok) break;
            scores(base, st1);
            products(base, st2, total == 1);
            for (int it = 0, of_head = 0; it < total; ++it, ++base) {
                const bool more = it + 1 < total, fine = of_head < w.fine;
                if (++of_head == w.per_head) of_head = 0;
                const int next1 = R1::after(st1), next2 = R2::after(st2);
                const uint64_t q = desc_mn(sbase + R1::at(st1), 0), g = desc_mn(sbase + R2::at(st2), 0);
                if (kAhead && more) {
                    if (!(ok = warp_wait(&bars.q_word, words & 1, abort))) break;
                    ++words;
                    scores(base + 1, next1);
                }
                if (!(ok = wait_turn(bars.a_ready, base, abort))) break;
                tc::tc_fence_after();
                chain_ts32(tV, tS(base), g, idG, it > 0, leader);
                if (fine) chain_ts32(tV, tS(base) + 16, g, idG, true, leader);
                if (!kAhead && more) scores(base + 1, next1);
                commit_by(&bars.empty[R2::bar(st2)], leader);
                if (!(ok = wait_turn(bars.b_ready, base, abort))) break;
                tc::tc_fence_after();
                chain_ts32(tK, tP, q, idG, it > 0, leader);
                if (fine) chain_ts32(tK, tP + 16, q, idG, true, leader);
                if (more) products(base + 1, next2, it + 2 == total);
                commit_by(&bars.empty[R1::bar(st1)], leader);
                if (!more) commit_by(&bars.done, leader);
                st1 = next1;
                st2 = next2;
            }
            ++own;
        }
        if (!ok || *abort) {   // no product in flight when the memory is given back
            int quit = 0;
            commit_by(&bars.drain, leader);
            warp_wait(&bars.drain, 0, &quit);
        }
    } else {
        const int part = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tc::tmem_lane_base(warp) + part * 32;
        const float sc = a.scale * kLog2e;
        const float2 sc2 = make_float2(sc, sc);
        for (int r = 0; ok && (ok = see_item(bars, r)) && bars.item[r & 1].total >= 0; ++r) {
            const volatile GradItem &w = bars.item[r & 1];   // read where it is needed, not kept
            const int total = w.total, begin = w.start * kTile, nq = w.nq;
            // this row's key is seen from this query on (where masked), and by the warp's rows all
            const int sees = a.causal ? w.row0 + row - (w.nk - nq) : INT_MIN / 2, all_see = sees + 31 - lane;
            int r0 = begin;
            auto turns = [&](auto fine, int number) {   // once for either kind of operands: a test in each turn costs 4%
            for (int it = 0; it < number; ++it, ++base) {
                const float *ls = stats + (base & 1) * 2 * kTile + part * 32, *de = ls + kTile;
                const int from = sees - r0 - part * 32;   // hidden columns before it
                const bool partly = all_see - r0 - part * 32 > 0;
                if ((r0 += kTile) >= nq) r0 = begin;
                ok = warp_wait(&bars.stats[base & 1], (base >> 1) & 1, abort) && wait_turn(bars.s_full, base, abort);
                if (!ok) break;
                tc::tc_fence_after();
                float2 p[16];
                {
                    float x[32];
                    tc::tmem_ld32(tS(base) + lanes, x);
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
                put_operand<decltype(fine)::value>(tS(base) + lanes, p);
                arrive_operand(&bars.a_ready[base & 1], lane);
                ok = wait_turn(bars.dp_full, base, abort);
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
                put_operand<decltype(fine)::value>(tP + lanes, p);
                arrive_operand(&bars.b_ready[base & 1], lane);
                if (lane == 0) tc::mbar_arrive(&bars.stats_read[base & 1]);
            }
            };
            for (int left = total; ok && left > 0; left -= w.per_head) {   // the group's heads
                turns(std::true_type(), w.fine);
                if (ok) turns(std::false_type(), w.per_head - w.fine);
            }
            if (ok && total > 0) ok = warp_wait(&bars.done, own++ & 1, abort);
            if (!ok) break;
            tc::tc_fence_after();
            // two groups of columns of dV, two of dK
            const int key = w.row0 + row;
            const bool is_k = part & 2, there = key < w.nk;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(is_k ? a.dk : a.dv) +
                                 ((w.k0 + key) * a.bt.Hkv + w.head) * (int64_t)D + (part & 1) * (D / 2);
            leave_item(bars, r, lane);
            store_columns<D / 2>((is_k ? tK : tV) + tc::tmem_lane_base(warp) + (part & 1) * (D / 2), dst,
                                 is_k ? a.scale : 1.f, total == 0, there);
        }
    }
    __syncwarp();
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
    using R1 = Ring<D, 0>;   // K
    using R2 = Ring<D, 1>;   // an item's tile of O, then V
    extern __shared__ __align__(1024) uint8_t smem[];
    GradBars &bars = *reinterpret_cast<GradBars *>(smem + C::kBars);
    const uint32_t sbase = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    next_may_start();
    const uint32_t tmem = grad_setup<D>(bars, {2, 17, 16, 18});
    if (tid == 32 && a.bt.Tk > 0)
        prefetch_map(&maps.q), prefetch_map(&maps.k), prefetch_map(&maps.v), prefetch_map(&maps.g), prefetch_map(&maps.o);
    wait_for_previous();
    zero_behind(static_cast<__nv_bfloat16 *>(a.dq), a.bt.cu_q, a.bt.n, a.bt.Tq, a.bt.Hq * D);

    volatile int *abort = &bars.abort;
    const uint32_t tS = tmem, tP = tmem + kTile, tQ = tmem + 3 * kTile;
    // Over all items: `base` turns and `own` items with turns before this one.  Turn j is key tile j: K is load
    // base + j of the first ring; of the second, O is load base + own, V load base + own + 1 + j.
    int base = 0, own = 0;
    bool ok = true;
    GradItem w;

    if (warp == 17) {
        int put1 = 0, put2 = 0;   // loads under way
        PlaceFrom from;
        for (int r = 0;; ++r) {
            int n, count, level;
            const int64_t index = item_index(r);
            w.total = -1;
            if (place_of(a.bt.cu_q, a.bt.n, a.bt.Tq, kTile, index / a.bt.Hq, lane, n, count, level, from)) {
                const Seq s = seq_of(a.bt, n);
                w.q0 = s.q0, w.k0 = s.k0, w.nq = s.nq, w.nk = s.nk;
                w.head = (int)(index % a.bt.Hq);
                w.row0 = (level - 1) * kTile;
                w.total = (keys_seen(s, min(w.row0 + kTile, s.nq) - 1, a.causal) + kTile - 1) / kTile;
                w.fine = keys_seen(s, w.row0, a.causal) <= kFineKeys;
            }
            if (!(ok = give_item(bars, w, r, lane)) || w.total < 0) break;
            if (w.total == 0) continue;
            const int hk = w.head / (a.bt.Hq / a.bt.Hkv);
            if (own > 0 && !(ok = warp_wait(&bars.own_empty, (own - 1) & 1, abort))) break;
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&bars.own_full, 2 * C::kTileBytes);
                tma_tile<D>(C::kOwn, smem, &maps.q, w.head, w.q0 + w.row0, &bars.own_full);
                tma_tile<D>(C::kOwn + C::kTileBytes, smem, &maps.g, w.head, w.q0 + w.row0, &bars.own_full);
            }
            auto load2 = [&](int m, const CUtensorMap *map, int head, int64_t row) {
                if (!R2::wait_free(bars, m)) return false;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&bars.full[R2::stage(m)], C::kTileBytes);
                    tma_tile<D>(R2::place(m), smem, map, head, row, &bars.full[R2::stage(m)]);
                }
                put2 = m + 1;
                return true;
            };
            ok = load2(base + own, &maps.o, w.head, w.q0 + w.row0);
            ++own;
            for (int j = 0; j < w.total && ok; ++j, ++base) {
                if (!(ok = R1::wait_free(bars, base))) break;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&bars.full[R1::stage(base)], C::kTileBytes);
                    tma_tile<D>(R1::place(base), smem, &maps.k, hk, w.k0 + (int64_t)j * kTile, &bars.full[R1::stage(base)]);
                }
                put1 = base + 1;
                ok = load2(base + own, &maps.v, hk, w.k0 + (int64_t)j * kTile);
            }
            if (!ok) break;
        }
        if (!ok && lane == 0) {   // leave no copy in flight
            int quit = 0;
            if (own > 0) bounded_wait(&bars.own_full, (own - 1) & 1, &quit);
            R1::drain(bars, put1);
            R2::drain(bars, put2);
        }
    } else if (warp == 18) {
        // Keys that are not there are summed over with weight zero (their values only masked).  The word on
        // the next K and V goes with the reading of this turn's scores.
        for (int r = 0; ok && (ok = take_item(bars, w, r, lane)) && w.total >= 0; ++r) {
            if (w.total == 0) continue;
            for (int j = 0; j <= w.total && ok; ++j) {
                const int n = base + j;
                if (j < w.total) {   // the last turn has no next one
                    ok = R1::watch(bars, smem, n, w.nk - j * kTile, lane) && R2::wait_full(bars, n + own + 1);
                    if (!ok) break;
                }
                if (lane == 0) tc::mbar_arrive(j == 0 ? &bars.first : &bars.a_ready[(n - 1) & 1]);
                if (j == 0) {   // O has been read, and dO by all but the products
                    ok = warp_wait(&bars.out_read, own & 1, abort);
                    if (ok && lane == 0) {
                        tc::mbar_arrive(&bars.empty[R2::stage(base + own)]);
                        tc::mbar_arrive(&bars.own_empty);
                    }
                } else {
                    ok = wait_turn(bars.a_ready, n - 1, abort);
                }
            }
            base += w.total;
            ++own;
        }
    } else if (warp == 16) {
        constexpr uint32_t idS = tc::make_idesc_bf16(kTile, kTile, false, false);
        constexpr uint32_t idG = tc::make_idesc_bf16(kTile, D, false, true);
        const uint32_t leader = elect_lane();
        const uint64_t dQ = desc_k(sbase + C::kOwn, 0), dG = desc_k(sbase + C::kOwn + C::kTileBytes, 0);
        int st1 = 0, st2 = 0;   // stages of this turn's K and of the next load of the second ring
        auto scores = [&](int n, int st, bool last) {   // S and dP; dP alternates between two places
            chain_ss<D>(tS, dQ, desc_k(sbase + R1::at(st), 0), idS, leader);
            commit_by(&bars.s_full[n & 1], leader);
            chain_ss<D>(tP + (n & 1) * kTile, dG, desc_k(sbase + R2::at(st2), 0), idS, leader);
            commit_by(&bars.dp_full[n & 1], leader);
            commit_by(&bars.empty[R2::bar(st2)], leader);
            if (last) commit_by(&bars.own_empty, leader);
            st2 = R2::after(st2);
        };
        for (int r = 0; ok && (ok = take_item(bars, w, r, lane)) && w.total >= 0; ++r) {
            const int total = w.total;
            if (total == 0) continue;
            ok = warp_wait(&bars.own_full, own & 1, abort) && warp_wait(&bars.first, own & 1, abort);
            if (!ok) break;
            st2 = R2::after(st2);   // O's
            scores(base, st1, total == 1);
            for (int j = 0; j < total; ++j, ++base) {
                const int next1 = R1::after(st1);
                const uint64_t k = desc_mn(sbase + R1::at(st1), 0);
                // the next scores as soon as these have been read
                if (!(ok = wait_turn(bars.a_ready, base, abort))) break;
                tc::tc_fence_after();
                if (j + 1 < total) scores(base + 1, next1, j + 2 == total);
                if (!(ok = wait_turn(bars.b_ready, base, abort))) break;
                tc::tc_fence_after();
                chain_ts32(tQ, tP + (base & 1) * kTile, k, idG, j > 0, leader);
                if (w.fine) chain_ts32(tQ, tP + (base & 1) * kTile + 16, k, idG, true, leader);
                commit_by(&bars.empty[R1::bar(st1)], leader);
                if (j + 1 == total) commit_by(&bars.done, leader);
                st1 = next1;
            }
            ++own;
        }
        if (!ok || *abort) {   // no product in flight when the memory is given back
            int quit = 0;
            commit_by(&bars.drain, leader);
            warp_wait(&bars.drain, 0, &quit);
        }
    } else if (warp < 16) {
        const int part = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tc::tmem_lane_base(warp) + part * 32;
        const float sc = a.scale * kLog2e;
        const float2 sc2 = make_float2(sc, sc);
        float *parts = reinterpret_cast<float *>(smem + C::kStats);
        for (int r = 0; ok && (ok = see_item(bars, r)) && bars.item[r & 1].total >= 0; ++r) {
            const volatile GradItem &w = bars.item[r & 1];   // read where it is needed, not kept
            const int total = w.total, qi = w.row0 + row;
            int seen, seen_all;   // keys that this row sees, and every row of the warp
            bool there;
            float ls = -CUDART_INF_F;
            int64_t at = 0;
            {
                const Seq s{0, 0, w.nq, w.nk};
                there = qi < s.nq;
                seen = there ? keys_seen(s, qi, a.causal) : 0;
                seen_all = qi - lane + 31 < s.nq ? keys_seen(s, qi - lane, a.causal) : 0;
                if (there) {
                    at = stat_at(a.bt, w.q0 + qi, w.head);
                    ls = a.lse[at] * kLog2e;
                }
                if (ls != -CUDART_INF_F) ls = -ls;
            }
            float de = 0.f;
            if (total > 0) {
                // delta = dO . O of this row, a quarter of the channels in each group, with O as exact as the
                // forward gives it: a delta from the rounded O alone errs by as much as rounding dS does
                uint4 rest[D / 32];
#pragma unroll
                for (int y = 0; y < D / 32; ++y)
                    rest[y] = a.rest && there ? reinterpret_cast<const uint4 *>(
                                                    static_cast<const __nv_bfloat16 *>(a.rest) +
                                                    ((w.q0 + qi) * a.bt.Hq + w.head) * (int64_t)D)[part * (D / 32) + y]
                                              : make_uint4(0, 0, 0, 0);
                ok = warp_wait(&bars.own_full, own & 1, abort) && R2::wait_full(bars, base + own);
                if (!ok) break;
                const uint8_t *g = smem + C::kOwn + C::kTileBytes, *o = smem + R2::place(base + own);
#pragma unroll
                for (int y = 0; y < D / 32; ++y) {
                    const int c = part * (D / 32) + y;
                    const uint32_t off = (c >> 3) * (kTile * 128) + tc::sw128(row, c & 7);
                    const uint4 u = *reinterpret_cast<const uint4 *>(g + off), v = *reinterpret_cast<const uint4 *>(o + off);
                    const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w},
                                   rs[4] = {rest[y].x, rest[y].y, rest[y].z, rest[y].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        de = fmaf(__uint_as_float(us[e] << 16), __uint_as_float(vs[e] << 16) + __uint_as_float(rs[e] << 16), de);
                        de = fmaf(__uint_as_float(us[e] & 0xffff0000u),
                                  __uint_as_float(vs[e] & 0xffff0000u) + __uint_as_float(rs[e] & 0xffff0000u), de);
                    }
                }
                parts[part * kTile + row] = de;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars.out_read);
                if (!(ok = warp_wait(&bars.out_read, own & 1, abort))) break;
                de = (parts[row] + parts[kTile + row]) + (parts[2 * kTile + row] + parts[3 * kTile + row]);
            }
            if (part == 0 && there) a.delta[at] = de;
            const float2 ls2 = make_float2(ls, ls), de2 = make_float2(-de, -de);
            auto turns = [&](auto fine) {
            for (int j = 0; j < total; ++j, ++base) {
                const uint32_t dp = tP + (base & 1) * kTile + lanes;
                const int limit = seen - j * kTile - part * 32;   // columns at or past it are hidden
                const bool partly = j * kTile + (part + 1) * 32 > seen_all;
                if (!(ok = wait_turn(bars.s_full, base, abort))) break;
                tc::tc_fence_after();
                float2 p[16];
                {
                    float x[32];
                    tc::tmem_ld32(tS + lanes, x);
                    tc::tmem_ld_wait();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bars.a_ready[base & 1]);
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[e] = fma2(make_float2(x[2 * e], x[2 * e + 1]), sc2, ls2);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) p[e] = make_float2(ex2_approx(p[e].x), ex2_approx(p[e].y));
                if (!(ok = wait_turn(bars.dp_full, base, abort))) break;
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
                put_operand<decltype(fine)::value>(dp, p);
                arrive_operand(&bars.b_ready[base & 1], lane);
            }
            };
            if (w.fine) turns(std::true_type());
            else turns(std::false_type());
            if (ok && total > 0) ok = warp_wait(&bars.done, own++ & 1, abort);
            if (!ok) break;
            tc::tc_fence_after();
            const int to = w.row0 + row;
            const bool write = to < w.nq;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.dq) + ((w.q0 + to) * a.bt.Hq + w.head) * (int64_t)D + part * (D / 4);
            leave_item(bars, r, lane);
            store_columns<D / 4>(tQ + tc::tmem_lane_base(warp) + part * (D / 4), dst, a.scale, total == 0, write);
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D> cudaError_t launch_prompt_grad_tc(const PromptArgs &a, int sms, cudaStream_t st) {
    using C = GradCfg<D>;
    cudaError_t e;
    // items, an upper bound
    const int64_t gk = a.bt.Tk == 0 ? 0 : max_tiles(a.bt.cu_k, a.bt.n, a.bt.Tk, kTile) * a.bt.Hkv;
    const int64_t gq = a.bt.Tq == 0 ? 0 : max_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq, kTile) * a.bt.Hq;
    // before the maps: it binds the device's context to this thread (autograd's may have none yet), which
    // their encoding needs
    if ((e = allow_smem(attn_grad_q_tc_kernel<D>, C::kSmem)) != cudaSuccess) return e;
    PromptMaps maps = {};
    if (a.bt.Tq > 0 && !encode_prompt_maps(maps, a, D)) return cudaErrorInvalidValue;
    if (gq > 0) {   // first: it forms the delta that the other reads
        if ((e = launch_behind(attn_grad_q_tc_kernel<D>, (unsigned)(gq < sms ? gq : sms), C::kThreads, C::kSmem, st, a,
                               maps)) != cudaSuccess)
            return e;
    }
    if (gk > 0) {
        if ((e = allow_smem(attn_grad_kv_tc_kernel<D>, C::kSmem)) != cudaSuccess) return e;
        return launch_behind(attn_grad_kv_tc_kernel<D>, (unsigned)(gk < sms ? gk : sms), C::kThreads, C::kSmem, st, a, maps);
    }
    return cudaSuccess;
}

}  // namespace attn
}  // namespace kda
