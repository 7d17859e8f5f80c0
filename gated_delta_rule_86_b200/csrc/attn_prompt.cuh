// attn_prompt.cuh -- attention over whole prompts and its gradient, fp32 arithmetic on CUDA cores.
//
//     S = scale Q K^T,  masked where the query does not see the key,  P = softmax(S),  O = P V,
//     lse_i = log sum_j exp(S_ij)
// in one pass over the keys with a running row maximum and sum.  With causal masking query i of a
// sequence of nq queries and nk keys sees keys j <= i + nk - nq; a row that sees none gives O = 0 and
// lse = -inf.  The gradient, from P_ij = exp(S_ij - lse_i) computed again:
//     delta_i = dO_i . O_i,   dP = dO V^T,   dS = P o (dP - delta),
//     dV = P^T dO,   dK = scale dS^T Q,   dQ = scale dS K.
// dK and dV are summed over the query heads of a group inside one block, dQ over the keys inside
// another, so there are no atomics: the same call gives the same bits.  (S and dP are computed in both,
// seven products in place of five.)
//
// fp32 inputs ask for fp32 accuracy, which the tensor cores' operands do not give; these kernels are
// bound by the FMA units and, for small batches, by the latency of a tile.  A block has ROWS rows of one
// head and walks tiles of 64 of the other side; thread (ty, tx) holds RPT x 4 scores, rows
// RPT ty and on, so a row's 16 threads lie in one half of a warp and its maximum and sum are four shuffles.
// Large batches have 64 rows a block and 4 a thread (16 products for 8 loads from shared memory), small
// ones 16 and 2 (4 warps; with 1 a thread and 8 warps shared memory is read more and the time is the same:
// B1 T256 H2 D64 14 us forward, 43 gradient in two launches, against 14 and 45).  The next tile is on its way (cp.async) while one is worked on.
#pragma once

#include "attn_append.cuh"
#include "attn_common.cuh"

namespace kda {
namespace attn {

struct PromptArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements from one token to the next
    Batch bt;
    bool causal;
    float scale;
    void *out;
    void *rest;                             // bf16: what rounding took from out, or null
    float *lse;                             // [B][Hq][Tq]
    // gradient only
    const void *d_out;
    float *delta;                           // workspace [B][Hq][Tq]
    void *dq, *dk, *dv;
};

// Place of a query's lse and delta: row = its row in the flattened [B * Tq] tensors.
__device__ __forceinline__ int64_t stat_at(const Batch &bt, int64_t row, int h) {
    const int64_t b = bt.cu_q ? 0 : row / bt.Tq;
    return (b * bt.Hq + h) * bt.Tq + (row - b * bt.Tq);
}

constexpr int kPT = 64;   // rows of a tile of the other side

template <int D> struct PromptCfg {
    static constexpr int kPitch = D + 4;           // floats of a staged row
    static constexpr int kTileF = kPT * kPitch;
    // own tiles of `rows` rows, `ring` tiles of the other side (two or three, twice), weights [rows][68], statistics
    static constexpr int smem(int rows, int own, int ring = 4) {
        return (own * rows * kPitch + ring * kTileF + rows * 68 + 2 * 2 * kPT) * 4 + 160;
    }
};

__device__ __forceinline__ void copy16(float *dst, const float *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Rows [r0, r0 + N) of a head into shared memory, zeros at or past `rows`.
template <int D, int N, int THREADS>
__device__ __forceinline__ void stage_rows(float *dst, const float *src, int64_t stride, int r0, int rows) {
#pragma unroll 4
    for (int i = threadIdx.x; i < N * D / 4; i += THREADS) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        const bool there = r0 + r < rows;
        copy16(dst + r * (D + 4) + c, src + (there ? (int64_t)(r0 + r) * stride + c : 0), there);
    }
}

// acc[i][j] += A[RPT ty + i] . B[tx + 16 j] over D channels (pitch D + 4)
template <int D, int RPT>
__device__ __forceinline__ void dot_rows(float (&acc)[RPT][4], const float *A, const float *B, int ty, int tx) {
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 a[RPT], b[4];
#pragma unroll
        for (int i = 0; i < RPT; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (RPT * ty + i) * (D + 4) + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * (D + 4) + c);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] += a[i].x * b[j].x + a[i].y * b[j].y + a[i].z * b[j].z + a[i].w * b[j].w;
    }
}

// acc[i][c] += sum_t W[RPT ty + i][t] X[t][channel c of tx]  (W pitch 68, X pitch D + 4).  APART: a tile's 64 products
// are summed by themselves first, since one sum over all tiles errs as the root of all its terms: dK over 16 heads of
// 1024 queries by 2.3e-6 of its size, and 4.5e-7 so.  It is free but for blocks of 16 rows (forward, heads of 128, 10%;
// dQ, 5%), which have the fewest terms and do without it where they sum over keys alone.
template <bool APART, int D, int RPT>
__device__ __forceinline__ void weigh_rows(float (&acc)[RPT][D / 16], const float *W, const float *X, int ty, int tx) {
    float tile[RPT][D / 16] = {};
    auto &sum = *[&] {
        if constexpr (APART) return &tile;
        else return &acc;
    }();
#pragma unroll 2
    for (int t = 0; t < kPT; t += 4) {
        float4 w[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) w[i] = *reinterpret_cast<const float4 *>(W + (RPT * ty + i) * 68 + t);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float x[D / 16];
#pragma unroll
            for (int c = 0; c < D / 16; c += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(X + (t + u) * (D + 4) + tx * 4 + (c / 4) * 64);
                x[c] = f.x, x[c + 1] = f.y, x[c + 2] = f.z, x[c + 3] = f.w;
            }
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float wi = u == 0 ? w[i].x : u == 1 ? w[i].y : u == 2 ? w[i].z : w[i].w;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) sum[i][c] += wi * x[c];
            }
        }
    }
    if constexpr (APART)
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[i][c] += tile[i][c];
}

// A thread's channels of one row: tx * 4 + {0 .. 3}, + 64 for the second four.
template <int D> __device__ __forceinline__ void write_row(float *dst, const float (&acc)[D / 16], int tx, float mul) {
#pragma unroll
    for (int c = 0; c < D / 16; c += 4)
        *reinterpret_cast<float4 *>(dst + tx * 4 + (c / 4) * 64) =
            make_float4(acc[c] * mul, acc[c + 1] * mul, acc[c + 2] * mul, acc[c + 3] * mul);
}

// A thread's weights into shared memory; a row's come from the half warp that reads them.
template <int RPT> __device__ __forceinline__ void put_weights(float *sp, const float (&x)[RPT][4], int ty, int tx) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sp[(RPT * ty + i) * 68 + tx + 16 * j] = x[i][j];
    __syncwarp();
}

template <int ROWS> struct RowsCfg {
    static constexpr int kPer = ROWS == 64 ? 4 : 2;        // rows of a thread
    static constexpr int kThreads = ROWS / kPer * 16;
};

template <int D, int ROWS>
__global__ void __launch_bounds__(RowsCfg<ROWS>::kThreads) attn_prompt_kernel(const PromptArgs a) {
    using C = PromptCfg<D>;
    constexpr int THREADS = RowsCfg<ROWS>::kThreads, RPT = RowsCfg<ROWS>::kPer;
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *ring = sq + ROWS * C::kPitch, *sp = ring + 4 * C::kTileF;
    int *scratch = reinterpret_cast<int *>(sp + ROWS * 68 + 4 * kPT);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, h = blockIdx.y;
    int n, t;
    if (!find_tile(a.bt.cu_q, a.bt.n, a.bt.Tq, ROWS, gridDim.x - 1 - blockIdx.x, scratch, n, t)) return;
    const Seq s = seq_of(a.bt, n);
    const int r0 = t * ROWS, hk = h / (a.bt.Hq / a.bt.Hkv);
    const float *q = static_cast<const float *>(a.q) + s.q0 * a.q_stride + (int64_t)h * D;
    const float *k = static_cast<const float *>(a.k) + s.k0 * a.k_stride + (int64_t)hk * D;
    const float *v = static_cast<const float *>(a.v) + s.k0 * a.v_stride + (int64_t)hk * D;
    const int end = keys_seen(s, min(r0 + ROWS, s.nq) - 1, a.causal);
    auto load = [&](int c0, int into) {
        if (c0 < end) {
            stage_rows<D, kPT, THREADS>(ring + 2 * into * C::kTileF, k, a.k_stride, c0, s.nk);
            stage_rows<D, kPT, THREADS>(ring + (2 * into + 1) * C::kTileF, v, a.v_stride, c0, s.nk);
        }
        copies_commit();
    };
    stage_rows<D, ROWS, THREADS>(sq, q, a.q_stride, r0, s.nq);
    load(0, 0);

    const float sc = a.scale * kLog2e;
    float m[RPT], l[RPT], o[RPT][D / 16];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        m[i] = -CUDART_INF_F;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
    }
    int at = 0;
    for (int c0 = 0; c0 < end; c0 += kPT, at ^= 1) {
        copies_wait();
        __syncthreads();
        load(c0 + kPT, at ^ 1);
        float x[RPT][4] = {};
        dot_rows<D, RPT>(x, sq, ring + 2 * at * C::kTileF, ty, tx);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int seen = keys_seen(s, r0 + RPT * ty + i, a.causal) - c0;
            float top = -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = tx + 16 * j < seen ? x[i][j] * sc : -CUDART_INF_F;
                top = fmaxf(top, x[i][j]);
            }
#pragma unroll
            for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m[i], top), base = mn == -CUDART_INF_F ? 0.f : mn;
            const float f = exp2f(m[i] - base);
            m[i] = mn;
            l[i] *= f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = exp2f(x[i][j] - base);
                l[i] += x[i][j];
            }
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[i][c] *= f;
        }
        put_weights(sp, x, ty, tx);
        weigh_rows<ROWS == 64, D, RPT>(o, sp, ring + (2 * at + 1) * C::kTileF, ty, tx);
    }
    copies_wait();
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = r0 + RPT * ty + i;
        float sum = l[i];
#pragma unroll
        for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (r >= s.nq) continue;
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        write_row<D>(static_cast<float *>(a.out) + ((s.q0 + r) * a.bt.Hq + h) * D, o[i], tx, inv);
        if (a.lse && tx == 0)
            a.lse[stat_at(a.bt, s.q0 + r, h)] =
                sum == 0.f ? -CUDART_INF_F : m[i] * 0.69314718055994531f + logf(sum);
    }
}

// P and dS of a tile: x (scores, log2 units) and y (dP) in, both out in place.
// `transposed`: rows of the thread's block are keys, columns queries.
template <int RPT>
__device__ __forceinline__ void grad_scores(float (&x)[RPT][4], float (&y)[RPT][4], const Seq &s, const float *lse2,
                                            const float *delta, int r0, int c0, int ty, int tx, bool causal,
                                            bool transposed) {
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int qi = transposed ? tx + 16 * j : RPT * ty + i, kj = transposed ? RPT * ty + i : tx + 16 * j;
            const bool seen = r0 + qi < s.nq && c0 + kj < keys_seen(s, r0 + qi, causal);
            const float p = seen ? exp2f(x[i][j] - lse2[qi]) : 0.f;
            x[i][j] = p;
            y[i][j] = seen ? p * (y[i][j] - delta[qi]) : 0.f;
        }
}

// lse (in log2 units; 0 for rows that see nothing) and delta (where DELTA) of N queries
template <int N, int THREADS, bool DELTA>
__device__ __forceinline__ void stage_stats(float *lse2, float *delta, const PromptArgs &a, const Seq &s, int r0, int h) {
    for (int i = threadIdx.x; i < N; i += THREADS) {
        const int r = r0 + i;
        float x = 0.f, y = 0.f;
        if (r < s.nq) {
            const int64_t at = stat_at(a.bt, s.q0 + r, h);
            x = a.lse[at] * kLog2e;
            if (DELTA) y = a.delta[at];
            if (x == -CUDART_INF_F) x = 0.f;
        }
        lse2[i] = x;
        if (DELTA) delta[i] = y;
    }
}

// Gradients of rows behind the last packed sequence: zero.  Normally there are none; every block takes its
// share, in 16-byte pieces (`row` elements each).
template <typename T> __device__ __forceinline__ void zero_behind(T *g, const int32_t *cu, int n, int T_, int row) {
    if (cu == nullptr) return;
    const int from = min(max(cu[n], 0), T_);
    const int64_t pieces = (int64_t)(T_ - from) * row * (int)sizeof(T) / 16;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, blocks = (int64_t)gridDim.x * gridDim.y;
    for (int64_t i = block * blockDim.x + threadIdx.x; i < pieces; i += blocks * blockDim.x)
        reinterpret_cast<uint4 *>(g + (int64_t)from * row)[i] = make_uint4(0, 0, 0, 0);
}

// dK and dV of ROWS keys (the index-th tile) of one head of the cache, over all query heads of its group.
// OWN_DELTA: delta is formed here from O, for a launch beside the queries' blocks.
template <int D, int ROWS, bool OWN_DELTA>
__device__ __forceinline__ void grad_kv(const PromptArgs &a, int64_t index, int hk) {
    using C = PromptCfg<D>;
    constexpr int THREADS = RowsCfg<ROWS>::kThreads, RPT = RowsCfg<ROWS>::kPer, TILES = OWN_DELTA ? 3 : 2;
    extern __shared__ __align__(16) float sm[];
    float *sk = sm, *sv = sk + ROWS * C::kPitch, *ring = sv + ROWS * C::kPitch, *sp = ring + 2 * TILES * C::kTileF,
          *stats = sp + ROWS * 68;   // lse and delta of two tiles
    int *scratch = reinterpret_cast<int *>(stats + 4 * kPT);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    int n, t;
    if (!find_tile(a.bt.cu_k, a.bt.n, a.bt.Tk, ROWS, index, scratch, n, t)) return;
    const Seq s = seq_of(a.bt, n);
    const int c0 = t * ROWS, group = a.bt.Hq / a.bt.Hkv;
    // the first tile of queries that sees key c0
    const int start = a.causal ? max(0, c0 - (s.nk - s.nq)) / kPT : 0;
    const int per_head = max(0, (s.nq + kPT - 1) / kPT - start), total = per_head * group;
    auto load = [&](int it, int into) {
        if (it < total) {
            const int h = hk * group + it / per_head, r0 = (start + it % per_head) * kPT;
            stage_rows<D, kPT, THREADS>(ring + TILES * into * C::kTileF,
                                        static_cast<const float *>(a.q) + s.q0 * a.q_stride + (int64_t)h * D, a.q_stride,
                                        r0, s.nq);
            stage_rows<D, kPT, THREADS>(ring + (TILES * into + 1) * C::kTileF,
                                        static_cast<const float *>(a.d_out) + (s.q0 * a.bt.Hq + h) * (int64_t)D,
                                        (int64_t)a.bt.Hq * D, r0, s.nq);
            if (OWN_DELTA)
                stage_rows<D, kPT, THREADS>(ring + (TILES * into + 2) * C::kTileF,
                                            static_cast<const float *>(a.out) + (s.q0 * a.bt.Hq + h) * (int64_t)D,
                                            (int64_t)a.bt.Hq * D, r0, s.nq);
            stage_stats<kPT, THREADS, !OWN_DELTA>(stats + 2 * into * kPT, stats + (2 * into + 1) * kPT, a, s, r0, h);
        }
        copies_commit();
    };
    stage_rows<D, ROWS, THREADS>(sk, static_cast<const float *>(a.k) + s.k0 * a.k_stride + (int64_t)hk * D, a.k_stride, c0,
                                 s.nk);
    stage_rows<D, ROWS, THREADS>(sv, static_cast<const float *>(a.v) + s.k0 * a.v_stride + (int64_t)hk * D, a.v_stride, c0,
                                 s.nk);
    load(0, 0);
    const float sc = a.scale * kLog2e;
    float gk[RPT][D / 16] = {}, gv[RPT][D / 16] = {};
    for (int it = 0; it < total; ++it) {
        const int at = it & 1, r0 = (start + it % per_head) * kPT;
        const float *sq = ring + TILES * at * C::kTileF, *sg = sq + C::kTileF;
        copies_wait();
        __syncthreads();
        load(it + 1, at ^ 1);
        if (OWN_DELTA) {
            constexpr int PER = THREADS / kPT;   // threads of a row
            const int r = tid / PER;
            const float *go = sg + r * C::kPitch, *oo = sg + C::kTileF + r * C::kPitch;
            float dot = 0.f;
#pragma unroll
            for (int c = (tid % PER) * 4; c < D; c += 4 * PER) {
                const float4 x = *reinterpret_cast<const float4 *>(go + c), y = *reinterpret_cast<const float4 *>(oo + c);
                dot += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
            }
#pragma unroll
            for (int d = PER / 2; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
            if (tid % PER == 0) stats[(2 * at + 1) * kPT + r] = dot;
        }
        float x[RPT][4] = {}, y[RPT][4] = {};
        dot_rows<D, RPT>(x, sk, sq, ty, tx);
        dot_rows<D, RPT>(y, sv, sg, ty, tx);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] *= sc;
        if (OWN_DELTA) __syncthreads();
        grad_scores(x, y, s, stats + 2 * at * kPT, stats + (2 * at + 1) * kPT, r0, c0, ty, tx, a.causal, true);
        put_weights(sp, x, ty, tx);
        weigh_rows<true, D, RPT>(gv, sp, sg, ty, tx);
        put_weights(sp, y, ty, tx);
        weigh_rows<true, D, RPT>(gk, sp, sq, ty, tx);
    }
    copies_wait();
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = c0 + RPT * ty + i;
        if (r >= s.nk) continue;
        const int64_t to = ((s.k0 + r) * a.bt.Hkv + hk) * D;
        write_row<D>(static_cast<float *>(a.dk) + to, gk[i], tx, a.scale);
        write_row<D>(static_cast<float *>(a.dv) + to, gv[i], tx, 1.f);
    }
}

template <int D, int ROWS>
__global__ void __launch_bounds__(RowsCfg<ROWS>::kThreads) attn_grad_kv_kernel(const PromptArgs a) {
    zero_behind(static_cast<float *>(a.dk), a.bt.cu_k, a.bt.n, a.bt.Tk, a.bt.Hkv * D);
    zero_behind(static_cast<float *>(a.dv), a.bt.cu_k, a.bt.n, a.bt.Tk, a.bt.Hkv * D);
    grad_kv<D, ROWS, false>(a, blockIdx.x, blockIdx.y);
}

// dQ of ROWS queries (the index-th tile) of one head; and their delta = dO . O, which the keys' kernel reads
// after this one.
template <int D, int ROWS> __device__ __forceinline__ void grad_q(const PromptArgs &a, int64_t index, int h) {
    using C = PromptCfg<D>;
    constexpr int THREADS = RowsCfg<ROWS>::kThreads, RPT = RowsCfg<ROWS>::kPer;
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *sg = sq + ROWS * C::kPitch, *ring = sg + ROWS * C::kPitch, *sp = ring + 4 * C::kTileF,
          *stats = sp + ROWS * 68;
    int *scratch = reinterpret_cast<int *>(stats + 4 * kPT);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    int n, t;
    if (!find_tile(a.bt.cu_q, a.bt.n, a.bt.Tq, ROWS, index, scratch, n, t)) return;
    const Seq s = seq_of(a.bt, n);
    const int r0 = t * ROWS, hk = h / (a.bt.Hq / a.bt.Hkv);
    const float *k = static_cast<const float *>(a.k) + s.k0 * a.k_stride + (int64_t)hk * D;
    const float *v = static_cast<const float *>(a.v) + s.k0 * a.v_stride + (int64_t)hk * D;
    const int end = keys_seen(s, min(r0 + ROWS, s.nq) - 1, a.causal);
    auto load = [&](int c0, int into) {
        if (c0 < end) {
            stage_rows<D, kPT, THREADS>(ring + 2 * into * C::kTileF, k, a.k_stride, c0, s.nk);
            stage_rows<D, kPT, THREADS>(ring + (2 * into + 1) * C::kTileF, v, a.v_stride, c0, s.nk);
        }
        copies_commit();
    };
    stage_rows<D, ROWS, THREADS>(sq, static_cast<const float *>(a.q) + s.q0 * a.q_stride + (int64_t)h * D, a.q_stride, r0,
                                 s.nq);
    stage_rows<D, ROWS, THREADS>(sg, static_cast<const float *>(a.d_out) + (s.q0 * a.bt.Hq + h) * (int64_t)D,
                                 (int64_t)a.bt.Hq * D, r0, s.nq);
    load(0, 0);
    copies_wait();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = RPT * ty + i;
        const bool there = r0 + r < s.nq;
        const float *o = static_cast<const float *>(a.out) + ((s.q0 + r0 + r) * a.bt.Hq + h) * (int64_t)D;
        float dot = 0.f;
#pragma unroll
        for (int c = tx * 4; c < D; c += 64) {
            const float4 x = there ? *reinterpret_cast<const float4 *>(o + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 y = *reinterpret_cast<const float4 *>(sg + r * C::kPitch + c);
            dot += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
        }
#pragma unroll
        for (int d = 8; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        if (tx == 0) {
            float lse = 0.f;
            if (there) {
                const int64_t to = stat_at(a.bt, s.q0 + r0 + r, h);
                a.delta[to] = dot;
                lse = a.lse[to] * kLog2e;
            }
            stats[r] = lse == -CUDART_INF_F ? 0.f : lse;
            stats[kPT + r] = dot;
        }
    }
    const float sc = a.scale * kLog2e;
    float gq[RPT][D / 16] = {};
    int at = 0;
    for (int c0 = 0; c0 < end; c0 += kPT, at ^= 1) {
        copies_wait();
        __syncthreads();
        load(c0 + kPT, at ^ 1);
        const float *sk = ring + 2 * at * C::kTileF, *sv = sk + C::kTileF;
        float x[RPT][4] = {}, y[RPT][4] = {};
        dot_rows<D, RPT>(x, sq, sk, ty, tx);
        dot_rows<D, RPT>(y, sg, sv, ty, tx);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] *= sc;
        grad_scores(x, y, s, stats, stats + kPT, r0, c0, ty, tx, a.causal, false);
        put_weights(sp, y, ty, tx);
        weigh_rows<ROWS == 64, D, RPT>(gq, sp, sk, ty, tx);
    }
    copies_wait();
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = r0 + RPT * ty + i;
        if (r < s.nq) write_row<D>(static_cast<float *>(a.dq) + ((s.q0 + r) * a.bt.Hq + h) * D, gq[i], tx, a.scale);
    }
}

template <int D, int ROWS>
__global__ void __launch_bounds__(RowsCfg<ROWS>::kThreads) attn_grad_q_kernel(const PromptArgs a) {
    zero_behind(static_cast<float *>(a.dq), a.bt.cu_q, a.bt.n, a.bt.Tq, a.bt.Hq * D);
    grad_q<D, ROWS>(a, gridDim.x - 1 - blockIdx.x, blockIdx.y);   // the last tiles see the most keys
}

// Both for small batches, side by side: neither fills the GPU.  The first blocks take the keys.  B1 T256 H2 D64:
// 29 us, 45 one after the other; T48 H4 D128 11 and 21; T1024 H2 D64 108 and 158.  (grad_rows has the limit.)
template <int D>
__global__ void __launch_bounds__(RowsCfg<16>::kThreads) attn_grad_both_kernel(const PromptArgs a, int kv_blocks) {
    zero_behind(static_cast<float *>(a.dk), a.bt.cu_k, a.bt.n, a.bt.Tk, a.bt.Hkv * D);
    zero_behind(static_cast<float *>(a.dv), a.bt.cu_k, a.bt.n, a.bt.Tk, a.bt.Hkv * D);
    zero_behind(static_cast<float *>(a.dq), a.bt.cu_q, a.bt.n, a.bt.Tq, a.bt.Hq * D);
    const int block = blockIdx.x;
    if (block < kv_blocks) grad_kv<D, 16, true>(a, block / a.bt.Hkv, block % a.bt.Hkv);
    else grad_q<D, 16>(a, (gridDim.x - 1 - block) / a.bt.Hq, (gridDim.x - 1 - block) % a.bt.Hq);
}

template <typename K> cudaError_t allow_smem(K kern, int bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// Rows of a block: 64, or 16 where blocks of 64 rows would leave SMs idle (a tile's work is then spread over
// four times the blocks, each done sooner, and costs more in all).  What counts is work: tiles of 64 rows, each by
// the quarters of its keys that it sees, a half under a causal mask (three quarters in short sequences).
inline int seen_quarters(const PromptArgs &a) {
    const int len = a.bt.cu_q ? a.bt.Tq / a.bt.n : a.bt.Tq;
    return !a.causal || a.bt.Tk >= 2 * (int64_t)a.bt.Tq ? 4 : len >= 512 ? 2 : 3;
}
inline int64_t likely_tiles(const int32_t *cu, int n, int T) {   // packed: the last tile of a sequence is half full
    return cu == nullptr ? max_tiles(cu, n, T, 64) : T / 64 + n / 2;
}
inline int64_t query_work(const PromptArgs &a) {
    return seen_quarters(a) * likely_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq) * a.bt.Hq;
}
inline int64_t key_work(const PromptArgs &a) {
    return seen_quarters(a) * likely_tiles(a.bt.cu_k, a.bt.n, a.bt.Tk) * a.bt.Hkv;
}
// Forward, us with 16 and with 64 rows (H heads of their own keys; causal unless said otherwise).  Heads of 64:
// T1024 H6 64 and 80, H8 81 and 80, T8192 H1 438 and 613, B4 T1024 H4 137 and 125; B8 T256 H4 29 and 23; not causal: T512
// H8 34 and 42, T1024 H5 101 and 80.  Heads of 128: T1024 H5 127 and 142, H6 144 and 142, H8 178 and 142; B4 T256 H4
// 36.8 and 38.7, B8 T256 H3 48 and 39; not causal: T512 H8 79 and 73, T1024 H8 304 and 142.
inline int prompt_rows(const PromptArgs &a, int d, int sms) {
    return 8 * query_work(a) < (int64_t)sms * (d == 64 ? 15 : 10) ? 16 : 64;
}
// Gradient: both halves in one launch of blocks of 16 rows, or one after the other.  In one launch, in two with 16 and
// with 64 rows, us, as above.  Heads of 64: T1024 H4 160, 203, 272; T1024 H6 234, 222, 272; T1024 H8 309, 289, 273; T8192
// H1 2197, 1539, 2115; B8 T256 H4 108, 95, 76; not causal: T512 H8 166, 111, 140, T1024 H8 589, 424, 272.  Heads of 128:
// T1024 H8 423, 558, 495; B8 T256 H3 114, 147, 131, H4 147, 180, 132; not causal: T512 H8 227, 245, 246, T1024 H5 534, 713, 481.
// Queries by 64 rows and keys by 16, B2 T1024 H16 of 2 heads of keys: 1172 (1195, 1255, 1502).
struct GradRows {
    bool one;   // one launch
    int q, k;
};
inline GradRows grad_rows(const PromptArgs &a, int d, int sms) {
    const int64_t q = query_work(a), k = key_work(a);
    return {a.bt.Tq > 0 && a.bt.Tk > 0 && 10 * (q + k) < (int64_t)sms * (d == 64 ? 23 : 40), 8 * q < (int64_t)sms * 15 ? 16 : 64,
            8 * k < (int64_t)sms * 15 ? 16 : 64};
}

template <int D, int ROWS> cudaError_t launch_prompt_rows(const PromptArgs &a, cudaStream_t st) {
    const int64_t tiles = max_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq, ROWS);
    constexpr int smem = PromptCfg<D>::smem(ROWS, 1);
    cudaError_t e = allow_smem(attn_prompt_kernel<D, ROWS>, smem);
    if (e != cudaSuccess) return e;
    attn_prompt_kernel<D, ROWS><<<dim3((unsigned)tiles, a.bt.Hq), RowsCfg<ROWS>::kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <int D> cudaError_t launch_prompt(const PromptArgs &a, int sms, cudaStream_t st) {
    if (a.bt.Tq == 0) return cudaSuccess;
    return prompt_rows(a, D, sms) == 16 ? launch_prompt_rows<D, 16>(a, st) : launch_prompt_rows<D, 64>(a, st);
}

template <int D, int ROWS> cudaError_t launch_grad_kv(const PromptArgs &a, cudaStream_t st) {
    constexpr int smem = PromptCfg<D>::smem(ROWS, 2);
    cudaError_t e = allow_smem(attn_grad_kv_kernel<D, ROWS>, smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = max_tiles(a.bt.cu_k, a.bt.n, a.bt.Tk, ROWS);
    attn_grad_kv_kernel<D, ROWS><<<dim3((unsigned)tiles, a.bt.Hkv), RowsCfg<ROWS>::kThreads, smem, st>>>(a);
    return cudaGetLastError();
}
template <int D, int ROWS> cudaError_t launch_grad_q(const PromptArgs &a, cudaStream_t st) {
    constexpr int smem = PromptCfg<D>::smem(ROWS, 2);
    cudaError_t e = allow_smem(attn_grad_q_kernel<D, ROWS>, smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = max_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq, ROWS);
    attn_grad_q_kernel<D, ROWS><<<dim3((unsigned)tiles, a.bt.Hq), RowsCfg<ROWS>::kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <int D> cudaError_t launch_prompt_grad(const PromptArgs &a, int sms, cudaStream_t st) {
    const GradRows rows = grad_rows(a, D, sms);
    if (rows.one) {
        constexpr int smem = PromptCfg<D>::smem(16, 2, 6);
        static_assert(smem <= 232448, "shared memory");
        const cudaError_t e = allow_smem(attn_grad_both_kernel<D>, smem);
        if (e != cudaSuccess) return e;
        const int64_t kv = max_tiles(a.bt.cu_k, a.bt.n, a.bt.Tk, 16) * a.bt.Hkv,
                      q = max_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq, 16) * a.bt.Hq;
        attn_grad_both_kernel<D><<<(unsigned)(kv + q), RowsCfg<16>::kThreads, smem, st>>>(a, (int)kv);
        return cudaGetLastError();
    }
    cudaError_t e = cudaSuccess;
    if (a.bt.Tq > 0)   // first: it forms the delta that the other reads
        e = rows.q == 16 ? launch_grad_q<D, 16>(a, st) : launch_grad_q<D, 64>(a, st);
    if (e == cudaSuccess && a.bt.Tk > 0) e = rows.k == 16 ? launch_grad_kv<D, 16>(a, st) : launch_grad_kv<D, 64>(a, st);
    return e;
}

}  // namespace attn
}  // namespace kda
