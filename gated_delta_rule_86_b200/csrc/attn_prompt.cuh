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
// bound by the FMA units.  Tiles of 64 x 64 scores; thread (ty, tx) of 16 x 16 holds rows
// 4 ty .. 4 ty + 3, so a row's 16 threads lie in one half of a warp and its maximum and sum are four
// shuffles.
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

constexpr int kPT = 64;         // queries and keys of a tile
constexpr int kPThreads = 256;

// Rows [r0, r0 + 64) of a token tensor's head into shared memory as fp32, row pitch D + 4; rows at or
// past `rows` are zero.
template <typename T, int D>
__device__ __forceinline__ void stage_rows(float *dst, const T *src, int64_t stride, int r0, int rows, float mul) {
    constexpr int VE = Vec16<T>::N;
    for (int i = threadIdx.x; i < kPT * D / VE; i += kPThreads) {
        const int r = i / (D / VE), c = i % (D / VE) * VE;
        float *d = dst + r * (D + 4) + c;
        if (r0 + r < rows) {
            const Vec16<T> x = load16(src + (int64_t)(r0 + r) * stride + c);
#pragma unroll
            for (int e = 0; e < VE; ++e) d[e] = to_f32(x.x[e]) * mul;
        } else {
#pragma unroll
            for (int e = 0; e < VE; ++e) d[e] = 0.f;
        }
    }
}

// acc[i][j] += A[4 ty + i] . B[tx + 16 j] over D channels (pitch D + 4)
template <int D> __device__ __forceinline__ void dot_rows(float (&acc)[4][4], const float *A, const float *B, int ty,
                                                          int tx) {
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (4 * ty + i) * (D + 4) + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * (D + 4) + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] += a[i].x * b[j].x + a[i].y * b[j].y + a[i].z * b[j].z + a[i].w * b[j].w;
    }
}

// acc[i][c] += sum_t W[4 ty + i][t] X[t][tx * D / 16 + c]  (W pitch 68, X pitch D + 4)
template <int D> __device__ __forceinline__ void weigh_rows(float (&acc)[4][D / 16], const float *W, const float *X,
                                                            int ty, int tx) {
#pragma unroll 2
    for (int t = 0; t < kPT; t += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4 *>(W + (4 * ty + i) * 68 + t);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float x[D / 16];
#pragma unroll
            for (int c = 0; c < D / 16; c += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(X + (t + u) * (D + 4) + tx * 4 + (c / 4) * 64);
                x[c] = f.x, x[c + 1] = f.y, x[c + 2] = f.z, x[c + 3] = f.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float wi = u == 0 ? w[i].x : u == 1 ? w[i].y : u == 2 ? w[i].z : w[i].w;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) acc[i][c] += wi * x[c];
            }
        }
    }
}

// Channel of a thread's c-th accumulator in weigh_rows.
__device__ __forceinline__ int weigh_channel(int tx, int c) { return tx * 4 + (c / 4) * 64 + c % 4; }

template <typename T, int D>
__device__ __forceinline__ void write_row(T *dst, const float (&acc)[D / 16], int tx, float mul) {
#pragma unroll
    for (int c = 0; c < D / 16; c += 4) {
        T *p = dst + weigh_channel(tx, c);
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = from_f32<T>(acc[c + e] * mul);
    }
}

template <int D> constexpr int prompt_smem(int tiles, int squares) {
    return (tiles * kPT * (D + 4) + squares * kPT * 68) * 4 + 160;
}

template <typename T, int D> __global__ void __launch_bounds__(kPThreads, 1) attn_prompt_kernel(const PromptArgs a) {
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *sk = sq + kPT * (D + 4), *sv = sk + kPT * (D + 4), *sp = sv + kPT * (D + 4);
    int *scratch = reinterpret_cast<int *>(sp + kPT * 68);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, h = blockIdx.y;
    int n, t;
    if (!find_tile(a.bt.cu_q, a.bt.n, a.bt.Tq, kPT, blockIdx.x, scratch, n, t)) return;
    const Seq s = seq_of(a.bt, n);
    const int r0 = t * kPT, hk = h / (a.bt.Hq / a.bt.Hkv);
    const T *q = static_cast<const T *>(a.q) + s.q0 * a.q_stride + (int64_t)h * D;
    const T *k = static_cast<const T *>(a.k) + s.k0 * a.k_stride + (int64_t)hk * D;
    const T *v = static_cast<const T *>(a.v) + s.k0 * a.v_stride + (int64_t)hk * D;
    stage_rows<T, D>(sq, q, a.q_stride, r0, s.nq, a.scale * kLog2e);

    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -CUDART_INF_F;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
    }
    const int end = keys_seen(s, min(r0 + kPT, s.nq) - 1, a.causal);
    for (int c0 = 0; c0 < end; c0 += kPT) {
        __syncthreads();
        stage_rows<T, D>(sk, k, a.k_stride, c0, s.nk, 1.f);
        stage_rows<T, D>(sv, v, a.v_stride, c0, s.nk, 1.f);
        __syncthreads();
        float x[4][4] = {};
        dot_rows<D>(x, sq, sk, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int seen = keys_seen(s, r0 + 4 * ty + i, a.causal) - c0;
            float top = -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (tx + 16 * j >= seen) x[i][j] = -CUDART_INF_F;
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
                const float p = exp2f(x[i][j] - base);
                l[i] += p;
                sp[(4 * ty + i) * 68 + tx + 16 * j] = p;
            }
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[i][c] *= f;
        }
        __syncwarp();   // a row's weights come from the half warp that reads them
        weigh_rows<D>(o, sp, sv, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * ty + i;
        float sum = l[i];
#pragma unroll
        for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (r >= s.nq) continue;
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        write_row<T, D>(static_cast<T *>(a.out) + ((s.q0 + r) * a.bt.Hq + h) * D, o[i], tx, inv);
        if (a.lse && tx == 0)
            a.lse[stat_at(a.bt, s.q0 + r, h)] =
                sum == 0.f ? -CUDART_INF_F : m[i] * 0.69314718055994531f + logf(sum);
    }
}

// delta_i = dO_i . O_i, one warp per (query, head).  Rows behind the last sequence get zero gradients
// here: no other kernel visits them.
template <typename T, int D> __global__ void __launch_bounds__(256) attn_delta_kernel(const PromptArgs a) {
    constexpr int VE = Vec16<T>::N;
    constexpr int LANES = D / VE;   // lanes of a row
    const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t rows_q = (int64_t)(a.bt.cu_q ? 1 : a.bt.n) * a.bt.Tq, rows_k = (int64_t)(a.bt.cu_q ? 1 : a.bt.n) * a.bt.Tk;
    const int64_t nq = rows_q * a.bt.Hq, nk = rows_k * a.bt.Hkv;
    float dot = 0.f;
    if (item < nq) {
        const int64_t row = item / a.bt.Hq;
        const Vec16<T> x = load16(static_cast<const T *>(a.d_out) + item * D + lane * VE);
        const Vec16<T> y = load16(static_cast<const T *>(a.out) + item * D + lane * VE);
#pragma unroll
        for (int e = 0; e < VE; ++e) dot += to_f32(x.x[e]) * to_f32(y.x[e]);
        if (a.bt.cu_q && row >= __ldg(a.bt.cu_q + a.bt.n)) {
            Vec16<T> z = {};
            store16(static_cast<T *>(a.dq) + item * D + lane * VE, z);
        }
    }
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (item < nq && lane == 0) a.delta[stat_at(a.bt, item / a.bt.Hq, (int)(item % a.bt.Hq))] = dot;
    if (a.bt.cu_k && item < nk && item / a.bt.Hkv >= __ldg(a.bt.cu_k + a.bt.n)) {
        Vec16<T> z = {};
        store16(static_cast<T *>(a.dk) + item * D + lane * VE, z);
        store16(static_cast<T *>(a.dv) + item * D + lane * VE, z);
    }
}

// P and dS of one 64 x 64 tile: x (scores, log2 units) and y (dP) in, both out in place.
// `transposed`: rows of the thread's block are keys, columns queries.
__device__ __forceinline__ void grad_scores(float (&x)[4][4], float (&y)[4][4], const Seq &s, const float *lse2,
                                            const float *delta, int r0, int c0, int ty, int tx, bool causal,
                                            bool transposed) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int qi = transposed ? tx + 16 * j : 4 * ty + i, kj = transposed ? 4 * ty + i : tx + 16 * j;
            const bool seen = r0 + qi < s.nq && c0 + kj < keys_seen(s, r0 + qi, causal);
            const float p = seen ? exp2f(x[i][j] - lse2[qi]) : 0.f;
            x[i][j] = p;
            y[i][j] = seen ? p * (y[i][j] - delta[qi]) : 0.f;
        }
}

// lse (in log2 units; 0 for rows that see nothing) and delta of 64 queries
__device__ __forceinline__ void stage_stats(float *lse2, float *delta, const PromptArgs &a, const Seq &s, int r0, int h) {
    if (threadIdx.x < kPT) {
        const int r = r0 + threadIdx.x;
        float x = 0.f, y = 0.f;
        if (r < s.nq) {
            const int64_t at = stat_at(a.bt, s.q0 + r, h);
            x = a.lse[at] * kLog2e;
            y = a.delta[at];
            if (x == -CUDART_INF_F) x = 0.f;
        }
        lse2[threadIdx.x] = x;
        delta[threadIdx.x] = y;
    }
}

// dK and dV of 64 keys of one head of the cache, over all query heads of its group.
template <typename T, int D> __global__ void __launch_bounds__(kPThreads, 1) attn_grad_kv_kernel(const PromptArgs a) {
    extern __shared__ __align__(16) float sm[];
    float *sk = sm, *sv = sk + kPT * (D + 4), *sq = sv + kPT * (D + 4), *sg = sq + kPT * (D + 4),
          *sp = sg + kPT * (D + 4);
    __shared__ float lse2[kPT], delta[kPT];
    int *scratch = reinterpret_cast<int *>(sp + kPT * 68);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, hk = blockIdx.y;
    int n, t;
    if (!find_tile(a.bt.cu_k, a.bt.n, a.bt.Tk, kPT, blockIdx.x, scratch, n, t)) return;
    const Seq s = seq_of(a.bt, n);
    const int c0 = t * kPT, group = a.bt.Hq / a.bt.Hkv;
    stage_rows<T, D>(sk, static_cast<const T *>(a.k) + s.k0 * a.k_stride + (int64_t)hk * D, a.k_stride, c0, s.nk, 1.f);
    stage_rows<T, D>(sv, static_cast<const T *>(a.v) + s.k0 * a.v_stride + (int64_t)hk * D, a.v_stride, c0, s.nk, 1.f);
    float gk[4][D / 16] = {}, gv[4][D / 16] = {};
    // the first query that sees key c0
    const int start = a.causal ? max(0, c0 - (s.nk - s.nq)) / kPT * kPT : 0;
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
        const T *q = static_cast<const T *>(a.q) + s.q0 * a.q_stride + (int64_t)h * D;
        const T *g = static_cast<const T *>(a.d_out) + (s.q0 * a.bt.Hq + h) * (int64_t)D;
        for (int r0 = start; r0 < s.nq; r0 += kPT) {
            __syncthreads();
            stage_rows<T, D>(sq, q, a.q_stride, r0, s.nq, 1.f);
            stage_rows<T, D>(sg, g, (int64_t)a.bt.Hq * D, r0, s.nq, 1.f);
            stage_stats(lse2, delta, a, s, r0, h);
            __syncthreads();
            float x[4][4] = {}, y[4][4] = {};
            dot_rows<D>(x, sk, sq, ty, tx);
            dot_rows<D>(y, sv, sg, ty, tx);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] *= a.scale * kLog2e;
            grad_scores(x, y, s, lse2, delta, r0, c0, ty, tx, a.causal, true);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sp[(4 * ty + i) * 68 + tx + 16 * j] = x[i][j];
            __syncwarp();
            weigh_rows<D>(gv, sp, sg, ty, tx);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sp[(4 * ty + i) * 68 + tx + 16 * j] = y[i][j];
            __syncwarp();
            weigh_rows<D>(gk, sp, sq, ty, tx);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = c0 + 4 * ty + i;
        if (r >= s.nk) continue;
        const int64_t at = ((s.k0 + r) * a.bt.Hkv + hk) * D;
        write_row<T, D>(static_cast<T *>(a.dk) + at, gk[i], tx, a.scale);
        write_row<T, D>(static_cast<T *>(a.dv) + at, gv[i], tx, 1.f);
    }
}

// dQ of 64 queries of one head.
template <typename T, int D> __global__ void __launch_bounds__(kPThreads, 1) attn_grad_q_kernel(const PromptArgs a) {
    extern __shared__ __align__(16) float sm[];
    float *sk = sm, *sv = sk + kPT * (D + 4), *sq = sv + kPT * (D + 4), *sg = sq + kPT * (D + 4),
          *sp = sg + kPT * (D + 4);
    __shared__ float lse2[kPT], delta[kPT];
    int *scratch = reinterpret_cast<int *>(sp + kPT * 68);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, h = blockIdx.y;
    int n, t;
    if (!find_tile(a.bt.cu_q, a.bt.n, a.bt.Tq, kPT, blockIdx.x, scratch, n, t)) return;
    const Seq s = seq_of(a.bt, n);
    const int r0 = t * kPT, hk = h / (a.bt.Hq / a.bt.Hkv);
    const T *k = static_cast<const T *>(a.k) + s.k0 * a.k_stride + (int64_t)hk * D;
    const T *v = static_cast<const T *>(a.v) + s.k0 * a.v_stride + (int64_t)hk * D;
    stage_rows<T, D>(sq, static_cast<const T *>(a.q) + s.q0 * a.q_stride + (int64_t)h * D, a.q_stride, r0, s.nq,
                     a.scale * kLog2e);
    stage_rows<T, D>(sg, static_cast<const T *>(a.d_out) + (s.q0 * a.bt.Hq + h) * (int64_t)D, (int64_t)a.bt.Hq * D, r0,
                     s.nq, 1.f);
    stage_stats(lse2, delta, a, s, r0, h);
    float gq[4][D / 16] = {};
    const int end = keys_seen(s, min(r0 + kPT, s.nq) - 1, a.causal);
    for (int c0 = 0; c0 < end; c0 += kPT) {
        __syncthreads();
        stage_rows<T, D>(sk, k, a.k_stride, c0, s.nk, 1.f);
        stage_rows<T, D>(sv, v, a.v_stride, c0, s.nk, 1.f);
        __syncthreads();
        float x[4][4] = {}, y[4][4] = {};
        dot_rows<D>(x, sq, sk, ty, tx);
        dot_rows<D>(y, sg, sv, ty, tx);
        grad_scores(x, y, s, lse2, delta, r0, c0, ty, tx, a.causal, false);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sp[(4 * ty + i) * 68 + tx + 16 * j] = y[i][j];
        __syncwarp();
        weigh_rows<D>(gq, sp, sk, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * ty + i;
        if (r < s.nq)
            write_row<T, D>(static_cast<T *>(a.dq) + ((s.q0 + r) * a.bt.Hq + h) * D, gq[i], tx, a.scale);
    }
}

template <typename K> cudaError_t allow_smem(K kern, int bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int D> cudaError_t launch_prompt(const PromptArgs &a, cudaStream_t st) {
    const int64_t tiles = max_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq, kPT);
    if (tiles == 0) return cudaSuccess;
    constexpr int smem = prompt_smem<D>(3, 1);
    cudaError_t e = allow_smem(attn_prompt_kernel<T, D>, smem);
    if (e != cudaSuccess) return e;
    attn_prompt_kernel<T, D><<<dim3((unsigned)tiles, a.bt.Hq), kPThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t launch_delta(const PromptArgs &a, cudaStream_t st) {
    constexpr int LANES = D / Vec16<T>::N;
    const int64_t rows = a.bt.cu_q ? 1 : a.bt.n;
    const int64_t items_q = rows * a.bt.Tq * a.bt.Hq, items_k = a.bt.cu_k ? rows * a.bt.Tk * a.bt.Hkv : 0;
    const int64_t items = items_q > items_k ? items_q : items_k;
    if (items == 0) return cudaSuccess;
    attn_delta_kernel<T, D><<<(unsigned)((items * LANES + 255) / 256), 256, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t launch_prompt_grad(const PromptArgs &a, cudaStream_t st) {
    cudaError_t e = launch_delta<T, D>(a, st);
    if (e != cudaSuccess) return e;
    constexpr int smem = prompt_smem<D>(4, 1);
    const int64_t tk = max_tiles(a.bt.cu_k, a.bt.n, a.bt.Tk, kPT), tq = max_tiles(a.bt.cu_q, a.bt.n, a.bt.Tq, kPT);
    if (tk > 0) {
        if ((e = allow_smem(attn_grad_kv_kernel<T, D>, smem)) != cudaSuccess) return e;
        attn_grad_kv_kernel<T, D><<<dim3((unsigned)tk, a.bt.Hkv), kPThreads, smem, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (tq > 0) {
        if ((e = allow_smem(attn_grad_q_kernel<T, D>, smem)) != cudaSuccess) return e;
        attn_grad_q_kernel<T, D><<<dim3((unsigned)tq, a.bt.Hq), kPThreads, smem, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace attn
}  // namespace kda
