// attn_append.cuh -- appends keys and values to a paged cache, rotating keys (and queries) by position.
//
// Token j of sequence n has position p = cache_lens[n] + j.  Its pairs of channels (x1, x2) turn by the
// angle a = p * inv_freq[i]:
//     x1' = x1 cos a - x2 sin a,    x2' = x2 cos a + x1 sin a,
// pair i being channels (i, i + r/2), or (2i, 2i + 1) when interleaved, of the first r channels; the
// rest, and v, are copied.  k' and v go to slot p % page_size of page table[n][p / page_size]; k' also
// to k_out where the prompt's own attention reads it, q' to q_out.
//
// The angle is formed in 64 bits: a far position times a frequency of order 1 has no fraction left in 32.
// It is reduced to a fraction of a turn there, and sine and cosine of that are taken in 32 bits (error
// below 2^-22 against the 2^-9 of the bf16 result).  One sine and cosine serve all heads of a token.
//
// Bound by memory: every byte is read once and written once, 16 bytes per thread and access: 8 prompts of
// 1024 to 16384 tokens, 32 + 8 heads of 128, k_out too: 192 us, 6.0 TB/s.  A step of 256 tokens takes 4.3 us,
// one of a single token 2.8: the launch and one round trip to memory each for lengths, pages and rows.
#pragma once

#include "attn_common.cuh"

namespace kda {
namespace attn {

struct AppendArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements from one token to the next
    const float *inv_freq;
    int rotary, interleaved;
    const int32_t *cu, *cache_lens;
    int n, T, Hq, Hkv;                      // T: tokens of a row (dense), or packed tokens
    int64_t tokens;                         // rows of the flattened token tensors
    Cache cache;
    void *q_out, *k_out;
};

constexpr int kAppendThreads = 256;

// sequence of a packed token: the last n with cu[n] <= token; -1 behind the last sequence
__device__ __forceinline__ int seq_of_token(const int32_t *cu, int n, int64_t token) {
    int lo = 0, hi = n;   // cu[lo] <= token < cu[hi], if there is such a pair
    if (token < cu[0] || token >= cu[n]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= token) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <typename T> struct Vec16 {
    static constexpr int N = 16 / sizeof(T);
    T x[N];
};

template <typename T> __device__ __forceinline__ Vec16<T> load16(const T *p) {
    union { uint4 u; Vec16<T> v; } c;
    c.u = *reinterpret_cast<const uint4 *>(p);
    return c.v;
}
template <typename T> __device__ __forceinline__ void store16(T *p, const Vec16<T> &v) {
    union { uint4 u; Vec16<T> v; } c;
    c.v = v;
    *reinterpret_cast<uint4 *>(p) = c.u;
}

// Six blocks per SM, 40 registers a thread: 192 us for the prompts above, with five (48 registers) 197, with
// seven, which spill, 248; two units of a thread under way at once (74 registers, three blocks) 249.
template <typename T, int D, int TOKENS>
__global__ void __launch_bounds__(kAppendThreads, 6) attn_append_kernel(const AppendArgs a) {
    constexpr int VE = Vec16<T>::N;      // elements of a 16-byte vector
    constexpr int UNITS = D / (2 * VE);  // a thread's share of a head: two vectors
    __shared__ float2 s_turn[TOKENS][D / 2];
    __shared__ int s_seq[TOKENS], s_pos[TOKENS];

    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * TOKENS;
    next_may_start();
    wait_for_previous();
    if (tid < TOKENS) {
        const int64_t t = t0 + tid;
        int seq = -1, pos = 0;
        if (t < a.tokens) {
            int64_t j;
            if (a.cu) {
                seq = seq_of_token(a.cu, a.n, t);
                j = seq < 0 ? 0 : t - a.cu[seq];
            } else {
                seq = (int)(t / a.T);
                j = t - (int64_t)seq * a.T;
            }
            if (seq >= 0) {
                const int have = a.cache_lens[seq];
                if (have < 0 || have + j > 0x7fffffff) seq = -1;   // an unused row of the batch
                else pos = (int)(have + j);
            }
        }
        s_seq[tid] = seq;
        s_pos[tid] = pos;
    }
    __syncthreads();
    const int pairs = a.rotary / 2;
    for (int i = tid; i < TOKENS * pairs; i += kAppendThreads) {
        const int tk = i / pairs, f = i - tk * pairs;
        const double turns = (double)s_pos[tk] * (double)a.inv_freq[f] * 0.15915494309189533577;   // / 2 pi
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        s_turn[tk][f] = make_float2(c, s);
    }
    __syncthreads();

    const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v);
    T *q_out = static_cast<T *>(a.q_out), *k_out = static_cast<T *>(a.k_out);
    const int heads = a.Hq + 2 * a.Hkv;   // queries, keys, values
    for (int i = tid; i < TOKENS * heads * UNITS; i += kAppendThreads) {
        const int u = i % UNITS, th = i / UNITS, h = th % heads, tk = th / heads;
        const int seq = s_seq[tk];
        if (seq < 0) continue;
        const int64_t t = t0 + tk;
        const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
        const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
        const T *src = is_q ? q + t * a.q_stride + (int64_t)h * D
                            : (is_v ? v + t * a.v_stride : k + t * a.k_stride) + (int64_t)hk * D;
        // the unit's two vectors: halves of pairs where the pair lies half the rotary width apart
        const int half = a.rotary / (2 * VE);
        const bool apart = !a.interleaved && u < half && !is_v;
        int c0, c1;
        if (a.interleaved || is_v) {
            c0 = 2 * u * VE;
            c1 = c0 + VE;
        } else if (u < half) {
            c0 = u * VE;
            c1 = c0 + half * VE;
        } else {
            c0 = 2 * u * VE;   // behind the rotated channels: 2 half + 2 (u - half)
            c1 = c0 + VE;
        }
        Vec16<T> x = load16(src + c0), y = load16(src + c1);
        if (apart) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float2 cs = s_turn[tk][c0 + e];
                const float p = to_f32(x.x[e]), r = to_f32(y.x[e]);
                x.x[e] = from_f32<T>(p * cs.x - r * cs.y);
                y.x[e] = from_f32<T>(r * cs.x + p * cs.y);
            }
        } else if (a.interleaved && !is_v) {
#pragma unroll
            for (int e = 0; e < VE; e += 2) {
                if (c0 + e < a.rotary) {
                    const float2 cs = s_turn[tk][(c0 + e) / 2];
                    const float p = to_f32(x.x[e]), r = to_f32(x.x[e + 1]);
                    x.x[e] = from_f32<T>(p * cs.x - r * cs.y);
                    x.x[e + 1] = from_f32<T>(r * cs.x + p * cs.y);
                }
                if (c1 + e < a.rotary) {
                    const float2 cs = s_turn[tk][(c1 + e) / 2];
                    const float p = to_f32(y.x[e]), r = to_f32(y.x[e + 1]);
                    y.x[e] = from_f32<T>(p * cs.x - r * cs.y);
                    y.x[e + 1] = from_f32<T>(r * cs.x + p * cs.y);
                }
            }
        }
        if (is_q) {
            T *dst = q_out + (t * a.Hq + h) * D;
            store16(dst + c0, x);
            store16(dst + c1, y);
            continue;
        }
        if (!is_v && k_out) {
            T *dst = k_out + (t * a.Hkv + hk) * D;
            store16(dst + c0, x);
            store16(dst + c1, y);
        }
        const int pos = s_pos[tk], col = pos >> a.cache.page_log2;
        int page = -1;
        if (col < a.cache.width) page = a.cache.table[seq * a.cache.row + col];
        if (page < 0 || page >= a.cache.num_pages) {
            record_device_error(kDevErrBadPage);
            continue;
        }
        const int64_t slot = ((int64_t)hk << a.cache.page_log2) + (pos & ((1 << a.cache.page_log2) - 1));
        T *dst = (is_v ? static_cast<T *>(a.cache.v) + page * a.cache.v_stride
                       : static_cast<T *>(a.cache.k) + page * a.cache.k_stride) + slot * D;
        store16(dst + c0, x);
        store16(dst + c1, y);
    }
}

template <typename T, int D> cudaError_t launch_append_d(const AppendArgs &a, int sms, cudaStream_t st) {
    // few tokens (8 an SM): one per block, so that they spread over the SMs; many: four, whose sines (up to 64 each)
    // keep all 256 threads busy at once.  One against four, 32 + 8 heads of 128: 3.3 and 5.7 us at 16 tokens,
    // 5.2 and 5.9 at 592, 8.4 and 11.7 at 1184, 15.2 and 12.9 at 2368, 98 and 77 at 16384.
    if (a.tokens <= (int64_t)sms * 8)
        return launch_behind(attn_append_kernel<T, D, 1>, (unsigned)a.tokens, kAppendThreads, 0, st, a);
    return launch_behind(attn_append_kernel<T, D, 4>, (unsigned)((a.tokens + 3) / 4), kAppendThreads, 0, st, a);
}

}  // namespace attn
}  // namespace kda
