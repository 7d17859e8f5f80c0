// attn_decode.cuh -- attention of one new token per sequence over a paged key-value cache: the schedule, the
// kernel for fp32 and the one that joins the parts.  (attn_decode_mma.cuh has the kernel for bf16.)
//
//     o_h = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q_h . k_j - m),   j = 0 .. seq_lens[b] - 1,
// one pass over the keys and values with a running maximum m and sum; the query heads of a group share
// a head of the cache, so a block handles up to GC of them against keys it has loaded once.
//
// Bound by memory: the cache is read once.  The work of all (sequence, head) pairs is one line of tiles
// of 64 tokens (bf16: 128), cut into equal shares, one per block: long and short sequences balance, and a single
// long sequence spreads over the whole GPU.  A share may begin and end inside a pair; such a pair's
// blocks leave (m, sum, o) in the workspace and a second small kernel joins them in a fixed order (no
// atomics: the same call gives the same bits).  The lengths stay on the device: every block works out its
// share from them.
//
// Inside a block each warp runs on its own: it takes 16 of a tile's 64 tokens and copies them through
// its own ring of stages (cp.async, rows looked up page by page, rows past the end or on a bad page
// filled with zeros), so there is no barrier but at the end of a pair, where the warps' results join.
#pragma once

#include "attn_common.cuh"
#include "tc_utils.cuh"

namespace kda {
namespace attn {

constexpr int kWarpTokens = 16;   // of a tile, per warp

struct DecodeArgs {
    const void *q;
    int64_t q_stride;   // elements from one sequence's query to the next's
    Cache cache;
    const int32_t *lens;
    int n, Hq, Hkv;
    int vheads;         // head groups of at most GC query heads: Hkv * ceil(Hq / Hkv / GC)
    float scale;
    void *out;
    float *lse;         // [n][Hq] or null
    float *part;        // workspace: 2 slots per block of [GC][D + 2]
    int blocks;         // blocks of the main kernel
    int per_pair;       // one block per (sequence, head group), no shares and no join
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Tokens of sequence b that there are: its length, at most what its row of the table can hold.
__host__ __device__ __forceinline__ int clip_len(const DecodeArgs &a, int len) {
    const int64_t most = (int64_t)a.cache.width << a.cache.page_log2;
    return (int)min((int64_t)max(len, 0), most);
}
__host__ __device__ __forceinline__ int decode_len(const DecodeArgs &a, int b) { return clip_len(a, a.lens[b]); }
// The same ahead of a kernel's wait: at GPU scope, so that no line that an SM kept from before is taken for it.
__device__ __forceinline__ int decode_len_early(const DecodeArgs &a, int b) {
    return clip_len(a, tc::ld_relaxed_gpu(a.lens + b));
}
// What a pair costs beside its tiles (its queries, the join of the warps), in tiles: it counts in the shares,
// or blocks with many short pairs would end long after the others.
constexpr int kPairCost = 2;
// Length of a pair on the line.
template <int TILE> __device__ __forceinline__ int units_of(int len) {
    return len > 0 ? (len + TILE - 1) / TILE + kPairCost : 0;
}
template <int TILE> __device__ __forceinline__ int decode_units(const DecodeArgs &a, int b) {
    return units_of<TILE>(decode_len(a, b));
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if (lane == 0) scratch[warp] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < warps; ++w) x += scratch[w];
    return x;
}

// The sequence that holds place `want` of the line (counted for one head group), and its begin.
template <int TILE>
__device__ __forceinline__ void find_sequence(const DecodeArgs &a, int64_t want, int64_t *scratch, int &seq,
                                              int64_t &before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int64_t at = 0;
    for (int base = 0; base < a.n; base += blockDim.x) {
        const int b = base + threadIdx.x;
        const int64_t mine = b < a.n ? decode_units<TILE>(a, b) : 0;
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        __syncthreads();
        if (lane == 31) scratch[warp] = upto;
        __syncthreads();
        int64_t off = at, all = 0;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) off += scratch[w];
            all += scratch[w];
        }
        if (want >= off + upto - mine && want < off + upto) {
            scratch[16] = b;
            scratch[17] = off + upto - mine;
        }
        at += all;
        if (want < at) break;
    }
    __syncthreads();
    seq = (int)scratch[16];
    before = scratch[17];
    __syncthreads();
}

// The line of `all` tiles in `blocks` shares that differ by one tile at most.
struct Shares {
    int64_t per, rem;   // the first `rem` shares have per + 1 tiles
    __device__ __forceinline__ Shares(int64_t all, int blocks) : per(all / blocks), rem(all % blocks) {}
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * per + min(c, rem); }
    // the share that holds tile t
    __device__ __forceinline__ int64_t of(int64_t t) const {
        const int64_t wide = rem * (per + 1);
        return t < wide ? t / (per + 1) : rem + (t - wide) / per;
    }
};

// Walks the tiles of a block's share of the line.
template <int TILE> struct Walk {
    int b, vh, tile, tiles, len;
    int64_t at, last;   // place on the line, the share's end
    // Works the share out from the lengths; false if it is empty.  Every thread of the block.
    __device__ __forceinline__ bool start(const DecodeArgs &a, int64_t *scratch) {
        if (a.per_pair) {
            b = blockIdx.x / a.vheads;
            vh = blockIdx.x % a.vheads;
            tile = 0;
            len = decode_len(a, b);
            tiles = (len + TILE - 1) / TILE;
            at = 0;
            last = tiles;
            return tiles > 0;
        }
        int64_t mine = 0;
        for (int n = threadIdx.x; n < a.n; n += blockDim.x) mine += decode_units<TILE>(a, n);
        const int64_t all = block_sum(mine, scratch) * a.vheads;
        const Shares sh(all, a.blocks);
        at = sh.begin(blockIdx.x);
        last = sh.begin(blockIdx.x + 1);
        if (at >= last) return false;
        int64_t before;
        find_sequence<TILE>(a, at / a.vheads, scratch, b, before);
        len = decode_len(a, b);
        tiles = (len + TILE - 1) / TILE;
        const int64_t in_seq = at - before * a.vheads;
        vh = (int)(in_seq / (tiles + kPairCost));
        tile = (int)(in_seq % (tiles + kPairCost));
        if (tile >= tiles) {   // the share begins behind a pair's last tile
            at -= tile - (tiles - 1);
            tile = tiles - 1;
            next(a);
        }
        return at < last;
    }
    __host__ __device__ __forceinline__ void next(const DecodeArgs &a) {
        ++at;
        if (++tile < tiles) return;
        at += kPairCost;
        tile = 0;
        if (++vh < a.vheads) return;
        vh = 0;
        do {   // behind the last sequence: any length, the caller stops there
            ++b;
            len = b < a.n ? decode_len(a, b) : TILE;
        } while (len == 0);
        tiles = (len + TILE - 1) / TILE;
    }
    __host__ __device__ __forceinline__ bool more() const { return at < last; }
};

template <int D, int GC> struct DecodeCfg {
    static constexpr int kRowBytes = D * 4;
    static constexpr int kStageBytes = 2 * kWarpTokens * kRowBytes;   // keys and values of a warp's tokens
    static constexpr int kStages = 3;
    static constexpr int kDecodeWarps = 4;
    static constexpr int kTile = kDecodeWarps * kWarpTokens;
    static constexpr int kRing = kDecodeWarps * kStages * kStageBytes;
    static constexpr int kQ = GC * D * 4;
    static constexpr int kP = kDecodeWarps * GC * kWarpTokens * 4;
    static constexpr int kJoin = kDecodeWarps * GC * (D + 2) * 4;
    static constexpr int kSmem = kRing + kQ + kP + kJoin + 160;
};

// What a block does for a pair without tokens where no join follows: zeros, lse -inf.
template <typename T, int D, int GC> __device__ __forceinline__ void write_empty(const DecodeArgs &a, int b, int vh) {
    const int group = a.Hq / a.Hkv, chunks = a.vheads / a.Hkv, hkv = vh / chunks, h0 = hkv * group + (vh % chunks) * GC;
    const int nh = min(GC, hkv * group + group - h0);
    T *out = static_cast<T *>(a.out) + ((int64_t)b * a.Hq + h0) * D;
    for (int e = threadIdx.x; e < nh * D; e += blockDim.x) out[e] = from_f32<T>(0.f);
    if (a.lse && threadIdx.x < nh) a.lse[(int64_t)b * a.Hq + h0 + threadIdx.x] = -CUDART_INF_F;
}

// A sequence longer than its row of the table is cut there, and reported.
__device__ __forceinline__ void check_len(const DecodeArgs &a, int b) {
    if (a.lens[b] > decode_len(a, b)) record_device_error(kDevErrBadPage);
}

// Copies a warp's 16 tokens of the tile at `w` into its stage; returns a mask of the valid ones.
template <typename T, int D, int TILE>
__device__ __forceinline__ uint32_t load_tokens(const DecodeArgs &a, const Walk<TILE> &w, int warp, int lane, int hkv,
                                                uint32_t stage) {
    constexpr int CH = D * (int)sizeof(T) / 16;   // 16-byte chunks of a row
    const int t0 = w.tile * TILE + warp * kWarpTokens;
    // lanes 0-15 look up their token's page
    const int tok = t0 + (lane & 15);
    int page = -1;
    if (tok < w.len) {
        page = a.cache.table[w.b * a.cache.row + (tok >> a.cache.page_log2)];
        if (page < 0 || page >= a.cache.num_pages) {
            record_device_error(kDevErrBadPage);
            page = -1;
        }
    }
    const uint32_t valid = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
    const int in_page = (1 << a.cache.page_log2) - 1;
#pragma unroll
    for (int i = 0; i < kWarpTokens * CH / 32; ++i) {
        const int r = (i * 32 + lane) / CH, c = (i * 32 + lane) % CH;
        const int pg = __shfl_sync(0xffffffffu, page, r);
        const int64_t slot = ((int64_t)hkv << a.cache.page_log2) + ((t0 + r) & in_page);
        const T *kr = static_cast<const T *>(a.cache.k), *vr = static_cast<const T *>(a.cache.v);
        if (pg >= 0) {
            kr += pg * a.cache.k_stride + slot * D;
            vr += pg * a.cache.v_stride + slot * D;
        }
        const uint32_t off = r * (CH * 16) + (((c & ~7) | ((c ^ r) & 7)) << 4);
        cp_async16(stage + off, kr + (pg >= 0 ? c * (16 / (int)sizeof(T)) : 0), pg >= 0);
        cp_async16(stage + kWarpTokens * CH * 16 + off, vr + (pg >= 0 ? c * (16 / (int)sizeof(T)) : 0), pg >= 0);
    }
    return valid;
}

// Channels [4 i, 4 i + 4) of a row staged by load_tokens.
template <int D> __device__ __forceinline__ float4 staged4(const float *rows, int r, int i) {
    return *reinterpret_cast<const float4 *>(reinterpret_cast<const char *>(rows) + r * (D * 4) +
                                             (((i & ~7) | ((i ^ r) & 7)) << 4));
}

template <int D, int GC>
__global__ void __launch_bounds__(DecodeCfg<D, GC>::kDecodeWarps * 32, 1) attn_decode_kernel(const DecodeArgs a) {
    using C = DecodeCfg<D, GC>;
    constexpr int kDecodeWarps = C::kDecodeWarps;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *s_q = reinterpret_cast<float *>(smem + C::kRing);
    float *s_join = s_q + GC * D + kDecodeWarps * GC * kWarpTokens;
    int64_t *scratch = reinterpret_cast<int64_t *>(smem + C::kRing + C::kQ + C::kP + C::kJoin);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *s_p = s_q + GC * D + warp * GC * kWarpTokens;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * C::kStages * C::kStageBytes;
    const uint8_t *ring_ptr = smem + warp * C::kStages * C::kStageBytes;

    if (a.per_pair) next_may_start();
    wait_for_previous();
    if (!a.per_pair) next_may_start();   // only now: the join reads the lengths before its own wait
    Walk<C::kTile> w;
    const bool work = w.start(a, scratch);
    if (a.per_pair && tid == 0) check_len(a, w.b);
    if (!work) {
        if (a.per_pair) write_empty<float, D, GC>(a, w.b, w.vh);
        return;
    }
    Walk<C::kTile> ahead = w;

    const int group = a.Hq / a.Hkv, chunks = a.vheads / a.Hkv;
    uint32_t valid[C::kStages];
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) valid[s] = 0;
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) {
        if (ahead.more()) {
            valid[s] = load_tokens<float, D, C::kTile>(a, ahead, warp, lane, ahead.vh / chunks, ring + s * C::kStageBytes);
            ahead.next(a);
        }
        cp_async_commit();
    }

    constexpr int CPL = D / 32;   // channels of a lane in the output
    float m[GC], l[GC], o[GC][CPL];
    const int row = lane & 15, half = lane >> 4;
    bool starts_inside = w.tile != 0;   // the first pair began in an earlier block
    bool fresh = true;
    int st = 0;
    while (w.more()) {
        const int hkv = w.vh / chunks, h0 = hkv * group + (w.vh % chunks) * GC;
        const int nh = min(GC, hkv * group + group - h0);
        if (fresh) {   // a new pair: its queries, scaled so that exp is 2^x
            __syncthreads();
            for (int e = tid; e < GC * D; e += blockDim.x) {
                const int g = e / D;
                s_q[e] = g < nh ? static_cast<const float *>(a.q)[w.b * a.q_stride + (int64_t)h0 * D + e] * (a.scale * kLog2e)
                                : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                m[g] = -CUDART_INF_F;
                l[g] = 0.f;
#pragma unroll
                for (int c = 0; c < CPL; ++c) o[g][c] = 0.f;
            }
            fresh = false;
        }
        // keep the ring full
        {
            const int into = (st + C::kStages - 1) % C::kStages;
            uint32_t got = 0;
            if (ahead.more()) {
                got = load_tokens<float, D, C::kTile>(a, ahead, warp, lane, ahead.vh / chunks, ring + into * C::kStageBytes);
                ahead.next(a);
            }
            cp_async_commit();
#pragma unroll
            for (int s = 0; s < C::kStages; ++s)
                if (s == into) valid[s] = got;
        }
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        uint32_t ok = 0;
#pragma unroll
        for (int s = 0; s < C::kStages; ++s)
            if (s == st) ok = valid[s];
        const float *ks = reinterpret_cast<const float *>(ring_ptr + st * C::kStageBytes);
        const float *vs = ks + kWarpTokens * D;

        // scores: lane (row, half) sums half of the channels of one key
        float s[GC];
#pragma unroll
        for (int g = 0; g < GC; ++g) s[g] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
            const int at = half * (D / 8) + c;
            const float4 kk = staged4<D>(ks, row, at);
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                const float4 qq = *reinterpret_cast<const float4 *>(s_q + g * D + 4 * at);
                s[g] += qq.x * kk.x + qq.y * kk.y + qq.z * kk.z + qq.w * kk.w;
            }
        }
        const bool live = (ok >> row) & 1;
#pragma unroll
        for (int g = 0; g < GC; ++g) {
            float x = s[g] + __shfl_xor_sync(0xffffffffu, s[g], 16);
            x = live ? x : -CUDART_INF_F;
            float top = x;
#pragma unroll
            for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m[g], top), base = mn == -CUDART_INF_F ? 0.f : mn;
            const float f = exp2f(m[g] - base), p = live ? exp2f(x - base) : 0.f;
            m[g] = mn;
            l[g] = l[g] * f + (half == 0 ? p : 0.f);   // a lane's own share of the sum
#pragma unroll
            for (int c = 0; c < CPL; ++c) o[g][c] *= f;
            if (half == 0) s_p[g * kWarpTokens + row] = p;
        }
        __syncwarp();
#pragma unroll 4
        for (int t = 0; t < kWarpTokens; ++t) {
            const float4 x = staged4<D>(vs, t, lane * CPL / 4);
            const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                const float p = s_p[g * kWarpTokens + t];
#pragma unroll
                for (int c = 0; c < CPL; ++c) o[g][c] += p * xs[CPL == 4 ? c : (lane & 1) * 2 + c];
            }
        }
        __syncwarp();

        st = (st + 1) % C::kStages;
        const Walk<C::kTile> cur = w;
        w.next(a);
        const bool end = !w.more();
        if (end || w.b != cur.b || w.vh != cur.vh) {
            // the end of this block's part of a pair: join the warps
            const bool ends_inside = cur.tile + 1 < cur.tiles;
            const bool whole = !starts_inside && !ends_inside;
            float *mine_j = s_join + warp * GC * (D + 2);
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                float sum = l[g];
#pragma unroll
                for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (lane == 0) {
                    mine_j[g * (D + 2)] = m[g];
                    mine_j[g * (D + 2) + 1] = sum;
                }
#pragma unroll
                for (int c = 0; c < CPL; ++c) mine_j[g * (D + 2) + 2 + lane * CPL + c] = o[g][c];
            }
            __syncthreads();
            // the first pair of a share leaves its part in slot 0, the last in slot 1
            float *part = a.part + ((int64_t)blockIdx.x * 2 + (starts_inside || !end ? 0 : 1)) * GC * (D + 2);
            for (int e = tid; e < nh * D; e += blockDim.x) {
                const int g = e / D, c = e % D;
                float top = -CUDART_INF_F;
#pragma unroll
                for (int k = 0; k < kDecodeWarps; ++k) top = fmaxf(top, s_join[(k * GC + g) * (D + 2)]);
                const float base = top == -CUDART_INF_F ? 0.f : top;
                float sum = 0.f, acc = 0.f;
#pragma unroll
                for (int k = 0; k < kDecodeWarps; ++k) {
                    const float *j = s_join + (k * GC + g) * (D + 2);
                    const float f = exp2f(j[0] - base);
                    sum += f * j[1];
                    acc += f * j[2 + c];
                }
                if (whole) {
                    const int64_t h = (int64_t)cur.b * a.Hq + h0 + g;
                    static_cast<float *>(a.out)[h * D + c] = sum > 0.f || sum != sum ? acc / sum : 0.f;
                    if (c == 0 && a.lse)
                        a.lse[h] = sum == 0.f ? -CUDART_INF_F : top * 0.69314718055994531f + logf(sum);
                } else {
                    part[g * (D + 2) + 2 + c] = acc;
                    if (c == 0) {
                        part[g * (D + 2)] = top;
                        part[g * (D + 2) + 1] = sum;
                    }
                }
            }
            __syncthreads();
            starts_inside = false;
            fresh = true;
        }
    }
    cp_async_wait<0>();
}

// Joins the parts of every pair that more than one block worked on, and writes the rows of sequences
// without a token (zeros, lse -inf).  One block per (sequence, head group), one warp per head; the parts
// of a head are read several at a time, since each read waits for L2.
constexpr int kJoinThreads = 256;
template <typename T, int D, int GC, int TILE>
__global__ void __launch_bounds__(kJoinThreads) attn_decode_join_kernel(const DecodeArgs a) {
    constexpr int CPL = D / 32;   // channels of a lane
    __shared__ int64_t scratch[20];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x / a.vheads, vh = blockIdx.x % a.vheads;
    next_may_start();
    // The lengths are older than the kernel before this one, which lets this one start when it has itself
    // waited for them, so they are complete in memory; the shares are worked out while it runs.
    int64_t all = 0, before = 0;
    for (int n = tid; n < a.n; n += blockDim.x) {
        const int t = units_of<TILE>(decode_len_early(a, n));
        all += t;
        if (n < b) before += t;
    }
    all = block_sum(all, scratch) * a.vheads;
    before = block_sum(before, scratch) * a.vheads;
    const int group = a.Hq / a.Hkv, chunks = a.vheads / a.Hkv, hkv = vh / chunks, h0 = hkv * group + (vh % chunks) * GC;
    const int nh = min(GC, hkv * group + group - h0);
    const int tiles = (decode_len_early(a, b) + TILE - 1) / TILE;
    const Shares sh(all, a.blocks);
    const int64_t s0 = before + (int64_t)vh * (tiles + kPairCost);
    const int c0 = tiles > 0 ? (int)sh.of(s0) : 0, c1 = tiles > 0 ? (int)sh.of(s0 + tiles - 1) : 0;
    wait_for_previous();
    if (tid == 0 && vh == 0) check_len(a, b);
    if (tiles == 0) {
        write_empty<T, D, GC>(a, b, vh);
        return;
    }
    if (c0 == c1) return;   // one block had it all and wrote the output
    for (int g = warp; g < nh; g += kJoinThreads / 32) {
        // the first block's part lies in its slot 0 if the pair began before its share; the others' in slot 0
        auto part_of = [&](int k) {
            return a.part + (((int64_t)k * 2 + (s0 < sh.begin(k) ? 0 : 1)) * GC + g) * (D + 2);
        };
        float top = -CUDART_INF_F, sum = 0.f, acc[CPL];
        for (int k = c0 + lane; k <= c1; k += 32) top = fmaxf(top, part_of(k)[0]);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == -CUDART_INF_F ? 0.f : top;
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc[c] = 0.f;
#pragma unroll 8
        for (int k = c0; k <= c1; ++k) {
            const float *p = part_of(k);
            const float f = exp2f(p[0] - base);
            sum += p[1] * f;
#pragma unroll
            for (int c = 0; c < CPL; c += 2) {
                const float2 x = *reinterpret_cast<const float2 *>(p + 2 + lane * CPL + c);
                acc[c] += x.x * f;
                acc[c + 1] += x.y * f;
            }
        }
        const int64_t h = (int64_t)b * a.Hq + h0 + g;
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            static_cast<T *>(a.out)[h * D + lane * CPL + c] = from_f32<T>(sum > 0.f || sum != sum ? acc[c] / sum : 0.f);
        if (lane == 0 && a.lse) a.lse[h] = sum == 0.f ? -CUDART_INF_F : top * 0.69314718055994531f + logf(sum);
    }
}

constexpr int kMaxDecodeBlocks = 1024;

// Blocks of the main kernel: one per SM, no more than there can be tiles.
inline int decode_blocks(const DecodeArgs &a, int tile, int sms) {
    const int64_t tokens = (int64_t)a.cache.width << a.cache.page_log2;
    const int64_t t = (int64_t)a.n * a.vheads * ((tokens + tile - 1) / tile);
    const int most = sms < kMaxDecodeBlocks ? sms : kMaxDecodeBlocks;
    return (int)(t < most ? t : most);
}

}  // namespace attn
}  // namespace kda
