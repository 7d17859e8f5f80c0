// attn_common.cuh -- what the softmax-attention kernels share: the batch's layout in memory, the
// paged cache's, and the lookup of a sequence's tiles.
#pragma once

#include <math_constants.h>

#include "kda_common.cuh"

namespace kda {
namespace attn {

// Recorded in the device error word when a page table names a page outside the pool, or a sequence
// is longer than its row of the table (mirrors KDA_ERR_BAD_PAGE).
constexpr int kDevErrBadPage = 5;

// Kernels of this family are launched so that they may start while the one before them in the stream still
// runs (programmatic dependent launch): their blocks come up, set up what is theirs alone, and wait there for
// the end of what is before them, ahead of their first access to memory.  A decode step's kernels are so
// short that coming up is a third of their time.
// What earlier kernels may have written is read by plain loads: the non-coherent ones (__ldg) are for data that no
// one writes while a kernel is resident, which does not hold for a kernel that comes up under its writer.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... A, typename... B>
cudaError_t launch_behind(void (*kern)(A...), unsigned grid, int threads, size_t smem, cudaStream_t st, const B &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The batch of a prompt call.  Dense: sequence n is row n of [B, T].  Packed (cu given): B == 1 and
// sequence n is tokens cu[n] .. cu[n + 1] - 1.
struct Batch {
    const int32_t *cu_q, *cu_k;   // cu_k == cu_q when the keys have no offsets of their own
    int n;                        // sequences
    int Tq, Tk;                   // tokens of a row (dense), or of the packed tensors
    int Hq, Hkv;
};

struct Seq {
    int64_t q0, k0;   // first query and key, as rows of the flattened [B * T] tensors
    int nq, nk;       // queries and keys
};

// Range [a, b) of sequence n, held inside the tensor whatever the offsets say.
__device__ __forceinline__ void seq_range(const int32_t *cu, int n, int T, int64_t &first, int &len) {
    if (cu == nullptr) {
        first = (int64_t)n * T;
        len = T;
        return;
    }
    const int a = min(max(cu[n], 0), T), b = min(max(cu[n + 1], a), T);
    first = a;
    len = b - a;
}

__device__ __forceinline__ Seq seq_of(const Batch &bt, int n) {
    Seq s;
    seq_range(bt.cu_q, n, bt.Tq, s.q0, s.nq);
    seq_range(bt.cu_k, n, bt.Tk, s.k0, s.nk);
    return s;
}

// Upper bound of the tiles of `tile` rows over all sequences, known on the host.
inline int64_t max_tiles(const int32_t *cu, int n, int T, int tile) {
    const int64_t per_row = ((int64_t)T + tile - 1) / tile;
    return cu == nullptr ? per_row * n : (int64_t)T / tile + n;
}

// The index-th tile of `tile` rows, counted through the sequences in order; false if there are fewer.
// Called by every thread of the block (it synchronises); `scratch` is 34 words of shared memory.
// A block of W warps looks at 32 W sequences at a time.
__device__ __forceinline__ bool find_tile(const int32_t *cu, int nseq, int T, int tile, int64_t index, int *scratch,
                                          int &seq, int &t) {
    if (cu == nullptr) {
        const int per_row = (T + tile - 1) / tile;
        if (per_row == 0 || index >= (int64_t)per_row * nseq) return false;
        seq = (int)(index / per_row);
        t = (int)(index % per_row);
        return true;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int64_t before = 0;
    if (threadIdx.x == 0) scratch[32] = -1;
    for (int base = 0; base < nseq; base += blockDim.x) {
        const int n = base + threadIdx.x;
        int mine = 0;
        if (n < nseq) {
            int64_t first;
            int len;
            seq_range(cu, n, T, first, len);
            mine = (len + tile - 1) / tile;
        }
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        __syncthreads();
        if (lane == 31) scratch[warp] = upto;
        __syncthreads();
        int64_t off = before, all = 0;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) off += scratch[w];
            all += scratch[w];
        }
        if (index >= off + upto - mine && index < off + upto) {
            scratch[32] = n;
            scratch[33] = (int)(index - (off + upto - mine));
        }
        before += all;
        if (index < before) break;
    }
    __syncthreads();
    seq = scratch[32];
    t = scratch[33];
    __syncthreads();
    return seq >= 0;
}

// The index-th tile in an order in which no tile comes before one of a higher level, the level of tile t of a
// sequence being t + 1 (with causal masking: the number of key tiles that it sees): items of about the same
// cost go out together, the largest first.  Gives the sequence, its number of tiles and the level; false if
// there are fewer tiles.  A whole warp.  Of more than 128 packed sequences the tiles come in the sequences' own
// order, each sequence's from its end; `from` then keeps the place from one call to the next, whose index may not be
// smaller.  (8192 sequences of 8 tokens, 16 + 4 heads of 64: 2.2 ms; 15.9 where every call looks through all sequences
// before its own.  129 ragged sequences of up to 4096 tokens take a tenth longer than 127 by levels: 539 and 493 us.)
struct PlaceFrom {
    int n0 = 0;            // 32 sequences are looked at together, these next
    int64_t before = 0;    // tiles of those before them
};
__device__ __forceinline__ bool place_of(const int32_t *cu, int nseq, int T, int tile, int64_t index, int lane, int &seq,
                                         int &count, int &level, PlaceFrom &from) {
    if (cu == nullptr) {
        count = (T + tile - 1) / tile;
        if (index >= (int64_t)count * nseq) return false;
        level = count - (int)(index / nseq);
        seq = (int)(index % nseq);
        return true;
    }
    constexpr int kHeld = 4;   // tile counts that a lane keeps: the levels are searched for up to 128 sequences
    int c[kHeld];
    auto tiles_of = [&](int n) {
        int64_t first;
        int len = 0;
        if (n < nseq) seq_range(cu, n, T, first, len);
        return (len + tile - 1) / tile;
    };
    if (nseq > 32 * kHeld) {
        for (; from.n0 < nseq; from.n0 += 32) {
            const int mine = tiles_of(from.n0 + lane);
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const int64_t end = from.before + upto;
            const uint32_t hit = __ballot_sync(0xffffffffu, index >= end - mine && index < end);
            if (hit) {
                const int at = __ffs(hit) - 1;
                seq = from.n0 + at;
                count = __shfl_sync(0xffffffffu, mine, at);
                level = (int)(__shfl_sync(0xffffffffu, end, at) - index);
                return true;
            }
            from.before += __shfl_sync(0xffffffffu, upto, 31);
        }
        return false;
    }
    int top = 0;
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
        c[x] = tiles_of(x * 32 + lane);
        top = max(top, c[x]);
    }
    top = __reduce_max_sync(0xffffffffu, (unsigned)top);
    auto above = [&](int l) {   // tiles of a level above l
        int sum = 0;
#pragma unroll
        for (int x = 0; x < kHeld; ++x) sum += max(0, c[x] - l);
        return (int64_t)__reduce_add_sync(0xffffffffu, sum);
    };
    if (index >= above(0)) return false;
    int lo = 0, hi = top;   // above(lo) > index >= above(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (above(mid) > index) lo = mid;
        else hi = mid;
    }
    level = hi;
    int k = (int)(index - above(hi));   // the k-th sequence with that level
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
        uint32_t have = __ballot_sync(0xffffffffu, c[x] >= level);
        const int number = __popc(have);
        if (k < number) {
            for (; k > 0; --k) have &= have - 1;
            const int at = __ffs(have) - 1;
            seq = x * 32 + at;
            count = __shfl_sync(0xffffffffu, c[x], at);
            return true;
        }
        k -= number;
    }
    return false;
}

// Keys that query `row` of a sequence sees, counted from the first: with causal masking query i sees keys
// j <= i + nk - nq, so that the last query sees the last key.
__device__ __forceinline__ int keys_seen(const Seq &s, int row, bool causal) {
    return causal ? min(s.nk, max(0, row + 1 + s.nk - s.nq)) : s.nk;
}

// A paged cache: [num_pages][Hkv][page_size][d], pages `k_stride` / `v_stride` elements apart.
struct Cache {
    void *k, *v;
    int64_t k_stride, v_stride;
    const int32_t *table;   // [sequences][width], rows `row` entries apart
    int64_t row;
    int width, num_pages, page_log2;
};

}  // namespace attn
}  // namespace kda
