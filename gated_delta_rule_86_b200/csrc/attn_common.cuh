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
    const int a = min(max(__ldg(cu + n), 0), T), b = min(max(__ldg(cu + n + 1), a), T);
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

// Keys [lo, hi) that some query of rows [r0, r1) of a sequence sees: with causal masking query i sees
// keys j <= i + nk - nq, so that the last query sees the last key.
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
