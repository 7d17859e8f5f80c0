// Test-only probe of parts of the attention kernels, from the kernels' own source.
#include <stdint.h>

#include "../../gated_delta_rule_86_b200/csrc/attn_decode_mma.cuh"
#include "../../gated_delta_rule_86_b200/csrc/attn_prompt_tc.cuh"

using namespace kda::attn;

namespace {

// The places of the line from (b, vh, 0) on, `count` of them, as a warp of the bf16 decode step walks them;
// returns how often the page that it was given is `marker`.
template <int TILE> int64_t walk(const DecodeArgs &a, int b, int vh, int64_t count, int warp, int32_t marker) {
    Walk<TILE> w = {};
    w.b = b;
    w.vh = vh;
    w.len = decode_len(a, b);
    w.tiles = (w.len + TILE - 1) / TILE;
    w.last = count;
    int64_t hits = 0;
    if (!w.more()) return 0;
    for (int page = first_page(a, w, warp);; page = next_page(a, w, warp)) {
        hits += page == marker;
        if (!w.more()) return hits;
    }
}

// The softmax warp and place (16 * place + warp) that gives up; none: -1.
__device__ int g_quit = -1;
struct QuitOne {
    static __device__ __forceinline__ bool gives_up(int warp, int place, volatile int *abort) {
        if (16 * place + warp != g_quit) return false;
        kda::record_device_error(kda::kDevErrTimeout);
        *abort = 1;
        return true;
    }
};

}  // namespace

// On the host, over host memory.
extern "C" int64_t attn_probe_walk(const int32_t *lens, int n, int vheads, const int32_t *table, int64_t row, int width,
                                   int page_log2, int b, int vh, int64_t count, int warp, int32_t marker) {
    DecodeArgs a = {};
    a.lens = lens;
    a.n = n;
    a.vheads = vheads;
    a.cache.table = table;
    a.cache.row = row;
    a.cache.width = width;
    a.cache.page_log2 = page_log2;
    return walk<DecodeMmaCfg<128, 8>::kTile>(a, b, vh, count, warp, marker);
}

// The prompt kernel with one softmax warp of every block giving up (see NoFault).  Synchronises; returns the
// device error word, which it clears, or -1 if a CUDA call failed.
extern "C" int attn_probe_give_up(int quit, int d, const void *q, const void *k, const void *v, int B, int T, int Hq, int Hkv,
                                  float scale, void *out) {
    PromptArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = (int64_t)Hq * d;
    a.k_stride = a.v_stride = (int64_t)Hkv * d;
    a.bt.n = B;
    a.bt.Tq = a.bt.Tk = T;
    a.bt.Hq = Hq;
    a.bt.Hkv = Hkv;
    a.causal = true;
    a.scale = scale;
    a.out = out;
    int sms = 0, word = 0;
    const int none = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, 0) != cudaSuccess) return -1;
    if (cudaMemcpyToSymbol(g_quit, &quit, sizeof(quit)) != cudaSuccess) return -1;
    if ((d == 64 ? launch_prompt_tc<64, QuitOne>(a, sms, nullptr) : launch_prompt_tc<128, QuitOne>(a, sms, nullptr)) !=
        cudaSuccess)
        return -1;
    if (cudaDeviceSynchronize() != cudaSuccess) return -1;
    if (cudaMemcpyFromSymbol(&word, kda::g_device_error, sizeof(word)) != cudaSuccess) return -1;
    if (cudaMemcpyToSymbol(kda::g_device_error, &none, sizeof(none)) != cudaSuccess) return -1;
    return word;
}

// Whether the decode step gives each pair a block of its own; on the host.
extern "C" int attn_probe_per_pair(int64_t pairs, int64_t tokens, int d, int bf16, int sms) {
    return decode_per_pair(pairs, tokens, d, bf16 != 0, sms);
}

// The rows of a block that fp32 prompts get: forward, gradient in one launch or not, its queries', its keys'; on the host.
extern "C" void attn_probe_rows(int d, int causal, int n, int Tq, int Tk, int Hq, int Hkv, int packed, int sms, int32_t *rows) {
    PromptArgs a = {};
    const int32_t offsets = 0;   // never looked into
    a.bt.cu_q = a.bt.cu_k = packed ? &offsets : nullptr;
    a.bt.n = n;
    a.bt.Tq = Tq;
    a.bt.Tk = Tk;
    a.bt.Hq = Hq;
    a.bt.Hkv = Hkv;
    a.causal = causal != 0;
    const GradRows g = grad_rows(a, d, sms);
    rows[0] = prompt_rows(a, d, sms);
    rows[1] = g.one;
    rows[2] = g.q;
    rows[3] = g.k;
}

namespace {
__global__ void powers(const float *x, float *y, int n) {   // n even
    const int i = 2 * (blockIdx.x * blockDim.x + threadIdx.x);
    if (i + 1 >= n) return;
    const float2 p = ex2_fma(make_float2(x[i], x[i + 1]));
    y[i] = p.x;
    y[i + 1] = p.y;
}
}  // namespace

// y[i] = 2^x[i] as the prompt kernel computes a part of its weights on the FMA units; n even.
extern "C" int attn_probe_powers(const float *x, float *y, int n) {
    powers<<<(n / 2 + 255) / 256, 256>>>(x, y, n);
    return cudaDeviceSynchronize() == cudaSuccess ? 0 : -1;
}
