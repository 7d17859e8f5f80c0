// attn_api.cuh -- host side of the softmax-attention entry points (declared in include/kda.h):
// argument validation, kernel selection and launch.  Included by kda_api.cu.
#pragma once

#include <cmath>

#include "../../include/kda.h"
#include "attn_append.cuh"
#include "attn_decode_mma.cuh"
#include "attn_grad_tc.cuh"
#include "attn_prompt.cuh"
#include "attn_prompt_tc.cuh"
#include "kda_chunk_tc.cuh"

namespace kda {
namespace attn {

inline bool aligned(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Types, heads and head size.  Unsupported values of valid arguments come last.
inline kda_status check_heads(int32_t Hq, int32_t Hkv, int32_t d, kda_dtype dtype) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d < 1) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)Hq * d > (1 << 24)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// Elements from one token to the next: 0 means dense.  Tokens may not overlap, and every row must keep
// the 16-byte alignment.
inline kda_status take_stride(int64_t &stride, int32_t heads, int32_t d, int esize) {
    if (stride == 0) stride = (int64_t)heads * d;
    if (stride < (int64_t)heads * d || stride * esize % 16 != 0 || stride > (int64_t(1) << 31))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

inline kda_status check_cache(Cache &c, void *k, void *v, int64_t k_stride, int64_t v_stride, int32_t num_pages,
                              int32_t page_size, const int32_t *table, int64_t table_stride, int32_t width,
                              int32_t Hkv, int32_t d, int esize) {
    if (!k || !v || !table || num_pages < 1 || page_size < 1 || width < 1) return KDA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(table, 4)) return KDA_ERR_INVALID_ARG;
    const int64_t dense = (int64_t)Hkv * page_size * d;
    if (k_stride == 0) k_stride = dense;
    if (v_stride == 0) v_stride = dense;
    if (k_stride < dense || v_stride < dense || k_stride * esize % 16 != 0 || v_stride * esize % 16 != 0)
        return KDA_ERR_INVALID_ARG;
    if (table_stride == 0) table_stride = width;
    if (table_stride < width) return KDA_ERR_INVALID_ARG;
    if ((page_size & (page_size - 1)) != 0 || page_size > (1 << 16)) return KDA_ERR_UNSUPPORTED;
    c.k = k;
    c.v = v;
    c.k_stride = k_stride;
    c.v_stride = v_stride;
    c.table = table;
    c.row = table_stride;
    c.width = width;
    c.num_pages = num_pages;
    c.page_log2 = 0;
    while ((1 << c.page_log2) < page_size) ++c.page_log2;
    return KDA_OK;
}

inline bool scale_ok(float s) { return std::isfinite(s) && s > 0.f; }

// The checks that the prompt calls share; fills the arguments' common part.
inline kda_status check_prompt(PromptArgs &a, const void *q, const void *k, const void *v, int64_t q_stride,
                               int64_t k_stride, int64_t v_stride, const int32_t *cu_q, const int32_t *cu_k,
                               int32_t num_seqs, int32_t B, int32_t Tq, int32_t Tk, int32_t Hq, int32_t Hkv, int32_t d,
                               int32_t causal, float scale, kda_dtype dtype, const void *out) {
    if (B < 1 || Tq < 0 || Tk < 0) return KDA_ERR_INVALID_ARG;
    if ((Tq > 0 && (!q || !out)) || (Tk > 0 && (!k || !v))) return KDA_ERR_INVALID_ARG;
    if (cu_k && !cu_q) return KDA_ERR_INVALID_ARG;
    if (cu_q) {
        if (B != 1 || num_seqs < 1 || !aligned(cu_q, 4) || !aligned(cu_k, 4)) return KDA_ERR_INVALID_ARG;
        if (!cu_k && Tk != Tq) return KDA_ERR_INVALID_ARG;
    }
    if (!scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, out};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    kda_status s = check_heads(Hq, Hkv, d, dtype);
    const kda_status heads = s;
    if (s == KDA_ERR_INVALID_ARG) return s;
    const int esize = dtype == KDA_F32 ? 4 : 2;
    if ((s = take_stride(q_stride, Hq, d, esize)) != KDA_OK) return s;
    if ((s = take_stride(k_stride, Hkv, d, esize)) != KDA_OK) return s;
    if ((s = take_stride(v_stride, Hkv, d, esize)) != KDA_OK) return s;
    if (heads != KDA_OK) return heads;
    const int64_t most = (int64_t)B * (Tq > Tk ? Tq : Tk) + (cu_q ? num_seqs : 0);
    if (most >= (int64_t(1) << 31) || Hq > 65535) return KDA_ERR_UNSUPPORTED;   // 32-bit rows and grid limits
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.bt.cu_q = cu_q;
    a.bt.cu_k = cu_q ? (cu_k ? cu_k : cu_q) : nullptr;
    a.bt.n = cu_q ? num_seqs : B;
    a.bt.Tq = Tq;
    a.bt.Tk = Tk;
    a.bt.Hq = Hq;
    a.bt.Hkv = Hkv;
    a.causal = causal != 0;
    a.scale = scale;
    return KDA_OK;
}

inline kda_status status_of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace attn
}  // namespace kda

extern "C" {

kda_status kda_kv_append(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                         int64_t v_stride, const float *inv_freq, int32_t rotary_dim, int32_t interleaved,
                         const int32_t *cu_seqlens, int32_t num_seqs, int32_t B, int32_t T, int32_t Hq, int32_t Hkv,
                         int32_t d, kda_dtype dtype, const int32_t *cache_lens, const int32_t *page_table,
                         int64_t table_stride, int32_t table_width, void *k_cache, void *v_cache,
                         int64_t k_page_stride, int64_t v_page_stride, int32_t num_pages, int32_t page_size,
                         void *q_out, void *k_out, void *stream) {
    using namespace kda::attn;
    if (B < 1 || T < 0 || !cache_lens || !aligned(cache_lens, 4)) return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!k || !v || (q != nullptr) != (q_out != nullptr))) return KDA_ERR_INVALID_ARG;
    if (cu_seqlens && (B != 1 || num_seqs < 1 || !aligned(cu_seqlens, 4))) return KDA_ERR_INVALID_ARG;
    if (rotary_dim < 0 || (rotary_dim > 0 && (!inv_freq || !aligned(inv_freq, 4)))) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, q_out, k_out};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    if (!q) Hq = Hkv;   // no queries to rotate: their head count says nothing
    const kda_status heads = check_heads(Hq, Hkv, d, dtype);
    if (heads == KDA_ERR_INVALID_ARG) return heads;
    if (rotary_dim > d || rotary_dim % 2 != 0) return KDA_ERR_INVALID_ARG;
    const int esize = dtype == KDA_F32 ? 4 : 2;
    AppendArgs a = {};
    kda_status s;
    if ((s = take_stride(q_stride, Hq, d, esize)) != KDA_OK) return s;
    if ((s = take_stride(k_stride, Hkv, d, esize)) != KDA_OK) return s;
    if ((s = take_stride(v_stride, Hkv, d, esize)) != KDA_OK) return s;
    if (q && q == q_out && q_stride != (int64_t)Hq * d) return KDA_ERR_INVALID_ARG;   // in place only where dense
    if ((s = check_cache(a.cache, k_cache, v_cache, k_page_stride, v_page_stride, num_pages, page_size, page_table,
                         table_stride, table_width, Hkv, d, esize)) != KDA_OK)
        return s;
    if (heads != KDA_OK) return heads;
    if (rotary_dim % 16 != 0) return KDA_ERR_UNSUPPORTED;   // half of it is whole 16-byte vectors
    if ((int64_t)B * T >= (int64_t(1) << 31)) return KDA_ERR_UNSUPPORTED;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.inv_freq = inv_freq;
    a.rotary = rotary_dim;
    a.interleaved = interleaved != 0;
    a.cu = cu_seqlens;
    a.cache_lens = cache_lens;
    a.n = cu_seqlens ? num_seqs : B;
    a.T = T;
    a.Hq = q ? Hq : 0;
    a.Hkv = Hkv;
    a.tokens = (int64_t)B * T;
    a.q_out = q_out;
    a.k_out = k_out;
    if (a.tokens == 0) return KDA_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = kda::device_sm_count();
    if (sms < 1) return KDA_ERR_CUDA;
    if (dtype == KDA_F32)
        return status_of(d == 64 ? launch_append_d<float, 64>(a, sms, st) : launch_append_d<float, 128>(a, sms, st));
    return status_of(d == 64 ? launch_append_d<__nv_bfloat16, 64>(a, sms, st)
                             : launch_append_d<__nv_bfloat16, 128>(a, sms, st));
}

kda_status kda_attn_decode_workspace_size(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int64_t max_tokens,
                                          kda_dtype dtype, size_t *bytes) {
    using namespace kda::attn;
    if (!bytes || B < 1 || max_tokens < 1) return KDA_ERR_INVALID_ARG;
    *bytes = 0;
    const kda_status s = check_heads(Hq, Hkv, d, dtype);
    if (s != KDA_OK) return s;
    *bytes = decode_workspace_bytes(B, Hq, Hkv, d, max_tokens, dtype == KDA_BF16, kda::device_sm_count());
    return KDA_OK;
}

kda_status kda_attn_decode_step(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                                int64_t k_page_stride, int64_t v_page_stride, int32_t num_pages, int32_t page_size,
                                const int32_t *page_table, int64_t table_stride, int32_t table_width,
                                const int32_t *seq_lens, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, float scale,
                                kda_dtype dtype, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                void *stream) {
    using namespace kda::attn;
    if (B < 1 || !q || !out || !seq_lens) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(seq_lens, 4) || !aligned(lse, 4)) return KDA_ERR_INVALID_ARG;
    if (!scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    const kda_status heads = check_heads(Hq, Hkv, d, dtype);
    if (heads == KDA_ERR_INVALID_ARG) return heads;
    const int esize = dtype == KDA_F32 ? 4 : 2;
    DecodeArgs a = {};
    kda_status s;
    if ((s = take_stride(q_stride, Hq, d, esize)) != KDA_OK) return s;
    if ((s = check_cache(a.cache, const_cast<void *>(k_cache), const_cast<void *>(v_cache), k_page_stride,
                         v_page_stride, num_pages, page_size, page_table, table_stride, table_width, Hkv, d, esize)) !=
        KDA_OK)
        return s;
    if (heads != KDA_OK) return heads;
    const int sms = kda::device_sm_count();
    const size_t need = decode_workspace_bytes(B, Hq, Hkv, d, (int64_t)table_width << a.cache.page_log2,
                                               dtype == KDA_BF16, sms);
    if (!aligned(workspace, 16) || (need > 0 && !workspace) || workspace_bytes < need) return KDA_ERR_INVALID_ARG;
    if ((int64_t)B * Hq > 0x7fffffff) return KDA_ERR_UNSUPPORTED;
    if (((int64_t)table_width << a.cache.page_log2) > 0x7fffffff - 1024) return KDA_ERR_UNSUPPORTED;
    a.q = q;
    a.q_stride = q_stride;
    a.lens = seq_lens;
    a.n = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.part = static_cast<float *>(workspace);
    if (sms < 1) return KDA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == KDA_F32)
        return status_of(d == 64 ? launch_attn_decode_f32<64>(a, sms, st) : launch_attn_decode_f32<128>(a, sms, st));
    return status_of(d == 64 ? launch_attn_decode_bf16<64>(a, sms, st) : launch_attn_decode_bf16<128>(a, sms, st));
}

kda_status kda_attn_fwd(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                        int64_t v_stride, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int32_t num_seqs,
                        int32_t B, int32_t Tq, int32_t Tk, int32_t Hq, int32_t Hkv, int32_t d, int32_t causal,
                        float scale, kda_dtype dtype, void *out, void *out_rest, float *lse, void *stream) {
    using namespace kda::attn;
    PromptArgs a = {};
    if (!aligned(lse, 4) || !aligned(out_rest, 16)) return KDA_ERR_INVALID_ARG;
    const kda_status s = check_prompt(a, q, k, v, q_stride, k_stride, v_stride, cu_seqlens_q, cu_seqlens_k, num_seqs,
                                      B, Tq, Tk, Hq, Hkv, d, causal, scale, dtype, out);
    if (s != KDA_OK) return s;
    if (out_rest && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    a.out = out;
    a.rest = out_rest;
    a.lse = lse;
    if (Tq == 0) return KDA_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = kda::device_sm_count();
    if (sms < 1) return KDA_ERR_CUDA;
    if (dtype == KDA_F32) return status_of(d == 64 ? launch_prompt<64>(a, sms, st) : launch_prompt<128>(a, sms, st));
    return status_of(d == 64 ? launch_prompt_tc<64>(a, sms, st) : launch_prompt_tc<128>(a, sms, st));
}

kda_status kda_attn_bwd_workspace_size(int32_t B, int32_t Tq, int32_t Hq, size_t *bytes) {
    if (!bytes || B < 1 || Tq < 0 || Hq < 1) return KDA_ERR_INVALID_ARG;
    *bytes = (size_t)B * Tq * Hq * sizeof(float);
    return KDA_OK;
}

kda_status kda_attn_bwd(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                        int64_t v_stride, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int32_t num_seqs,
                        int32_t B, int32_t Tq, int32_t Tk, int32_t Hq, int32_t Hkv, int32_t d, int32_t causal,
                        float scale, kda_dtype dtype, const void *out, const void *out_rest, const float *lse,
                        const void *d_out, void *dq, void *dk, void *dv, void *workspace, size_t workspace_bytes,
                        void *stream) {
    using namespace kda::attn;
    PromptArgs a = {};
    const kda_status s = check_prompt(a, q, k, v, q_stride, k_stride, v_stride, cu_seqlens_q, cu_seqlens_k, num_seqs,
                                      B, Tq, Tk, Hq, Hkv, d, causal, scale, dtype, out);
    if (s != KDA_OK) return s;
    if ((Tq > 0 && (!lse || !d_out || !dq)) || (Tk > 0 && (!dk || !dv))) return KDA_ERR_INVALID_ARG;
    if (out_rest && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {out_rest, d_out, dq, dk, dv, workspace};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    if (!aligned(lse, 4)) return KDA_ERR_INVALID_ARG;
    if (Tq > 0 && (!workspace || workspace_bytes < (size_t)B * Tq * Hq * sizeof(float))) return KDA_ERR_INVALID_ARG;
    a.out = const_cast<void *>(out);
    a.rest = const_cast<void *>(out_rest);
    a.lse = const_cast<float *>(lse);
    a.d_out = d_out;
    a.delta = static_cast<float *>(workspace);
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = kda::device_sm_count();
    if (sms < 1) return KDA_ERR_CUDA;
    if (dtype == KDA_F32)
        return status_of(d == 64 ? launch_prompt_grad<64>(a, sms, st) : launch_prompt_grad<128>(a, sms, st));
    return status_of(d == 64 ? launch_prompt_grad_tc<64>(a, sms, st) : launch_prompt_grad_tc<128>(a, sms, st));
}

}  // extern "C"
