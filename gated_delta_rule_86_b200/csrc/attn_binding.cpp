// attn_binding.cpp -- the Python binding of the softmax-attention calls of include/kda.h.
//
// Argument marshalling only: checks, outputs and workspaces from torch's allocator, pointers and the
// device's current stream to libkda_b200.so.  It is native because a decode step takes 3 to 7 us on the GPU
// and the same steps in Python took 10 us more on the host than the launch itself; the gradient's half
// runs on autograd's thread without the interpreter.
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/variable.h>
#include <torch/extension.h>

#include <cmath>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/kda.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

// A library call's status that is not KDA_OK; becomes the package's KdaError in Python.
struct StatusError : std::runtime_error {
    int status;
    std::string call;
    StatusError(int s, const char *c)
        : std::runtime_error(std::string(c) + " failed: " + kda_status_string(static_cast<kda_status>(s))),
          status(s), call(c) {}
};

void check(kda_status s, const char *call) {
    if (s != KDA_OK) throw StatusError(s, call);
}

template <typename... A> [[noreturn]] void bad_value(const A &...a) {
    std::ostringstream s;
    (s << ... << a);
    throw py::value_error(s.str());
}
template <typename... A> [[noreturn]] void bad_type(const A &...a) {
    std::ostringstream s;
    (s << ... << a);
    throw py::type_error(s.str());
}

kda_dtype code_of(const Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return KDA_BF16;
    if (t.scalar_type() == at::kFloat) return KDA_F32;
    bad_type("unsupported dtype ", t.scalar_type(), "; use torch.float32 or torch.bfloat16");
}

void same(const Tensor &t, const Tensor &x) {
    if (x.scalar_type() != t.scalar_type())
        bad_type("all token tensors and the cache must share one dtype: got ", x.scalar_type(), " beside ",
                 t.scalar_type());
    if (x.device() != t.device())
        bad_value("all tensors of a call must be on one device: got ", x.device(), " beside ", t.device());
}

void on_gpu(const Tensor &t) {
    if (!t.is_cuda()) bad_value("softmax attention takes CUDA tensors");
}

// A one-dimensional int32 tensor of n entries (any number: -1) on the call's device, dense.
Tensor ints(const Tensor &t, const char *name, int64_t n, const Tensor &beside) {
    if (t.scalar_type() != at::kInt || t.dim() != 1) bad_type(name, " must be a one-dimensional int32 tensor");
    if (n >= 0 && t.size(0) != n) bad_value(name, " must have ", n, " entries");
    if (t.device() != beside.device()) bad_value(name, " must be on the device of the other tensors");
    return t.contiguous();
}

bool aligned(const Tensor &t) { return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0; }

// A token tensor [B, T, H, d] as the kernels can read it, and the elements from one token to the next: where
// it is, if its heads are dense and its tokens an even, aligned distance apart; a copy otherwise.
std::pair<Tensor, int64_t> tokens(const Tensor &t) {
    const int64_t B = t.size(0), T = t.size(1), H = t.size(2), d = t.size(3);
    int64_t step = H * d;
    Tensor x = t;
    if (!t.is_contiguous()) {
        int64_t st = T == 1 ? t.stride(0) : t.stride(1);   // one token per row: the rows are the tokens
        if (T > 1 && B > 1 && t.stride(0) != T * st) st = 0;
        if (t.stride(3) != 1 || (H > 1 && t.stride(2) != d) || st < step || st * t.element_size() % 16 != 0 || B * T < 2)
            x = t.contiguous();
        else
            step = st;
    }
    if (!aligned(x)) {
        x = x.clone(at::MemoryFormat::Contiguous);
        step = H * d;
    }
    return {x, step};
}

Tensor out_like(const Tensor &like) { return at::empty(like.sizes(), like.options()); }

Tensor take_out(const OptTensor &out, const Tensor &like) {
    if (!out) return out_like(like);
    if (out->sizes() != like.sizes() || out->scalar_type() != like.scalar_type() || out->device() != like.device() ||
        !out->is_contiguous() || !aligned(*out))
        bad_value("out must be a contiguous ", like.scalar_type(), " tensor of shape ", like.sizes(), " on ", like.device());
    return *out;
}

void *ptr(const Tensor &t) { return t.data_ptr(); }
void *ptr(const OptTensor &t) { return t ? t->data_ptr() : nullptr; }
const int32_t *int_ptr(const OptTensor &t) { return t ? t->data_ptr<int32_t>() : nullptr; }
float *float_ptr(const OptTensor &t) { return t ? t->data_ptr<float>() : nullptr; }

// The device of a call, current while it lives, and its current stream.
struct On {
    c10::cuda::CUDAGuard guard;
    void *stream;
    explicit On(const Tensor &t)
        : guard(t.device()), stream(c10::cuda::getCurrentCUDAStream(t.device().index()).stream()) {}
};

float scale_of(const std::optional<double> &scale, int64_t d) {
    return scale ? static_cast<float>(*scale) : static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
}

int32_t i32(int64_t x) {
    if (x > 0x7fffffff) bad_value("a size of ", x, " is beyond 32 bits");
    return static_cast<int32_t>(x);
}

// ---- prompts ------------------------------------------------------------------------------------

struct Prompt {
    Tensor q, k, v;
    OptTensor cu, cu_k;
    int64_t qs, ks, vs;
    int32_t n, B, Tq, Tk, Hq, Hkv, d, causal;
    float scale;
    kda_dtype dtype;
};

Prompt prompt_args(const Tensor &q, const Tensor &k, const Tensor &v, const OptTensor &cu, const OptTensor &cu_k,
                   bool causal, const std::optional<double> &scale) {
    if (q.dim() != 4 || k.dim() != 4 || k.sizes() != v.sizes())
        bad_value("q must be [B, Tq, Hq, d] and k, v [B, Tk, Hkv, d]");
    Prompt p;
    p.B = i32(q.size(0)), p.Tq = i32(q.size(1)), p.Hq = i32(q.size(2)), p.d = i32(q.size(3));
    p.Tk = i32(k.size(1)), p.Hkv = i32(k.size(2));
    if (k.size(0) != p.B || k.size(3) != p.d) bad_value("k and v must be [B, Tk, Hkv, d] with q's B and d");
    if (p.Hkv == 0 || p.Hq % p.Hkv != 0)
        bad_value("the ", p.Hq, " query heads must be a multiple of the ", p.Hkv, " heads of k and v");
    if (!cu && cu_k) bad_value("cu_seqlens_k needs cu_seqlens");
    if (cu && !cu_k && p.Tk != p.Tq) bad_value("packed k and v of another length than q need cu_seqlens_k");
    p.n = 0;
    if (cu) {
        p.cu = ints(*cu, "cu_seqlens", -1, q);
        p.n = i32(p.cu->size(0) - 1);
        if (cu_k) p.cu_k = ints(*cu_k, "cu_seqlens_k", p.n + 1, q);
        if (p.B != 1 || p.n < 1) bad_value("cu_seqlens requires B == 1 and at least two offsets");
    }
    same(q, k);
    same(q, v);
    p.dtype = code_of(q);
    on_gpu(q);
    std::tie(p.q, p.qs) = tokens(q);
    std::tie(p.k, p.ks) = tokens(k);
    std::tie(p.v, p.vs) = tokens(v);
    p.causal = causal;
    p.scale = scale_of(scale, p.d);
    return p;
}

// (out, lse, rest); the rest only with the lse, and for bf16 alone
std::tuple<Tensor, Tensor, Tensor> fwd(const Tensor &q, const Tensor &k, const Tensor &v, const OptTensor &cu,
                                       const OptTensor &cu_k, bool causal, const std::optional<double> &scale,
                                       const OptTensor &out, bool want_lse, bool want_rest) {
    const Prompt p = prompt_args(q, k, v, cu, cu_k, causal, scale);
    Tensor o = take_out(out, q), lse, rest;
    if (want_rest && p.dtype == KDA_BF16) rest = out_like(q);
    if (want_lse) lse = at::empty({p.B, p.Hq, p.Tq}, q.options().dtype(at::kFloat));
    const On on(q);
    check(kda_attn_fwd(ptr(p.q), ptr(p.k), ptr(p.v), p.qs, p.ks, p.vs, int_ptr(p.cu), int_ptr(p.cu_k), p.n, p.B, p.Tq,
                       p.Tk, p.Hq, p.Hkv, p.d, p.causal, p.scale, p.dtype, ptr(o), rest.defined() ? ptr(rest) : nullptr,
                       want_lse ? lse.data_ptr<float>() : nullptr, on.stream),
          "kda_attn_fwd");
    return {o, lse, rest};
}

std::tuple<Tensor, Tensor, Tensor> bwd(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &out,
                                       const Tensor &lse, const Tensor &d_out, const OptTensor &cu, const OptTensor &cu_k,
                                       bool causal, const std::optional<double> &scale, const OptTensor &rest) {
    const Prompt p = prompt_args(q, k, v, cu, cu_k, causal, scale);
    if (rest && rest->sizes() != q.sizes()) bad_value("out_rest must have q's shape");
    if (rest) same(q, *rest);
    if (rest && p.dtype != KDA_BF16) bad_type("out_rest goes with bf16 alone");
    if (out.sizes() != q.sizes() || d_out.sizes() != q.sizes() || lse.dim() != 3 || lse.size(0) != p.B ||
        lse.size(1) != p.Hq || lse.size(2) != p.Tq)
        bad_value("out and d_out must have q's shape, and lse [B, Hq, Tq]");
    if (lse.scalar_type() != at::kFloat) bad_type("lse must be float32");
    if (lse.device() != q.device()) bad_value("lse must be on the device of the other tensors");
    same(q, out);
    same(q, d_out);
    const Tensor o = tokens(out.contiguous()).first, l = lse.contiguous(), g = tokens(d_out.contiguous()).first;
    OptTensor re;
    if (rest) re = tokens(rest->contiguous()).first;
    Tensor dq = out_like(q), dk = out_like(k), dv = out_like(k);
    const On on(q);
    size_t bytes = 0;
    check(kda_attn_bwd_workspace_size(p.B, p.Tq, p.Hq, &bytes), "kda_attn_bwd_workspace_size");
    Tensor ws = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
    check(kda_attn_bwd(ptr(p.q), ptr(p.k), ptr(p.v), p.qs, p.ks, p.vs, int_ptr(p.cu), int_ptr(p.cu_k), p.n, p.B, p.Tq,
                       p.Tk, p.Hq, p.Hkv, p.d, p.causal, p.scale, p.dtype, ptr(o), ptr(re), l.data_ptr<float>(), ptr(g), ptr(dq),
                       ptr(dk), ptr(dv), ptr(ws), bytes, on.stream),
          "kda_attn_bwd");
    return {dq, dk, dv};
}

// A leaf's gradient is added on the stream on which the first graph that uses the leaf was built, for as long
// as that graph lives.  While it lives elsewhere, a captured backward pass would have to wait for a stream
// that is not part of the capture: the process ends in that wait, so the call is refused before.
void check_capture(const Tensor &t) {
    if (!t.requires_grad() || !t.is_leaf()) return;
    const auto sum = torch::autograd::impl::try_get_grad_accumulator(t);
    if (!sum) return;
    const c10::cuda::CUDAGuard guard(t.device());
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return;
    TORCH_CHECK(sum->input_metadata(0).stream() == c10::cuda::getCurrentCUDAStream(t.device().index()).unwrap(),
                "kda_attn under capture: an autograd graph of the same leaves lives on another stream; free it first, "
                "or capture kda_attn_fwd and kda_attn_bwd");
}

// A tangent of forward-mode differentiation would be dropped where no input asks for a gradient.
void check_no_tangent(const Tensor &t) {
    TORCH_CHECK_NOT_IMPLEMENTED(!t._fw_grad(0).defined(), "kda_attn has no forward-mode derivative: an input carries a tangent");
}

// kda_attn_fwd with kda_attn_bwd as its gradient.
struct Attention : torch::autograd::Function<Attention> {
    static Tensor forward(torch::autograd::AutogradContext *ctx, const Tensor &q, const Tensor &k, const Tensor &v,
                          const OptTensor &cu, const OptTensor &cu_k, bool causal, const std::optional<double> &scale) {
        auto [out, lse, rest] = fwd(q, k, v, cu, cu_k, causal, scale, std::nullopt, true, true);
        ctx->save_for_backward({q, k, v, out, lse, cu.value_or(Tensor()), cu_k.value_or(Tensor()), rest});
        ctx->saved_data["causal"] = causal;
        ctx->saved_data["scale"] = scale ? c10::IValue(*scale) : c10::IValue();
        return out;
    }
    static torch::autograd::variable_list backward(torch::autograd::AutogradContext *ctx,
                                                   torch::autograd::variable_list grads) {
        TORCH_CHECK(!at::GradMode::is_enabled(),
                    "kda_attn is differentiable once: its gradient has none (create_graph=True)");
        const auto s = ctx->get_saved_variables();
        const auto opt = [](const Tensor &t) { return t.defined() ? OptTensor(t) : OptTensor(); };
        const auto scale = ctx->saved_data["scale"];
        Tensor dq, dk, dv;
        if (grads[0].defined())
            std::tie(dq, dk, dv) =
                bwd(s[0], s[1], s[2], s[3], s[4], grads[0], opt(s[5]), opt(s[6]), ctx->saved_data["causal"].toBool(),
                    scale.isNone() ? std::optional<double>() : std::optional<double>(scale.toDouble()), opt(s[7]));
        return {dq, dk, dv, Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

// ---- the paged cache ----------------------------------------------------------------------------

struct Paged {
    int64_t k_step, v_step, row;   // elements between pages, entries between rows of the table
    int32_t pages, heads, size, d, width;
    Tensor table;
};

int64_t page_step(const Tensor &c) {
    const int64_t dense = c.size(1) * c.size(2) * c.size(3);
    if (c.is_contiguous()) return dense;
    // the cache is used in place: no copy can stand in for it
    if (c.stride(3) != 1 || (c.size(2) > 1 && c.stride(2) != c.size(3)) ||
        (c.size(1) > 1 && c.stride(1) != c.size(2) * c.size(3)))
        bad_value("a page of the cache must be dense; pages may lie apart");
    if (c.size(0) < 2) return dense;
    if (c.stride(0) < dense)   // 0 among them, which the library would take for dense
        bad_value("the pages of a cache must not overlap: they lie ", c.stride(0), " elements apart and hold ", dense);
    return c.stride(0);
}

Paged cache_args(const Tensor &k_cache, const Tensor &v_cache, const Tensor &table, int64_t n) {
    if (k_cache.dim() != 4 || v_cache.sizes() != k_cache.sizes())
        bad_value("k_cache and v_cache must be [num_pages, Hkv, page_size, d]");
    Paged c;
    c.pages = i32(k_cache.size(0)), c.heads = i32(k_cache.size(1)), c.size = i32(k_cache.size(2)), c.d = i32(k_cache.size(3));
    c.k_step = page_step(k_cache);
    c.v_step = page_step(v_cache);
    if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != n)
        bad_value("page_table must be an int32 tensor [", n, ", pages of a sequence]");
    if (table.device() != k_cache.device()) bad_value("page_table must be on the device of the cache");
    c.width = i32(table.size(1));
    c.table = table;
    if (!table.is_contiguous() && ((c.width > 1 && table.stride(1) != 1) || (n > 1 && table.stride(0) < c.width)))
        c.table = table.contiguous();
    c.row = n > 1 ? c.table.stride(0) : c.width;
    return c;
}

std::pair<OptTensor, OptTensor> kv_append(const Tensor &k, const Tensor &v, const Tensor &k_cache, const Tensor &v_cache,
                                          const Tensor &page_table, const Tensor &cache_lens, const OptTensor &inv_freq,
                                          const OptTensor &q, const OptTensor &cu_seqlens, bool interleaved, bool return_k,
                                          const OptTensor &q_out) {
    if (at::GradMode::is_enabled() && (k.requires_grad() || v.requires_grad() || (q && q->requires_grad())) &&
        PyErr_WarnEx(PyExc_UserWarning,
                     "kda_kv_append has no gradient: its results do not lead back to inputs that require one "
                     "(call it under torch.no_grad() where that is meant)", 1) != 0)
        throw py::error_already_set();   // where warnings are errors
    if (k.dim() != 4 || v.sizes() != k.sizes()) bad_value("k and v must be [B, T, Hkv, d]");
    const int32_t B = i32(k.size(0)), T = i32(k.size(1)), Hkv = i32(k.size(2)), d = i32(k.size(3));
    const int64_t n = cu_seqlens ? cu_seqlens->numel() - 1 : B;
    if (cu_seqlens && (B != 1 || n < 1)) bad_value("cu_seqlens requires B == 1 and at least two offsets");
    const Paged c = cache_args(k_cache, v_cache, page_table, n);
    if (c.heads != Hkv || c.d != d)
        bad_value("the cache holds ", c.heads, " heads of ", c.d, " channels, k and v ", Hkv, " of ", d);
    same(k, v);
    same(k, k_cache);
    same(k, v_cache);
    const kda_dtype dtype = code_of(k);
    on_gpu(k);
    const Tensor lens = ints(cache_lens, "cache_lens", n, k);
    OptTensor cu;
    if (cu_seqlens) cu = ints(*cu_seqlens, "cu_seqlens", -1, k);
    OptTensor freq;
    int32_t rotary = 0;
    if (inv_freq) {
        if (inv_freq->scalar_type() != at::kFloat || inv_freq->dim() != 1)
            bad_type("inv_freq must be a one-dimensional float32 tensor");
        if (inv_freq->device() != k.device()) bad_value("inv_freq must be on the device of the other tensors");
        freq = inv_freq->contiguous();
        rotary = i32(2 * freq->size(0));
    }
    const auto [kt, ks] = tokens(k);
    const auto [vt, vs] = tokens(v);
    OptTensor qt, qo, ko;
    int64_t qs = 0;
    int32_t Hq = 0;
    if (q) {
        if (q->dim() != 4 || q->size(0) != B || q->size(1) != T || q->size(3) != d || Hkv == 0 || q->size(2) % Hkv != 0)
            bad_value("q must be [B, T, Hq, d] with Hq a multiple of Hkv");
        same(k, *q);
        Hq = i32(q->size(2));
        qo = take_out(q_out, *q);
        std::tie(qt, qs) = tokens(*q);
    } else if (q_out) {
        bad_value("q_out needs q");
    }
    if (return_k) ko = out_like(k);
    const On on(k);
    check(kda_kv_append(ptr(qt), ptr(kt), ptr(vt), qs, ks, vs, float_ptr(freq), rotary, interleaved, int_ptr(cu), i32(n), B,
                        T, Hq, Hkv, d, dtype, lens.data_ptr<int32_t>(), c.table.data_ptr<int32_t>(), c.row, c.width,
                        ptr(k_cache), ptr(v_cache), c.k_step, c.v_step, c.pages, c.size, ptr(qo), ptr(ko), on.stream),
          "kda_kv_append");
    return {qo, ko};
}

std::pair<Tensor, Tensor> decode_step(const Tensor &q, const Tensor &k_cache, const Tensor &v_cache,
                                      const Tensor &page_table, const Tensor &seq_lens,
                                      const std::optional<double> &scale, const OptTensor &out, bool want_lse) {
    if (q.dim() != 3) bad_value("q must be [B, Hq, d]");
    const int32_t B = i32(q.size(0)), Hq = i32(q.size(1)), d = i32(q.size(2));
    const Paged c = cache_args(k_cache, v_cache, page_table, B);
    if (c.d != d || c.heads == 0 || Hq % c.heads != 0)
        bad_value("q of ", Hq, " heads of ", d, " channels does not go with a cache of ", c.heads, " of ", c.d);
    const Tensor lens = ints(seq_lens, "seq_lens", B, q);
    same(q, k_cache);
    same(q, v_cache);
    const kda_dtype dtype = code_of(q);
    on_gpu(q);
    Tensor qt = q;
    int64_t qs = static_cast<int64_t>(Hq) * d;
    if (!q.is_contiguous() || !aligned(q)) std::tie(qt, qs) = tokens(q.unsqueeze(1));
    Tensor o = take_out(out, q), lse, ws;
    if (want_lse) lse = at::empty({B, Hq}, q.options().dtype(at::kFloat));
    const On on(q);
    size_t bytes = 0;
    check(kda_attn_decode_workspace_size(B, Hq, c.heads, d, std::max<int64_t>(1, int64_t(c.width) * c.size), dtype, &bytes),
          "kda_attn_decode_workspace_size");
    if (bytes) ws = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
    check(kda_attn_decode_step(ptr(qt), qs, ptr(k_cache), ptr(v_cache), c.k_step, c.v_step, c.pages, c.size,
                               c.table.data_ptr<int32_t>(), c.row, c.width, lens.data_ptr<int32_t>(), B, Hq, c.heads, d,
                               scale_of(scale, d), dtype, ptr(o), want_lse ? lse.data_ptr<float>() : nullptr,
                               bytes ? ptr(ws) : nullptr, bytes, on.stream),
          "kda_attn_decode_step");
    return {o, lse};
}

}  // namespace

PYBIND11_MODULE(_attention, m) {
    m.doc() = "Native binding of the softmax-attention calls; see gated_delta_rule_86_b200.attention.";
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const StatusError &e) {
            const py::object type = py::module_::import("gated_delta_rule_86_b200._lib").attr("KdaError");
            const py::object error = type(e.status, e.call);
            PyErr_SetObject(type.ptr(), error.ptr());
        }
    });
    m.def("fwd", [](const Tensor &q, const Tensor &k, const Tensor &v, const OptTensor &cu, const OptTensor &cu_k, bool causal,
                    std::optional<double> scale, const OptTensor &out, bool return_lse, bool return_rest) -> py::object {
        auto [o, lse, rest] = fwd(q, k, v, cu, cu_k, causal, scale, out, return_lse, return_rest);
        if (!return_lse && !return_rest) return py::cast(o);
        py::list all;
        all.append(o);
        if (return_lse) all.append(lse);
        if (return_rest) all.append(rest.defined() ? py::cast(rest) : py::none());
        return py::tuple(all);
    });
    m.def("bwd", &bwd);
    m.def("attn", [](const Tensor &q, const Tensor &k, const Tensor &v, const OptTensor &cu, const OptTensor &cu_k, bool causal,
                     std::optional<double> scale) {
        for (const Tensor *t : {&q, &k, &v}) check_no_tangent(*t);
        const bool graph = at::GradMode::is_enabled() && (q.requires_grad() || k.requires_grad() || v.requires_grad());
        if (!graph) return std::get<0>(fwd(q, k, v, cu, cu_k, causal, scale, std::nullopt, false, false));
        for (const Tensor *t : {&q, &k, &v}) check_capture(*t);
        return Attention::apply(q, k, v, cu, cu_k, causal, scale);
    });
    m.def("kv_append", &kv_append);
    m.def("decode_step", [](const Tensor &q, const Tensor &kc, const Tensor &vc, const Tensor &table, const Tensor &lens,
                            std::optional<double> scale, const OptTensor &out, bool return_lse) -> py::object {
        auto [o, lse] = decode_step(q, kc, vc, table, lens, scale, out, return_lse);
        if (return_lse) return py::make_tuple(o, lse);
        return py::cast(o);
    });
    m.def("tokens", &tokens);
    m.attr("built_for") = KDA_BUILT_FOR;   // read from the file by the build
}
