// binding.cpp -- native Python binding of the cache and cross-attention entry points
// (include/ra.h): checks of shapes, types and layouts, allocation of outputs and workspace
// on the current stream, one library call; and cross attention's autograd node.
//
// A decode step calls these once per token and layer, where the time that a call takes on
// the host is the time that it takes: through ctypes an append took 16 us and a training
// step's forward and backward 130 us (90 of them for handing a Python backward to
// autograd's thread), against 3 and 26 us on the GPU.  The computation is the library's;
// nothing here launches a kernel of torch's, but for a copy where an incoming gradient is
// not dense and the zeros of a backward without queries.  A call without a single token or query
// returns empty results; the C ABI takes sizes from one up.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/utils/pybind.h>

#include <string>
#include <tuple>

#include "../../include/ra.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

struct RaStatus : std::runtime_error {
    int status;
    RaStatus(int s, const std::string& message) : std::runtime_error(message), status(s) {}
};

void check(ra_status s) {
    if (s != RA_OK)
        throw RaStatus(s, "ra status " + std::to_string((int)s) + ": " + ra_last_error());
}

[[noreturn]] void refuse(const std::string& message) { throw py::value_error(message); }

std::string str(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}

// Token rows [..., H, D] whose heads are dense.
void check_rows(const Tensor& t, const char* name, at::Device device) {
    if (t.scalar_type() != at::kBFloat16 || t.device() != device)
        refuse(std::string(name) + " must be a bf16 tensor on " + device.str());
    const int64_t n = t.dim();
    if (n < 2 || t.stride(n - 1) != 1 || (t.size(n - 2) > 1 && t.stride(n - 2) != t.size(n - 1)))
        refuse(std::string(name) + ": the heads of a token must be dense");
}

const int* ints(const Tensor& t, const char* name, at::Device device, at::IntArrayRef shape) {
    if (t.scalar_type() != at::kInt || t.device() != device || !t.is_contiguous())
        refuse(std::string(name) + " must be a contiguous int32 tensor on " + device.str());
    if (t.sizes() != shape)
        refuse(std::string(name) + " must have shape " + str(shape) + ", not " + str(t.sizes()));
    return t.const_data_ptr<int>();
}

void check_dense(const Tensor& t, const char* name, at::Device device, at::IntArrayRef shape,
                 at::ScalarType type) {
    if (t.scalar_type() != type || t.device() != device || !t.is_contiguous() ||
        t.sizes() != shape)
        refuse(std::string(name) + " must be a contiguous " + at::toString(type) +
               " tensor of shape " + str(shape) + " on " + device.str());
}

void check_cuda(const Tensor& t) {
    if (!t.is_cuda()) refuse("the tensors must be on a CUDA device");
}

int narrow(int64_t v, const char* name) {
    if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
    return (int)v;
}

ra_dtype dtype_of(at::ScalarType t) {
    if (t == at::kBFloat16) return RA_BF16;
    if (t == at::kFloat) return RA_FP32;
    refuse("unsupported dtype " + std::string(at::toString(t)));
}

void* stream_of(const Tensor& t) {
    return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
}

// Elements between tokens; the dense value where there is one at most.
int64_t token_stride(const Tensor& t, int64_t dim) {
    return t.size(dim) > 1 ? t.stride(dim) : t.size(dim + 1) * t.size(dim + 2);
}

struct Cache {
    int n_pages, page_size, H_kv, D;
    int64_t stride;
};

Cache check_cache(const Tensor& k, const Tensor& v, at::Device device) {
    if (k.dim() != 4 || k.sizes() != v.sizes())
        refuse("k_pages and v_pages must both be [n_pages, page_size, H_kv, D]");
    check_rows(k, "k_pages", device);
    check_rows(v, "v_pages", device);
    const int64_t n = k.size(0), ps = k.size(1), row = k.size(2) * k.size(3);
    if (ps > 1 && (k.stride(1) != row || v.stride(1) != row))
        refuse("the rows of a page must be dense");
    if (n > 1 && k.stride(0) != v.stride(0))
        refuse("k_pages and v_pages must have the same page stride");
    return {narrow(n, "n_pages"), narrow(ps, "page_size"), narrow(k.size(2), "H_kv"),
            narrow(k.size(3), "D"), n > 1 ? k.stride(0) : ps * row};
}

struct Batch {
    int B, max_pages;
    const int *cu, *lens, *tables;
};

Batch check_batch(const Tensor& cu, const Tensor& lens, const Tensor& tables, at::Device device) {
    if (tables.dim() != 2) refuse("block_tables must be [B, max_pages]");
    const int64_t B = tables.size(0);
    return {narrow(B, "B"), narrow(tables.size(1), "max_pages"),
            ints(cu, "cu_tokens", device, {B + 1}), ints(lens, "seq_lens", device, {B}),
            ints(tables, "block_tables", device, {B, tables.size(1)})};
}

// The caller's workspace, or a new one, on the current stream.
Tensor workspace_of(const OptTensor& given, int64_t need, const Tensor& like) {
    if (given) {
        if (given->device() != like.device() || !given->is_contiguous())
            refuse("workspace must be a contiguous tensor on " + like.device().str());
        return *given;
    }
    return need > 0 ? at::empty({need}, like.options().dtype(at::kByte)) : Tensor();
}
void* ptr(const Tensor& t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }
int64_t bytes(const Tensor& t) { return t.defined() ? (int64_t)t.nbytes() : 0; }

Tensor result_of(const OptTensor& given, const char* name, at::IntArrayRef shape,
                 at::ScalarType type, const Tensor& like) {
    if (!given) return at::empty(shape, like.options().dtype(type));
    check_dense(*given, name, like.device(), shape, given->scalar_type());
    return *given;
}

// ------------------------------------------------------------------ append
std::optional<Tensor> paged_kv_append(const OptTensor& q, const Tensor& k, const Tensor& v,
                                      const Tensor& k_pages, const Tensor& v_pages,
                                      const Tensor& cu_tokens, const Tensor& seq_lens,
                                      const Tensor& block_tables, const OptTensor& inv_freq,
                                      int64_t max_tokens, int64_t pos_offset, bool interleaved,
                                      const OptTensor& q_out) {
    check_cuda(k);
    const at::Device dev = k.device();
    const c10::cuda::CUDAGuard guard(dev);
    const Cache c = check_cache(k_pages, v_pages, dev);
    if (k.dim() != 3 || k.size(1) != c.H_kv || k.size(2) != c.D || v.sizes() != k.sizes())
        refuse("k and v must be [N, H_kv, D] with the cache's heads");
    check_rows(k, "k", dev);
    check_rows(v, "v", dev);
    const int64_t N = k.size(0);
    const Batch b = check_batch(cu_tokens, seq_lens, block_tables, dev);
    int rot = 0;
    const float* inv = nullptr;
    if (inv_freq) {
        check_dense(*inv_freq, "inv_freq", dev, {inv_freq->numel()}, at::kFloat);
        rot = narrow(2 * inv_freq->numel(), "rot_dim");
        inv = inv_freq->const_data_ptr<float>();
    }
    int H_q = 0;
    std::optional<Tensor> out;
    if (q) {
        if (q->dim() != 3 || q->size(0) != N || q->size(2) != c.D) refuse("q must be [N, H_q, D]");
        check_rows(*q, "q", dev);
        H_q = narrow(q->size(1), "H_q");
        if (q_out) {
            if (q_out->sizes() != q->sizes()) refuse("q_out must have q's shape");
            check_rows(*q_out, "q_out", dev);
            out = *q_out;
        } else {
            out = at::empty(q->sizes(), q->options());
        }
    }
    if (N == 0) return out;  // a step without tokens
    check(ra_paged_kv_append(
        q ? q->const_data_ptr() : nullptr, k.const_data_ptr(), v.const_data_ptr(),
        q ? token_stride(*q, 0) : 0, token_stride(k, 0), token_stride(v, 0), b.cu, b.lens,
        b.tables, inv, b.B, narrow(N, "N"), narrow(std::min(max_tokens, N), "max_tokens"), H_q,
        c.H_kv, c.D, rot, interleaved, narrow(pos_offset, "pos_offset"), c.page_size, c.n_pages,
        b.max_pages, c.stride, RA_BF16, out ? out->mutable_data_ptr() : nullptr,
        out ? token_stride(*out, 0) : 0, k_pages.mutable_data_ptr(), v_pages.mutable_data_ptr(),
        stream_of(k)));
    return out;
}

// ------------------------------------------------------------------ prefix attention
std::tuple<Tensor, Tensor> prefix_attn_fwd(
    const Tensor& q, const Tensor& k_pages, const Tensor& v_pages, const Tensor& cu_tokens,
    const Tensor& seq_lens, const Tensor& block_tables, int64_t max_tokens,
    std::optional<int64_t> max_len, const OptTensor& prefix_table, int64_t prefix_len,
    std::optional<double> scale, at::ScalarType out_dtype, const OptTensor& out,
    const OptTensor& lse, const OptTensor& workspace) {
    check_cuda(q);
    const at::Device dev = q.device();
    const c10::cuda::CUDAGuard guard(dev);
    const Cache c = check_cache(k_pages, v_pages, dev);
    if (q.dim() != 3 || q.size(2) != c.D)
        refuse("q must be [N, H_q, D] with the cache's head dimension");
    check_rows(q, "q", dev);
    const int64_t N = q.size(0);
    const int H_q = narrow(q.size(1), "H_q"), plen = narrow(prefix_len, "prefix_len");
    const Batch b = check_batch(cu_tokens, seq_lens, block_tables, dev);
    const int* table = nullptr;
    if (plen > 0) {
        if (!prefix_table || prefix_table->numel() * c.page_size < plen)
            refuse("prefix_table must name ceil(prefix_len / page_size) pages");
        table = ints(*prefix_table, "prefix_table", dev, {prefix_table->numel()});
    }
    const int ml = narrow(max_len ? *max_len : (int64_t)b.max_pages * c.page_size, "max_len");
    const int mt = narrow(std::min(max_tokens, N), "max_tokens"), n = narrow(N, "N");
    const Tensor o = result_of(out, "out", q.sizes(), out_dtype, q);
    const Tensor l = result_of(lse, "lse", {H_q, N}, at::kFloat, q);
    if (N == 0) return {o, l};  // a step without tokens
    const Tensor ws = workspace_of(
        workspace,
        ra_prefix_attn_workspace(b.B, n, mt, ml, plen, H_q, c.H_kv, c.D, c.page_size), q);
    check(ra_prefix_attn_fwd(q.const_data_ptr(), token_stride(q, 0), k_pages.const_data_ptr(),
                             v_pages.const_data_ptr(), b.cu, b.lens, b.tables, table, plen, b.B,
                             n, mt, ml, H_q, c.H_kv, c.D, c.page_size, c.n_pages, b.max_pages,
                             c.stride, scale ? (float)*scale : (float)(1.0 / std::sqrt((double)c.D)),
                             RA_BF16, dtype_of(o.scalar_type()), o.mutable_data_ptr(),
                             l.mutable_data_ptr<float>(), ptr(ws), bytes(ws), stream_of(q)));
    return {o, l};
}

// ------------------------------------------------------------------ cross attention
struct Cross {
    int B, Lq, Lk, H_q, H_kv, D;
    int64_t qt, qb, kt, kb;
    const int* lens;
    float scale;
};

Cross check_cross(const Tensor& q, const Tensor& k, const Tensor& v, const OptTensor& kv_lens,
                  std::optional<double> scale) {
    const at::Device dev = q.device();
    if (q.dim() != 4 || k.dim() != 4 || k.sizes() != v.sizes())
        refuse("q must be [B, Lq, H_q, D], k and v [B, Lk, H_kv, D]");
    check_rows(q, "q", dev);
    check_rows(k, "k", dev);
    check_rows(v, "v", dev);
    const int64_t B = q.size(0), Lk = k.size(1);
    if (k.size(0) != B || k.size(3) != q.size(3))
        refuse("q, k and v must have the same batch and head dimension");
    Cross c;
    c.B = narrow(B, "B");
    c.Lq = narrow(q.size(1), "Lq");
    c.Lk = narrow(Lk, "Lk");
    c.H_q = narrow(q.size(2), "H_q");
    c.H_kv = narrow(k.size(2), "H_kv");
    c.D = narrow(q.size(3), "D");
    c.qt = token_stride(q, 1);
    c.kt = token_stride(k, 1);
    c.qb = B > 1 ? q.stride(0) : c.Lq * c.qt;
    c.kb = B > 1 ? k.stride(0) : Lk * c.kt;
    if ((Lk > 1 && v.stride(1) != c.kt) || (B > 1 && v.stride(0) != c.kb))
        refuse("k and v must have the same strides");
    c.lens = kv_lens ? ints(*kv_lens, "kv_lens", dev, {B}) : nullptr;
    c.scale = scale ? (float)*scale : (float)(1.0 / std::sqrt((double)c.D));
    return c;
}

std::tuple<Tensor, Tensor> cross_attn_fwd(const Tensor& q, const Tensor& k, const Tensor& v,
                                          const OptTensor& kv_lens, std::optional<double> scale,
                                          at::ScalarType out_dtype, const OptTensor& out,
                                          const OptTensor& lse, const OptTensor& workspace) {
    check_cuda(q);
    const c10::cuda::CUDAGuard guard(q.device());
    const Cross c = check_cross(q, k, v, kv_lens, scale);
    const Tensor o = result_of(out, "out", q.sizes(), out_dtype, q);
    const Tensor l = result_of(lse, "lse", {c.B, c.H_q, c.Lq}, at::kFloat, q);
    if (q.numel() == 0) return {o, l};
    const Tensor ws = workspace_of(
        workspace, ra_cross_attn_workspace(c.B, c.Lq, c.Lk, c.H_q, c.H_kv, c.D), q);
    check(ra_cross_attn_fwd(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), c.lens,
                            c.B, c.Lq, c.Lk, c.H_q, c.H_kv, c.D, c.qt, c.qb, c.kt, c.kb, c.scale,
                            RA_BF16, dtype_of(o.scalar_type()), o.mutable_data_ptr(),
                            l.mutable_data_ptr<float>(), ptr(ws), bytes(ws), stream_of(q)));
    return {o, l};
}

std::tuple<Tensor, Tensor, Tensor> cross_attn_bwd(const Tensor& q, const Tensor& k,
                                                  const Tensor& v, const Tensor& out,
                                                  const Tensor& lse, const Tensor& dout,
                                                  const OptTensor& kv_lens,
                                                  std::optional<double> scale,
                                                  at::ScalarType grad_dtype,
                                                  const OptTensor& workspace) {
    check_cuda(q);
    const at::Device dev = q.device();
    const c10::cuda::CUDAGuard guard(dev);
    const Cross c = check_cross(q, k, v, kv_lens, scale);
    check_dense(out, "out", dev, q.sizes(), at::kBFloat16);
    check_dense(dout, "dout", dev, q.sizes(), at::kBFloat16);
    check_dense(lse, "lse", dev, {c.B, c.H_q, c.Lq}, at::kFloat);
    const ra_dtype gd = dtype_of(grad_dtype);
    const auto opt = q.options().dtype(grad_dtype);
    if (q.numel() == 0)
        return {at::empty(q.sizes(), opt), at::zeros(k.sizes(), opt), at::zeros(k.sizes(), opt)};
    const Tensor dq = at::empty(q.sizes(), opt), dk = at::empty(k.sizes(), opt),
                 dv = at::empty(k.sizes(), opt);
    const Tensor ws =
        workspace_of(workspace, ra_cross_attn_bwd_workspace(c.B, c.Lq, c.H_q, c.D, gd), q);
    check(ra_cross_attn_bwd(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), c.lens,
                            out.const_data_ptr(), lse.const_data_ptr<float>(),
                            dout.const_data_ptr(), c.B, c.Lq, c.Lk, c.H_q, c.H_kv, c.D, c.qt,
                            c.qb, c.kt, c.kb, c.scale, RA_BF16, gd, dq.mutable_data_ptr(),
                            dk.mutable_data_ptr(), dv.mutable_data_ptr(), ptr(ws), bytes(ws),
                            stream_of(q)));
    return {dq, dk, dv};
}

// Gradients that a graph of their own is asked for (create_graph): a second derivative is
// refused when it is taken; without this node it would silently lack this operator's part.
// q, k and v are arguments so that the node lies on the way to them.
struct OnceDifferentiable : torch::autograd::Function<OnceDifferentiable> {
    static torch::autograd::variable_list forward(torch::autograd::AutogradContext*,
                                                  const Tensor& dq, const Tensor& dk,
                                                  const Tensor& dv, const Tensor&,
                                                  const Tensor&, const Tensor&) {
        return {dq.detach(), dk.detach(), dv.detach()};
    }
    static torch::autograd::variable_list backward(torch::autograd::AutogradContext*,
                                                   torch::autograd::variable_list) {
        refuse("cross_attention can be differentiated once");
    }
};

// The forward keeps q, k, v, O (bf16), the LSE and the key counts; gradients come in bf16,
// summed in fp32 and rounded once.
struct CrossAttention : torch::autograd::Function<CrossAttention> {
    static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& q, const Tensor& k,
                          const Tensor& v, const OptTensor& kv_lens, double scale) {
        auto [o, lse] = cross_attn_fwd(q, k, v, kv_lens, scale, at::kBFloat16, {}, {}, {});
        ctx->save_for_backward({q, k, v, o, lse, kv_lens ? *kv_lens : Tensor()});
        ctx->saved_data["scale"] = scale;
        return o;
    }
    static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                   torch::autograd::variable_list grads) {
        const auto s = ctx->get_saved_variables();
        const OptTensor lens = s[5].defined() ? OptTensor(s[5]) : OptTensor();
        auto [dq, dk, dv] =
            cross_attn_bwd(s[0], s[1], s[2], s[3], s[4], grads[0].contiguous(), lens,
                           ctx->saved_data["scale"].toDouble(), at::kBFloat16, {});
        if (at::GradMode::is_enabled()) {
            const auto g = OnceDifferentiable::apply(dq, dk, dv, s[0], s[1], s[2]);
            return {g[0], g[1], g[2], Tensor(), Tensor()};
        }
        return {dq, dk, dv, Tensor(), Tensor()};
    }
};

Tensor cross_attention(const Tensor& q, const Tensor& k, const Tensor& v,
                       const OptTensor& kv_lens, double scale) {
    return CrossAttention::apply(q, k, v, kv_lens, scale);
}

}  // namespace

PYBIND11_MODULE(_ra_torch, m) {
    static py::object error_class;
    m.def("set_error_class", [](py::object cls) { error_class = std::move(cls); });
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const RaStatus& e) {
            const std::string what = e.what();
            const py::object x = error_class(e.status, what.substr(what.find(": ") + 2));
            PyErr_SetObject(error_class.ptr(), x.ptr());
        }
    });
    py::module_::import("atexit").attr("register")(
        py::cpp_function([]() { error_class.release().dec_ref(); }));
    // the calls keep the GIL: they take a few microseconds and wait for nothing
    m.def("paged_kv_append", &paged_kv_append);
    m.def("prefix_attn_fwd", &prefix_attn_fwd);
    m.def("cross_attn_fwd", &cross_attn_fwd);
    m.def("cross_attn_bwd", &cross_attn_bwd);
    m.def("cross_attention", &cross_attention);
    // the checks alone, for tests without a GPU
    m.def("check_cache", [](const Tensor& k, const Tensor& v) {
        const Cache c = check_cache(k, v, k.device());
        return std::make_tuple(c.n_pages, c.page_size, c.H_kv, c.D, c.stride);
    });
    m.def("check_batch", [](const Tensor& cu, const Tensor& lens, const Tensor& tables) {
        const Batch b = check_batch(cu, lens, tables, tables.device());
        return std::make_tuple(b.B, b.max_pages);
    });
    m.def("check_cross", [](const Tensor& q, const Tensor& k, const Tensor& v,
                            const OptTensor& lens) {
        const Cross c = check_cross(q, k, v, lens, {});
        return std::make_tuple(c.B, c.Lq, c.Lk, c.H_q, c.H_kv, c.D, c.qt, c.qb, c.kt, c.kb);
    });
}
