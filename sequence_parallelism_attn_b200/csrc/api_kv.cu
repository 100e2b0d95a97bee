// api_kv.cu -- the entry points over a K/V cache and an encoder's states: argument
// validation and dispatch.  Nothing is launched unless every argument check passes.
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>
#include <string>
#include "kv_internal.h"
#include "../../include/ra.h"

namespace {

ra_status fail(ra_status s, const std::string& msg) { return (ra_status)ra::set_last_error(s, msg); }

ra_status cuda_fail(cudaError_t e, const char* what) {
    return fail(RA_ERR_CUDA, std::string(what) + ": " + cudaGetErrorName(e) + " (" +
                                 cudaGetErrorString(e) + ")");
}

bool aligned(const void* p, unsigned n) {
    return p && (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0;
}

// Tokens and heads of a call fit the 32-bit indices of the kernels.
constexpr long long kMaxTokens = 1ll << 24, kMaxKeys = 1ll << 30, kMaxSequences = 1ll << 28;

ra_status check_heads(int H_q, int H_kv, int D, ra_dtype dtype) {
    if (H_kv < 1 || H_q < 1 || D < 1) return fail(RA_ERR_INVALID, "H_q, H_kv and D must be >= 1");
    if (H_q % H_kv != 0) return fail(RA_ERR_INVALID, "H_q must be a multiple of H_kv");
    if (dtype != RA_BF16 && dtype != RA_FP32) return fail(RA_ERR_INVALID, "bad dtype");
    if (dtype != RA_BF16) return fail(RA_ERR_UNSUPPORTED, "the cache operators take bf16");
    if (D != 64 && D != 128) return fail(RA_ERR_UNSUPPORTED, "D must be 64 or 128");
    return RA_OK;
}

ra_status check_stride(long long stride, long long dense, const char* name) {
    if (stride < dense) return fail(RA_ERR_INVALID, std::string(name) + " below the dense size");
    if (stride % 8 != 0)
        return fail(RA_ERR_INVALID, std::string(name) + " must be a multiple of 8 elements");
    return RA_OK;
}

ra_status check_batch(const int* cu, const int* lens, const int* tables, int B, int n_tokens,
                      int max_tokens) {
    if (B < 1 || n_tokens < 1 || max_tokens < 1)
        return fail(RA_ERR_INVALID, "B, n_tokens and max_tokens must be >= 1");
    if (n_tokens > kMaxTokens || max_tokens > n_tokens || B > kMaxSequences)
        return fail(RA_ERR_INVALID,
                    "n_tokens must be <= 2^24, max_tokens <= n_tokens and B <= 2^28");
    if (!aligned(cu, 4) || !aligned(lens, 4) || !aligned(tables, 4))
        return fail(RA_ERR_INVALID,
                    "cu_tokens, seq_lens and block_tables must be non-null and 4-byte aligned");
    return RA_OK;
}

ra_status check_cache(const void* k, const void* v, int page_size, int n_pages, int max_pages,
                      long long page_stride, int H_kv, int D) {
    if (!aligned(k, 16) || !aligned(v, 16))
        return fail(RA_ERR_INVALID, "k_pages and v_pages must be non-null and 16-byte aligned");
    if (page_size < 1 || n_pages < 1 || max_pages < 1)
        return fail(RA_ERR_INVALID, "page_size, n_pages and max_pages must be >= 1");
    return check_stride(page_stride, (long long)page_size * H_kv * D, "page_stride");
}

ra_status check_results(float scale, ra_dtype out_dtype, const void* out, const float* lse) {
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(RA_ERR_INVALID, "scale must be finite and > 0");
    if (out_dtype != RA_BF16 && out_dtype != RA_FP32) return fail(RA_ERR_INVALID, "bad out_dtype");
    if (!aligned(out, 16) || !aligned(lse, 16))
        return fail(RA_ERR_INVALID, "out and lse must be non-null and 16-byte aligned");
    return RA_OK;
}

ra_status check_workspace(const void* ws, long long bytes, long long need) {
    if (need > 0 && (!aligned(ws, 16) || bytes < need))
        return fail(RA_ERR_INVALID, "workspace must be 16-byte aligned and at least " +
                                        std::to_string(need) + " bytes");
    return RA_OK;
}

#define RA_CHECK(call)                   \
    do {                                 \
        const ra_status st_ = (call);    \
        if (st_ != RA_OK) return st_;    \
    } while (0)

}  // namespace

extern "C" {

ra_status ra_paged_kv_append(const void* q, const void* k, const void* v, long long q_tstride,
                             long long k_tstride, long long v_tstride, const int* cu_tokens,
                             const int* seq_lens, const int* block_tables, const float* inv_freq,
                             int B, int n_tokens, int max_tokens, int H_q, int H_kv, int D,
                             int rot_dim, int interleaved, int pos_offset, int page_size,
                             int n_pages, int max_pages, long long page_stride, ra_dtype dtype,
                             void* q_out, long long q_out_tstride, void* k_pages, void* v_pages,
                             void* stream) {
    if (H_q < 0) return fail(RA_ERR_INVALID, "H_q must be >= 0");
    RA_CHECK(check_heads(H_q > 0 ? H_q : H_kv, H_kv, D, dtype));
    RA_CHECK(check_batch(cu_tokens, seq_lens, block_tables, B, n_tokens, max_tokens));
    RA_CHECK(check_cache(k_pages, v_pages, page_size, n_pages, max_pages, page_stride, H_kv, D));
    if (!aligned(k, 16) || !aligned(v, 16) || (H_q > 0 && (!aligned(q, 16) || !aligned(q_out, 16))))
        return fail(RA_ERR_INVALID, "q, k, v and q_out must be non-null and 16-byte aligned");
    if (H_q > 0) {
        RA_CHECK(check_stride(q_tstride, (long long)H_q * D, "q_tstride"));
        RA_CHECK(check_stride(q_out_tstride, (long long)H_q * D, "q_out_tstride"));
        if (q == q_out && q_tstride != q_out_tstride)
            return fail(RA_ERR_INVALID, "q_out may be q only with the same token stride");
    }
    RA_CHECK(check_stride(k_tstride, (long long)H_kv * D, "k_tstride"));
    RA_CHECK(check_stride(v_tstride, (long long)H_kv * D, "v_tstride"));
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0)
        return fail(RA_ERR_INVALID, "rot_dim must be a multiple of 16 in [0, D]");
    if (rot_dim > 0 && !aligned(inv_freq, 4))
        return fail(RA_ERR_INVALID, "inv_freq must be non-null and 4-byte aligned");
    if (interleaved != 0 && interleaved != 1)
        return fail(RA_ERR_INVALID, "interleaved must be 0 or 1");
    if (pos_offset < 0) return fail(RA_ERR_INVALID, "pos_offset must be >= 0");
    ra::AppendArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_tstride = q_tstride;
    a.k_tstride = k_tstride;
    a.v_tstride = v_tstride;
    a.q_out_tstride = q_out_tstride;
    a.cu = cu_tokens;
    a.lens = seq_lens;
    a.tables = block_tables;
    a.inv_freq = inv_freq;
    a.B = B;
    a.n_tokens = n_tokens;
    a.max_tokens = max_tokens;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.rot = rot_dim;
    a.interleaved = interleaved;
    a.pos_offset = pos_offset;
    a.page_size = page_size;
    a.n_pages = n_pages;
    a.max_pages = max_pages;
    a.page_stride = page_stride;
    a.q_out = q_out;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.stream = (cudaStream_t)stream;
    const cudaError_t e = ra::launch_paged_append(a);
    return e == cudaSuccess ? RA_OK : cuda_fail(e, "paged append launch");
}

long long ra_prefix_attn_workspace(int B, int n_tokens, int max_tokens, int max_len,
                                   int prefix_len, int H_q, int H_kv, int D, int page_size) {
    if (B < 1 || n_tokens < 1 || max_tokens < 1 || max_len < 1 || prefix_len < 0 || H_kv < 1 ||
        H_q < 1 || H_q % H_kv != 0 || D < 1 || page_size < 1)
        return 0;
    return ra::plan_kv(B, n_tokens, max_tokens, max_len, prefix_len, H_q, H_kv, D, 1, page_size)
        .workspace;
}

ra_status ra_prefix_attn_fwd(const void* q, long long q_tstride, const void* k_pages,
                             const void* v_pages, const int* cu_tokens, const int* seq_lens,
                             const int* block_tables, const int* prefix_table, int prefix_len,
                             int B, int n_tokens, int max_tokens, int max_len, int H_q, int H_kv,
                             int D, int page_size, int n_pages, int max_pages,
                             long long page_stride, float scale, ra_dtype in_dtype,
                             ra_dtype out_dtype, void* out, float* lse, void* workspace,
                             long long workspace_bytes, void* stream) {
    RA_CHECK(check_heads(H_q, H_kv, D, in_dtype));
    RA_CHECK(check_batch(cu_tokens, seq_lens, block_tables, B, n_tokens, max_tokens));
    RA_CHECK(check_cache(k_pages, v_pages, page_size, n_pages, max_pages, page_stride, H_kv, D));
    RA_CHECK(check_results(scale, out_dtype, out, lse));
    if (!aligned(q, 16)) return fail(RA_ERR_INVALID, "q must be non-null and 16-byte aligned");
    RA_CHECK(check_stride(q_tstride, (long long)H_q * D, "q_tstride"));
    if (prefix_len < 0 || prefix_len > kMaxKeys)
        return fail(RA_ERR_INVALID, "prefix_len must be in [0, 2^30]");
    if (prefix_len > 0 && !aligned(prefix_table, 4))
        return fail(RA_ERR_INVALID, "prefix_table must be non-null and 4-byte aligned");
    if (max_len < 1 || max_len > kMaxKeys || max_len > (long long)max_pages * page_size)
        return fail(RA_ERR_INVALID, "max_len must be in [1, min(2^30, max_pages * page_size)]");
    ra::KvArgs a;
    a.q = q;
    a.q_tstride = q_tstride;
    a.q_bstride = 0;
    a.k = k_pages;
    a.v = v_pages;
    a.kv_tstride = (long long)H_kv * D;
    a.page_stride = page_stride;
    a.cu = cu_tokens;
    a.lens = seq_lens;
    a.tables = block_tables;
    a.prefix_table = prefix_table;
    a.prefix_len = prefix_len;
    a.B = B;
    a.n_tokens = n_tokens;
    a.max_tokens = max_tokens;
    a.max_len = max_len;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.page_size = page_size;
    a.n_pages = n_pages;
    a.max_pages = max_pages;
    a.causal = 1;
    a.scale = scale;
    a.out_bf16 = out_dtype == RA_BF16;
    a.out = out;
    a.lse = lse;
    a.workspace = workspace;
    a.stream = (cudaStream_t)stream;
    const ra::KvPlan plan =
        ra::plan_kv(B, n_tokens, max_tokens, max_len, prefix_len, H_q, H_kv, D, 1, page_size);
    if ((long long)n_tokens * H_q > 0x7fffffffLL || plan.blocks > 0x7fffffffLL)
        return fail(RA_ERR_INVALID, "problem too large for one launch");
    RA_CHECK(check_workspace(workspace, workspace_bytes, plan.workspace));
    const char* why = "prefix attention launch";
    const cudaError_t e = ra::launch_kv(a, plan, ra::wait_limit_ns(), &why);
    return e == cudaSuccess ? RA_OK : cuda_fail(e, why);
}

long long ra_cross_attn_workspace(int B, int Lq, int Lk, int H_q, int H_kv, int D) {
    if (B < 1 || Lq < 1 || Lk < 1 || H_kv < 1 || H_q < 1 || H_q % H_kv != 0 || D < 1 ||
        (long long)B * Lq > kMaxTokens)
        return 0;
    return ra::plan_kv(B, B * Lq, Lq, Lk, 0, H_q, H_kv, D, 0, Lk).workspace;
}

// The sizes and strides that cross attention's forward and backward share.
static ra_status check_cross(const void* q, const void* k, const void* v, const int* kv_lens,
                             int B, int Lq, int Lk, int H_q, int H_kv, int D, long long q_tstride,
                             long long q_bstride, long long kv_tstride, long long kv_bstride,
                             ra_dtype in_dtype) {
    RA_CHECK(check_heads(H_q, H_kv, D, in_dtype));
    if (B < 1 || Lq < 1 || Lk < 1) return fail(RA_ERR_INVALID, "B, Lq and Lk must be >= 1");
    if ((long long)B * Lq > kMaxTokens || Lk > kMaxKeys)
        return fail(RA_ERR_INVALID, "B * Lq must be <= 2^24 and Lk <= 2^30");
    if ((long long)B * Lq * H_q > 0x7fffffffLL)
        return fail(RA_ERR_INVALID, "problem too large for one launch");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16))
        return fail(RA_ERR_INVALID, "q, k and v must be non-null and 16-byte aligned");
    if (kv_lens && !aligned(kv_lens, 4))
        return fail(RA_ERR_INVALID, "kv_lens must be 4-byte aligned");
    RA_CHECK(check_stride(q_tstride, (long long)H_q * D, "q_tstride"));
    RA_CHECK(check_stride(kv_tstride, (long long)H_kv * D, "kv_tstride"));
    RA_CHECK(check_stride(q_bstride, (Lq - 1) * q_tstride + (long long)H_q * D, "q_bstride"));
    return check_stride(kv_bstride, (Lk - 1) * kv_tstride + (long long)H_kv * D, "kv_bstride");
}

ra_status ra_cross_attn_fwd(const void* q, const void* k, const void* v, const int* kv_lens, int B,
                            int Lq, int Lk, int H_q, int H_kv, int D, long long q_tstride,
                            long long q_bstride, long long kv_tstride, long long kv_bstride,
                            float scale, ra_dtype in_dtype, ra_dtype out_dtype, void* out,
                            float* lse, void* workspace, long long workspace_bytes, void* stream) {
    RA_CHECK(check_cross(q, k, v, kv_lens, B, Lq, Lk, H_q, H_kv, D, q_tstride, q_bstride,
                         kv_tstride, kv_bstride, in_dtype));
    RA_CHECK(check_results(scale, out_dtype, out, lse));
    ra::KvArgs a;
    a.q = q;
    a.q_tstride = q_tstride;
    a.q_bstride = q_bstride;
    a.k = k;
    a.v = v;
    a.kv_tstride = kv_tstride;
    a.page_stride = kv_bstride;
    a.cu = nullptr;
    a.lens = kv_lens;
    a.tables = nullptr;
    a.prefix_table = nullptr;
    a.prefix_len = 0;
    a.B = B;
    a.n_tokens = B * Lq;
    a.max_tokens = Lq;
    a.max_len = Lk;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.page_size = Lk;
    a.n_pages = B;
    a.max_pages = 1;
    a.causal = 0;
    a.scale = scale;
    a.out_bf16 = out_dtype == RA_BF16;
    a.out = out;
    a.lse = lse;
    a.workspace = workspace;
    a.stream = (cudaStream_t)stream;
    const ra::KvPlan plan = ra::plan_kv(B, B * Lq, Lq, Lk, 0, H_q, H_kv, D, 0, Lk);
    RA_CHECK(check_workspace(workspace, workspace_bytes, plan.workspace));
    if (plan.blocks > 0x7fffffffLL)
        return fail(RA_ERR_INVALID, "problem too large for one launch");
    const char* why = "cross attention launch";
    const cudaError_t e = ra::launch_kv(a, plan, ra::wait_limit_ns(), &why);
    return e == cudaSuccess ? RA_OK : cuda_fail(e, why);
}

long long ra_cross_attn_bwd_workspace(int B, int Lq, int H_q, int D, ra_dtype grad_dtype) {
    if (B < 1 || Lq < 1 || H_q < 1 || D < 1) return 0;
    const long long rows = ((long long)B * Lq * H_q + 3) / 4 * 4;
    return 4 * (rows + (grad_dtype == RA_BF16 ? rows * D : 0));
}

ra_status ra_cross_attn_bwd(const void* q, const void* k, const void* v, const int* kv_lens,
                            const void* out, const float* lse, const void* dout, int B, int Lq,
                            int Lk, int H_q, int H_kv, int D, long long q_tstride,
                            long long q_bstride, long long kv_tstride, long long kv_bstride,
                            float scale, ra_dtype in_dtype, ra_dtype grad_dtype, void* dq,
                            void* dk, void* dv, void* workspace, long long workspace_bytes,
                            void* stream) {
    RA_CHECK(check_cross(q, k, v, kv_lens, B, Lq, Lk, H_q, H_kv, D, q_tstride, q_bstride,
                         kv_tstride, kv_bstride, in_dtype));
    RA_CHECK(check_results(scale, grad_dtype, out, lse));
    if (!aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16))
        return fail(RA_ERR_INVALID, "dout, dq, dk and dv must be non-null and 16-byte aligned");
    if ((long long)B * H_kv * ((Lk + 127) / 128) > 0x7fffffffLL)
        return fail(RA_ERR_INVALID, "problem too large for one launch");
    RA_CHECK(check_workspace(workspace, workspace_bytes,
                             ra_cross_attn_bwd_workspace(B, Lq, H_q, D, grad_dtype)));
    ra::CrossBwdArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.dout = dout;
    a.lse = lse;
    a.kv_lens = kv_lens;
    a.B = B;
    a.Lq = Lq;
    a.Lk = Lk;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.D = D;
    a.q_tstride = q_tstride;
    a.q_bstride = q_bstride;
    a.kv_tstride = kv_tstride;
    a.kv_bstride = kv_bstride;
    a.scale = scale;
    a.grad_bf16 = grad_dtype == RA_BF16;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.workspace = (float*)workspace;
    a.stream = (cudaStream_t)stream;
    const char* why = "cross attention backward launch";
    const cudaError_t e =
        ra::launch_cross_bwd(a, ra::wait_limit_ns(), ra::bwd_deterministic(), &why);
    return e == cudaSuccess ? RA_OK : cuda_fail(e, why);
}

}  // extern "C"
