// cross_bwd.cu -- the backward of cross attention: the key-stationary tensor-core backward
// in its cross form (attn_bwd_sm100.cu), and the rounding of its fp32 dQ where the caller
// wants bf16 gradients (dQ is a sum over key tiles, so it is rounded once, when complete).
#include "kv_internal.h"
#include "sm100_ptx.cuh"

namespace ra {
namespace {

// 8 values per thread: 32 bytes read, 16 written; bound by memory (most of it L2: the
// backward has just written dQ).
__global__ void __launch_bounds__(256) round_bf16_kernel(const float4* __restrict__ in,
                                                         uint4* __restrict__ out, long long n8) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    const float4 a = in[2 * i], b = in[2 * i + 1];
    out[i] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                        pack_bf16x2(b.z, b.w));
}

}  // namespace

cudaError_t launch_cross_bwd(const CrossBwdArgs& c, unsigned long long wait_limit_ns,
                             int deterministic, const char** why) {
    const long long rows = (long long)c.B * c.H_q * c.Lq, n = rows * c.D;
    const void* k[1] = {c.k};
    const void* v[1] = {c.v};
    float* dk[1] = {(float*)c.dk};
    float* dv[1] = {(float*)c.dv};
    AttnBwdArgs a;
    a.q = c.q;
    a.k_chunks = k;
    a.v_chunks = v;
    a.out = c.out;
    a.lse = c.lse;
    a.dout = c.dout;
    a.P = 1;
    a.B = c.B;
    a.H_q = c.H_q;
    a.H_kv = c.H_kv;
    a.Lc = c.Lk;
    a.D = c.D;
    a.q_bstride = c.q_bstride;
    a.kv_bstride = c.kv_bstride;
    a.scale = c.scale;
    a.causal = 0;
    a.workspace = c.workspace;
    a.dq = c.grad_bf16 ? c.workspace + (rows + 3) / 4 * 4 : (float*)c.dq;
    a.dk_chunks = dk;
    a.dv_chunks = dv;
    a.deterministic = deterministic;
    a.cross_Lq = c.Lq;
    a.kv_lens = c.kv_lens;
    a.q_tstride = c.q_tstride;
    a.kv_tstride = c.kv_tstride;
    a.grad_bf16 = c.grad_bf16;
    a.stream = c.stream;
    const cudaError_t e = launch_attn_bwd_sm100(a, wait_limit_ns, why);
    if (e != cudaSuccess || !c.grad_bf16) return e;
    const long long n8 = n / 8;
    round_bf16_kernel<<<(unsigned)((n8 + 255) / 256), 256, 0, c.stream>>>(
        (const float4*)a.dq, (uint4*)c.dq, n8);
    return cudaGetLastError();
}

}  // namespace ra
