// paged_append.cu -- K and V of new tokens into a paged cache, with the position rotation
// applied to q and k on the way.
//
// Token i of sequence b (of its n_b new tokens, the last n_b of its length len_b) sits at
// p = len_b - n_b + i of the sequence's own keys and at sequence position pos_offset + p.
// With angle_j = (pos_offset + p) * inv_freq_j, the pair (x, y) of a head's elements
// (j, j + R/2), or (2j, 2j+1) interleaved, becomes (x cos - y sin, y cos + x sin); elements
// from R on are copied.  The product is formed and reduced to turns in 64 bits (one multiply
// and one subtraction): a 32-bit product loses 2^-24 of an angle of up to millions of
// radians.  The fraction that is left, at most half a turn, is exact enough in 32 bits
// (relative 2^-24) for sincospif.
//
// What bounds it: memory (every vector is read and written once); a small call, the latency of
// length -> page -> store.  Four tokens to a block, so that a thread has eight 16-byte loads in
// flight, and they are issued before the places and angles are worked out: 396 MB (16 thousand
// tokens of 32 + 2 x 8 heads of 128) take 65 us, 6.1 TB/s; loading after them took 72 us.
#include <cuda_bf16.h>
#include "kv_internal.h"

namespace ra {

__device__ unsigned int g_append_error_word = 0;

namespace {

constexpr int kTokens = 4;  // tokens per block
constexpr long long kNoPlace = -1, kNoToken = -2;  // of a token's row in the cache

struct AppendParams {
    AppendArgs a;
    int tiles;  // blocks per sequence (the flat form: 0)
};

__device__ __forceinline__ void rotate2(uint32_t& xy_lo, uint32_t& xy_hi, float2 cs0, float2 cs1) {
    // elements (lo of xy_lo with lo of xy_hi) by cs0, (hi with hi) by cs1
    const float x0 = __uint_as_float(xy_lo << 16), x1 = __uint_as_float(xy_lo & 0xffff0000u);
    const float y0 = __uint_as_float(xy_hi << 16), y1 = __uint_as_float(xy_hi & 0xffff0000u);
    const __nv_bfloat162 a =
        __floats2bfloat162_rn(x0 * cs0.x - y0 * cs0.y, x1 * cs1.x - y1 * cs1.y);
    const __nv_bfloat162 b =
        __floats2bfloat162_rn(y0 * cs0.x + x0 * cs0.y, y1 * cs1.x + x1 * cs1.y);
    xy_lo = *reinterpret_cast<const uint32_t*>(&a);
    xy_hi = *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t rotate1(uint32_t xy, float2 cs) {
    const float x = __uint_as_float(xy << 16), y = __uint_as_float(xy & 0xffff0000u);
    const __nv_bfloat162 a = __floats2bfloat162_rn(x * cs.x - y * cs.y, y * cs.x + x * cs.y);
    return *reinterpret_cast<const uint32_t*>(&a);
}

// One thread moves two 16-byte vectors of one head: the two halves of 8 rotated pairs, or
// neighbours.  Units of a token: (H_q + 2 H_kv) heads x D/16.
//
// A block has up to four tokens of one sequence or, FLAT, any four rows next to each other,
// whose sequences it looks up: B x max_tokens / 4 blocks are too many where few sequences have
// that many tokens.
template <int D, bool FLAT>
__global__ void __launch_bounds__(384) append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int UPH = D / 16;
    const AppendArgs& a = p.a;
    __shared__ float2 cs[kTokens][D / 2];
    __shared__ long long row_off[kTokens];  // element offset of the token's row in the cache
    __shared__ int place[kTokens];  // FLAT: the token's place among its sequence's own keys
    int b = 0, t0 = 0, len = 0, n = 0, row0, nt;  // row0: the first token's row
    if (FLAT) {
        row0 = (int)blockIdx.x * kTokens;
        nt = min(a.n_tokens - row0, kTokens);
        if (blockIdx.x == 0)
            for (int e = threadIdx.x; e < a.B; e += blockDim.x)
                if (token_rows(a.cu, e, a.n_tokens, a.max_tokens).bad)
                    atomicOr(&g_append_error_word, kKvErrTokens);
    } else {
        b = blockIdx.x / p.tiles;
        t0 = (blockIdx.x % p.tiles) * kTokens;
        const TokenRows rows = token_rows(a.cu, b, a.n_tokens, a.max_tokens);
        len = max(a.lens[b], 0);
        n = rows.n;
        row0 = rows.first + t0;
        if (threadIdx.x == 0 && t0 == 0 && rows.bad) atomicOr(&g_append_error_word, kKvErrTokens);
        nt = min(n - t0, kTokens);
        if (nt <= 0) return;
    }
    // a unit's vectors, loaded before the places and angles are worked out
    const int units = (a.H_q + 2 * a.H_kv) * UPH, ru = a.rot / 16;
    uint4 x[kTokens], y[kTokens];
    int v0 = 0, v1 = 0;
    auto load = [&](int u) {
        const int head = u / UPH, j = u % UPH;
        const bool is_q = head < a.H_q, is_v = head >= a.H_q + a.H_kv;
        const int h = is_q ? head : (is_v ? head - a.H_q - a.H_kv : head - a.H_q);
        const uint16_t* src = (const uint16_t*)(is_q ? a.q : (is_v ? a.v : a.k));
        const long long stride = is_q ? a.q_tstride : (is_v ? a.v_tstride : a.k_tstride);
        const bool halves = !a.interleaved && j < ru;  // the two halves of 8 rotated pairs
        v0 = halves ? j : 2 * j;
        v1 = halves ? j + ru : 2 * j + 1;
#pragma unroll
        for (int t = 0; t < kTokens; ++t)
            if (t < nt) {
                const uint4* r =
                    reinterpret_cast<const uint4*>(src + (long long)(row0 + t) * stride + h * D);
                x[t] = r[v0];
                y[t] = r[v1];
            }
    };
    if (threadIdx.x < units) load(threadIdx.x);
    // the place of token t of the block in the cache: kNoPlace, or kNoToken where the row is none
    auto locate = [&](int t, int b, int pos) {
        long long off = kNoPlace;
        if (pos >= 0) {
            const int slot = pos / a.page_size;
            if (slot >= a.max_pages) {
                atomicOr(&g_append_error_word, kKvErrLength);
            } else {
                const int page = a.tables[(long long)b * a.max_pages + slot];
                if (page < 0 || page >= a.n_pages)
                    atomicOr(&g_append_error_word, kKvErrPage);
                else
                    off = (long long)page * a.page_stride +
                          (long long)(pos - slot * a.page_size) * a.H_kv * D;
            }
        } else {
            atomicOr(&g_append_error_word, kKvErrLength);
        }
        row_off[t] = off;
    };
    if (FLAT) {
        for (int t = threadIdx.x >> 5; t < nt; t += blockDim.x >> 5) {
            const int tok = row0 + t, e = find_sequence(a.cu, a.B, tok);
            const TokenRows rows = token_rows(a.cu, e, a.n_tokens, a.max_tokens);
            const int i = tok - rows.first, pos = max(a.lens[e], 0) - rows.n + i;
            if ((threadIdx.x & 31) == 0) {
                place[t] = pos;
                if (i >= 0 && i < min(rows.n, a.max_tokens)) locate(t, e, pos);
                else row_off[t] = kNoToken;
            }
        }
        __syncthreads();
    } else if (threadIdx.x < nt) {
        locate(threadIdx.x, b, len - n + t0 + (int)threadIdx.x);
    }
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
        const int t = i / half, j = i - t * half;
        const double pos = (double)a.pos_offset + (double)(FLAT ? place[t] : len - n + t0 + t);
        double turns = pos * (double)a.inv_freq[j] * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= rint(turns);
        float s, c;
        sincospif((float)(2.0 * turns), &s, &c);
        cs[t][j] = make_float2(c, s);
    }
    __syncthreads();
    for (int u = threadIdx.x; u < units; u += blockDim.x) {
        if (u >= blockDim.x) load(u);
        const int head = u / UPH, j = u % UPH;
        const bool is_q = head < a.H_q, is_v = head >= a.H_q + a.H_kv;
        const int h = is_q ? head : (is_v ? head - a.H_q - a.H_kv : head - a.H_q);
        const bool turned = !is_v && j < ru;
#pragma unroll
        for (int t = 0; t < kTokens; ++t)
            if (t < nt) {
                if (turned) {
                    uint32_t* xs = reinterpret_cast<uint32_t*>(&x[t]);
                    uint32_t* ys = reinterpret_cast<uint32_t*>(&y[t]);
                    if (a.interleaved) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            xs[e] = rotate1(xs[e], cs[t][8 * j + e]);
                            ys[e] = rotate1(ys[e], cs[t][8 * j + 4 + e]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            rotate2(xs[e], ys[e], cs[t][8 * j + 2 * e], cs[t][8 * j + 2 * e + 1]);
                    }
                }
                uint4* w = nullptr;
                if (is_q) {
                    if (!FLAT || row_off[t] != kNoToken)
                        w = reinterpret_cast<uint4*>((uint16_t*)a.q_out +
                                                     (long long)(row0 + t) * a.q_out_tstride + h * D);
                } else if (row_off[t] >= 0)
                    w = reinterpret_cast<uint4*>((uint16_t*)(is_v ? a.v_pages : a.k_pages) +
                                                 row_off[t] + h * D);
                if (w) {
                    w[v0] = x[t];
                    w[v1] = y[t];
                }
            }
    }
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a) {
    cache_kernels_in_use();
    AppendParams p;
    p.a = a;
    p.tiles = (a.max_tokens + kTokens - 1) / kTokens;
    const int units = (a.H_q + 2 * a.H_kv) * (a.D / 16);
    const int threads = units >= 384 ? 384 : ((units + 31) / 32) * 32;
    // Flat where at least half of the blocks by sequence would be empty.  Measured, us on the GPU,
    // by sequence and flat (32 + 2 x 8 heads of 128): 16 and 1 tokens in turn, 128 sequences, 8.2,
    // 7.0; 1000 and 500, 8 sequences, 27.7, 33.1 (the look-up comes before a block's stores); 255
    // single tokens and one of 2000 (128,000 blocks against 564) flat 11.8, of which 9 are memory's.
    const long long flat = (a.n_tokens + kTokens - 1) / kTokens;
    if ((long long)p.tiles * a.B >= 2 * (flat + a.B)) {
        p.tiles = 0;
        const unsigned rows = (unsigned)flat;
        if (a.D == 128) append_kernel<128, true><<<rows, threads, 0, a.stream>>>(p);
        else append_kernel<64, true><<<rows, threads, 0, a.stream>>>(p);
        return cudaGetLastError();
    }
    const unsigned grid = (unsigned)((long long)p.tiles * a.B);  // < 2 (2^22 + 2^28)
    if (a.D == 128) append_kernel<128, false><<<grid, threads, 0, a.stream>>>(p);
    else append_kernel<64, false><<<grid, threads, 0, a.stream>>>(p);
    return cudaGetLastError();
}

cudaError_t read_and_clear_append_error(unsigned int* value) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_append_error_word, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    if (*value) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_append_error_word, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace ra
