// kv_rows.cu -- attention of few query rows over many keys: the single-token form of the
// paged, prefix and cross attention.
//
// A block takes 16 or 32 query rows (tokens x the query heads that share a kv head), one kv
// head and one range of keys, either of the prefix that every sequence sees (rows of the
// whole batch, so the prefix is read once) or of one sequence's own keys.  Its four warps
// take the range's 16-key groups in turn, each warp with its own running softmax state
// (maximum m, sum l, output O, all fp32) and its own ring of cp.async stages, so no warp
// waits for another until the range is done; the four states are then merged by
//   m* = max m_w,   O = sum 2^(m_w - m*) O_w / sum 2^(m_w - m*) l_w
// and written as one partial result (O, log2-sum) of the rows, or as the final one where
// the call has a single range.  The combine kernel merges a row's partials the same way.
//
// What bounds it: 16 rows need 4 D flops per key against 4 D bytes of K and V, far below the
// machine's balance, so it runs at the rate at which K and V arrive.  Hence mma.sync on
// 16-row fragments (a tcgen05 tile has at least 64 rows) and the deep per-warp rings.
#include <cuda_bf16.h>
#include <cmath>
#include "kv_internal.h"
#include "sm100_ptx.cuh"

namespace ra {

__device__ unsigned int g_kv_error_word = 0;

namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 16;  // keys of a warp's group
constexpr float kRescale = 8.0f;  // log2 units: the maximum may lag by 2^8

struct RowsParams {
    KvArgs a;
    KvPlan p;
    int group;
    float scale_log2;
    float* part_o;    // [split][token][head][D]
    float* part_lse;  // [split][token][head], log2
    unsigned items_p;  // blocks over the prefix, the first of the grid
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int MT>
struct RCfg {
    static constexpr int STAGES = D == 128 ? 3 : 4;
    static constexpr int GROUP_BYTES = kKeys * D * 2;          // K or V of one group
    static constexpr int WARP_BYTES = STAGES * 2 * GROUP_BYTES;
    static constexpr int SMEM = kWarps * WARP_BYTES;
    static constexpr int ROWS = MT * 16;
    static constexpr int PITCH = D + 4;  // floats of a row in the merge buffer
    static_assert(kWarps * ROWS * PITCH * 4 + kWarps * ROWS * 12 <= SMEM, "merge buffer");
};

// Byte offset of 16-byte chunk c of row r, chunks permuted within a row so that the eight
// rows of an ldmatrix fall on different banks.
template <int D>
__device__ __forceinline__ uint32_t sw(int r, int c) {
    return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

// A row's place: token index, head, output index (token * H_q + head) or -1.
struct Row {
    int tok, head;
};

// PAGED: keys found through a page table (else dense batch rows).  One page holds whole
// 16-key groups where PAGE16, else every key is looked up.
template <int D, int MT, bool PAGE16>
__global__ void __launch_bounds__(kWarps * 32, 2) kv_rows_kernel(const __grid_constant__ RowsParams p) {
    using C = RCfg<D, MT>;
    extern __shared__ __align__(128) uint8_t smem[];
    const KvArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ---- which rows and keys
    unsigned item = blockIdx.x;
    const bool is_prefix = item < p.items_p;
    int b = 0, split, tile, g, tok0, n_tok, chunk, part;
    int len;
    const int* table;
    if (is_prefix) {
        tile = item % p.p.tiles_p;
        item /= p.p.tiles_p;
        g = item % a.H_kv;
        split = item / a.H_kv;
        tok0 = 0;
        n_tok = a.cu ? min(a.cu[a.B], a.n_tokens) : a.n_tokens;
        len = a.prefix_len;
        chunk = p.p.chunk_p;
        table = a.prefix_table;
        part = split;
    } else {
        item -= p.items_p;
        tile = item % p.p.tiles_o;
        item /= p.p.tiles_o;
        g = item % a.H_kv;
        item /= a.H_kv;
        split = item % p.p.splits_o;
        b = item / p.p.splits_o;
        if (a.cu) {
            tok0 = max(a.cu[b], 0);
            n_tok = min(a.cu[b + 1], a.n_tokens) - tok0;
            if (n_tok > a.max_tokens && threadIdx.x == 0 && split == 0)
                atomicOr(&g_kv_error_word, kKvErrTokens);
        } else {
            tok0 = b * a.max_tokens;
            n_tok = a.max_tokens;
        }
        len = a.lens ? max(a.lens[b], 0) : a.max_len;
        if (len > a.max_len) {
            if (threadIdx.x == 0 && split == 0) atomicOr(&g_kv_error_word, kKvErrLength);
            len = a.max_len;
        }
        chunk = p.p.chunk_o;
        table = a.tables ? a.tables + (long long)b * a.max_pages : nullptr;
        part = p.p.parts_p + split;
    }
    const int n_rows = n_tok * p.group;
    const int row0 = tile * C::ROWS;
    if (row0 >= n_rows) return;
    const int k_begin = split * chunk;
    int k_end = min(k_begin + chunk, len);
    const bool causal = a.causal && !is_prefix;
    // the latest key that any of the block's rows sees
    if (causal) {
        const int last_tok = min((row0 + C::ROWS - 1) / p.group, n_tok - 1);
        k_end = min(k_end, len - n_tok + last_tok + 1);
    }
    const int n_groups = k_end > k_begin ? (k_end - k_begin + kKeys - 1) / kKeys : 0;
    const int n_mine = (n_groups - warp + kWarps - 1) / kWarps;  // groups warp, warp + 4, ...

    // ---- Q fragments, straight from global memory
    const int r_lo = lane >> 2, c_lo = (lane & 3) * 2;
    uint32_t qf[MT][D / 16][4];
    int limit[MT][2];  // keys below it are seen
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int row = row0 + mt * 16 + r_lo + 8 * hf;
            const bool ok = row < n_rows;
            const int t = ok ? row / p.group : 0;
            const int head = g * p.group + (ok ? row - t * p.group : 0);
            limit[mt][hf] = !ok ? 0 : (causal ? min(k_end, len - n_tok + t + 1) : k_end);
            const long long off = (a.cu ? (long long)(tok0 + t) * a.q_tstride
                                        : (long long)b * a.q_bstride + (long long)t * a.q_tstride) +
                                  (long long)head * D;
            const uint32_t* q32 = reinterpret_cast<const uint32_t*>((const uint16_t*)a.q + off);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qf[mt][kk][hf] = ok ? q32[(kk * 16 + c_lo) / 2] : 0u;
                qf[mt][kk][2 + hf] = ok ? q32[(kk * 16 + c_lo + 8) / 2] : 0u;
            }
        }
    int min_limit = k_end;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        min_limit = min(min_limit, min(limit[mt][0], limit[mt][1]));
    min_limit = __reduce_min_sync(0xffffffffu, min_limit);

    // ---- loads: group i of this warp is keys k_begin + 16 (warp + 4 i) ..
    const uint32_t ring = smem_u32(smem) + warp * C::WARP_BYTES;
    int page_reg = 0;  // lane l: page of this warp's group 32 (i / 32) + l
    auto look_up = [&](int key) -> int {
        int page = table[key / a.page_size];
        if (page < 0 || page >= a.n_pages) {
            atomicOr(&g_kv_error_word, kKvErrPage);
            page = 0;
        }
        return page;
    };
    auto load = [&](int i) {
        if (PAGE16 && table && (i & 31) == 0) {
            const int ii = i + lane;
            if (ii < n_mine) page_reg = look_up(k_begin + kKeys * (warp + kWarps * ii));
        }
        if (i < n_mine) {
            const int key0 = k_begin + kKeys * (warp + kWarps * i);
            const uint32_t st = ring + (i % C::STAGES) * 2 * C::GROUP_BYTES;
            long long base = 0;
            if (PAGE16) {
                if (table) {
                    const int page = __shfl_sync(0xffffffffu, page_reg, i & 31);
                    base = (long long)page * a.page_stride +
                           (long long)(key0 % a.page_size) * a.kv_tstride;
                } else {
                    base = (long long)b * a.page_stride + (long long)key0 * a.kv_tstride;
                }
            }
            constexpr int CPR = D / 8;          // 16-byte chunks per row
            constexpr int RPI = 32 / CPR;       // rows per instruction
#pragma unroll
            for (int r0 = 0; r0 < kKeys; r0 += RPI) {
                const int r = r0 + lane / CPR, c = lane % CPR;
                const bool ok = key0 + r < k_end;  // keys past the end: zeros, never read
                long long off;
                if (PAGE16) {
                    off = base + (long long)r * a.kv_tstride;
                } else {
                    const int key = ok ? key0 + r : key0;
                    off = (long long)look_up(key) * a.page_stride +
                          (long long)(key % a.page_size) * a.kv_tstride;
                }
                off += (long long)g * D + c * 8;
                if (PAGE16 && !ok) off = base;  // a valid address; nothing is read from it
                cp_async16(st + sw<D>(r, c), (const uint16_t*)a.k + off, ok);
                cp_async16(st + C::GROUP_BYTES + sw<D>(r, c), (const uint16_t*)a.v + off, ok);
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) load(i);

    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2], lu[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            m[mt][hf] = -INFINITY;
            l[mt][hf] = lu[mt][hf] = 0.f;
        }
    }
    const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row of this lane's address
    for (int i = 0; i < n_mine; ++i) {
        cp_wait<C::STAGES - 2>();
        __syncwarp();
        load(i + C::STAGES - 1);
        const uint32_t kst = ring + (i % C::STAGES) * 2 * C::GROUP_BYTES;
        const uint32_t vst = kst + C::GROUP_BYTES;
        float s[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][n][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t kf[4];
            ldsm4(kf, kst + sw<D>((mi >> 1) * 8 + mr, kk * 2 + (mi & 1)));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                mma16816(s[mt][0], qf[mt][kk], kf[0], kf[1]);
                mma16816(s[mt][1], qf[mt][kk], kf[2], kf[3]);
            }
        }
        const int key0 = k_begin + kKeys * (warp + kWarps * i);
        if (key0 + kKeys > min_limit) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (key0 + n * 8 + c_lo + (e & 1) >= limit[mt][e >> 1])
                            s[mt][n][e] = -INFINITY;
        }
        uint32_t pf[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float alpha[2];
            bool grew = false;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float mx = fmaxf(fmaxf(s[mt][0][2 * hf], s[mt][0][2 * hf + 1]),
                                 fmaxf(s[mt][1][2 * hf], s[mt][1][2 * hf + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float m_new = mx * p.scale_log2;
                alpha[hf] = 1.f;
                // the maximum is moved only when it grew by more than 2^8 (the sums use the
                // same stale maximum, so the result is the same)
                if (m_new - m[mt][hf] > kRescale) {
                    alpha[hf] = ex2_approx(m[mt][hf] - m_new);
                    m[mt][hf] = m_new;
                    grew = true;
                }
                const float neg = m[mt][hf] == -INFINITY ? 0.f : -m[mt][hf];
                float sum = 0.f, used = 0.f;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = ex2_approx(fmaf(s[mt][n][2 * hf], p.scale_log2, neg));
                    const float p1 = ex2_approx(fmaf(s[mt][n][2 * hf + 1], p.scale_log2, neg));
                    const uint32_t pp = pack_bf16x2(p0, p1);
                    pf[mt][2 * n + hf] = pp;
                    sum += p0 + p1;
                    used += __uint_as_float(pp << 16) + __uint_as_float(pp & 0xffff0000u);
                }
                l[mt][hf] = l[mt][hf] * alpha[hf] + sum;
                lu[mt][hf] = lu[mt][hf] * alpha[hf] + used;
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[mt][n][0] *= alpha[0];
                    o[mt][n][1] *= alpha[0];
                    o[mt][n][2] *= alpha[1];
                    o[mt][n][3] *= alpha[1];
                }
            }
        }
#pragma unroll
        for (int nn = 0; nn < D / 16; ++nn) {
            uint32_t vf[4];
            ldsm4_t(vf, vst + sw<D>((mi & 1) * 8 + mr, nn * 2 + (mi >> 1)));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                mma16816(o[mt][2 * nn], pf[mt], vf[0], vf[1]);
                mma16816(o[mt][2 * nn + 1], pf[mt], vf[2], vf[3]);
            }
        }
        __syncwarp();
    }
    cp_wait<0>();
    __syncthreads();

    // ---- merge the warps' states through shared memory
    float* so = reinterpret_cast<float*>(smem);               // [warp][row][PITCH]
    float* sm = so + kWarps * C::ROWS * C::PITCH;             // [warp][row][3]: m, l, lu
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int off = 1; off <= 2; off <<= 1) {
                l[mt][hf] += __shfl_xor_sync(0xffffffffu, l[mt][hf], off);
                lu[mt][hf] += __shfl_xor_sync(0xffffffffu, lu[mt][hf], off);
            }
            const int r = mt * 16 + r_lo + 8 * hf;
            float* w = so + (warp * C::ROWS + r) * C::PITCH;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2*>(w + n * 8 + c_lo) =
                    make_float2(o[mt][n][2 * hf], o[mt][n][2 * hf + 1]);
            if ((lane & 3) == 0) {
                float* x = sm + (warp * C::ROWS + r) * 3;
                x[0] = m[mt][hf];
                x[1] = l[mt][hf];
                x[2] = lu[mt][hf];
            }
        }
    __syncthreads();
    constexpr int TPR = D / 4;  // threads per row
    for (int r = threadIdx.x / TPR; r < C::ROWS; r += kWarps * 32 / TPR) {
        const int row = row0 + r, c = (threadIdx.x % TPR) * 4;
        if (row >= n_rows) break;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[(w * C::ROWS + r) * 3]);
        float ls = 0.f, lus = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        // a row that saw nothing has every m = -inf and every sum 0; a NaN score leaves m
        // at -inf as well but makes the sums NaN, which must come through
        const float ms = mm == -INFINITY ? 0.f : mm;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float* x = sm + (w * C::ROWS + r) * 3;
            const float f = ex2_approx(x[0] - ms);
            ls += f * x[1];
            lus += f * x[2];
            const float4 v =
                *reinterpret_cast<const float4*>(so + (w * C::ROWS + r) * C::PITCH + c);
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
        }
        const float inv = lus == 0.f ? 0.f : 1.f / lus;
        const float lse2 = ls == 0.f ? -INFINITY : ms + log2f(ls);
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const int t = row / p.group, head = g * p.group + row - t * p.group;
        const long long orow = (long long)(tok0 + t) * a.H_q + head;
        if (p.p.direct) {
            if (a.out_bf16)
                *reinterpret_cast<uint2*>((uint16_t*)a.out + orow * D + c) =
                    make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            else
                *reinterpret_cast<float4*>((float*)a.out + orow * D + c) = acc;
            if (c == 0) {
                const long long li = a.cu ? (long long)head * a.n_tokens + tok0 + t
                                          : ((long long)b * a.H_q + head) * a.max_tokens + t;
                a.lse[li] = lse2 * 0.69314718055994530942f;
            }
        } else {
            const long long pr = (long long)part * a.n_tokens * a.H_q + orow;
            if (lse2 != -INFINITY)
                *reinterpret_cast<float4*>(p.part_o + pr * D + c) = acc;
            if (c == 0) p.part_lse[pr] = lse2;
        }
    }
}

// One warp per row: its partials' log2 sums give the weights, and the weighted outputs are
// added up in ascending order of the splits (the same bits on every call).
template <int D>
__global__ void __launch_bounds__(128) kv_combine_kernel(const __grid_constant__ RowsParams p) {
    const KvArgs& a = p.a;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)a.n_tokens * a.H_q;
    if (row >= rows) return;
    const int tok = (int)(row / a.H_q), head = (int)(row - (long long)tok * a.H_q);
    if (a.cu && tok >= a.cu[a.B]) return;  // rows behind the last sequence stay as they were
    const int ns = p.p.parts_p + p.p.parts_o;
    float mm = -INFINITY;
    for (int s = lane; s < ns; s += 32) mm = fmaxf(mm, p.part_lse[s * rows + row]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, off));
    constexpr int V = D / 32;  // values per lane
    float acc[V], sum = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    const float ms = mm == -INFINITY ? 0.f : mm;  // (a NaN partial comes through as NaN)
    for (int s = 0; s < ns; ++s) {
        const float w = ex2_approx(p.part_lse[s * rows + row] - ms);
        if (w == 0.f) continue;  // an empty partial has no output either
        sum += w;
        const float* src = p.part_o + (s * rows + row) * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(w, src[e], acc[e]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= inv;
    if (a.out_bf16) {
        uint32_t* dst = reinterpret_cast<uint32_t*>((uint16_t*)a.out + row * D + lane * V);
#pragma unroll
        for (int e = 0; e < V; e += 2) dst[e / 2] = pack_bf16x2(acc[e], acc[e + 1]);
    } else {
        float* dst = (float*)a.out + row * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) dst[e] = acc[e];
    }
    if (lane == 0) {
        long long li;
        if (a.cu) {
            li = (long long)head * a.n_tokens + tok;
        } else {
            const int b = tok / a.max_tokens, t = tok - b * a.max_tokens;
            li = ((long long)b * a.H_q + head) * a.max_tokens + t;
        }
        a.lse[li] = sum == 0.f ? -INFINITY : (ms + log2f(sum)) * 0.69314718055994530942f;
    }
}

template <int D, int MT, bool PAGE16>
cudaError_t launch_rows(const RowsParams& p, unsigned grid) {
    using C = RCfg<D, MT>;
    auto k = kv_rows_kernel<D, MT, PAGE16>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    k<<<grid, kWarps * 32, C::SMEM, p.a.stream>>>(p);
    return cudaGetLastError();
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Keys per split: about `target` blocks in all, no split under 128 keys (four warps of two
// groups), a multiple of 64.
int chunk_for(long long blocks_per_split, int keys, long long target) {
    long long splits = target / (blocks_per_split > 0 ? blocks_per_split : 1);
    if (splits < 1) splits = 1;
    long long chunk = (keys + splits - 1) / splits;
    chunk = (chunk + 63) / 64 * 64;
    return (int)(chunk < 128 ? 128 : chunk);
}

}  // namespace

namespace {

// The tile kernel's share of a plan over `units` (batch rows) x H_kv heads, `tokens` tokens
// and `keys` keys each: row blocks, and the number of key ranges that takes the least time
// by a plain model (a wave of 148 blocks costs a range's key tiles and three more for
// filling and draining; partials are written and read at 5 TB/s).
void plan_tiles(long long units, int H_kv, int group, int tokens, int keys, int D,
                long long part_bytes, bool joined, int& chunk, int& splits, int& blocks,
                int& ksplit, int& parts) {
    const int tpt = 128 / group, tiles = ceil_div(tokens, tpt);
    ksplit = tiles == 1;
    blocks = ksplit ? 1 : ceil_div(tiles, 2);
    const int kt = ceil_div(keys, 128);
    const double tile_us = (D == 128 ? 2.2 : 1.5) * (ksplit ? 0.6 : 1.0);
    double best = 0;
    splits = 0;
    for (int s = 1; s <= kt && s <= 512; ++s) {
        const int per = ceil_div(kt, s);
        if (s > 1 && ceil_div(kt, per) != s) continue;  // the same ranges as fewer splits
        const double waves = (double)ceil_div(units * H_kv * blocks * s, kSms);
        const int np = s * (1 + ksplit);
        const double join = np > 1 || joined ? 2.0 * np * part_bytes / 5e6 : 0.0;
        const double us = waves * (per + 3) * tile_us + join + (np > 1 && !joined ? 3.0 : 0.0);
        if (splits == 0 || us < best) {
            best = us;
            splits = s;
        }
    }
    chunk = ceil_div(kt, splits) * 128;
    parts = splits * (1 + ksplit);
}

}  // namespace

KvPlan plan_kv(int B, int n_tokens, int max_tokens, int max_len, int prefix_len, int H_q,
               int H_kv, int D, int paged, int page_size) {
    KvPlan p = {};
    const int group = H_q / H_kv;
    const long long rows_o = (long long)max_tokens * group, rows_p = (long long)n_tokens * group;
    // the tile kernel takes whole groups of heads, and pages that divide its 128-key tiles
    const bool tiles_ok =
        group <= 128 && (!paged || (page_size >= 8 && (page_size & (page_size - 1)) == 0));
    const long long part_bytes = (long long)n_tokens * H_q * (D + 1) * 4;
    p.kind_p = prefix_len == 0 ? kKvNone : (tiles_ok && rows_p > 32 ? kKvTiles : kKvRows);
    p.kind_o = tiles_ok && rows_o > 32 ? kKvTiles : kKvRows;
    const long long rows_most = p.kind_p == kKvRows && rows_p > rows_o ? rows_p
                                : p.kind_o == kKvRows                  ? rows_o
                                                                       : rows_p;
    p.mt = rows_most > 16 ? 2 : 1;
    const int R = 16 * p.mt;
    if (p.kind_p == kKvRows) {
        p.tiles_p = ceil_div(rows_p, R);
        p.chunk_p = chunk_for((long long)H_kv * p.tiles_p, prefix_len, 4LL * kSms);
        p.splits_p = p.parts_p = ceil_div(prefix_len, p.chunk_p);
    } else if (p.kind_p == kKvTiles) {
        plan_tiles(1, H_kv, group, n_tokens, prefix_len, D, part_bytes, true, p.chunk_p,
                   p.splits_p, p.tiles_p, p.ksplit_p, p.parts_p);
    }
    if (p.kind_o == kKvRows) {
        p.tiles_o = ceil_div(rows_o, R);
        p.chunk_o = chunk_for((long long)B * H_kv * p.tiles_o, max_len, 8LL * kSms);
        p.splits_o = p.parts_o = ceil_div(max_len, p.chunk_o);
    } else {
        plan_tiles(B, H_kv, group, max_tokens, max_len, D, part_bytes, p.kind_p != kKvNone,
                   p.chunk_o, p.splits_o, p.tiles_o, p.ksplit_o, p.parts_o);
    }
    p.direct = p.parts_p + p.parts_o == 1;
    const long long bp = (long long)p.splits_p * H_kv * p.tiles_p,
                    bo = (long long)B * p.splits_o * H_kv * p.tiles_o;
    p.blocks = bp + bo;
    p.workspace = p.direct ? 0 : (p.parts_p + p.parts_o) * part_bytes;
    return p;
}

cudaError_t launch_kv(const KvArgs& a, const KvPlan& plan, unsigned long long wait_limit_ns,
                      const char** why) {
    cudaError_t e = cudaSuccess;
    if (plan.kind_p == kKvTiles || plan.kind_o == kKvTiles) {
        e = launch_kv_tiles(a, plan, wait_limit_ns, why);
        if (e != cudaSuccess) return e;
    }
    RowsParams p;
    p.a = a;
    p.p = plan;
    p.group = a.H_q / a.H_kv;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    const long long rows = (long long)a.n_tokens * a.H_q;
    p.part_o = (float*)a.workspace;
    p.part_lse = p.part_o + (long long)(plan.parts_p + plan.parts_o) * rows * a.D;
    p.items_p = plan.kind_p == kKvRows
                    ? (unsigned)((long long)plan.splits_p * a.H_kv * plan.tiles_p)
                    : 0;
    const unsigned grid =
        p.items_p + (plan.kind_o == kKvRows
                         ? (unsigned)((long long)a.B * plan.splits_o * a.H_kv * plan.tiles_o)
                         : 0);
    if (grid > 0) {
        const bool page16 = !a.tables || a.page_size % kKeys == 0;
        if (a.D == 128) {
            if (plan.mt == 1)
                e = page16 ? launch_rows<128, 1, true>(p, grid) : launch_rows<128, 1, false>(p, grid);
            else
                e = page16 ? launch_rows<128, 2, true>(p, grid) : launch_rows<128, 2, false>(p, grid);
        } else {
            if (plan.mt == 1)
                e = page16 ? launch_rows<64, 1, true>(p, grid) : launch_rows<64, 1, false>(p, grid);
            else
                e = page16 ? launch_rows<64, 2, true>(p, grid) : launch_rows<64, 2, false>(p, grid);
        }
    }
    if (e != cudaSuccess || plan.direct) return e;
    const unsigned cg = (unsigned)((rows + 3) / 4);
    if (a.D == 128) kv_combine_kernel<128><<<cg, 128, 0, a.stream>>>(p);
    else kv_combine_kernel<64><<<cg, 128, 0, a.stream>>>(p);
    return cudaGetLastError();
}

cudaError_t read_and_clear_kv_error(unsigned int* value) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_kv_error_word, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    if (*value) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_kv_error_word, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace ra
