// kv_rows.cuh -- what the kernels for few query rows share: parameters, cp.async and
// mma.sync wrappers, and the softmax state of 16 or 32 rows that a warp carries through its
// groups of keys.
#pragma once
#include <cmath>
#include "kv_internal.h"
#include "sm100_ptx.cuh"

namespace ra {

constexpr int kWarps = 4;
// Keys of a group: 8 KB of K and V either way.  At D = 64 a group of 16 spent as much on the
// softmax's latencies as on its bytes (5.5 TB/s in the long run, against 6.2 at D = 128).
constexpr int group_keys(int D) { return D == 64 ? 32 : 16; }
constexpr float kRescale = 8.0f;  // log2 units: the maximum may lag by 2^8

struct RowsParams {
    KvArgs a;
    KvPlan p;
    int group;
    FastDiv dgroup, dpage, dheads, dtokens;  // by group, page_size, H_q, max_tokens
    float scale_log2;
    float* part_o;    // the tile kernel's partials: [part][token][head][D]
    float* part_lse;  // [part][token][head], log2
    float* slot_o;    // the rows kernel's: [slot][row of the tile][D]
    float* slot_lse;  // [slot][row of the tile], log2
    int2* meta;       // per j: first slot, number of slots
};

// kv_cluster.cu: prefix and own keys by clusters of blocks, without partial results.
cudaError_t launch_kv_cluster(const RowsParams& p);

__device__ __forceinline__ int fdiv(int n, const FastDiv& f) {
    return (int)((__umulhi((uint32_t)n, f.mul) + (uint32_t)n) >> f.shift);
}
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

constexpr int kBlocksPerSm = 2;  // resident, by registers and by the rings' 96 KB

template <int D, int MT>
struct RCfg {
    static constexpr int STAGES = 3;
    static constexpr int KEYS = group_keys(D);
    static constexpr int GROUP_BYTES = KEYS * D * 2;           // K or V of one group
    static constexpr int WARP_BYTES = STAGES * 2 * GROUP_BYTES;
    static constexpr int SMEM = kWarps * WARP_BYTES;
    static constexpr int ROWS = MT * 16;
};

// Byte offset of 16-byte chunk c of row r, chunks permuted within a row so that the eight
// rows of an ldmatrix fall on different banks.
template <int D>
__device__ __forceinline__ uint32_t sw(int r, int c) {
    return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

// A sequence of the batch, or (b = -1) the prefix, as the rows kernels see it.
struct Seq {
    int b, tok0, n_tok, len, groups, tiles;  // groups: key groups of one head and tile
    const int* table;
};

// Where the rows kernel's row tiles of sequence b (first token row: first) start, of each kv
// head's in the batch: b times the most that a sequence has or, packed, by the token rows before
// (a sequence's tiles hold its rows and start at most one tile behind the last one's end), so
// that their number follows the batch's tokens and not B times the longest run.  Sequences
// without tokens need none: min(b, first) of those before have some, at most.
__device__ __forceinline__ int first_tile(const RowsParams& p, int b, int first) {
    const int before = min(b, first);
    return p.p.packed ? first * p.group / (16 * p.p.mt) + before : before * p.p.tiles_o;
}

// A warp's rows: their Q fragments, how far each sees, and the running softmax state.  Lane l
// holds rows l/4 and l/4 + 8 of each 16-row fragment, columns 2 (l % 4) and the next of every 8.
template <int D, int MT>
struct RowState {
    static constexpr int kKeys = group_keys(D), NT = kKeys / 8, H16 = kKeys / 16, R = MT * 16;
    uint32_t qf[MT][D / 16][4];
    int limit[MT][2];  // keys below it are seen
    int min_limit;
    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2], lu[MT][2];

    // Rows R * tile .. of kv head g of sequence s, and an empty state.
    __device__ __forceinline__ void start(const RowsParams& p, const Seq& s, int g, int tile,
                                          bool causal) {
        const KvArgs& a = p.a;
        const int lane = threadIdx.x & 31, r_lo = lane >> 2, c_lo = (lane & 3) * 2;
        min_limit = s.len;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int row = tile * R + mt * 16 + r_lo + 8 * hf;
                const bool ok = row < s.n_tok * p.group;
                const int t = ok ? fdiv(row, p.dgroup) : 0;
                const int head = g * p.group + (ok ? row - t * p.group : 0);
                limit[mt][hf] = ok && causal ? min(s.len, s.len - s.n_tok + t + 1)
                                             : s.len;
                min_limit = min(min_limit, limit[mt][hf]);
                const long long off =
                    (a.cu ? (long long)(s.tok0 + t) * a.q_tstride
                          : (long long)s.b * a.q_bstride + (long long)t * a.q_tstride) +
                    (long long)head * D;
                const uint32_t* q32 =
                    reinterpret_cast<const uint32_t*>((const uint16_t*)a.q + off);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    qf[mt][kk][hf] = ok ? q32[(kk * 16 + c_lo) / 2] : 0u;
                    qf[mt][kk][2 + hf] = ok ? q32[(kk * 16 + c_lo + 8) / 2] : 0u;
                }
                m[mt][hf] = -INFINITY;
                l[mt][hf] = lu[mt][hf] = 0.f;
            }
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
        }
        min_limit = __reduce_min_sync(0xffffffffu, min_limit);
    }

    // One group of keys: scores, softmax, output.  kst, vst: its K and V in shared memory;
    // key0: the first key's index, to be held against the rows' limits.
    __device__ __forceinline__ void attend(const RowsParams& p, uint32_t kst, uint32_t vst,
                                           int key0) {
        const int lane = threadIdx.x & 31, c_lo = (lane & 3) * 2;
        const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: this lane's matrix and row
        // two accumulation chains (even and odd steps of D) of a 16-key group where registers
        // allow: with two warps to a scheduler the products' latency shows
        constexpr int CHAINS = D == 128 && MT == 1 ? 2 : 1;
        float s[MT][NT][4], s_odd[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][n][e] = s_odd[mt][n][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int h = 0; h < H16; ++h) {
                uint32_t kf[4];
                ldsm4(kf, kst + sw<D>(16 * h + (mi >> 1) * 8 + mr, kk * 2 + (mi & 1)));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float(&acc)[NT][4] = CHAINS == 2 && (kk & 1) ? s_odd[mt] : s[mt];
                    mma16816(acc[2 * h], qf[mt][kk], kf[0], kf[1]);
                    mma16816(acc[2 * h + 1], qf[mt][kk], kf[2], kf[3]);
                }
            }
        if (CHAINS == 2)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][n][e] += s_odd[mt][n][e];
        if (key0 + kKeys > min_limit) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (key0 + n * 8 + c_lo + (e & 1) >= limit[mt][e >> 1])
                            s[mt][n][e] = -INFINITY;
        }
        uint32_t pf[MT][H16][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float alpha[2];
            bool grew = false;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float mx = fmaxf(s[mt][0][2 * hf], s[mt][0][2 * hf + 1]);
#pragma unroll
                for (int n = 1; n < NT; ++n) mx = fmax3(mx, s[mt][n][2 * hf], s[mt][n][2 * hf + 1]);
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
                for (int n = 0; n < NT; ++n) {
                    const float p0 = ex2_approx(fmaf(s[mt][n][2 * hf], p.scale_log2, neg));
                    const float p1 = ex2_approx(fmaf(s[mt][n][2 * hf + 1], p.scale_log2, neg));
                    // weights are rounded to bf16 for the tensor cores; l_used sums them as
                    // they are used, so that the weights applied to V add up to one
                    const uint32_t pp = pack_bf16x2(p0, p1);
                    pf[mt][n >> 1][2 * (n & 1) + hf] = pp;
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
        for (int h = 0; h < H16; ++h)
#pragma unroll
            for (int nn = 0; nn < D / 16; ++nn) {
                uint32_t vf[4];
                ldsm4_t(vf, vst + sw<D>(16 * h + (mi & 1) * 8 + mr, nn * 2 + (mi >> 1)));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mma16816(o[mt][2 * nn], pf[mt][h], vf[0], vf[1]);
                    mma16816(o[mt][2 * nn + 1], pf[mt][h], vf[2], vf[3]);
                }
            }
    }
};

}  // namespace ra
