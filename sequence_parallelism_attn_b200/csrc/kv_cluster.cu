// kv_cluster.cu -- attention of few query rows over a moderate number of keys, where the time
// of a call is latency: one kernel, without partial results in memory.
//
// A cluster of up to eight blocks takes one (sequence, kv head), whose rows (32 at most) are
// one row tile.  Its warps share out the groups of the prefix's keys and of the sequence's own,
// each warp with a ring and a softmax state as in kv_rows.cu; a block merges its four states in shared memory, the
// cluster's blocks read one another's merged states through distributed shared memory, each
// for its part of the rows, and write the result.  Every sequence reads the prefix for itself
// (from L2 after the first): with few sequences, or a short prefix, that costs less than the
// 5 us of a second kernel and the scan of the batch that kv_rows.cu needs.  4 sequences of 33
// .. 300 keys behind 1000 (2 kv heads of 64) take 6.2 us, by kv_rows.cu and its combine 9.6.
// With 17 to 32 rows of D = 128 the state and Q need more than the 255 registers: 52 to 80 bytes
// are spilled.
#include "kv_rows.cuh"

namespace ra {

__device__ unsigned int g_kv_cluster_error_word = 0;

namespace {

template <int D, int MT>
struct CCfg : RCfg<D, MT> {
    using B = RCfg<D, MT>;
    static constexpr int PITCH = D + 4;  // floats of a row of a state
    // after the keys: the warps' states [warp][row][PITCH] and sums [warp][row][4] (m, l, lu),
    // then the block's merged state and sums, which the cluster reads
    static constexpr int OFF_SUMS = kWarps * B::ROWS * PITCH * 4;
    static constexpr int OFF_OWN = OFF_SUMS + kWarps * B::ROWS * 16;
    static constexpr int OFF_OWN_SUMS = OFF_OWN + B::ROWS * PITCH * 4;
    static_assert(OFF_OWN_SUMS + B::ROWS * 16 <= B::SMEM, "the states fit in the rings");
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}
__device__ __forceinline__ uint32_t remote(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_remote(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int D, int MT, bool PAGE16>
__global__ void __launch_bounds__(kWarps * 32, 2)
    kv_cluster_kernel(const __grid_constant__ RowsParams p) {
    using C = CCfg<D, MT>;
    constexpr int R = C::ROWS, kKeys = C::KEYS, H16 = kKeys / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    const KvArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), n_ranks = (int)cluster_size();
    const int j = (int)(blockIdx.x / (unsigned)n_ranks), g = j % a.H_kv;

    Seq s;
    s.b = j / a.H_kv;
    const bool reports = rank == 0 && threadIdx.x == 0 && g == 0;
    if (a.cu) {
        const TokenRows rows = token_rows(a.cu, s.b, a.n_tokens, a.max_tokens);
        if (rows.bad && reports) atomicOr(&g_kv_cluster_error_word, kKvErrTokens);
        s.tok0 = rows.first;
        s.n_tok = min(rows.n, a.max_tokens);
    } else {
        s.tok0 = s.b * a.max_tokens;
        s.n_tok = a.max_tokens;
    }
    if (s.n_tok == 0) return;  // the same for the whole cluster
    s.len = a.lens ? max(a.lens[s.b], 0) : a.max_len;
    if (s.len > a.max_len) {
        if (reports) atomicOr(&g_kv_cluster_error_word, kKvErrLength);
        s.len = a.max_len;
    }
    s.table = a.tables ? a.tables + (long long)s.b * a.max_pages : nullptr;
    s.tiles = s.groups = 0;

    // this warp's groups: [lo, lo + cnt) of the prefix's, then the sequence's own
    const int gp = (a.prefix_len + kKeys - 1) / kKeys, go = (s.len + kKeys - 1) / kKeys;
    const int per = (gp + go + kWarps * n_ranks - 1) / (kWarps * n_ranks);
    const int lo = (rank * kWarps + warp) * per;
    const int cnt = max(min(gp + go - lo, per), 0);

    const uint32_t ring = smem_u32(smem) + warp * C::WARP_BYTES;
    int page_reg = 0, page_at = -1;  // lane l: page of 16 keys, number l from group page_at on
    auto look_up = [&](const int* table, int key) -> int {
        int page = table[fdiv(key, p.dpage)];
        if (page < 0 || page >= a.n_pages) {
            atomicOr(&g_kv_cluster_error_word, kKvErrPage);
            page = 0;
        }
        return page;
    };
    auto load = [&](int i) {
        if (i < cnt) {
            const int gi = lo + i;
            const bool pre = gi < gp;
            const int key0 = (pre ? gi : gi - gp) * kKeys, len = pre ? a.prefix_len : s.len;
            const int* table = pre ? a.prefix_table : s.table;
            const uint32_t st = ring + (i % C::STAGES) * 2 * C::GROUP_BYTES;
            if (PAGE16 && s.table && (page_at < 0 || gi - page_at >= 32 / H16)) {
                page_at = gi;
                const int lg = gi + lane / H16;  // the lane's group, and its 16 keys in it
                const bool lp = lg < gp;
                const int key = (lp ? lg : lg - gp) * kKeys + (lane % H16) * 16;
                page_reg = lg < gp + go && key < (lp ? a.prefix_len : s.len)
                               ? look_up(lp ? a.prefix_table : s.table, key)
                               : 0;
            }
            constexpr int CPR = D / 8;     // 16-byte chunks per row
            constexpr int RPI = 32 / CPR;  // rows per instruction
#pragma unroll
            for (int h = 0; h < H16; ++h) {
                const int first = key0 + 16 * h;
                long long base = 0;
                if (PAGE16) {
                    if (s.table) {
                        const int page =
                            __shfl_sync(0xffffffffu, page_reg, (gi - page_at) * H16 + h);
                        base = (long long)page * a.page_stride +
                               (long long)(first - fdiv(first, p.dpage) * a.page_size) * a.kv_tstride;
                    } else {
                        base = (long long)s.b * a.page_stride + (long long)first * a.kv_tstride;
                    }
                    if (first >= len) base = 0;  // no key there: nothing is read
                }
#pragma unroll
                for (int r0 = 0; r0 < 16; r0 += RPI) {
                    const int r = r0 + lane / CPR, c = lane % CPR;
                    const bool ok = first + r < len;  // keys past the end: zeros, not read
                    long long off;
                    if (PAGE16) {
                        off = base + (ok ? (long long)r * a.kv_tstride : 0);
                    } else {
                        const int key = ok ? first + r : key0;
                        off = (long long)look_up(table, key) * a.page_stride +
                              (long long)(key - fdiv(key, p.dpage) * a.page_size) * a.kv_tstride;
                    }
                    off += (long long)g * D + c * 8;
                    const uint32_t dst = st + sw<D>(16 * h + r, c);
                    cp_async16(dst, (const uint16_t*)a.k + off, ok);
                    cp_async16(dst + C::GROUP_BYTES, (const uint16_t*)a.v + off, ok);
                }
            }
        }
        cp_commit();
    };

    RowState<D, MT> r;
    int own_limit[MT][2], own_min = 0;
    bool own = false;
    for (int i = 1 - C::STAGES; i < max(cnt, 1); ++i) {
        if (i == 0) {  // the rows' Q, behind the first loads
            r.start(p, s, g, 0, a.causal);
            own_min = r.min_limit;
            r.min_limit = a.prefix_len;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    own_limit[mt][hf] = r.limit[mt][hf];
                    r.limit[mt][hf] = a.prefix_len;  // all of the prefix is seen
                }
        }
        if (i >= cnt) break;
        if (i >= 0) {
            cp_wait<C::STAGES - 2>();
            __syncwarp();
        }
        load(i + C::STAGES - 1);
        if (i < 0) continue;
        const int gi = lo + i;
        if (!own && gi >= gp) {
            own = true;
            r.min_limit = own_min;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) r.limit[mt][hf] = own_limit[mt][hf];
        }
        const uint32_t kst = ring + (i % C::STAGES) * 2 * C::GROUP_BYTES;
        r.attend(p, kst, kst + C::GROUP_BYTES, (own ? gi - gp : gi) * kKeys);
        __syncwarp();
    }
    cp_wait<0>();
    __syncthreads();

    // ---- the block's four states into one
    float* states = reinterpret_cast<float*>(smem);
    float4* sums = reinterpret_cast<float4*>(smem + C::OFF_SUMS);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int off = 1; off <= 2; off <<= 1) {
                r.l[mt][hf] += __shfl_xor_sync(0xffffffffu, r.l[mt][hf], off);
                r.lu[mt][hf] += __shfl_xor_sync(0xffffffffu, r.lu[mt][hf], off);
            }
            const int row = mt * 16 + (lane >> 2) + 8 * hf;
            float* w = states + (warp * R + row) * C::PITCH + (lane & 3) * 2;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2*>(w + n * 8) =
                    make_float2(r.o[mt][n][2 * hf], r.o[mt][n][2 * hf + 1]);
            if ((lane & 3) == 0)
                sums[warp * R + row] = make_float4(r.m[mt][hf], r.l[mt][hf], r.lu[mt][hf], 0.f);
        }
    __syncthreads();
    constexpr int TPR = D / 4, RPP = kWarps * 32 / TPR;  // threads per row, rows per pass
    const int c4 = threadIdx.x % TPR;
    // (where no state has a finite maximum the sums are 0, or a NaN that has to come through)
    const int rows = s.n_tok * p.group;  // <= R
    for (int row = threadIdx.x / TPR; row < rows; row += RPP) {
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sums[w * R + row].x);
        const float top = mm == -INFINITY ? 0.f : mm;
        float l = 0.f, lu = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 x = sums[w * R + row];
            const float f = ex2_approx(x.x - top);  // 0 for -inf; 0 * NaN stays NaN
            const float4 v = *reinterpret_cast<const float4*>(states + (w * R + row) * C::PITCH +
                                                              c4 * 4);
            l = fmaf(f, x.y, l);
            lu = fmaf(f, x.z, lu);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
        }
        *reinterpret_cast<float4*>(smem + C::OFF_OWN + (row * C::PITCH + c4 * 4) * 4) = acc;
        if (c4 == 0)
            *reinterpret_cast<float4*>(smem + C::OFF_OWN_SUMS + row * 16) =
                make_float4(mm, l, lu, 0.f);
    }
    __syncwarp();
    cluster_sync();

    // ---- the cluster's states into the result: each block takes its part of the rows
    const uint32_t own_at = smem_u32(smem) + C::OFF_OWN, sums_at = smem_u32(smem) + C::OFF_OWN_SUMS;
    for (int row = rank * RPP + threadIdx.x / TPR; row < rows; row += n_ranks * RPP) {
        float mm = -INFINITY;
        for (int q = 0; q < n_ranks; ++q)
            mm = fmaxf(mm, ld_remote(remote(sums_at + row * 16, q)).x);
        const float top = mm == -INFINITY ? 0.f : mm;
        float l = 0.f, lu = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = 0; q < n_ranks; ++q) {
            const float4 x = ld_remote(remote(sums_at + row * 16, q));
            const float4 v = ld_remote(remote(own_at + (row * C::PITCH + c4 * 4) * 4, q));
            const float f = ex2_approx(x.x - top);
            l = fmaf(f, x.y, l);
            lu = fmaf(f, x.z, lu);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
        }
        const float inv = lu == 0.f ? 0.f : 1.f / lu;
        const int t = fdiv(row, p.dgroup), head = g * p.group + row - t * p.group;
        const long long orow = (long long)(s.tok0 + t) * a.H_q + head;
        if (a.out_bf16)
            *reinterpret_cast<uint2*>((uint16_t*)a.out + orow * D + c4 * 4) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                           pack_bf16x2(acc.z * inv, acc.w * inv));
        else
            *reinterpret_cast<float4*>((float*)a.out + orow * D + c4 * 4) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (c4 == 0) {
            const long long li = a.cu ? (long long)head * a.n_tokens + s.tok0 + t
                                      : ((long long)s.b * a.H_q + head) * a.max_tokens + t;
            a.lse[li] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994530942f;
        }
    }
    __syncwarp();
    cluster_sync();  // no block ends while another reads its state
}

template <int D, int MT, bool PAGE16>
cudaError_t launch(const RowsParams& p) {
    auto k = kv_cluster_kernel<D, MT, PAGE16>;
    constexpr int smem = RCfg<D, MT>::SMEM;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.p.blocks);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = p.a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.p.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, p);
}

}  // namespace

cudaError_t launch_kv_cluster(const RowsParams& p) {
    const bool page16 = !p.a.tables || p.a.page_size % 16 == 0;
    if (p.a.D == 128) {
        if (p.p.mt == 1) return page16 ? launch<128, 1, true>(p) : launch<128, 1, false>(p);
        return page16 ? launch<128, 2, true>(p) : launch<128, 2, false>(p);
    }
    if (p.p.mt == 1) return page16 ? launch<64, 1, true>(p) : launch<64, 1, false>(p);
    return page16 ? launch<64, 2, true>(p) : launch<64, 2, false>(p);
}

cudaError_t read_and_clear_kv_cluster_error(unsigned int* value) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_kv_cluster_error_word, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    if (*value) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_kv_cluster_error_word, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace ra
