// kv_rows.cu -- attention of few query rows over many keys: the single-token form of the
// paged, prefix and cross attention, and the joining of every form's partial results.
//
// Work is counted in groups of 16 keys (32 at D = 64) of (sequence, kv head, row tile) -- row
// tiles of 16 or 32 rows, tokens x the query heads that share the kv head -- laid end to end:
// the prefix first (rows of the whole batch, so its keys are read once), then every
// sequence's own keys.  The resident warps (four to a block, two blocks to an SM) each take an
// equal stretch of that line, whatever the sequences' lengths, and run it as one stream: a
// ring of cp.async stages that is filled across the borders between heads and sequences, and
// a softmax state (maximum m, sum l, output O, all fp32) that is written out as a partial
// result at each border.  No warp waits for another.  A first form with a block per key range
// and a merge of its four warps' states took 82 us where this takes 74 (12 sequences of 1001
// .. 16384 keys, 8 kv heads of 128, 427 MB): its blocks spent some 4 us each on starting,
// filling and merging.
//
// Up to four neighbouring kv heads are walked side by side by as many warps (each head's row
// of a token is 128 or 256 bytes; apart, 16 heads of 64 were read at 5.4 TB/s over 786 MB,
// side by side at 6.2).  Walker w's piece of the j-th (sequence, heads, tile) is partial slot
// w + j of each head (along the line one of the two grows at every border, so no slot is used
// twice), and the pieces of one j lie next to each other; the warp that has its first key
// notes where and how many.
//
// What bounds it: 16 rows need 4 D flops per key against 4 D bytes of K and V, far below the
// machine's balance, so it runs at the rate at which K and V arrive (6.2 TB/s over 786 MB).  The
// keys of the prefix are read once for each tile of 16 or 32 of the batch's rows.  A tile of 32
// rows of D = 128 needs more than the 255 registers: 114 to 142 bytes are spilled.
// Hence mma.sync on 16-row fragments (a tcgen05 tile has at least 64 rows) and the deep
// per-warp rings.
#include <cmath>
#include <cstring>
#include "kv_rows.cuh"

namespace ra {

__device__ unsigned int g_kv_error_word = 0;

namespace {

template <int R, int KEYS>
__device__ __forceinline__ Seq get_seq(const RowsParams& p, int b) {
    const KvArgs& a = p.a;
    Seq s;
    s.b = b;
    if (b < 0) {
        s.tok0 = 0;
        s.n_tok = a.cu ? min(a.cu[a.B], a.n_tokens) : a.n_tokens;
        s.len = p.p.kind_p == kKvRows ? a.prefix_len : 0;
        s.table = a.prefix_table;
    } else {
        if (a.cu) {
            const TokenRows rows = token_rows(a.cu, b, a.n_tokens, a.max_tokens);
            s.tok0 = rows.first;
            s.n_tok = min(rows.n, a.max_tokens);
            if (p.p.few && rows.n > p.p.few) s.n_tok = 0;  // the tile kernel's
        } else {
            s.tok0 = b * a.max_tokens;
            s.n_tok = a.max_tokens;
        }
        s.len = a.lens ? min(max(a.lens[b], 0), a.max_len) : a.max_len;
        s.table = a.tables ? a.tables + (long long)b * a.max_pages : nullptr;
    }
    s.groups = (s.len + KEYS - 1) / KEYS;
    s.tiles = s.n_tok > 0 ? (s.n_tok * p.group + R - 1) / R : 0;
    return s;
}

// A place on the line: a key group of a (sequence, head, tile).
struct Place {
    Seq s;
    int g, tile, key;  // key: group index
};

template <int R, int KEYS>
__device__ __forceinline__ void next_piece(const RowsParams& p, Place& x) {
    x.key = 0;
    if (++x.tile < x.s.tiles) return;
    x.tile = 0;
    if (++x.g < (p.a.H_kv >> p.p.heads_log)) return;
    x.g = 0;
    do {
        x.s = get_seq<R, KEYS>(p, x.s.b + 1);
    } while (x.s.groups * x.s.tiles == 0 && x.s.b + 1 < p.a.B);
}

// PAGE16: a page holds whole runs of 16 keys (or the keys are dense); else every key is looked
// up by itself.
template <int D, int MT, bool PAGE16>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm)
    kv_rows_kernel(const __grid_constant__ RowsParams p) {
    using C = RCfg<D, MT>;
    constexpr int R = C::ROWS, kKeys = C::KEYS, H16 = kKeys / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    const KvArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // 2^hl neighbouring warps walk the line together, each for one of as many neighbouring
    // kv heads: a token's heads lie side by side in memory and are then read side by side
    const int hl = p.p.heads_log, hs = warp & ((1 << hl) - 1);
    const int wid = (int)(blockIdx.x * kWarps + warp) >> hl;
    const int n_warps = (int)(gridDim.x * kWarps) >> hl;

    // ---- this warp's stretch of the line: [f0, f0 + cnt).  Every warp adds up the batch for
    // itself (entry 0 the prefix, entry e sequence e - 1), then looks for the entry that its
    // stretch starts in.
    // (the host has checked that the whole line is shorter than 2^31 groups)
    Place x;
    int cnt = 0;
    auto weight = [&](int e) -> unsigned {
        if (e > a.B) return 0;
        const Seq s = get_seq<R, C::KEYS>(p, e - 1);
        return (unsigned)(s.groups * s.tiles * (a.H_kv >> hl));
    };
    unsigned w = weight(lane), total = w;
#pragma unroll 4
    for (int e0 = 32; e0 <= a.B; e0 += 32) total += weight(e0 + lane);
    total = __reduce_add_sync(0xffffffffu, total);
    const unsigned per =
        max((total + n_warps - 1) / n_warps, (unsigned)p.p.min_groups);
    const unsigned f0 = per * wid;
    // (a stretch that starts past the end is empty; the product may wrap there)
    if (wid < (int)((total + per - 1) / per)) {
        cnt = (int)min(per, total - f0);
        unsigned at = 0;
#pragma unroll 1
        for (int e0 = 0; e0 <= a.B; e0 += 32) {
            if (e0 > 0) w = weight(e0 + lane);
            unsigned incl = w;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            const unsigned sum = __shfl_sync(0xffffffffu, incl, 31);
            if (at + sum > f0) {
                const int l = __ffs(__ballot_sync(0xffffffffu, at + incl > f0)) - 1;
                const unsigned rel = f0 - at - __shfl_sync(0xffffffffu, incl - w, l);
                x.s = get_seq<R, C::KEYS>(p, e0 + l - 1);
                const unsigned piece = rel / (unsigned)x.s.groups;
                x.key = (int)(rel - piece * (unsigned)x.s.groups);
                x.g = (int)(piece / (unsigned)x.s.tiles);
                x.tile = (int)piece - x.g * x.s.tiles;
                break;
            }
            at += sum;
        }
    }
    if (cnt == 0) {
        if (blockIdx.x == 0) pdl_wait();
        return;
    }

    // ---- the loads run ahead of the products on a place of their own
    const uint32_t ring = smem_u32(smem) + warp * C::WARP_BYTES;
    Place y = x;
    int page_reg = 0, page_at = -1;  // lane l: page of the piece's 16 keys number page_at + l
    auto look_up = [&](const int* table, int key) -> int {
        int page = table[fdiv(key, p.dpage)];
        if (page < 0 || page >= a.n_pages) {
            atomicOr(&g_kv_error_word, kKvErrPage);
            page = 0;
        }
        return page;
    };
    auto load = [&](int i) {
        if (i < cnt) {
            const int key0 = y.key * kKeys;
            const uint32_t st = ring + (i % C::STAGES) * 2 * C::GROUP_BYTES;
            if (PAGE16 && y.s.table && (page_at < 0 || y.key * H16 - page_at >= 32)) {
                page_at = y.key * H16;
                const int key = (page_at + lane) * 16;
                page_reg = key < y.s.len ? look_up(y.s.table, key) : 0;
            }
            constexpr int CPR = D / 8;     // 16-byte chunks per row
            constexpr int RPI = 32 / CPR;  // rows per instruction
#pragma unroll
            for (int h = 0; h < H16; ++h) {
                const int first = key0 + 16 * h;
                long long base = 0;
                if (PAGE16) {
                    if (y.s.table) {
                        const int page =
                            __shfl_sync(0xffffffffu, page_reg, y.key * H16 + h - page_at);
                        base = (long long)page * a.page_stride +
                               (long long)(first - fdiv(first, p.dpage) * a.page_size) * a.kv_tstride;
                    } else {
                        base = (long long)y.s.b * a.page_stride + (long long)first * a.kv_tstride;
                    }
                    if (first >= y.s.len) base = 0;  // no key there: nothing is read
                }
#pragma unroll
                for (int r0 = 0; r0 < 16; r0 += RPI) {
                    const int r = r0 + lane / CPR, c = lane % CPR;
                    const bool ok = first + r < y.s.len;  // keys past the end: zeros, not read
                    long long off;
                    if (PAGE16) {
                        off = base + (ok ? (long long)r * a.kv_tstride : 0);
                    } else {
                        const int key = ok ? first + r : key0;
                        off = (long long)look_up(y.s.table, key) * a.page_stride +
                              (long long)(key - fdiv(key, p.dpage) * a.page_size) * a.kv_tstride;
                    }
                    off += (long long)((y.g << hl) + hs) * D + c * 8;
                    const uint32_t dst = st + sw<D>(16 * h + r, c);
                    cp_async16(dst, (const uint16_t*)a.k + off, ok);
                    cp_async16(dst + C::GROUP_BYTES, (const uint16_t*)a.v + off, ok);
                }
            }
            if (++y.key == y.s.groups && i + 1 < cnt) {
                next_piece<R, C::KEYS>(p, y);
                page_at = -1;
            }
        }
        cp_commit();
    };
    RowState<D, MT> r;
    bool fresh = true;
    // the slot of the piece that x is in: a share of the slots to each of the warp group's heads
    auto slot_of = [&]() {
        const int jq = x.s.b < 0 ? x.g * p.p.tiles_p + x.tile
                                 : (p.p.j_own >> hl) +
                                       first_tile(p, x.s.b, x.s.tok0) * (a.H_kv >> hl) +
                                       x.g * x.s.tiles + x.tile;
        return hs * ((int)p.p.slots >> hl) + wid + jq;
    };
    for (int i = 1 - C::STAGES; i < cnt; ++i) {
        // (the first steps, below 0, only fill the ring)
        if (i >= 0 && fresh) {  // a new piece: its Q fragments, an empty state
            fresh = false;
            r.start(p, x.s, (x.g << hl) + hs, x.tile, a.causal && x.s.b >= 0);
            if (x.key == 0 && lane == 0) {  // the piece that starts this j: note its slots
                const unsigned last = (f0 + i + x.s.groups - 1) / per;
                const int g = (x.g << hl) + hs;
                const int j = x.s.b < 0 ? g * p.p.tiles_p + x.tile
                                        : p.p.j_own + first_tile(p, x.s.b, x.s.tok0) * a.H_kv +
                                              g * x.s.tiles + x.tile;
                p.meta[j] = make_int2(slot_of(), (int)last - wid + 1);
            }
        }
        if (i >= 0) {
            cp_wait<C::STAGES - 2>();
            __syncwarp();
        }
        load(i + C::STAGES - 1);
        if (i < 0) continue;
        const uint32_t kst = ring + (i % C::STAGES) * 2 * C::GROUP_BYTES;
        const uint32_t vst = kst + C::GROUP_BYTES;
        r.attend(p, kst, vst, x.key * kKeys);
        // ---- the piece's end: its partial result
        const bool border = x.key + 1 == x.s.groups;
        if (border || i + 1 == cnt) {
            const long long slot = (long long)slot_of() * R;
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
                    if (x.tile * R + row < x.s.n_tok * p.group) {
                        // no key seen: every m is -inf and every sum 0 (a NaN score leaves m
                        // as it was but makes the sums NaN, which must come through)
                        const float lr = r.l[mt][hf], mr = r.m[mt][hf];
                        const float inv = r.lu[mt][hf] == 0.f ? 0.f : 1.f / r.lu[mt][hf];
                        float* dst = p.slot_o + (slot + row) * D + (lane & 3) * 2;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
                            *reinterpret_cast<float2*>(dst + n * 8) =
                                make_float2(r.o[mt][n][2 * hf] * inv, r.o[mt][n][2 * hf + 1] * inv);
                        if ((lane & 3) == 0)
                            p.slot_lse[slot + row] =
                                lr == 0.f ? -INFINITY
                                          : (mr == -INFINITY ? 0.f : mr) + log2f(lr);
                    }
                }
            fresh = true;
        }
        ++x.key;
        if (border && i + 1 < cnt) next_piece<R, C::KEYS>(p, x);
        __syncwarp();
    }
    pdl_launch_dependents();
    // one block stays until the tile kernel has ended, so that the end of this grid means
    // the end of both; the others make room for the blocks that have not started yet
    if (blockIdx.x == 0) pdl_wait();
}

// One warp per row: its partials' log2 sums give the weights, one lane each, and the
// weighted outputs are added up in the splits' order (the same bits on every call), 16 bytes
// a lane: whole rows of D = 128, two partials at a time of D = 64.  It lives on latency (a
// row's partials are some KB in L2), so eight partials' loads are in flight at once.  Where
// few rows have many partials each (WPR = 8), a block's eight warps share a row's partials
// and merge their sums: 2 sequences of 16 rows behind 11705 keys, 366 partials to a row,
// took 55 us with one warp to a row.  SEARCH: a row's sequence is found by a search 32 ways at
// a time: of a mixed batch, whose rows belong to the rows kernel or to the tile kernel by their
// sequence's tokens, and of a ragged one, where B x the most tokens are far more than the rows.
template <int D, int WPR, bool SEARCH>
__global__ void __launch_bounds__(256) kv_combine_kernel(const __grid_constant__ RowsParams p) {
    const KvArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int idx = WPR == 8 ? (int)blockIdx.x : (int)blockIdx.x * 8 + warp;  // < 2^31 + 8
    const long long rows = (long long)a.n_tokens * a.H_q;
    const int R = 16 * p.p.mt;
    // the row: by token, or by (sequence, its token) where the rows kernel took the own keys
    const int i_tok = fdiv(idx, p.dheads), head = idx - i_tok * a.H_q;
    int b = 0, t = 0, tok = i_tok;
    bool live;
    // rows before the first sequence's and from the last one's end on stay as they are
    const int begin = a.cu ? max(a.cu[0], 0) : 0;
    const int end = a.cu ? min(a.cu[a.B], a.n_tokens) : a.n_tokens;
    bool few = !SEARCH && p.p.kind_o == kKvRows;  // the own keys are the rows kernel's
    int n_tok = a.max_tokens, first_tok = tok;    // (few) the sequence's tokens, its first row
    if (SEARCH) {
        if (!p.p.few && blockIdx.x == 0 && warp == 0)  // (a mixed batch: the tile kernel reports)
            for (int e = lane; e < a.B; e += 32)
                if (token_rows(a.cu, e, a.n_tokens, a.max_tokens).bad)
                    atomicOr(&g_kv_error_word, kKvErrTokens);
        live = tok >= begin && tok < end;
        if (live) {
            b = find_sequence(a.cu, a.B, tok);
            const TokenRows rows_b = token_rows(a.cu, b, a.n_tokens, a.max_tokens);
            first_tok = rows_b.first;
            n_tok = min(rows_b.n, a.max_tokens);
            t = tok - first_tok;
            few = !p.p.few || rows_b.n <= p.p.few;
            live = t >= 0 && t < n_tok && (few || !p.p.direct);
        }
    } else if (p.p.kind_o == kKvRows) {
        b = fdiv(i_tok, p.dtokens);
        t = i_tok - b * a.max_tokens;
        live = b < a.B;
        if (live && a.cu) {
            const TokenRows rows_b = token_rows(a.cu, b, a.n_tokens, a.max_tokens);
            if (rows_b.bad && t == 0 && head == 0 && lane == 0)
                atomicOr(&g_kv_error_word, kKvErrTokens);
            first_tok = rows_b.first;
            n_tok = min(rows_b.n, a.max_tokens);
            tok = first_tok + t;
            live = t < rows_b.n && tok < end;
        } else {
            first_tok = b * a.max_tokens;
        }
    } else {
        live = tok >= begin && tok < end;
    }
    if (!live) {
        pdl_wait();  // the end of this grid has to mean the end of those before it
        return;
    }
    const long long row = (long long)tok * a.H_q + head;
    const int g = fdiv(head, p.dgroup), hh = head - g * p.group;
    // two runs of partials: the prefix's, then the own keys'
    int n1 = 0, n2 = 0;
    const float *o1 = nullptr, *o2 = nullptr, *l1 = nullptr, *l2 = nullptr;
    long long s1 = rows, s2 = rows;  // rows between a run's partials
    int len = 0;
    if (few) {
        len = a.lens ? a.lens[b] : a.max_len;
        if (len > a.max_len && t == 0 && head == 0 && lane == 0)
            atomicOr(&g_kv_error_word, kKvErrLength);
    }
    pdl_wait();
    auto slots_of = [&](int j) {  // in bounds even if the batch changed under the call
        int2 x = p.meta[j];
        x.x = min(max(x.x, 0), (int)p.p.slots - 1);
        x.y = min(max(x.y, 0), (int)p.p.slots - x.x);
        return x;
    };
    if (p.p.kind_p == kKvTiles) {
        n1 = p.p.parts_p;
        o1 = p.part_o + row * D;
        l1 = p.part_lse + row;
    } else if (p.p.kind_p == kKvRows) {
        const int r = tok * p.group + hh;
        const int2 mt = slots_of(g * p.p.tiles_p + r / R);
        n1 = mt.y;
        s1 = R;
        o1 = p.slot_o + ((long long)mt.x * R + r % R) * D;
        l1 = p.slot_lse + (long long)mt.x * R + r % R;
    }
    if (!few) {
        n2 = p.p.parts_o;
        o2 = p.part_o + (p.p.parts_p * rows + row) * D;
        l2 = p.part_lse + p.p.parts_p * rows + row;
    } else if (len > 0) {
        const int r = t * p.group + hh;
        const int2 mt = slots_of(p.p.j_own + first_tile(p, b, first_tok) * a.H_kv +
                                 g * ((n_tok * p.group + R - 1) / R) + r / R);
        n2 = mt.y;
        s2 = R;
        o2 = p.slot_o + ((long long)mt.x * R + r % R) * D;
        l2 = p.slot_lse + (long long)mt.x * R + r % R;
    }
    // this warp's partials: [from, ns)
    const int all = n1 + n2, share = (all + WPR - 1) / WPR;
    const int from = WPR == 8 ? warp * share : 0, ns = WPR == 8 ? min(from + share, all) : all;
    auto lse_of = [&](int s) { return s < n1 ? l1[s * s1] : l2[(s - n1) * s2]; };
    const float first = from + lane < ns ? lse_of(from + lane) : -INFINITY;
    float mm = first;
    for (int s = from + lane + 32; s < ns; s += 32) mm = fmaxf(mm, lse_of(s));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, off));
    const float ms = mm == -INFINITY ? 0.f : mm;  // (a NaN partial comes through as NaN)
    constexpr int LPR = D / 4;    // lanes of a row
    constexpr int PAR = 32 / LPR;  // partials at a time
    const int sub = lane / LPR, c = (lane % LPR) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int base = from; base < ns; base += 32) {
        const float x = base == from ? first
                        : base + lane < ns ? lse_of(base + lane) : -INFINITY;
        const float w = ex2_approx(x - ms);
        sum += w;
        const int m = min(32, ns - base);
        for (int j = 0; j < m; j += 8 * PAR) {
            float wj[8];
            float4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int k = j + u * PAR + sub;
                wj[u] = __shfl_sync(0xffffffffu, w, k & 31);
                if (k >= m) wj[u] = 0.f;
                v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (wj[u] != 0.f) {  // an empty partial adds nothing
                    const int q = base + k;
                    v[u] = *reinterpret_cast<const float4*>(
                        (q < n1 ? o1 + q * s1 * D : o2 + (q - n1) * s2 * D) + c);
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                acc.x = fmaf(wj[u], v[u].x, acc.x);
                acc.y = fmaf(wj[u], v[u].y, acc.y);
                acc.z = fmaf(wj[u], v[u].z, acc.z);
                acc.w = fmaf(wj[u], v[u].w, acc.w);
            }
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (PAR == 2) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
    }
    float top = ms;  // what the weights are relative to
    if (WPR == 8) {
        __shared__ float4 s_acc[8][LPR];
        __shared__ float s_m[8], s_sum[8];
        if (sub == 0) s_acc[warp][c / 4] = acc;
        if (lane == 0) {
            s_m[warp] = mm;
            s_sum[warp] = sum;
        }
        __syncthreads();
        if (warp > 0) return;
        float m8 = s_m[0];
#pragma unroll
        for (int w = 1; w < 8; ++w) m8 = fmaxf(m8, s_m[w]);
        top = m8 == -INFINITY ? 0.f : m8;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            // a warp without a finite maximum summed relative to 0 (nothing, or a NaN)
            const float f = s_m[w] == -INFINITY ? 1.f : ex2_approx(s_m[w] - top);
            const float4 v = s_acc[w][c / 4];
            sum = fmaf(f, s_sum[w], sum);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (sub == 0) {
        if (a.out_bf16)
            *reinterpret_cast<uint2*>((uint16_t*)a.out + row * D + c) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                           pack_bf16x2(acc.z * inv, acc.w * inv));
        else
            *reinterpret_cast<float4*>((float*)a.out + row * D + c) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    if (lane == 0) {
        long long li;
        if (a.cu) {
            li = (long long)head * a.n_tokens + tok;
        } else {
            const int bb = fdiv(tok, p.dtokens), tt = tok - bb * a.max_tokens;
            li = ((long long)bb * a.H_q + head) * a.max_tokens + tt;
        }
        a.lse[li] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
    }
}

// Launches the second or a later kernel of a call: with `overlap` its blocks may start once
// the kernel before it has no block left to start (programmatic dependent launch).  The rows
// kernel reads nothing that the tile kernel writes, and waits for it only before it ends;
// the combine waits before it reads.
template <typename K>
cudaError_t launch_pdl(K kernel, const RowsParams& p, unsigned grid, int threads, int smem,
                       cudaStream_t stream, bool overlap) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int MT, bool PAGE16>
cudaError_t launch_rows(const RowsParams& p, unsigned grid, bool after_tiles) {
    using C = RCfg<D, MT>;
    auto k = kv_rows_kernel<D, MT, PAGE16>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, p, grid, kWarps * 32, C::SMEM, p.a.stream, after_tiles);
}

template <int D>
auto pick_combine(const KvPlan& p) {
    if (p.search)
        return p.wide_combine ? kv_combine_kernel<D, 8, true> : kv_combine_kernel<D, 1, true>;
    return p.wide_combine ? kv_combine_kernel<D, 8, false> : kv_combine_kernel<D, 1, false>;
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// The tile kernel's share of a plan over `units` (batch rows) x H_kv heads, `tokens` tokens
// (`all_tokens` in all where the units differ, else 0) and `keys` keys each: row blocks, and the
// length of a key range, by a plain model.
//   - A block costs its key tiles and three more for filling and draining, at tile_us each.
//   - A row block's keys are cut into ranges of `per` tiles and a shorter last one; the full
//     ranges come first in the grid, so the short ones fill up the SMs that a last wave of
//     full ones leaves idle (128 row blocks of 128 key tiles on 148 SMs: 113 + 15 tiles
//     instead of 128).
//   - Partials are written and read at 5 TB/s.
//   - rows_bytes: what the rows kernel reads beside it.  Its blocks start on every SM that
//     the tile kernel leaves free, at some 45 GB/s of keys to an SM, and take the others as
//     they become free; so where the tile kernel fits in less than a wave, fewer and longer
//     ranges can be the better choice.
void plan_tiles(long long units, int H_kv, int group, int tokens, int all_tokens, int keys, int D,
                long long part_bytes, bool joined, double rows_bytes, int& chunk, int& splits,
                int& blocks, int& ksplit, int& parts) {
    const int tpt = 128 / group, tiles = ceil_div(tokens, tpt);
    ksplit = tiles == 1;
    blocks = ksplit ? 1 : ceil_div(tiles, 2);
    const int kt = ceil_div(keys, 128);
    const long long items = all_tokens ? (long long)H_kv * ceil_div(all_tokens, ksplit ? tpt : 2 * tpt)
                                       : units * H_kv * blocks;
    // (a row tile's empty warps cost nothing, a half-empty block still its MMAs)
    const double fill = all_tokens ? 1.0 : (double)tokens * group / (256.0 * blocks);
    const double tile_us = (D == 128 ? 2.2 : 1.8) * (ksplit ? 0.6 : 0.6 + 0.4 * fill);
    const double rows_sm_us = rows_bytes / 45e3;
    double best = 0;
    int best_per = 0;
    auto consider = [&](int per) {
        const int s = ceil_div(kt, per), rest = kt - (s - 1) * per;
        const long long longs = items * (rest == per ? s : s - 1), q = longs / kSms,
                        r = longs % kSms;
        const long long shorts = rest == per ? 0 : items;
        const int cl = per + 3, cs = rest + 3;
        // full ranges wave by wave, then the short ones on the SMs that are free first
        double end = (double)(q + (r > 0)) * cl;
        if (shorts > 0) {
            const long long idle = kSms - r, fit = idle * (r > 0 ? cl / cs : 0);
            const long long over = shorts - fit;
            if (over > 0) end += (double)ceil_div(over, kSms) * cs;
        }
        const double us = end * tile_us;
        const double busy = ((double)longs * cl + (double)shorts * cs) * tile_us;
        const double left = rows_sm_us - (us * kSms - busy);
        const int np = s * (1 + ksplit);
        const double join = np > 1 || joined ? 2.0 * np * part_bytes / 5e6 : 0.0;
        const double all = us + (left > 0 ? left / kSms : 0.0) + join +
                           (np > 1 && !joined ? 3.0 : 0.0);
        if (best_per == 0 || all < best) {
            best = all;
            best_per = per;
        }
    };
    const long long most = 4LL * kSms / items > 64 ? 4LL * kSms / items : 64;
    for (int s = 1; s <= kt && s <= most; ++s) consider(ceil_div(kt, s));
    const int step = kt / 64 + 1;
    for (int per = kt - 1; per > kt / 2; per -= step) consider(per);
    splits = ceil_div(kt, best_per);
    chunk = best_per * 128;
    parts = splits * (1 + ksplit);
}

// Whether clusters of blocks take the call: every (sequence, kv head) one, as many blocks to
// each as run beside one another (two an SM, up to the portable eight; a cluster's blocks share
// one of the GPCs of some 18 SMs, so 28 clusters of eight fit, not 37).  Measured, us, for J
// (sequence, head) pairs of D = 128 with equal lengths, clusters against rows + combine:
//   J = 2:  2048 keys 7.0, 8.9    8192 keys 14.4, 11.7
//   J = 64: 512 keys 7.2, 9.3     2048 keys 15.8, 17.7     8192 keys 44, 50
// which is about 4.5 + the larger of 0.62 a group of a warp and the keys at 6.2 TB/s, against
// 8.5 + the keys at 6 TB/s.  The cluster's time is that of the longest sequence, the rows
// kernel's that of the whole batch (whose lengths are not known here: 0.75 of their bound), and
// only the clusters read the prefix anew for every sequence.
bool plan_cluster(int B, long long rows, bool tiles_p, int max_len, int prefix_len, int H_kv, int D,
                  KvPlan& p) {
    const long long js = (long long)B * H_kv;
    int c = 8;
    while (c > 1 && js * c > (c == 8 ? 224 : c == 4 ? 272 : kBlocksPerSm * kSms)) c /= 2;
    if (js * c > kBlocksPerSm * kSms) return false;
    const long long go = ceil_div(max_len, group_keys(D)), gp = ceil_div(prefix_len, group_keys(D));
    const double mb = 8192e-6;  // of a group
    const double steps = 0.62 * ceil_div(go + gp, kWarps * c), read = js * (go + gp) * mb / 6.2;
    const double cluster = 4.5 + (steps > read ? steps : read);
    const double other = 8.5 + 0.75 * js * go * mb / 6.0 + H_kv * gp * mb / 6.0 +
                         (tiles_p ? 4.0 : 0.0);  // the tile kernel beside, for the prefix
    if (cluster > other) return false;
    p = KvPlan{};
    p.kind_o = kKvCluster;
    p.mt = rows > 16 ? 2 : 1;
    p.cluster = c;
    p.direct = 1;
    p.blocks = js * c;
    return true;
}

KvPlan make_plan(int B, int n_tokens, int max_tokens, int max_len, int prefix_len, int H_q,
                 int H_kv, int D, int paged, int page_size) {
    KvPlan p = {};
    const int group = H_q / H_kv;
    const long long rows_o = (long long)max_tokens * group, rows_p = (long long)n_tokens * group;
    // the tile kernel takes whole groups of heads, and pages that divide its 128-key tiles
    const bool tiles_ok =
        group <= 128 && (!paged || (page_size >= 8 && (page_size & (page_size - 1)) == 0));
    // The most rows to leave to mma.sync: 32, but over many keys at D = 128 only 16, where the
    // second fragment's products, softmax and spilled registers (some 130 bytes a thread) are the
    // bound.  Measured, us on the GPU, 8 tokens of 4 heads to a kv head (8 of 128), rows kernel or
    // clusters against the tile kernel:
    //   keys           300         600         1024        1500        2000
    //   1 sequence     10.4, 12.4  12.4, 12.5  12.5, 12.5  14.5, 14.5  16.4, 16.6
    //   8 sequences    16.5, 14.5  16.6, 15.3  18.6, 16.6  22.7, 18.6  26.8, 20.7
    //   32 sequences   22.7, 28.9  31.7, 35.0  60.1, 43.5  74.5, 55.4  88.5, 65.6
    // (8000 keys, calls: 23.7, 17.1;  77.7, 48.6;  234, 199) and 4 sequences of 8 rows behind a
    // prefix: 8000 keys 25.0, 18.8    64000 keys 75.5, 55.0.  Below 1024 keys neither is the
    // better for all batches: the rule goes by the keys alone, and 8 sequences of 300 lose 2 us.
    // At D = 64 (4 tokens of 8 heads to a kv head, 4 of them) 32 sequences over 8000 keys 63, 87.
    auto most_rows = [&](int keys) { return tiles_ok && D == 128 && keys >= 1024 ? 16 : 32; };
    const bool many = rows_o > most_rows(max_len);
    if (!many && rows_o <= 32 &&
        plan_cluster(B, rows_o, prefix_len > 0 && rows_p > most_rows(prefix_len), max_len,
                     prefix_len, H_kv, D, p))
        return p;
    const long long part_bytes = (long long)n_tokens * H_q * (D + 1) * 4;
    p.kind_p = prefix_len == 0                                             ? kKvNone
               : tiles_ok && (many || rows_p > most_rows(prefix_len)) ? kKvTiles
                                                                           : kKvRows;
    p.kind_o = tiles_ok && many ? kKvTiles : kKvRows;
    // A step of a serving loop may hold tokens of running sequences and a new prompt: where a
    // sequence has at most 0.6 of the most tokens on average, those with few go to the rows
    // kernel (16 rows, a fragment's; 32 where a token alone has more than 16), the others to
    // the tile kernel, whose grid is then the row blocks that n_tokens can make, not B times
    // the most.  Measured, us, tile kernel alone against both (32 / 8 heads of 128):
    //   63 single tokens over 4096 keys, a prompt of 1000: 308, 200    1 and 500: 64, 36
    //   255 single tokens over 500 keys, one of 2000: 745, 197
    //   300, 200, 100 and 50 over 300 .. 2000 keys (0.54 of the most): 56, 55
    //   32 of 9, 8, 7, 1 in turn over 2000 (0.69): 60, 74    16 of 100 and 200 (0.75): 102, 134
    // With more than 32 heads to a kv head a single token is the tile kernel's too: it takes all,
    // packed (255 single tokens over 500 keys and one of 2000, 64 heads on one of
    // 128: 1129 us by B times the most blocks, packed 168).
    const int few = group <= 16 ? 16 / group : 32 / group;
    bool packed = false;
    if (p.kind_o == kKvTiles && paged && few < max_tokens &&
        5ll * n_tokens <= 3ll * B * max_tokens) {
        packed = true;
        p.few = few;
        if (few > 0) p.kind_o = kKvMixed;
    }
    const long long rows_most = p.kind_o == kKvMixed                       ? few * group
                                : p.kind_p == kKvRows && rows_p > rows_o ? rows_p
                                : p.kind_o == kKvRows                  ? rows_o
                                                                       : rows_p;
    p.mt = rows_most > 16 ? 2 : 1;
    const int R = 16 * p.mt;
    long long groups = 0;   // the rows kernel's work, at most
    long long tiles_b = 0;  // its row tiles of the sequences, of a kv head, at most
    const long long some = B < n_tokens ? B : n_tokens;  // sequences with tokens, at most
    if (p.kind_p == kKvRows) {
        p.tiles_p = ceil_div(rows_p, R);
        groups += (long long)ceil_div(prefix_len, group_keys(D)) * p.tiles_p * H_kv;
    } else if (p.kind_p == kKvTiles) {
        // own keys beside it: somewhat over half of their bound
        const double own = p.kind_o != kKvTiles ? 0.6 * B * (double)max_len * H_kv * D * 4 : 0.0;
        plan_tiles(1, H_kv, group, n_tokens, 0, prefix_len, D, part_bytes, true, own, p.chunk_p,
                   p.splits_p, p.tiles_p, p.ksplit_p, p.parts_p);
    }
    if (p.kind_o == kKvRows) {
        p.tiles_o = ceil_div(rows_o, R);
        tiles_b = some * p.tiles_o;
        if (tiles_b > rows_p / R + some) {
            p.packed = 1;
            tiles_b = rows_p / R + some;
        }
        groups += tiles_b * ceil_div(max_len, group_keys(D)) * H_kv;
    } else if (!packed) {
        plan_tiles(B, H_kv, group, max_tokens, 0, max_len, D, part_bytes, p.kind_p != kKvNone, 0.0,
                   p.chunk_o, p.splits_o, p.tiles_o, p.ksplit_o, p.parts_o);
    } else {
        const double own = few > 0 ? 0.6 * B * (double)max_len * H_kv * D * 4 : 0.0;
        plan_tiles(B, H_kv, group, max_tokens, n_tokens, max_len, D, part_bytes,
                   p.kind_p != kKvNone, own, p.chunk_o, p.splits_o, p.tiles_o, p.ksplit_o,
                   p.parts_o);
        // sum of ceil(n_b / block) over the sequences of more than `few` tokens
        const int block = (p.ksplit_o ? 1 : 2) * (128 / group), most = n_tokens / (few + 1);
        p.row_blocks_t = n_tokens / block + (B < most ? B : most);
        p.tiles_o = 1;
        tiles_b = few > 0 ? some : 0;
        groups += tiles_b * ceil_div(max_len, group_keys(D)) * H_kv;
    }
    p.direct = p.kind_p == kKvNone && p.parts_o == 1;
    p.blocks = (p.kind_p == kKvTiles ? (long long)p.splits_p * H_kv * p.tiles_p : 0) +
               (p.kind_o == kKvTiles && !packed ? (long long)B * p.splits_o * H_kv * p.tiles_o : 0) +
               (long long)p.row_blocks_t * p.splits_o * H_kv;
    long long bytes = p.direct ? 0 : (p.parts_p + p.parts_o) * part_bytes;
    if (groups > 0) {
        // A stretch costs its groups, every partial of a row some of the combine's time: with
        // G groups in the longest run of keys, about sqrt(G / 16) groups are the least worth
        // a warp (1, 2, 4 groups, a call of 1000 + 300 keys: 10.7, 10.0, 10.9 us).
        const int longest = ceil_div(p.kind_p == kKvRows && prefix_len > max_len ? prefix_len
                                                                                 : max_len,
                                     group_keys(D));
        p.min_groups = 2;
        while ((p.min_groups + 1) * (p.min_groups + 1) * 16 <= longest && p.min_groups < 16)
            ++p.min_groups;
        const long long least = (long long)p.min_groups * kWarps;
        const long long blocks = (groups + least - 1) / least;
        const int most = kBlocksPerSm * kSms;
        p.row_blocks = (int)(blocks < most ? blocks : most);
        long long per = groups / (p.row_blocks * kWarps);  // of a full batch
        if (per < p.min_groups) per = p.min_groups;
        // The combine: a warp to a row (444 blocks of eight resident), or a block to a row
        // (296 resident) with an eighth of the steps of eight partials, at some 0.8 us a step
        // beside 2 us a block.  24 x 8 tokens of 16 heads with 16 partials: 3 us or 24 us; 32
        // rows with 366: 40 us or 5 us.
        const double steps = (double)(longest / per + 1 + p.parts_p) / 8;
        // by token rows where at least half of the rows by sequence would be none's
        p.search = p.few > 0 || (paged && 2ll * n_tokens <= (long long)B * max_tokens);
        const long long rows = (p.search ? (long long)n_tokens : (long long)B * max_tokens) * H_q;
        const double narrow = ceil_div(rows, 8 * 3 * kSms) *
                              (2.0 + 0.8 * steps);
        const double wide = ceil_div(rows, 2 * kSms) *
                            (2.0 + 0.1 * steps);
        p.wide_combine = wide < narrow;
        p.heads_log = H_kv % 4 == 0 ? 2 : H_kv % 2 == 0 ? 1 : 0;
        p.j_own = p.kind_p == kKvRows ? H_kv * p.tiles_p : 0;
        const long long js = p.j_own + tiles_b * H_kv;
        p.slots = (long long)p.row_blocks * kWarps + js;
        bytes += p.slots * R * (D + 1) * 4 + js * 8 + 32;
        if (p.blocks < p.slots) p.blocks = p.slots;
        if (p.blocks < rows) p.blocks = rows;
        if (p.blocks < groups) p.blocks = groups;
    }
    p.workspace = bytes;
    return p;
}

}  // namespace

// A plan depends on the sizes alone; a call asks for it twice (workspace, launch) and a
// decode loop asks with the same sizes again, so the thread's last one is kept.
KvPlan plan_kv(int B, int n_tokens, int max_tokens, int max_len, int prefix_len, int H_q,
               int H_kv, int D, int paged, int page_size) {
    static thread_local int last[10] = {};
    static thread_local KvPlan plan;
    const int key[10] = {B, n_tokens, max_tokens, max_len, prefix_len, H_q, H_kv, D, paged + 1,
                         page_size};
    if (std::memcmp(key, last, sizeof key) != 0) {
        plan = make_plan(B, n_tokens, max_tokens, max_len, prefix_len, H_q, H_kv, D, paged,
                         page_size);
        std::memcpy(last, key, sizeof key);
    }
    return plan;
}

cudaError_t launch_kv(const KvArgs& a, const KvPlan& plan, unsigned long long wait_limit_ns,
                      const char** why) {
    cache_kernels_in_use();
    cudaError_t e = cudaSuccess;
    const bool tiled = plan.kind_p == kKvTiles || plan.kind_o == kKvTiles || plan.few;
    if (tiled) {
        e = launch_kv_tiles(a, plan, wait_limit_ns, why);
        if (e != cudaSuccess) return e;
    }
    RowsParams p;
    p.a = a;
    p.p = plan;
    p.group = a.H_q / a.H_kv;
    p.dgroup = make_fastdiv((uint32_t)p.group);
    p.dpage = make_fastdiv((uint32_t)a.page_size);
    p.dheads = make_fastdiv((uint32_t)a.H_q);
    p.dtokens = make_fastdiv((uint32_t)a.max_tokens);
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    if (plan.kind_o == kKvCluster) {
        *why = "cluster attention launch";
        return launch_kv_cluster(p);
    }
    const long long rows = (long long)a.n_tokens * a.H_q;
    p.part_o = (float*)a.workspace;
    const int parts = plan.direct ? 0 : plan.parts_p + plan.parts_o;
    p.part_lse = p.part_o + parts * rows * a.D;
    if (plan.row_blocks > 0) {
        float* after = p.part_lse + parts * rows;
        p.slot_o = (float*)(((uintptr_t)after + 15) & ~(uintptr_t)15);
        p.slot_lse = p.slot_o + plan.slots * 16 * plan.mt * a.D;
        p.meta = (int2*)(p.slot_lse + plan.slots * 16 * plan.mt);
        const unsigned grid = (unsigned)plan.row_blocks;
        const bool page16 = !a.tables || a.page_size % 16 == 0;
        if (a.D == 128) {
            if (plan.mt == 1)
                e = page16 ? launch_rows<128, 1, true>(p, grid, tiled)
                           : launch_rows<128, 1, false>(p, grid, tiled);
            else
                e = page16 ? launch_rows<128, 2, true>(p, grid, tiled)
                           : launch_rows<128, 2, false>(p, grid, tiled);
        } else {
            if (plan.mt == 1)
                e = page16 ? launch_rows<64, 1, true>(p, grid, tiled)
                           : launch_rows<64, 1, false>(p, grid, tiled);
            else
                e = page16 ? launch_rows<64, 2, true>(p, grid, tiled)
                           : launch_rows<64, 2, false>(p, grid, tiled);
        }
    }
    if (e != cudaSuccess || (plan.direct && !plan.few)) return e;
    const long long out_rows =
        plan.kind_o == kKvRows && !plan.search ? (long long)a.B * a.max_tokens * a.H_q : rows;
    const unsigned cg = (unsigned)(plan.wide_combine ? out_rows : (out_rows + 7) / 8);
    auto k = a.D == 128 ? pick_combine<128>(plan) : pick_combine<64>(plan);
    return launch_pdl(k, p, cg, 256, 0, a.stream, true);
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
