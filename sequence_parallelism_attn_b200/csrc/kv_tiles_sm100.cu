// kv_tiles_sm100.cu -- attention of many query rows over a cache's or an encoder's keys on
// the Blackwell tensor cores: the prefix that a batch shares (rows of the whole batch), the
// own keys of sequences with many new tokens, and cross attention.
//
// Rows: the tokens x the query heads that share a kv head, 128 / group tokens (rounded
// down) to a 128-row tile, loaded by one TMA box per 64 columns, so K and V are read once
// for all of a group's heads.  A block takes two such tiles over one range of keys; where
// there is a single tile in all, the block's two softmax warpgroups take its even and odd
// key tiles instead, as two partial results.  Partials are joined by kv_rows.cu's combine.
// Keys come in 128-row tiles from a dense batch row (one box) or from pages (a box per
// page, or per 128 rows of one); the boxes' page ids are read one tile ahead by the lanes
// that issue them.  Rows past the range's last key are zeroed in V's tile before it is
// published (they may hold anything, and 0 * NaN is not 0); their scores are masked.
//
// Roles, tensor memory and the order of the MMAs are those of attn_sm100.cu.  In units
// u = 0, 1, 2, ... that alternate between the warpgroups (unit u: warpgroup u & 1, key tile
// u / 2, or u where the warpgroups share a row tile), the MMA thread issues
//   S(0), S(1), then for every u:  S(u + 2) once S(u + 1) was read,  PV(u) once P(u) is there
// with one score buffer, two P and two O regions.  What bounds it: with two full row tiles
// the softmax and the tensor core (256 rows x 4 D flops per 4 D bytes): a key tile takes 2.5
// us at D = 128 and 1.93 us at D = 64, where one row to a thread leaves the softmax's latency
// in sight (MUFU 34%, issue slots 29% busy); a block costs some 6 us beside its key tiles.
// Below 128 rows the rate at which K and V arrive.  1000 tokens of 32 heads behind 16384 keys
// of 8 heads of 128: 310 us, 870 TFLOP/s, at the power cap.  Up to 60 bytes a thread are
// spilled (16 to 60 by instance).  The prefix's keys are read once for each row block.
//
// Every wait is bounded, as in attn_sm100.cu.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <cmath>
#include <cstdint>
#include "kv_internal.h"
#include "sm100_ptx.cuh"

namespace ra {

__device__ unsigned int g_kv_tile_error_word = 0;  // waits: bits 0-3; cache errors: << 8

namespace {

constexpr int kThreads = 384;
constexpr uint32_t kRegsLaunch = 168, kRegsSoftmax = 192, kRegsOther = 120;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsOther == kThreads * kRegsLaunch,
              "register split must use exactly the launch allocation");
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpLoadV = 10;
constexpr int kBM = 128, kBN = 128;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr unsigned kErrProducer = 1u, kErrMma = 2u, kErrSoftmax = 4u, kErrDrain = 8u;

struct __align__(64) TileParams {
    CUtensorMap tm_q, tm_k, tm_v;
    KvArgs a;
    int group, tpt;  // query heads per kv head, tokens per row tile
    int box;         // rows of a K/V box (128 where dense)
    int page_shift;  // log2 of the page size (paged)
    int chunk_p, splits_p, blocks_p, ksplit_p, part_p;  // prefix: keys per split, ...
    int chunk_o, splits_o, blocks_o, ksplit_o, part_o;  // own keys; first partial index
    unsigned items_p;
    int few;         // the packed form: sequences of more tokens
    int direct;
    float scale_log2;
    float* parts;    // [part][token][head][D]
    float* parts_lse;
    unsigned long long wait_limit_ns;
};

template <int D>
struct Cfg {
    static constexpr int TILE = kBM * D * 2;
    static constexpr int NKB = D / 64;
    static constexpr int BLK = kBM * 128;
    static constexpr int NSK = (D == 128) ? 3 : 4;
    static constexpr int NSV = (D == 128) ? 2 : 4;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = 2 * TILE;
    static constexpr int OFF_V = OFF_K + NSK * TILE;
    static constexpr int OFF_BAR = OFF_V + NSV * TILE;
    // q_full, k_full[NSK], k_empty[NSK], v_full[NSV], v_empty[NSV], s_full[2], p_full[2],
    // o_full[2], drain, s_free[2], pv_done[2], v_land
    static constexpr int N_BARS = 1 + 2 * NSK + 2 * NSV + 12;
    static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;  // tmem base, abort flag
    static constexpr int SMEM = OFF_MISC + 16 + 1024;      // + alignment slack
    static constexpr int BAR_Q = 0;
    __host__ __device__ static constexpr int bar_kf(int s) { return 1 + s; }
    __host__ __device__ static constexpr int bar_ke(int s) { return 1 + NSK + s; }
    __host__ __device__ static constexpr int bar_vf(int s) { return 1 + 2 * NSK + s; }
    __host__ __device__ static constexpr int bar_ve(int s) { return 1 + 2 * NSK + NSV + s; }
    static constexpr int B0 = 1 + 2 * NSK + 2 * NSV;
    __host__ __device__ static constexpr int bar_sf(int w) { return B0 + w; }
    __host__ __device__ static constexpr int bar_pf(int w) { return B0 + 2 + w; }
    __host__ __device__ static constexpr int bar_of(int w) { return B0 + 4 + w; }
    static constexpr int BAR_DRAIN = B0 + 6;
    __host__ __device__ static constexpr int bar_sfree(int w) { return B0 + 7 + w; }
    __host__ __device__ static constexpr int bar_pvd(int w) { return B0 + 9 + w; }
    static constexpr int BAR_LAND = B0 + 11;
    static constexpr uint32_t S_COL = 0, P_COL0 = 128, P_COL1 = 192;
    static constexpr uint32_t O_COL0 = 256, O_COL1 = 256 + D;
    static_assert(BAR_LAND == N_BARS - 1, "barrier count");
    static_assert(O_COL1 + D <= kTmemCols, "tensor memory budget");
    static_assert(SMEM <= 232448, "shared memory budget");
};

__device__ __forceinline__ void raise_abort(volatile int* abort_flag, unsigned code) {
    *abort_flag = 1;
    atomicOr(&g_kv_tile_error_word, code);
}

__device__ __forceinline__ bool wait1(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                      unsigned long long limit, unsigned code) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 15u) == 0) {
            if (*abort_flag) return false;
            if (global_timer_ns() - t0 > limit) {
                raise_abort(abort_flag, code);
                return false;
            }
        }
    }
}

// Bounded wait that ignores the abort flag: used to drain work this thread started.
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           unsigned long long limit) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 15u) == 0 && global_timer_ns() - t0 > limit) {
            raise_abort(abort_flag, kErrDrain);
            return false;
        }
    }
}

// Warp-uniform bounded wait (every lane polls; the give-up decision is lane 0's).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned long long limit, unsigned code) {
    const unsigned FULL = 0xffffffffu;
    bool done = mbar_try_wait(bar, parity);
    if (__all_sync(FULL, done)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (!done) done = mbar_try_wait(bar, parity);
        if (__all_sync(FULL, done)) return true;
        if ((it & 15u) == 0) {
            int stop = 0;
            if ((threadIdx.x & 31) == 0) {
                if (*abort_flag) stop = 1;
                else if (global_timer_ns() - t0 > limit) {
                    raise_abort(abort_flag, code);
                    stop = 1;
                }
            }
            if (__shfl_sync(FULL, stop, 0)) return false;
        }
    }
}

// A block's work.
struct Item {
    int b, g, part;        // batch row (0 for the prefix), kv head, first partial index
    int tok0, n_tok;       // the phase's tokens: first row of q, count
    int t0;                // first token of the block's first row tile
    int k_begin, k_hi, n;  // first key, end of the keys any of its rows sees, key tiles
    int lim0;              // the causal limit of the phase's token 0 (keys below it are seen)
    int causal, ksplit;
    const int* table;      // page ids, null where dense
};

// PACKED: own keys of sequences with more than `few` tokens only, their row blocks counted
// through the batch (an instance of its own: the search costs the softmax registers).
template <bool PACKED>
__device__ __forceinline__ bool make_item(const TileParams& p, Item& x) {
    const KvArgs& a = p.a;
    unsigned item = blockIdx.x;
    int len, chunk, split, blk;
    if (item < p.items_p) {
        blk = item % p.blocks_p;
        item /= p.blocks_p;
        x.g = item % a.H_kv;
        split = item / a.H_kv;
        x.b = 0;
        x.tok0 = 0;
        x.n_tok = min(a.cu[a.B], a.n_tokens);
        len = a.prefix_len;
        chunk = p.chunk_p;
        x.table = a.prefix_table;
        x.causal = 0;
        x.ksplit = p.ksplit_p;
        x.part = p.part_p + split * (1 + x.ksplit);
    } else {
        item -= p.items_p;
        if (PACKED) {
            // the item-th row block of the sequences with many tokens: every warp adds up
            // their blocks; the first block's first warp looks at the whole batch, to report
            const bool report = item == 0 && threadIdx.x < 32;
            const int lane = threadIdx.x & 31, size = p.ksplit_o ? p.tpt : 2 * p.tpt;
            x.g = item % a.H_kv;
            item /= a.H_kv;
            split = item % p.splits_o;
            const int r = (int)(item / p.splits_o);
            int at = 0;
            x.b = -1;
            blk = 0;
#pragma unroll 1
            for (int e0 = 0; e0 < a.B && (x.b < 0 || report); e0 += 256) {
                int w[8], all = 0;  // 256 sequences' loads in flight at once
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = e0 + 32 * i + lane;
                    w[i] = 0;
                    if (e < a.B) {
                        const TokenRows rows = token_rows(a.cu, e, a.n_tokens, a.max_tokens);
                        if (rows.n > p.few) w[i] = (min(rows.n, a.max_tokens) + size - 1) / size;
                        if (report && rows.bad)
                            atomicOr(&g_kv_tile_error_word, kKvErrTokens << 8);
                    }
                    all += w[i];
                }
                all = __reduce_add_sync(0xffffffffu, all);
                if (x.b >= 0 || at + all <= r) {
                    at += all;
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int sum = __reduce_add_sync(0xffffffffu, w[i]);
                    if (x.b < 0 && at + sum > r) {
                        int incl = w[i];
#pragma unroll
                        for (int off = 1; off < 32; off <<= 1) {
                            const int y = __shfl_up_sync(0xffffffffu, incl, off);
                            if (lane >= off) incl += y;
                        }
                        const int l = __ffs(__ballot_sync(0xffffffffu, at + incl > r)) - 1;
                        x.b = e0 + 32 * i + l;
                        blk = r - at - __shfl_sync(0xffffffffu, incl - w[i], l);
                    }
                    at += sum;
                }
            }
            if (x.b < 0) return false;
        } else {
            blk = item % p.blocks_o;
            item /= p.blocks_o;
            x.g = item % a.H_kv;
            item /= a.H_kv;
            split = item % p.splits_o;
            x.b = item / p.splits_o;
        }
        const bool first = threadIdx.x == 0 && split == 0;
        if (a.cu) {
            const TokenRows rows = token_rows(a.cu, x.b, a.n_tokens, a.max_tokens);
            if (first && rows.bad) atomicOr(&g_kv_tile_error_word, kKvErrTokens << 8);
            x.tok0 = rows.first;
            x.n_tok = rows.n;
        } else {
            x.tok0 = x.b * a.max_tokens;
            x.n_tok = a.max_tokens;
        }
        len = a.lens ? max(a.lens[x.b], 0) : a.max_len;
        if (len > a.max_len) {
            if (first) atomicOr(&g_kv_tile_error_word, kKvErrLength << 8);
            len = a.max_len;
        }
        chunk = p.chunk_o;
        x.table = a.tables ? a.tables + (long long)x.b * a.max_pages : nullptr;
        x.causal = a.causal;
        x.ksplit = p.ksplit_o;
        x.part = p.part_o + split * (1 + x.ksplit);
    }
    const int per_block = x.ksplit ? p.tpt : 2 * p.tpt;
    x.t0 = blk * per_block;
    if (x.t0 >= x.n_tok) return false;
    x.lim0 = len - x.n_tok + 1;
    x.k_begin = split * chunk;
    x.k_hi = min(x.k_begin + chunk, len);
    if (x.causal) x.k_hi = min(x.k_hi, x.lim0 + min(x.t0 + per_block, x.n_tok) - 1);
    x.n = x.k_hi > x.k_begin ? (x.k_hi - x.k_begin + kBN - 1) / kBN : 0;
    return true;
}

// K/V producer: one warp streams the K tiles (and first the Q tiles) or the V tiles.
template <int D, bool IS_K>
__device__ __forceinline__ void producer(const TileParams& p, uint32_t base, const Item& x,
                                         volatile int* abort_flag) {
    using C = Cfg<D>;
    constexpr int NS = IS_K ? C::NSK : C::NSV;
    const KvArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    auto bar = [&](int i) { return base + C::OFF_BAR + 8u * (uint32_t)i; };
    auto bar_full = [&](int s) { return bar(IS_K ? C::bar_kf(s) : C::bar_vf(s)); };
    auto bar_empty = [&](int s) { return bar(IS_K ? C::bar_ke(s) : C::bar_ve(s)); };
    const uint32_t ring = base + (IS_K ? C::OFF_K : C::OFF_V);
    const CUtensorMap* map = IS_K ? &p.tm_k : &p.tm_v;
    const unsigned long long lim = p.wait_limit_ns;
    int armed[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) armed[s] = -1;

    if (IS_K && lane == 0) {
        const int tiles = x.ksplit ? 1 : 2;
        const uint32_t bytes = (uint32_t)(p.tpt * p.group) * 128u * C::NKB;
        mbar_arrive_expect_tx(bar(C::BAR_Q), tiles * bytes);
        for (int w = 0; w < tiles; ++w)
            for (int kb = 0; kb < C::NKB; ++kb)
                tma_load_4d(base + C::OFF_Q + w * C::TILE + kb * C::BLK, &p.tm_q, bar(C::BAR_Q),
                            kb * 64, x.g * p.group,
                            (a.cu ? x.tok0 : 0) + x.t0 + w * p.tpt, a.cu ? 0 : x.b);
    }
    // this lane's box of the tile at key0: its page (read a tile ahead)
    auto look_up = [&](int key0) -> int {
        const int key = key0 + lane * p.box;
        if (!x.table || lane * p.box >= kBN || key >= x.k_hi) return 0;
        const int page = x.table[key >> p.page_shift];
        if (page >= 0 && page < a.n_pages) return page;
        atomicOr(&g_kv_tile_error_word, kKvErrPage << 8);
        return 0;
    };
    int page = look_up(x.k_begin);
    bool ok = true;
    for (int jt = 0; jt < x.n; ++jt) {
        const int slot = jt % NS, key0 = x.k_begin + jt * kBN;
        const int rows = min(kBN, x.k_hi - key0);
        const int nb = x.table ? (rows + p.box - 1) / p.box : 1;
        if (jt >= NS &&
            !wait_warp(bar_empty(slot), ((jt / NS) - 1) & 1, abort_flag, lim, kErrProducer)) {
            ok = false;
            break;
        }
        const bool tail = !IS_K && rows < kBN;  // the last tile: rows behind the keys
        const uint32_t fb = tail ? bar(C::BAR_LAND) : bar_full(slot);
        if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)(nb * p.box) * 128u * C::NKB);
        __syncwarp();
        if (lane < nb) {
            const int key = key0 + lane * p.box;
            const int row = x.table ? key & ((1 << p.page_shift) - 1) : key;
            const int pg = x.table ? page : x.b;
#pragma unroll
            for (int kb = 0; kb < C::NKB; ++kb)
                tma_load_4d(ring + slot * C::TILE + kb * C::BLK + lane * p.box * 128, map, fb,
                            kb * 64, x.g, row, pg);
        }
        page = look_up(key0 + kBN);
        if (tail) {
            const bool landed = wait_warp(fb, 0, abort_flag, lim, kErrProducer);
            if (!landed) {
                if (lane == 0) wait_drain(fb, 0, abort_flag, lim);
                ok = false;
                break;
            }
            // a row of a swizzle block is 128 consecutive bytes whatever the swizzle
            for (int kb = 0; kb < C::NKB; ++kb)
                for (int i = lane; i < (kBN - rows) * 8; i += 32)
                    st_shared_v4(ring + slot * C::TILE + kb * C::BLK + rows * 128 + i * 16, 0, 0,
                                 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_full(slot));
        }
        armed[slot] = jt;
    }
    // Drain: every copy this warp started must have landed before the CTA exits.
    if (lane == 0) {
        if (IS_K) wait_drain(bar(C::BAR_Q), 0, abort_flag, lim);
#pragma unroll
        for (int s = 0; s < NS; ++s)
            if (armed[s] >= 0) wait_drain(bar_full(s), (armed[s] / NS) & 1, abort_flag, lim);
    }
    __syncwarp();
}

template <int D>
__device__ __forceinline__ void mma_issuer(const TileParams& p, uint32_t base, uint32_t tmem,
                                           const Item& x, volatile int* abort_flag) {
    using C = Cfg<D>;
    auto bar = [&](int i) { return base + C::OFF_BAR + 8u * (uint32_t)i; };
    const unsigned long long lim = p.wait_limit_ns;
    constexpr uint32_t IDESC_S = idesc_bf16_f32(kBM, kBN, 0);  // K-major Q and K
    constexpr uint32_t IDESC_O = idesc_bf16_f32(kBM, D, 1);    // V is MN-major (D contiguous)
    const uint64_t dq0 = desc_sw128(base + C::OFF_Q, 16, 1024);
    const uint64_t dk0 = desc_sw128(base + C::OFF_K, 16, 1024);
    const uint64_t dv0 = desc_sw128(base + C::OFF_V, C::BLK, 1024);
    auto issue_s = [&](int w, int slot) {
        const uint64_t dq = dq0 + (uint64_t)((w * C::TILE) >> 4);
        const uint64_t dk = dk0 + (uint64_t)((slot * C::TILE) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * C::BLK + (kk % 4) * 32) >> 4;
            mma_ss(tmem + C::S_COL, dq + off, dk + off, IDESC_S, kk > 0 ? 1u : 0u);
        }
    };
    auto issue_pv = [&](int w, int slot, bool acc) {
        const uint64_t dv = dv0 + (uint64_t)((slot * C::TILE) >> 4);
        const uint32_t o = tmem + (w ? C::O_COL1 : C::O_COL0);
        const uint32_t pp = tmem + (w ? C::P_COL1 : C::P_COL0);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
            mma_ts(o, pp + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), IDESC_O,
                   (acc || kk > 0) ? 1u : 0u);
    };
    const int ks = x.ksplit;
    const int U = ks ? x.n : 2 * x.n;
    bool issued = false;
    // S of unit u: its key tile has landed (tile u / 2's first unit waits for it)
    auto unit_s = [&](int u) -> bool {
        const int tile = ks ? u : u >> 1, slot = tile % C::NSK, w = u & 1;
        if ((ks || w == 0) &&
            !wait1(bar(C::bar_kf(slot)), (tile / C::NSK) & 1, abort_flag, lim, kErrMma))
            return false;
        tc_fence_after();
        issue_s(ks ? 0 : w, slot);
        issued = true;
        tc_commit(bar(C::bar_sf(w)));
        if (ks || w == 1) tc_commit(bar(C::bar_ke(slot)));
        return true;
    };
    if (U > 0 && wait1(bar(C::BAR_Q), 0, abort_flag, lim, kErrMma) && unit_s(0)) {
        bool go = true;
        // S(u) goes into S once S(u - 1) has been read out of it
        if (U > 1) go = wait1(bar(C::bar_sfree(0)), 0, abort_flag, lim, kErrMma) && unit_s(1);
        for (int u = 0; go && u < U; ++u) {
            const int w = u & 1, i = u >> 1;
            if (u + 2 < U) {
                const int v = u + 1;
                if (!wait1(bar(C::bar_sfree(v & 1)), (v >> 1) & 1, abort_flag, lim, kErrMma) ||
                    !unit_s(u + 2))
                    break;
            }
            const int tile = ks ? u : i, slot = tile % C::NSV;
            if ((ks || w == 0) &&
                !wait1(bar(C::bar_vf(slot)), (tile / C::NSV) & 1, abort_flag, lim, kErrMma))
                break;
            if (!wait1(bar(C::bar_pf(w)), i & 1, abort_flag, lim, kErrMma)) break;
            tc_fence_after();
            issue_pv(w, slot, i > 0);
            tc_commit(bar(C::bar_pvd(w)));
            if (ks || w == 1) tc_commit(bar(C::bar_ve(slot)));
            if (u + 2 >= U) tc_commit(bar(C::bar_of(w)));
        }
    }
    if (issued) {  // every MMA this thread issued completes before TMEM is released
        tc_commit(bar(C::BAR_DRAIN));
        wait_drain(bar(C::BAR_DRAIN), 0, abort_flag, lim);
    }
}

template <int D>
__device__ __forceinline__ void softmax_wg(const TileParams& p, uint32_t base, uint32_t tmem,
                                           const Item& x, int wg, volatile int* abort_flag) {
    using C = Cfg<D>;
    const KvArgs& a = p.a;
    auto bar = [&](int i) { return base + C::OFF_BAR + 8u * (uint32_t)i; };
    const unsigned long long lim = p.wait_limit_ns;
    const unsigned FULL = 0xffffffffu;
    const int wr = (threadIdx.x >> 5) & 3;  // warp within the warpgroup = TMEM lane quarter
    const int lane = threadIdx.x & 31;
    // this thread's row: token t of the phase, query head hh of the group
    const int row = wr * 32 + lane;
    const int tl = row / p.group, hh = row - tl * p.group;
    const int tile_t0 = x.t0 + (x.ksplit ? 0 : wg * p.tpt);
    const int t = tile_t0 + tl;
    const bool row_ok = tl < p.tpt && t < x.n_tok;
    const bool live = __any_sync(FULL, row_ok);
    // keys below `limit` are seen; the tile's smallest limit is its first token's
    const int limit = x.causal && row_ok ? min(x.k_hi, x.lim0 + t) : x.k_hi;
    const int limit_min = x.causal ? min(x.k_hi, x.lim0 + tile_t0) : x.k_hi;
    const uint32_t lane_off = (uint32_t)(wr * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::S_COL;
    const uint32_t tP = tmem + lane_off + (wg ? C::P_COL1 : C::P_COL0);
    const uint32_t tO = tmem + lane_off + (wg ? C::O_COL1 : C::O_COL0);
    const float sl2 = p.scale_log2;
    const int cnt = x.ksplit ? (x.n - wg + 1) / 2 : x.n;

    // l_run: sum of the fp32 weights, which gives the LSE.  l_used: sum of the weights as they
    // meet V, rounded to bf16, which divides O, so that the weights applied add up to one.  With
    // l_run for both, a quarter of the loop's instructions would go, but where a key takes most
    // of the weight (256 times the others' at most while the maximum lags), or values are much
    // alike, O would be off by that weight's own rounding, 2^-9 instead of the sums' 2^-13.
    float m_run = -INFINITY, l_run = 0.f, l_used = 0.f;
    bool ok = true;
    for (int i = 0; i < cnt; ++i) {
        if (!wait_warp(bar(C::bar_sf(wg)), i & 1, abort_flag, lim, kErrSoftmax)) {
            ok = false;
            break;
        }
        __syncwarp();
        if (!live) {
            // none of the warp's rows is a token's: it keeps the barriers' count and leaves
            // the exponentials to the others (its rows of P and O are never read).  Waiting
            // for PV(i-1) keeps its arrival out of the phase before.
            tc_fence_before();
            mbar_arrive(bar(C::bar_sfree(wg)));
            if (i > 0 &&
                !wait_warp(bar(C::bar_pvd(wg)), (i - 1) & 1, abort_flag, lim, kErrSoftmax)) {
                ok = false;
                break;
            }
            __syncwarp();
            mbar_arrive(bar(C::bar_pf(wg)));
            continue;
        }
        tc_fence_after();
        uint64_t s2[64];  // the row's 128 scores as pairs (2i, 2i+1)
        tmem_ld128_pairs(tS, s2);
        tc_fence_before();
        mbar_arrive(bar(C::bar_sfree(wg)));
        const int key0 = x.k_begin + (x.ksplit ? 2 * i + wg : i) * kBN;
        if (key0 + kBN > limit_min) {
            const int c_hi = limit - 1 - key0;
#pragma unroll
            for (int e = 0; e < 64; ++e) {
                float u, v;
                f2_unpack(s2[e], u, v);
                if (2 * e > c_hi) u = -INFINITY;
                if (2 * e + 1 > c_hi) v = -INFINITY;
                s2[e] = f2_pack(u, v);
            }
        }
        float mx0, mx1, mx2, mx3;
        {
            float u, v;
            f2_unpack(s2[0], u, v); mx0 = fmaxf(u, v);
            f2_unpack(s2[1], u, v); mx1 = fmaxf(u, v);
            f2_unpack(s2[2], u, v); mx2 = fmaxf(u, v);
            f2_unpack(s2[3], u, v); mx3 = fmaxf(u, v);
#pragma unroll
            for (int e = 4; e < 64; e += 4) {
                f2_unpack(s2[e], u, v); mx0 = fmax3(mx0, u, v);
                f2_unpack(s2[e + 1], u, v); mx1 = fmax3(mx1, u, v);
                f2_unpack(s2[e + 2], u, v); mx2 = fmax3(mx2, u, v);
                f2_unpack(s2[e + 3], u, v); mx3 = fmax3(mx3, u, v);
            }
        }
        const float m_new = fmaxf(m_run, fmaxf(fmax3(mx0, mx1, mx2), mx3) * sl2);
        float alpha = 1.f;
        bool resc = false;
        if (i == 0) {
            m_run = m_new;
        } else if (m_new - m_run > kRescaleThreshold) {
            alpha = ex2_approx(m_run - m_new);
            m_run = m_new;
            resc = true;
        }
        const float neg_m = (m_run == -INFINITY) ? 0.f : -m_run;
        const uint64_t sl2x2 = f2_pack(sl2, sl2), negm_x2 = f2_pack(neg_m, neg_m);
        uint64_t sum_a = 0, sum_b = 0, used_a = 0, used_b = 0;  // (0.f, 0.f) pairs
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int c2 = 0; c2 < 32; ++c2) {
                if (c2 & 1)
                    pk[c2] = softmax_pair(s2[half * 32 + c2], sl2x2, negm_x2, sum_b, used_b);
                else
                    pk[c2] = softmax_pair(s2[half * 32 + c2], sl2x2, negm_x2, sum_a, used_a);
            }
            if (half == 0 && i > 0) {  // P(i-1) there has been read by PV(i-1)
                if (!wait_warp(bar(C::bar_pvd(wg)), (i - 1) & 1, abort_flag, lim, kErrSoftmax)) {
                    ok = false;
                    break;
                }
                __syncwarp();
                tc_fence_after();
            }
            tmem_st32(tP + half * 32, pk);
        }
        if (!ok) break;
        float s0, s1, u0, u1;
        f2_unpack(f2_add(sum_a, sum_b), s0, s1);
        f2_unpack(f2_add(used_a, used_b), u0, u1);
        l_run = l_run * alpha + (s0 + s1);
        l_used = l_used * alpha + (u0 + u1);
        if (__any_sync(FULL, resc)) {
#pragma unroll
            for (int cb = 0; cb < D / 32; ++cb) {
                uint32_t o[32];
                tmem_ld32(tO + cb * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(tO + cb * 32, o);
            }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::bar_pf(wg)));
    }
    if (ok && cnt > 0 && !wait_warp(bar(C::bar_of(wg)), 0, abort_flag, lim, kErrSoftmax)) ok = false;
    if (!ok) return;
    __syncwarp();
    tc_fence_after();

    // no key seen: l = 0; a NaN score comes through as a NaN sum
    const float inv_l = l_used == 0.f ? 0.f : 1.f / l_used;
    const float lse2 = l_run == 0.f ? -INFINITY
                                    : (m_run == -INFINITY ? 0.f : m_run) + lg2_approx(l_run);
    const int head = x.g * p.group + hh;
    const long long orow = (long long)(x.tok0 + t) * a.H_q + head;
    const long long prow = (long long)(x.part + (x.ksplit ? wg : 0)) * a.n_tokens * a.H_q + orow;
    const bool bf16 = p.direct && a.out_bf16;
#pragma unroll
    for (int cb = 0; cb < D / 32; ++cb) {
        uint32_t o[32];
        if (cnt > 0) {
            tmem_ld32(tO + cb * 32, o);
            tmem_wait_ld();
        }
        if (row_ok) {
            if (cnt == 0 || l_run == 0.f) {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0;
            }
            if (!bf16) {
                float* dst_row = p.direct ? (float*)a.out + orow * D : p.parts + prow * D;
                float4* dst = reinterpret_cast<float4*>(dst_row + cb * 32);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[e] = make_float4(__uint_as_float(o[4 * e]) * inv_l,
                                         __uint_as_float(o[4 * e + 1]) * inv_l,
                                         __uint_as_float(o[4 * e + 2]) * inv_l,
                                         __uint_as_float(o[4 * e + 3]) * inv_l);
            } else {
                uint4* dst = reinterpret_cast<uint4*>((uint16_t*)a.out + orow * D + cb * 32);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w[4];
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        w[f] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * f]) * inv_l,
                                           __uint_as_float(o[8 * e + 2 * f + 1]) * inv_l);
                    dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
        __syncwarp();
    }
    if (row_ok) {
        if (p.direct) {
            const long long li = a.cu ? (long long)head * a.n_tokens + x.tok0 + t
                                      : ((long long)x.b * a.H_q + head) * a.max_tokens + t;
            a.lse[li] = lse2 * 0.69314718055994530942f;
        } else {
            p.parts_lse[prow] = lse2;
        }
    }
}

template <int D, bool PACKED>
__global__ void __launch_bounds__(kThreads, 1) kv_tiles_sm100(const __grid_constant__ TileParams p) {
    using C = Cfg<D>;
    Item x;
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&p.tm_q);
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    pdl_launch_dependents();  // the rows kernel, which waits for this one only at its end
    if (!make_item<PACKED>(p, x)) return;  // the same for every thread of the block
    extern __shared__ uint8_t smem_raw[];
    uint32_t base = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (base & 1023u)) & 1023u;
    base += pad;
    uint8_t* smem = smem_raw + pad;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    auto bar = [&](int i) { return base + C::OFF_BAR + 8u * (uint32_t)i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(bar(C::BAR_Q), 1);
        for (int s = 0; s < C::NSK; ++s) {
            mbar_init(bar(C::bar_kf(s)), 1);
            mbar_init(bar(C::bar_ke(s)), 1);
        }
        for (int s = 0; s < C::NSV; ++s) {
            mbar_init(bar(C::bar_vf(s)), 1);
            mbar_init(bar(C::bar_ve(s)), 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar(C::bar_sf(w)), 1);
            mbar_init(bar(C::bar_pf(w)), 4 * 32);
            mbar_init(bar(C::bar_of(w)), 1);
            mbar_init(bar(C::bar_sfree(w)), 4 * 32);
            mbar_init(bar(C::bar_pvd(w)), 1);
        }
        mbar_init(bar(C::BAR_DRAIN), 1);
        mbar_init(bar(C::BAR_LAND), 1);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == kWarpMma) {
        __syncwarp();
        tmem_alloc(base + C::OFF_MISC, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (warp >= 8) {
        regs_decrease<kRegsOther>();
        if (warp == kWarpLoad) producer<D, true>(p, base, x, abort_flag);
        else if (warp == kWarpLoadV) producer<D, false>(p, base, x, abort_flag);
        else if (warp == kWarpMma && lane == 0) mma_issuer<D>(p, base, tmem, x, abort_flag);
    } else {
        regs_increase<kRegsSoftmax>();
        softmax_wg<D>(p, base, tmem, x, warp >> 2, abort_flag);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) {
        __syncwarp();
        tmem_dealloc(tmem, kTmemCols);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// bf16 [n3][n2][n1][D] with element strides s2, s3: boxes of 64 columns x b1 x b2, 128-byte
// swizzle, zero fill.
bool encode(CUtensorMap* m, const void* ptr, int D, long long n1, long long n2, long long n3,
            long long s2, long long s3, int b1, int b2) {
    auto enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)n1, (cuuint64_t)n2, (cuuint64_t)n3};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)s2 * 2, (cuuint64_t)s3 * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool PACKED>
cudaError_t launch(const TileParams& p, unsigned grid, const char** why) {
    auto k = kv_tiles_sm100<D, PACKED>;
    // the register split assumes the launch allocation: a raise beyond it would never complete
    static const int regs = [] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, kv_tiles_sm100<D, PACKED>) == cudaSuccess ? fa.numRegs : -1;
    }();
    if (regs != (int)kRegsLaunch) {
        *why = "tile kernel compiled with a register count its register split does not assume";
        return cudaErrorInvalidKernelImage;
    }
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    k<<<grid, kThreads, Cfg<D>::SMEM, p.a.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_tiles(const KvArgs& a, const KvPlan& plan, unsigned long long wait_limit_ns,
                            const char** why) {
    const cudaError_t ctx = ensure_context();
    if (ctx != cudaSuccess) return ctx;
    TileParams p;
    p.a = a;
    p.group = a.H_q / a.H_kv;
    p.tpt = kBM / p.group;
    p.box = kBN;
    p.page_shift = 0;
    if (a.tables) {
        while ((1 << p.page_shift) < a.page_size) ++p.page_shift;
        if (a.page_size < kBN) p.box = a.page_size;
    }
    const bool has_p = plan.kind_p == kKvTiles;
    p.chunk_p = plan.chunk_p;
    p.splits_p = plan.splits_p;
    p.blocks_p = plan.tiles_p;
    p.ksplit_p = plan.ksplit_p;
    p.part_p = 0;
    p.chunk_o = plan.chunk_o;
    p.splits_o = plan.splits_o;
    p.blocks_o = plan.tiles_o;
    p.ksplit_o = plan.ksplit_o;
    p.part_o = plan.parts_p;
    p.items_p = has_p ? (unsigned)((long long)plan.splits_p * a.H_kv * plan.tiles_p) : 0;
    const long long grid =
        p.items_p +
        (plan.row_blocks_t         ? (long long)plan.row_blocks_t
         : plan.kind_o == kKvTiles ? (long long)a.B * plan.tiles_o
                                   : 0) *
            plan.splits_o * a.H_kv;
    p.few = plan.few;
    p.direct = plan.direct;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    p.parts = (float*)a.workspace;
    p.parts_lse = p.parts + (long long)(plan.parts_p + plan.parts_o) * a.n_tokens * a.H_q * a.D;
    p.wait_limit_ns = wait_limit_ns;
    const long long q_rows = a.cu ? a.n_tokens : a.max_tokens, q_b = a.cu ? 1 : a.B;
    const long long q_bs = a.cu ? q_rows * a.q_tstride : a.q_bstride;
    if (!encode(&p.tm_q, a.q, a.D, a.H_q, q_rows, q_b, a.q_tstride, q_bs, p.group, p.tpt) ||
        !encode(&p.tm_k, a.k, a.D, a.H_kv, a.page_size, a.n_pages, a.kv_tstride, a.page_stride, 1,
                p.box) ||
        !encode(&p.tm_v, a.v, a.D, a.H_kv, a.page_size, a.n_pages, a.kv_tstride, a.page_stride, 1,
                p.box)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    const unsigned n = (unsigned)grid;
    if (plan.row_blocks_t)
        return a.D == 128 ? launch<128, true>(p, n, why) : launch<64, true>(p, n, why);
    return a.D == 128 ? launch<128, false>(p, n, why) : launch<64, false>(p, n, why);
}

cudaError_t read_and_clear_kv_tile_error(unsigned int* value, bool all) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_kv_tile_error_word, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    const unsigned int kept = all ? 0u : *value & ~255u;
    if (*value != kept)
        e = cudaMemcpyToSymbol(g_kv_tile_error_word, &kept, sizeof(unsigned int));
    return e;
}

}  // namespace ra
