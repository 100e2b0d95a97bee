// kv_internal.h -- what the operators over a K/V cache share: attention of new tokens over
// a paged cache (with a prefix that the whole batch sees) or over an encoder's states, and
// the append that fills the cache.  Arguments are validated by api_kv.cu.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>
#include "ra_internal.h"

namespace ra {

constexpr int kSms = 148;  // a B200's SMs: the work split is planned for them, not queried

// Bits of the device's cache error word (read and cleared by ra_sync_status).
constexpr unsigned kKvErrTokens = 1u, kKvErrLength = 2u, kKvErrPage = 4u;

// Called by every launch of the cache kernels (a captured one too): from the first on,
// ra_sync_status reads their error words, at 13 us each.
void cache_kernels_in_use();

// Sequence b's token rows: the first, and their number, kept within the token tensors
// whatever cu holds; bad where it was outside the call's bounds.
struct TokenRows {
    int first, n;
    bool bad;
};
__device__ __forceinline__ TokenRows token_rows(const int* cu, int b, int n_tokens,
                                                int max_tokens) {
    const int c0 = cu[b], c1 = cu[b + 1];
    TokenRows r;
    r.first = min(max(c0, 0), n_tokens);
    r.n = max(min(c1, n_tokens), r.first) - r.first;
    r.bad = c0 < 0 || c1 < c0 || c1 > n_tokens || c1 - c0 > max_tokens;
    return r;
}

// A whole warp: the last of B sequences that starts at or before the token (0 where none does),
// 32 ways at a time.
__device__ __forceinline__ int find_sequence(const int* cu, int B, int tok) {
    int b = 0, hi = B;
    while (hi - b > 1) {
        const int step = (hi - b + 31) / 32, e = b + (int)(threadIdx.x & 31) * step;
        const unsigned le = __ballot_sync(0xffffffffu, e < hi && cu[e] <= tok);
        if (le) b += (31 - __clz(le)) * step;
        hi = min(hi, b + step);
    }
    return b;
}

struct AppendArgs {
    const void *q, *k, *v;
    long long q_tstride, k_tstride, v_tstride, q_out_tstride;  // elements between tokens
    const int *cu, *lens, *tables;
    const float* inv_freq;
    int B, n_tokens, max_tokens, H_q, H_kv, D, rot, interleaved, pos_offset;
    int page_size, n_pages, max_pages;
    long long page_stride;  // elements
    void *q_out, *k_pages, *v_pages;
    cudaStream_t stream;
};
cudaError_t launch_paged_append(const AppendArgs& a);
cudaError_t read_and_clear_append_error(unsigned int* value);

// Queries and keys of one call.  Tokens of sequence b: cu[b] .. cu[b+1]-1 (ragged, cu given)
// or Lq tokens of batch row b (cu null).  Keys of sequence b: its own lens[b] keys (all
// max_len where lens is null) found through its page table (tables given) or in its dense
// batch row (tables null: page b, of page_stride elements), and before them the prefix.
struct KvArgs {
    const void* q;
    long long q_tstride, q_bstride;  // elements; q_bstride only where cu is null
    const void *k, *v;
    long long kv_tstride, page_stride;  // elements between tokens, between pages (batch rows)
    const int *cu, *lens, *tables, *prefix_table;
    int prefix_len, B, n_tokens, max_tokens, max_len;
    int H_q, H_kv, D;
    int page_size, n_pages, max_pages;
    int causal;  // own keys: new token i of n sees keys up to len - n + i
    float scale;
    int out_bf16;
    void* out;
    float* lse;
    void* workspace;
    cudaStream_t stream;
};

// How a call is split.  The prefix and the sequences' own keys are each taken by one of two
// kernels, or both by a third (kKvCluster): the tile kernel in ranges of `chunk` keys, each a
// partial result of its rows (two where its warpgroups share a row tile), or the rows kernel,
// whose warps share the keys out evenly among themselves.  The combine kernel joins the partials.
// kKvMixed (own keys): a ragged batch of long and short runs of new tokens, the rows kernel
// for sequences of up to `few` tokens, the tile kernel for the others.
constexpr int kKvNone = 0, kKvRows = 1, kKvTiles = 2, kKvCluster = 3, kKvMixed = 4;
struct KvPlan {
    int kind_p, chunk_p, splits_p, tiles_p, ksplit_p, parts_p;  // the prefix
    int kind_o, chunk_o, splits_o, tiles_o, ksplit_o, parts_o;  // own keys
    int mt;                       // rows kernel: 16-row fragments of a row tile
    int row_blocks, j_own;        // its grid; index of the first (sequence, head, tile)
    int heads_log;                // log2 of the kv heads that its warps take side by side
    int min_groups, wide_combine; // fewest key groups of a warp; eight warps join a row
    int packed, search;           // its row tiles counted by token rows; the combine's rows too
    long long slots;              // its partial slots
    int few;                      // kKvMixed (0 elsewhere)
    int row_blocks_t;             // packed own keys of the tile kernel: its row blocks, at most
    int cluster;                  // kKvCluster (own keys and prefix together): its blocks
    int direct;                   // a single part: results written without partials
    long long blocks, workspace;  // largest index of a launch (to be below 2^31), bytes
};
// paged: keys in pages of page_size (else dense batch rows).
KvPlan plan_kv(int B, int n_tokens, int max_tokens, int max_len, int prefix_len, int H_q,
               int H_kv, int D, int paged, int page_size);
// Everything of a plan: the tile kernel's part, the rows kernel's, the combine.
cudaError_t launch_kv(const KvArgs& a, const KvPlan& p, unsigned long long wait_limit_ns,
                      const char** why);
cudaError_t launch_kv_tiles(const KvArgs& a, const KvPlan& p, unsigned long long wait_limit_ns,
                            const char** why);
// The tile kernel's word: waits that ran out in bits 0 - 7, cache errors above them, which are
// left as they are unless all is set.
cudaError_t read_and_clear_kv_tile_error(unsigned int* value, bool all);
cudaError_t read_and_clear_kv_cluster_error(unsigned int* value);

struct CrossBwdArgs {
    const void *q, *k, *v, *out, *dout;
    const float* lse;
    const int* kv_lens;
    int B, Lq, Lk, H_q, H_kv, D;
    long long q_tstride, q_bstride, kv_tstride, kv_bstride;
    float scale;
    int grad_bf16;
    void *dq, *dk, *dv;
    float* workspace;  // Delta [B][H_q][Lq], then (bf16 gradients) dQ in fp32
    cudaStream_t stream;
};
cudaError_t launch_cross_bwd(const CrossBwdArgs& a, unsigned long long wait_limit_ns,
                             int deterministic, const char** why);
cudaError_t read_and_clear_kv_error(unsigned int* value);

}  // namespace ra
