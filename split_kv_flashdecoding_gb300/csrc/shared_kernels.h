// shared_kernels.h -- parameters and launchers of shared-prefix decode
// attention (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fd.h"
#include "plan_rule.h"

namespace fd {

constexpr int kSharedTile = 128;       // keys of a tile: rows of a K or V buffer
constexpr int kSharedQRows = 128;      // query rows of one tensor-core tile
constexpr int kSharedBlockRows = 256;  // query rows of one CTA: two such tiles

// The most steps of a stream that O accumulates over in tensor memory.  The
// tensor cores cut the sum of products and accumulator off (they do not round
// it), which with a tile's 16 products takes about 2.5e-7 of O: 37 tiles in a row
// left it short by 1.1e-5, more than its fp32 type says.  So a stream with more
// steps adds O up in global memory, where fp32 sums round, in runs of equal length
// of up to kFlush steps, and starts anew (256 x 64 heads behind 32768 keys, 37
// steps: none 275 us and 1.1e-5, one flush 285 and 5.9e-6, three 299 and 3.3e-6).
constexpr int kFlush = 20;

FD_HD int32_t shared_run(int32_t steps)   // steps between flushes
{
    const int32_t runs = (steps + kFlush - 1) / kFlush;
    return runs > 0 ? (steps + runs - 1) / runs : 1;
}

// Splits of a prefix of `len` keys for chunk length `chunk` (a multiple of
// kSharedTile), and their length: equal within the prefix, whole tiles.
FD_HD int32_t shared_splits(int32_t len, int32_t chunk)
{
    return len > 0 ? (len - 1) / chunk + 1 : 0;
}

FD_HD int32_t shared_split_len(int32_t len, int32_t splits)
{
    const int32_t even = (len - 1) / splits + 1;
    return (even + kSharedTile - 1) / kSharedTile * kSharedTile;
}

struct SharedParams {
    const uint16_t *q;               // bf16 [B, Hq, D]
    const int32_t *req_indptr;       // [P+1] requests of each prefix
    const int32_t *prefix_indptr;    // [P+1] key rows (ragged) or page-list entries (paged)
    const int32_t *prefix_last_len;  // paged: keys of each prefix's last page
    const int32_t *prefix_indices;   // paged: page of each entry
    const float *k_scale, *v_scale;  // FP8: [Hkv]
    float *partial_o;                // [rows, D]
    float *partial_lse;              // [rows]
    float *flush;                    // [items, 2, D / 4, 128, 4]; not used where no stream has over kFlush steps
    float *o, *lse;                  // [B, Hq, D], [B, Hq]; hold the suffix states when has_suffix
    int *status;
    int32_t batch, num_qo_heads, num_kv_heads, group;
    int32_t num_prefixes, chunk, num_items, num_partial_rows;
    int32_t prefix_rows;             // ragged: rows of K/V; paged: entries of prefix_indices
    int32_t page_size, num_pages;    // page_size 0: ragged
    int32_t box_rows;                // paged: rows of a page box
    int32_t has_suffix;
    // the requests' own keys, to check them against the plan's capacity (null: none)
    const int32_t *suffix_indptr, *suffix_last_len;
    int32_t max_suffix_tokens;
    float scale;                     // softmax scale
    int64_t timeout_ns;
};

struct SharedMaps {
    CUtensorMap k, v;
};

// Stage 1 over the prefixes (p.num_items CTAs) and the merge with the suffix
// states.
cudaError_t launch_shared(const SharedMaps &maps, const SharedParams &p, int kv_type, cudaStream_t stream);

}  // namespace fd
