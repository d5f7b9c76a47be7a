// prefill_kernels.h -- parameters and launchers of attention of many query tokens a
// request over an INT8 paged cache (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fd.h"
#include "plan_rule.h"

namespace fd {

constexpr int kPrefillTile = 128;       // keys of a tile
constexpr int kPrefillRows = 256;       // query rows of one CTA: two tensor-core tiles

// The most keys of one item.  The tensor cores cut the sum of products and
// accumulator off, 2.5e-7 of O a tile: 5e-4 over this many, a quarter of the rounding
// of a bf16 output.
constexpr int kPrefillMostKeys = 2048 * kPrefillTile;

// Splits of a request's `len` keys for chunk length `chunk` (a multiple of
// kPrefillTile), at least one, and their length: equal, whole tiles.
FD_HD int32_t prefill_splits(int32_t len, int32_t chunk)
{
    return len > chunk ? (len - 1) / chunk + 1 : 1;
}

FD_HD int32_t prefill_split_len(int32_t len, int32_t splits)
{
    const int32_t even = len > 0 ? (len - 1) / splits + 1 : 1;
    return (even + kPrefillTile - 1) / kPrefillTile * kPrefillTile;
}

struct PrefillParams {
    const uint16_t *q;               // bf16, token stride q_stride, heads contiguous
    int64_t q_stride;                // elements
    const int32_t *q_indptr;         // [B+1] tokens of each request
    const int32_t *page_indptr, *last_len, *page_indices;
    const int8_t *k, *v;             // [num_pages, page_size, Hkv, D]
    const float *k_scale, *v_scale;  // [num_pages, scale_heads]
    uint16_t *o;                     // bf16 [num_tokens, Hq, D]
    float *lse;                      // [num_tokens, Hq], or null
    float *partial_o, *partial_lse;  // rows of requests with several splits
    int *status;
    int32_t batch, num_tokens, num_qo_heads, num_kv_heads, group, group_log2;
    int32_t page_size, num_pages, page_entries, scale_heads;
    int32_t causal, chunk, num_items, num_partial_rows, merge_rows;
    float scale;
    int64_t timeout_ns;
};

// Stage 1 (p.num_items CTAs), and the merge of the requests with several splits.
cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t stream);

}  // namespace fd
