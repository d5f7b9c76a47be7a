// cache_kernels.h -- parameters and launchers of the kernels that write and
// rearrange a paged cache (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fd.h"

namespace fd {

// Rotary positions and the write of new keys and values into a paged cache.
struct AppendParams {
    const uint16_t *q;           // bf16, token stride q_stride, heads contiguous; null: no queries
    const uint16_t *k, *v;
    uint16_t *q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;   // elements
    void *k_pages, *v_pages;
    const float *k_scale, *v_scale;   // FP8: [Hkv], read
    // written: INT4 [Hkv][num_pages * page_size]; INT8 [num_pages][scale_heads], read too
    float *k_scale_out, *v_scale_out;
    const int32_t *append_indptr, *kv_page_indptr, *kv_last_page_len, *kv_page_indices, *positions;
    int *status;
    int32_t batch, num_tokens, num_qo_heads, num_kv_heads, page_size, num_pages, num_page_entries;
    int32_t tokens_per_cta;
    int32_t scale_heads, page_ctas, blocks_per_page;   // INT8
    fd_rope_info rope;           // rotary_dim 0: no rotation
};

cudaError_t launch_append(const AppendParams &p, int kv_type, cudaStream_t stream);

// Page copies within each of several pools.
constexpr int kMaxPools = 128;
struct CopyPagesParams {
    uint8_t *pool[kMaxPools];
    int64_t page_bytes[kMaxPools];
    const int32_t *src, *dst;
    int *status;                 // may be null
    int32_t num_pages, num_copies, segments;
};
constexpr int kCopySegment = 16384;   // bytes of a page that one CTA copies

cudaError_t launch_copy_pages(const CopyPagesParams &p, int num_pools, cudaStream_t stream);

// Scratch of fork and compact behind the workspace header.
struct PagesScratch {
    int *info;           // [16] counts of the call, see pages_kernel.cu
    int *block_count;    // [blocks]
    int *list;           // [num_pages] ranks of the moving pages (compact); free pages, a bit each (fork)
    int *child_rank;     // [max_batch] fresh pages before each child's (fork)
    int *child_copy;     // [max_batch] 1: its last page is a copy of its parent's
};
constexpr int kPagesPerBlock = 1024;
constexpr int kMaxTableBatch = 32768;   // requests of a fork's tables (their index in shared memory)

struct ForkParams {
    const int32_t *parent, *page_indptr, *last_len, *indices, *new_indptr, *refs_in;
    int32_t *refs_out, *new_indices, *copy_src, *copy_dst;
    int *status;
    int32_t old_batch, new_batch, page_size, num_pages, old_entries, new_entries, blocks;
    PagesScratch s;
};
cudaError_t launch_fork(const ForkParams &p, cudaStream_t stream);

struct CompactParams {
    const int32_t *refs_in, *indices;
    int32_t *refs_out, *new_indices, *copy_src, *copy_dst;
    int *status;
    int32_t num_pages, entries, limit, max_moves, blocks;
    PagesScratch s;
};
cudaError_t launch_compact(const CompactParams &p, cudaStream_t stream);

}  // namespace fd
