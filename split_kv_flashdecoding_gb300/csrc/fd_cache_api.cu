// fd_cache_api.cu -- the C entry points that write and rearrange a paged
// cache: rotary positions and append, page copies, forks and compaction.  See
// include/fd.h for the contract of each.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "api_util.h"
#include "cache_kernels.h"
#include "fd.h"
#include "kernels.h"
#include "stage1.h"

using fd::aligned;
using fd::as_stream;
using fd::round_up;

namespace {

constexpr int kHeadDim = 128;

// The fraction of `turns` as a 64-bit fixed-point number.
uint64_t turns_to_fixed(double turns)
{
    const double f = turns - floor(turns);
    const double hi = floor(ldexp(f, 32));
    const double lo = floor(ldexp(ldexp(f, 32) - hi, 32));
    return ((uint64_t)hi << 32) + (uint64_t)lo;
}

// Whether two lists share memory.
bool overlap(const int32_t *a, int64_t na, const int32_t *b, int64_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + nb * sizeof(int32_t) && y < x + na * sizeof(int32_t);
}

bool finite_positive(double x)
{
    return x > 0 && x <= 1e300;
}

}  // namespace

extern "C" int fd_plan_rope(int head_dim, int rotary_dim, const fd_rope_config *config, fd_rope_info *info)
{
    if (!info || !config || !finite_positive(config->base) || config->base < 1.0)
        return FD_ERR_INVALID_ARG;
    const double base = config->base, factor = config->factor, trained_len = config->trained_len;
    const double low = config->low, high = config->high;
    const int scaling = config->scaling;
    if (head_dim != kHeadDim || rotary_dim % 16 != 0)
        return FD_ERR_UNSUPPORTED;
    if (rotary_dim <= 0 || rotary_dim > head_dim)
        return FD_ERR_INVALID_ARG;
    if (scaling != FD_ROPE_PLAIN && scaling != FD_ROPE_LINEAR && scaling != FD_ROPE_BANDS &&
        scaling != FD_ROPE_YARN)
        return FD_ERR_INVALID_ARG;
    if (scaling != FD_ROPE_PLAIN && !(finite_positive(factor) && factor >= 1.0))
        return FD_ERR_INVALID_ARG;
    const bool bands = scaling == FD_ROPE_BANDS, yarn = scaling == FD_ROPE_YARN;
    if ((bands || yarn) && !(finite_positive(trained_len) && finite_positive(low) && finite_positive(high) &&
                             low < high))
        return FD_ERR_INVALID_ARG;
    if (yarn && base <= 1.0)
        return FD_ERR_INVALID_ARG;

    memset(info, 0, sizeof *info);
    info->head_dim = head_dim;
    info->rotary_dim = rotary_dim;
    info->interleaved = config->interleaved != 0;
    info->gain = yarn ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    const double two_pi = 6.283185307179586476925;
    // YaRN: the pair whose wavelength makes n turns over the trained length
    auto pair_of = [&](double turns) {
        return rotary_dim * log(trained_len / (turns * two_pi)) / (2.0 * log(base));
    };
    double first = 0, last = 1;
    if (yarn) {
        first = floor(pair_of(high));
        last = ceil(pair_of(low));
        first = first < 0 ? 0 : first;
        last = last > rotary_dim - 1 ? rotary_dim - 1 : last;
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rotary_dim);
        double keep = 1.0;   // share of the unscaled frequency
        if (scaling == FD_ROPE_LINEAR) {
            keep = 0.0;
        } else if (bands) {
            keep = (trained_len * f / two_pi - low) / (high - low);
        } else if (yarn) {
            const double width = last - first < 1e-3 ? 1e-3 : last - first;
            keep = 1.0 - (i - first) / width;
        }
        keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
        if (scaling != FD_ROPE_PLAIN)
            f = f * keep + f / factor * (1.0 - keep);
        info->step[i] = turns_to_fixed(f / two_pi);
    }
    return FD_OK;
}

namespace {

int append(int batch, int num_tokens, int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
           int num_pages, const fd_rope_info *rope, const void *q, int64_t q_stride, const void *k,
           int64_t k_stride, const void *v, int64_t v_stride, const int32_t *append_indptr_dev,
           const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
           const int32_t *kv_page_indices_dev, int num_page_entries, const int32_t *positions_dev, void *q_out,
           int64_t q_out_stride, void *k_pages, void *v_pages, const float *k_scale, const float *v_scale,
           float *k_scale_out, float *v_scale_out, int kv_type, void *workspace, int64_t workspace_bytes,
           void *stream)
{
    if (batch < 0 || num_tokens < 0 || num_qo_heads < 0 || num_kv_heads <= 0 || num_page_entries < 0)
        return FD_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || page_size <= 0 || page_size % 16 != 0 || num_qo_heads > 4096 ||
        num_kv_heads > 4096)
        return FD_ERR_UNSUPPORTED;
    if (num_pages <= 0 || (int64_t)num_pages * page_size > INT32_MAX)
        return FD_ERR_INVALID_ARG;
    if (rope && (rope->head_dim != head_dim || rope->rotary_dim <= 0 || rope->rotary_dim > head_dim ||
                 rope->rotary_dim % 16 != 0))
        return FD_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < FD_WORKSPACE_HEADER_BYTES)
        return FD_ERR_WORKSPACE;
    if (!aligned(workspace, 16))
        return FD_ERR_INVALID_ARG;
    if (batch == 0 || num_tokens == 0)
        return FD_OK;
    const bool has_q = num_qo_heads > 0;
    if ((has_q && (!q || !q_out)) || !k || !v || !k_pages || !v_pages || !append_indptr_dev ||
        !kv_page_indptr_dev || !kv_last_page_len_dev || !kv_page_indices_dev)
        return FD_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) ||
        !aligned(v_pages, 16) || !aligned(append_indptr_dev, 4) || !aligned(kv_page_indptr_dev, 4) ||
        !aligned(kv_last_page_len_dev, 4) || !aligned(kv_page_indices_dev, 4) || !aligned(positions_dev, 4))
        return FD_ERR_INVALID_ARG;
    // a token's heads must not overlap the next token's, and 16-byte chunks stay aligned
    const int64_t q_row = (int64_t)num_qo_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
    if ((has_q && (q_stride < q_row || q_out_stride < q_row || q_stride % 8 || q_out_stride % 8)) ||
        k_stride < kv_row || v_stride < kv_row || k_stride % 8 || v_stride % 8)
        return FD_ERR_INVALID_ARG;
    // The rotated queries may go over the queries themselves; elsewhere they would
    // change what other threads still read.
    const bool in_place = q_out == q && (q_out_stride == q_stride || num_tokens == 1);
    if (has_q && ((!in_place && fd::rows_overlap(q_out, q_row, q_out_stride, q, q_row, q_stride, num_tokens)) ||
                  fd::rows_overlap(q_out, q_row, q_out_stride, k, kv_row, k_stride, num_tokens) ||
                  fd::rows_overlap(q_out, q_row, q_out_stride, v, kv_row, v_stride, num_tokens)))
        return FD_ERR_INVALID_ARG;
    if (kv_type == fd::kKvTypeFp8 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)))
        return FD_ERR_INVALID_ARG;
    if ((kv_type == fd::kKvTypeInt4 || kv_type == fd::kKvTypeInt8) &&
        (!k_scale_out || !v_scale_out || !aligned(k_scale_out, 4) || !aligned(v_scale_out, 4)))
        return FD_ERR_INVALID_ARG;

    if (kv_type == fd::kKvTypeInt8 && (int64_t)num_tokens * (num_kv_heads + 2) > INT32_MAX)   // its grid
        return FD_ERR_INVALID_ARG;

    fd::AppendParams p;
    memset(&p, 0, sizeof p);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_scale_out = k_scale_out;
    p.v_scale_out = v_scale_out;
    p.scale_heads = fd::scale_heads(num_kv_heads);
    p.append_indptr = append_indptr_dev;
    p.kv_page_indptr = kv_page_indptr_dev;
    p.kv_last_page_len = kv_last_page_len_dev;
    p.kv_page_indices = kv_page_indices_dev;
    p.positions = positions_dev;
    p.status = static_cast<int *>(workspace);
    p.batch = batch;
    p.num_tokens = num_tokens;
    p.num_qo_heads = num_qo_heads;
    p.num_kv_heads = num_kv_heads;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.num_page_entries = num_page_entries;
    if (rope)
        p.rope = *rope;
    return fd::launch_append(p, kv_type, as_stream(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

}  // namespace

extern "C" int fd_append_paged(int batch, int num_tokens, int num_qo_heads, int num_kv_heads, int head_dim,
                               int page_size, int num_pages, const fd_rope_info *rope, const void *q,
                               int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                               int64_t v_stride, const int32_t *append_indptr_dev,
                               const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
                               const int32_t *kv_page_indices_dev, int num_page_entries,
                               const int32_t *positions_dev, void *q_out, int64_t q_out_stride, void *k_pages,
                               void *v_pages, void *workspace, int64_t workspace_bytes, void *stream)
{
    return append(batch, num_tokens, num_qo_heads, num_kv_heads, head_dim, page_size, num_pages, rope, q,
                  q_stride, k, k_stride, v, v_stride, append_indptr_dev, kv_page_indptr_dev,
                  kv_last_page_len_dev, kv_page_indices_dev, num_page_entries, positions_dev, q_out,
                  q_out_stride, k_pages, v_pages, nullptr, nullptr, nullptr, nullptr, fd::kKvTypeBf16, workspace,
                  workspace_bytes, stream);
}

extern "C" int fd_append_paged_fp8(int batch, int num_tokens, int num_qo_heads, int num_kv_heads, int head_dim,
                                   int page_size, int num_pages, const fd_rope_info *rope, const void *q,
                                   int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                   int64_t v_stride, const int32_t *append_indptr_dev,
                                   const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
                                   const int32_t *kv_page_indices_dev, int num_page_entries,
                                   const int32_t *positions_dev, void *q_out, int64_t q_out_stride,
                                   void *k_pages_fp8, void *v_pages_fp8, const float *k_scale,
                                   const float *v_scale, void *workspace, int64_t workspace_bytes, void *stream)
{
    return append(batch, num_tokens, num_qo_heads, num_kv_heads, head_dim, page_size, num_pages, rope, q,
                  q_stride, k, k_stride, v, v_stride, append_indptr_dev, kv_page_indptr_dev,
                  kv_last_page_len_dev, kv_page_indices_dev, num_page_entries, positions_dev, q_out,
                  q_out_stride, k_pages_fp8, v_pages_fp8, k_scale, v_scale, nullptr, nullptr, fd::kKvTypeFp8,
                  workspace, workspace_bytes, stream);
}

extern "C" int fd_append_paged_int4(int batch, int num_tokens, int num_qo_heads, int num_kv_heads, int head_dim,
                                    int page_size, int num_pages, const fd_rope_info *rope, const void *q,
                                    int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                    int64_t v_stride, const int32_t *append_indptr_dev,
                                    const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
                                    const int32_t *kv_page_indices_dev, int num_page_entries,
                                    const int32_t *positions_dev, void *q_out, int64_t q_out_stride,
                                    void *k_pages_int4, void *v_pages_int4, float *k_scale, float *v_scale,
                                    void *workspace, int64_t workspace_bytes, void *stream)
{
    return append(batch, num_tokens, num_qo_heads, num_kv_heads, head_dim, page_size, num_pages, rope, q,
                  q_stride, k, k_stride, v, v_stride, append_indptr_dev, kv_page_indptr_dev,
                  kv_last_page_len_dev, kv_page_indices_dev, num_page_entries, positions_dev, q_out,
                  q_out_stride, k_pages_int4, v_pages_int4, nullptr, nullptr, k_scale, v_scale, fd::kKvTypeInt4,
                  workspace, workspace_bytes, stream);
}

extern "C" int fd_append_paged_int8(int batch, int num_tokens, int num_qo_heads, int num_kv_heads, int head_dim,
                                    int page_size, int num_pages, const fd_rope_info *rope, const void *q,
                                    int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                    int64_t v_stride, const int32_t *append_indptr_dev,
                                    const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
                                    const int32_t *kv_page_indices_dev, int num_page_entries,
                                    const int32_t *positions_dev, void *q_out, int64_t q_out_stride,
                                    void *k_pages_int8, void *v_pages_int8, float *k_scale, float *v_scale,
                                    void *workspace, int64_t workspace_bytes, void *stream)
{
    return append(batch, num_tokens, num_qo_heads, num_kv_heads, head_dim, page_size, num_pages, rope, q,
                  q_stride, k, k_stride, v, v_stride, append_indptr_dev, kv_page_indptr_dev,
                  kv_last_page_len_dev, kv_page_indices_dev, num_page_entries, positions_dev, q_out,
                  q_out_stride, k_pages_int8, v_pages_int8, nullptr, nullptr, k_scale, v_scale, fd::kKvTypeInt8,
                  workspace, workspace_bytes, stream);
}

extern "C" int fd_copy_pages(int num_pools, void *const *pools, const int64_t *page_bytes, int num_pages,
                             int num_copies, const int32_t *src_dev, const int32_t *dst_dev, void *workspace,
                             int64_t workspace_bytes, void *stream)
{
    if (num_pools < 0 || num_pages < 0 || num_copies < 0 || (num_pools > 0 && (!pools || !page_bytes)))
        return FD_ERR_INVALID_ARG;
    if (workspace && workspace_bytes < FD_WORKSPACE_HEADER_BYTES)
        return FD_ERR_WORKSPACE;
    if (!aligned(workspace, 16))
        return FD_ERR_INVALID_ARG;
    auto segments = [](int64_t bytes) { return (bytes - 1) / fd::kCopySegment + 1; };
    for (int i = 0; i < num_pools; ++i) {   // all of them, before the first is copied
        if (!pools[i] || !aligned(pools[i], 16) || page_bytes[i] <= 0 || page_bytes[i] % 16 != 0 ||
            (num_copies > 0 && segments(page_bytes[i]) > INT32_MAX / num_copies))
            return FD_ERR_INVALID_ARG;
    }
    if (num_pools == 0 || num_copies == 0 || num_pages == 0)
        return FD_OK;
    if (!src_dev || !dst_dev || !aligned(src_dev, 4) || !aligned(dst_dev, 4))
        return FD_ERR_INVALID_ARG;
    fd::CopyPagesParams p;
    p.src = src_dev;
    p.dst = dst_dev;
    p.status = static_cast<int *>(workspace);
    p.num_pages = num_pages;
    p.num_copies = num_copies;
    for (int i0 = 0; i0 < num_pools; i0 += fd::kMaxPools) {
        const int n = num_pools - i0 < fd::kMaxPools ? num_pools - i0 : fd::kMaxPools;
        int64_t most = 0;
        for (int i = 0; i < n; ++i) {
            p.pool[i] = static_cast<uint8_t *>(pools[i0 + i]);
            p.page_bytes[i] = page_bytes[i0 + i];
            most = page_bytes[i0 + i] > most ? page_bytes[i0 + i] : most;
        }
        p.segments = (int32_t)segments(most);
        if (fd::launch_copy_pages(p, n, as_stream(stream)) != cudaSuccess)
            return FD_ERR_CUDA;
    }
    return FD_OK;
}

namespace {

// The most pages that a cache can have (16 keys each, key rows are 32-bit numbers).
constexpr int kMaxPages = INT32_MAX / 16;

int page_blocks(int num_pages)
{
    return (num_pages + fd::kPagesPerBlock - 1) / fd::kPagesPerBlock;
}

// header | the tickets of other calls, left as they are | info (256 bytes) | block counts |
// list [num_pages] | child arrays [max_batch] x 2
fd::PagesScratch pages_scratch(void *workspace, int num_pages, int max_batch)
{
    uint8_t *w = static_cast<uint8_t *>(workspace) + FD_WORKSPACE_HEADER_BYTES + fd::kTicketBytes;
    fd::PagesScratch s;
    s.info = reinterpret_cast<int *>(w);
    s.block_count = reinterpret_cast<int *>(w += 256);
    s.list = reinterpret_cast<int *>(w += round_up((int64_t)page_blocks(num_pages) * 4, 256));
    s.child_rank = reinterpret_cast<int *>(w += round_up((int64_t)num_pages * 4, 256));
    s.child_copy = reinterpret_cast<int *>(w += round_up((int64_t)max_batch * 4, 256));
    return s;
}

}  // namespace

extern "C" int fd_pages_workspace_bytes(int num_pages, int new_batch, int64_t *bytes)
{
    if (!bytes || num_pages < 0 || num_pages > kMaxPages || new_batch < 0)
        return FD_ERR_INVALID_ARG;
    *bytes = FD_WORKSPACE_HEADER_BYTES + fd::kTicketBytes + 256 + round_up((int64_t)page_blocks(num_pages) * 4, 256) +
             round_up((int64_t)num_pages * 4, 256) + 2 * round_up((int64_t)new_batch * 4, 256);
    return FD_OK;
}

extern "C" int fd_fork_pages(int old_batch, int new_batch, int page_size, int num_pages,
                             const int32_t *parent_dev, const int32_t *kv_page_indptr_dev,
                             const int32_t *kv_last_page_len_dev, const int32_t *kv_page_indices_dev,
                             int num_page_entries, const int32_t *new_page_indptr_dev, int new_page_entries,
                             const int32_t *page_refs_dev, int32_t *new_page_indices_dev, int32_t *new_page_refs_dev,
                             int32_t *copy_src_dev, int32_t *copy_dst_dev, void *workspace,
                             int64_t workspace_bytes, void *stream)
{
    if (old_batch < 0 || new_batch < 0 || num_pages <= 0 || num_pages > kMaxPages || num_page_entries < 0 || new_page_entries < 0 ||
        page_size <= 0)
        return FD_ERR_INVALID_ARG;
    if (old_batch > fd::kMaxTableBatch || new_batch > fd::kMaxTableBatch)
        return FD_ERR_UNSUPPORTED;
    int64_t need;
    fd_pages_workspace_bytes(num_pages, new_batch, &need);
    if (!workspace || workspace_bytes < need)
        return FD_ERR_WORKSPACE;
    if (!page_refs_dev || !new_page_refs_dev)
        return FD_ERR_INVALID_ARG;
    if ((old_batch > 0 && (!kv_page_indptr_dev || !kv_last_page_len_dev)) ||
        (num_page_entries > 0 && !kv_page_indices_dev))
        return FD_ERR_INVALID_ARG;
    if ((new_batch > 0 && (!parent_dev || !new_page_indptr_dev || !copy_src_dev || !copy_dst_dev)) ||
        (new_page_entries > 0 && !new_page_indices_dev))
        return FD_ERR_INVALID_ARG;
    if (new_page_refs_dev != page_refs_dev && overlap(new_page_refs_dev, num_pages, page_refs_dev, num_pages))
        return FD_ERR_INVALID_ARG;
    if (overlap(new_page_indices_dev, new_page_entries, kv_page_indices_dev, num_page_entries))
        return FD_ERR_INVALID_ARG;   // a child's table is read after another's is written
    const void *ptrs[] = {parent_dev, kv_page_indptr_dev, kv_last_page_len_dev, kv_page_indices_dev,
                          new_page_indptr_dev, page_refs_dev, new_page_indices_dev, new_page_refs_dev,
                          copy_src_dev, copy_dst_dev};
    for (const void *x : ptrs)
        if (!aligned(x, 4))
            return FD_ERR_INVALID_ARG;
    if (!aligned(workspace, 16))
        return FD_ERR_INVALID_ARG;
    fd::ForkParams p;
    p.parent = parent_dev;
    p.page_indptr = kv_page_indptr_dev;
    p.last_len = kv_last_page_len_dev;
    p.indices = kv_page_indices_dev;
    p.new_indptr = new_page_indptr_dev;
    p.refs_in = page_refs_dev;
    p.refs_out = new_page_refs_dev;
    p.new_indices = new_page_indices_dev;
    p.copy_src = copy_src_dev;
    p.copy_dst = copy_dst_dev;
    p.status = static_cast<int *>(workspace);
    p.old_batch = old_batch;
    p.new_batch = new_batch;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.old_entries = num_page_entries;
    p.new_entries = new_page_entries;
    p.blocks = page_blocks(num_pages);
    p.s = pages_scratch(workspace, num_pages, new_batch);
    return fd::launch_fork(p, as_stream(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

extern "C" int fd_compact_pages(int num_pages, const int32_t *page_refs_dev, const int32_t *kv_page_indices_dev,
                                int num_page_entries, int limit, int max_moves, int32_t *new_page_indices_dev,
                                int32_t *new_page_refs_dev, int32_t *copy_src_dev, int32_t *copy_dst_dev,
                                void *workspace, int64_t workspace_bytes, void *stream)
{
    if (num_pages <= 0 || num_pages > kMaxPages || num_page_entries < 0 || limit < 0 || max_moves < 0)
        return FD_ERR_INVALID_ARG;
    int64_t need;
    fd_pages_workspace_bytes(num_pages, 0, &need);
    if (!workspace || workspace_bytes < need)
        return FD_ERR_WORKSPACE;
    if (!page_refs_dev || !new_page_refs_dev || (num_page_entries > 0 && (!kv_page_indices_dev || !new_page_indices_dev)) ||
        (max_moves > 0 && (!copy_src_dev || !copy_dst_dev)))
        return FD_ERR_INVALID_ARG;
    // in place, entry by entry, or apart
    if ((new_page_indices_dev != kv_page_indices_dev &&
         overlap(new_page_indices_dev, num_page_entries, kv_page_indices_dev, num_page_entries)) ||
        (new_page_refs_dev != page_refs_dev && overlap(new_page_refs_dev, num_pages, page_refs_dev, num_pages)))
        return FD_ERR_INVALID_ARG;
    const void *ptrs[] = {page_refs_dev, kv_page_indices_dev, new_page_indices_dev, new_page_refs_dev,
                          copy_src_dev, copy_dst_dev};
    for (const void *x : ptrs)
        if (!aligned(x, 4))
            return FD_ERR_INVALID_ARG;
    if (!aligned(workspace, 16))
        return FD_ERR_INVALID_ARG;
    fd::CompactParams p;
    p.refs_in = page_refs_dev;
    p.indices = kv_page_indices_dev;
    p.refs_out = new_page_refs_dev;
    p.new_indices = new_page_indices_dev;
    p.copy_src = copy_src_dev;
    p.copy_dst = copy_dst_dev;
    p.status = static_cast<int *>(workspace);
    p.num_pages = num_pages;
    p.entries = num_page_entries;
    p.limit = limit;
    p.max_moves = max_moves;
    p.blocks = page_blocks(num_pages);
    p.s = pages_scratch(workspace, num_pages, 0);
    return fd::launch_compact(p, as_stream(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}
