// fd_prefill_api.cu -- the C entry points of attention of many query tokens a request
// over an INT8 paged cache: the plan (host only) and the launches.  See include/fd.h
// for the contract.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "api_util.h"
#include "fd.h"
#include "prefill_kernels.h"
#include "stage1.h"

using fd::aligned;
using fd::as_stream;
using fd::round_up;

namespace {

constexpr int kHeadDim = 128;
constexpr int kMaxSlots = 1024;   // SMs the plan can balance over
constexpr int kMostMerged = INT32_MAX - 64;   // the merge's grid counts rows up to its last CTA's

// The plan's view of its requests.
struct Requests {
    int batch, num_qo_heads, num_kv_heads, causal;
    const int32_t *q_indptr, *page_indptr, *last_len;
    int32_t page_size;

    int64_t tokens(int b) const
    {
        return (int64_t)q_indptr[b + 1] - q_indptr[b];
    }
    int64_t keys(int b) const
    {
        const int64_t n = (int64_t)page_indptr[b + 1] - page_indptr[b];
        return n <= 0 ? n : (n - 1) * page_size + last_len[b];
    }
    int64_t blocks(int b) const
    {
        return (tokens(b) * (num_qo_heads / num_kv_heads) + fd::kPrefillRows - 1) / fd::kPrefillRows;
    }
};

struct PlanSize {
    int64_t items, rows, merge;
};

PlanSize size_of(const Requests &x, int32_t chunk)
{
    PlanSize z{0, 0, 0};
    for (int b = 0; b < x.batch; ++b) {
        if (x.tokens(b) <= 0)
            continue;
        const int64_t splits = fd::prefill_splits((int32_t)x.keys(b), chunk);
        z.items += splits * x.blocks(b) * x.num_kv_heads;
        if (splits > 1) {
            z.merge += x.tokens(b) * x.num_qo_heads;
            z.rows += splits * x.tokens(b) * x.num_qo_heads;
        }
    }
    return z;
}

// Costs in SM cycles: a 128-key tile of one and of two 128-row tiles, a CTA's start
// and end, a partial row's write and read over all SMs, the merge's launch.
constexpr int64_t kTileOne = 2300, kTileTwo = 3120, kItemCost = 20000;
constexpr double kRowCost = 0.25, kMergeCost = 6000;

// Time of the grid for chunk length c: its CTAs go, in launch order, to the SM that
// is free first.
double grid_time(const Requests &x, int32_t chunk, int slots)
{
    int64_t heap[kMaxSlots];
    for (int i = 0; i < slots; ++i)
        heap[i] = 0;
    const auto later = [](int64_t a, int64_t b) { return a > b; };
    const int group = x.num_qo_heads / x.num_kv_heads;
    for (int b = 0; b < x.batch; ++b) {
        const int64_t tokens = x.tokens(b), keys = x.keys(b), rows = tokens * group;
        if (tokens <= 0)
            continue;
        const int32_t splits = fd::prefill_splits((int32_t)keys, chunk);
        const int64_t len = fd::prefill_split_len((int32_t)keys, splits);
        for (int64_t block = x.blocks(b) - 1; block >= 0; --block) {
            const int64_t row0 = block * fd::kPrefillRows, mine = std::min<int64_t>(rows - row0, fd::kPrefillRows);
            const int64_t end = x.causal ? std::min(keys, keys - tokens + (row0 + mine - 1) / group + 1) : keys;
            for (int32_t s = 0; s < splits; ++s) {
                const int64_t here = std::max<int64_t>(0, std::min(end - s * len, len));
                const int64_t tiles = (here + fd::kPrefillTile - 1) / fd::kPrefillTile;
                const int64_t cost = kItemCost + tiles * (mine > fd::kPrefillRows / 2 ? kTileTwo : kTileOne);
                for (int h = 0; h < x.num_kv_heads; ++h) {
                    std::pop_heap(heap, heap + slots, later);
                    heap[slots - 1] += cost;
                    std::push_heap(heap, heap + slots, later);
                }
            }
        }
    }
    const PlanSize z = size_of(x, chunk);
    return (double)*std::max_element(heap, heap + slots) + (double)z.rows * kRowCost + (z.merge ? kMergeCost : 0);
}

// The chunk length: one split a request, or for grids of up to 1, 2, .. 8 waves of
// CTAs (one an SM) the shortest chunk that fits, whichever has the shortest time.
int32_t choose_chunk(const Requests &x, int num_sms)
{
    int64_t longest = 1;
    for (int b = 0; b < x.batch; ++b)
        longest = std::max(longest, x.tokens(b) > 0 ? x.keys(b) : 0);
    const int slots = std::min(num_sms, kMaxSlots);
    const int32_t most = (int32_t)std::min<int64_t>((longest + fd::kPrefillTile - 1) / fd::kPrefillTile,
                                                    fd::kPrefillMostKeys / fd::kPrefillTile);
    int32_t best = most;
    // many more items than waves already: nothing to gain from splits
    if (size_of(x, most * fd::kPrefillTile).items > 16LL * slots)
        return most * fd::kPrefillTile;
    double best_time = grid_time(x, most * fd::kPrefillTile, slots);
    int32_t last = most;
    for (int waves = 1; waves <= 8; ++waves) {
        int32_t lo = 1, hi = most;   // in tiles; items fall as the chunk grows
        while (lo < hi) {
            const int32_t mid = lo + (hi - lo) / 2;
            if (size_of(x, mid * fd::kPrefillTile).items <= (int64_t)waves * slots)
                hi = mid;
            else
                lo = mid + 1;
        }
        if (lo == last)
            continue;
        last = lo;
        const double t = grid_time(x, lo * fd::kPrefillTile, slots);
        if (t < best_time) {
            best_time = t;
            best = lo;
        }
    }
    return best * fd::kPrefillTile;
}

// Workspace of a plan: header | tickets of other calls, left as they are | partial LSE |
// partial O.
int64_t prefill_bytes(int64_t rows)
{
    return FD_WORKSPACE_HEADER_BYTES + fd::kTicketBytes + round_up(rows * 4, 256) + rows * kHeadDim * 4;
}

}  // namespace

extern "C" int fd_plan_prefill_paged(int batch, int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                                     const int32_t *q_indptr_host, const int32_t *kv_page_indptr_host,
                                     const int32_t *kv_last_page_len_host, int causal, int num_sms, int chunk,
                                     fd_prefill_plan *plan)
{
    if (!plan || batch < 0 || num_qo_heads <= 0 || num_kv_heads <= 0 || num_qo_heads % num_kv_heads != 0 ||
        !q_indptr_host || !kv_page_indptr_host || (batch > 0 && !kv_last_page_len_host))
        return FD_ERR_INVALID_ARG;
    const int group = num_qo_heads / num_kv_heads;
    if (head_dim != kHeadDim || page_size <= 0 || page_size % 16 != 0 || num_qo_heads > 4096 ||
        (group != 1 && group != 2 && group != 4 && group != 8))
        return FD_ERR_UNSUPPORTED;
    if (num_sms < 0 || chunk < 0 || chunk % fd::kPrefillTile != 0 || chunk > fd::kPrefillMostKeys)
        return FD_ERR_INVALID_ARG;
    if (q_indptr_host[0] != 0 || kv_page_indptr_host[0] != 0)
        return FD_ERR_INVALID_ARG;
    const Requests x{batch, num_qo_heads, num_kv_heads, causal != 0, q_indptr_host, kv_page_indptr_host,
                     kv_last_page_len_host, page_size};
    for (int b = 0; b < batch; ++b) {
        if (x.tokens(b) < 0 || kv_page_indptr_host[b + 1] < kv_page_indptr_host[b])
            return FD_ERR_INVALID_ARG;
        if (kv_page_indptr_host[b + 1] > kv_page_indptr_host[b] &&
            (kv_last_page_len_host[b] < 1 || kv_last_page_len_host[b] > page_size))
            return FD_ERR_INVALID_ARG;
        if (x.keys(b) > INT32_MAX - fd::kPrefillTile)
            return FD_ERR_INVALID_ARG;
    }
    if ((int64_t)q_indptr_host[batch] * group > INT32_MAX - fd::kPrefillRows)
        return FD_ERR_INVALID_ARG;
    if (num_sms == 0) {
        const int rc = fd_num_sms(-1, &num_sms);
        if (rc != FD_OK)
            return rc;
    }
    if (chunk == 0)
        chunk = choose_chunk(x, num_sms);
    const PlanSize z = size_of(x, chunk);
    // CTAs and rows are counted in 32 bits (what lies in a row, and its bytes, in 64)
    if (z.items > INT32_MAX || z.rows > INT32_MAX || z.merge > kMostMerged)
        return FD_ERR_UNSUPPORTED;
    memset(plan, 0, sizeof *plan);
    plan->batch = batch;
    plan->num_tokens = q_indptr_host[batch];
    plan->num_qo_heads = num_qo_heads;
    plan->num_kv_heads = num_kv_heads;
    plan->head_dim = head_dim;
    plan->page_size = page_size;
    plan->causal = causal != 0;
    plan->chunk = chunk;
    plan->num_items = (int32_t)z.items;
    plan->num_partial_rows = (int32_t)z.rows;
    plan->num_merged_rows = (int32_t)z.merge;
    plan->num_page_entries = kv_page_indptr_host[batch];
    plan->workspace_bytes = prefill_bytes(z.rows);
    plan->timeout_ns = FD_DEFAULT_TIMEOUT_NS;
    return FD_OK;
}

extern "C" int fd_prefill_paged_int8(const fd_prefill_plan *plan, int num_pages, const int32_t *q_indptr_dev,
                                     const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
                                     const int32_t *kv_page_indices_dev, const void *q, int64_t q_stride,
                                     const void *k_pages_int8, const void *v_pages_int8, const float *k_scale,
                                     const float *v_scale, float scale, void *o, float *lse, void *workspace,
                                     int64_t workspace_bytes, void *stream)
{
    if (!plan)
        return FD_ERR_INVALID_ARG;
    const fd_prefill_plan &x = *plan;
    if (x.batch < 0 || x.num_tokens < 0 || x.num_qo_heads <= 0 || x.num_kv_heads <= 0 ||
        x.num_qo_heads % x.num_kv_heads != 0 || x.num_items < 0 || x.num_partial_rows < 0 || x.num_merged_rows < 0 ||
        x.num_merged_rows > x.num_partial_rows || x.num_merged_rows > kMostMerged || x.num_page_entries < 0 || x.chunk <= 0 ||
        x.chunk % fd::kPrefillTile != 0 || x.workspace_bytes < prefill_bytes(x.num_partial_rows))
        return FD_ERR_INVALID_ARG;
    const int group = x.num_qo_heads / x.num_kv_heads;
    if (x.head_dim != kHeadDim || x.page_size <= 0 || x.page_size % 16 != 0 || x.num_qo_heads > 4096 ||
        (group != 1 && group != 2 && group != 4 && group != 8))
        return FD_ERR_UNSUPPORTED;
    if ((int64_t)x.num_tokens * group > INT32_MAX - fd::kPrefillRows)
        return FD_ERR_INVALID_ARG;
    // O may go over the queries themselves, which a CTA has read before it writes; elsewhere
    // it would change what others still read.
    const int64_t row = (int64_t)x.num_qo_heads * kHeadDim;
    if (q && o && x.num_items > 0 && !(o == q && (q_stride == row || x.num_tokens == 1)) &&
        fd::rows_overlap(o, row, row, q, row, q_stride, x.num_tokens))
        return FD_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < x.workspace_bytes)
        return FD_ERR_WORKSPACE;
    if (!aligned(workspace, 16))
        return FD_ERR_INVALID_ARG;
    if (x.num_items == 0)
        return FD_OK;
    if (!q || !o || !q_indptr_dev || !kv_page_indptr_dev || !kv_last_page_len_dev ||
        (x.num_page_entries > 0 && (!kv_page_indices_dev || !k_pages_int8 || !v_pages_int8 || !k_scale || !v_scale)))
        return FD_ERR_INVALID_ARG;
    if (num_pages < 0 || (x.num_page_entries > 0 && num_pages == 0) || (int64_t)num_pages * x.page_size > INT32_MAX)
        return FD_ERR_INVALID_ARG;
    if (!(scale - scale == 0.f))   // finite
        return FD_ERR_INVALID_ARG;
    if (q_stride < (int64_t)x.num_qo_heads * kHeadDim || q_stride % 8 != 0)
        return FD_ERR_INVALID_ARG;
    const void *p16[] = {q, k_pages_int8, v_pages_int8, o};
    for (const void *y : p16)
        if (!aligned(y, 16))
            return FD_ERR_INVALID_ARG;
    const void *p4[] = {lse, q_indptr_dev, kv_page_indptr_dev, kv_last_page_len_dev, kv_page_indices_dev, k_scale,
                        v_scale};
    for (const void *y : p4)
        if (!aligned(y, 4))
            return FD_ERR_INVALID_ARG;
    fd::PrefillParams p;
    memset(&p, 0, sizeof p);
    p.q = static_cast<const uint16_t *>(q);
    p.q_stride = q_stride;
    p.q_indptr = q_indptr_dev;
    p.page_indptr = kv_page_indptr_dev;
    p.last_len = kv_last_page_len_dev;
    p.page_indices = kv_page_indices_dev;
    p.k = static_cast<const int8_t *>(k_pages_int8);
    p.v = static_cast<const int8_t *>(v_pages_int8);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.o = static_cast<uint16_t *>(o);
    p.lse = lse;
    uint8_t *ws = static_cast<uint8_t *>(workspace) + FD_WORKSPACE_HEADER_BYTES + fd::kTicketBytes;
    p.partial_lse = reinterpret_cast<float *>(ws);
    p.partial_o = reinterpret_cast<float *>(ws + round_up((int64_t)x.num_partial_rows * 4, 256));
    p.status = static_cast<int *>(workspace);
    p.batch = x.batch;
    p.num_tokens = x.num_tokens;
    p.num_qo_heads = x.num_qo_heads;
    p.num_kv_heads = x.num_kv_heads;
    p.group = group;
    p.group_log2 = group == 8 ? 3 : group / 2;
    p.page_size = x.page_size;
    p.num_pages = num_pages;
    p.page_entries = x.num_page_entries;
    p.scale_heads = fd::scale_heads(x.num_kv_heads);
    p.causal = x.causal != 0;
    p.chunk = x.chunk;
    p.num_items = x.num_items;
    p.num_partial_rows = x.num_partial_rows;
    p.merge_rows = x.num_merged_rows;
    p.scale = scale;
    p.timeout_ns = x.timeout_ns;
    return fd::launch_prefill(p, as_stream(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}
