// fd_shared_api.cu -- the C entry points of shared-prefix decode attention:
// the plan (host only) and the launches.  See include/fd.h for the contract.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "api_util.h"
#include "fd.h"
#include "kernels.h"
#include "shared_kernels.h"
#include "stage1.h"

using fd::aligned;
using fd::as_stream;
using fd::round_up;

namespace {

constexpr int kHeadDim = 128;
constexpr int kMaxSlots = 1024;   // SMs the plan can balance over

// The plan's view of its prefixes: requests and keys of prefix g.
struct Prefixes {
    int count;
    const int32_t *req_indptr;
    const int32_t *indptr;      // keys, or page-list entries when page_size > 0
    const int32_t *last_len;
    int32_t page_size;

    int64_t reqs(int g) const
    {
        return (int64_t)req_indptr[g + 1] - req_indptr[g];
    }
    int64_t keys(int g) const
    {
        const int64_t n = (int64_t)indptr[g + 1] - indptr[g];
        return page_size == 0 || n <= 0 ? n : (n - 1) * page_size + last_len[g];
    }
};

struct PlanSize {
    int64_t items, rows;
};

PlanSize size_of(const Prefixes &x, int num_qo_heads, int num_kv_heads, int32_t chunk)
{
    PlanSize z{0, 0};
    for (int g = 0; g < x.count; ++g) {
        const int64_t reqs = x.reqs(g), keys = x.keys(g);
        if (reqs <= 0 || keys <= 0)
            continue;
        const int64_t rows = reqs * (num_qo_heads / num_kv_heads);
        const int64_t blocks = (rows + fd::kSharedBlockRows - 1) / fd::kSharedBlockRows;
        const int64_t splits = fd::shared_splits((int32_t)keys, chunk);
        z.items += splits * blocks * num_kv_heads;
        z.rows += splits * reqs * num_qo_heads;
    }
    return z;
}

// Costs in SM cycles: a 128-key tile of one and of two 128-row tiles, a CTA's
// start and end, and a partial row's write and read over all SMs.
constexpr int64_t kTileOne = 2200, kTileTwo = 3800, kItemCost = 7000;
constexpr double kRowCost = 0.25;

// Time of the grid for chunk length c: its CTAs go, in launch order, to the
// SM that is free first.
double grid_time(const Prefixes &x, int num_qo_heads, int num_kv_heads, int32_t chunk, int slots)
{
    int64_t heap[kMaxSlots];
    for (int i = 0; i < slots; ++i)
        heap[i] = 0;
    double rows_total = 0;
    for (int g = 0; g < x.count; ++g) {
        const int64_t reqs = x.reqs(g), keys = x.keys(g);
        if (reqs <= 0 || keys <= 0)
            continue;
        const int64_t rows = reqs * (num_qo_heads / num_kv_heads);
        const int64_t blocks = (rows + fd::kSharedBlockRows - 1) / fd::kSharedBlockRows;
        const int32_t splits = fd::shared_splits((int32_t)keys, chunk);
        const int32_t len = fd::shared_split_len((int32_t)keys, splits);
        rows_total += (double)splits * reqs * num_qo_heads;
        for (int32_t s = 0; s < splits; ++s) {
            const int64_t tiles = (std::min<int64_t>(keys - (int64_t)s * len, len) + fd::kSharedTile - 1) / fd::kSharedTile;
            for (int64_t i = 0; i < blocks * num_kv_heads; ++i) {
                const int64_t last = rows - (blocks - 1) * fd::kSharedBlockRows;
                const bool two = i % blocks < blocks - 1 || last > fd::kSharedQRows;
                std::pop_heap(heap, heap + slots, [](int64_t a, int64_t b) { return a > b; });
                heap[slots - 1] += kItemCost + tiles * (two ? kTileTwo : kTileOne);
                std::push_heap(heap, heap + slots, [](int64_t a, int64_t b) { return a > b; });
            }
        }
    }
    return (double)*std::max_element(heap, heap + slots) + rows_total * kRowCost;
}

// The chunk length: for grids of up to 1, 2, .. 8 waves of CTAs (one an SM),
// the shortest chunk that fits, and of these the one with the shortest time.
int32_t choose_chunk(const Prefixes &x, int num_qo_heads, int num_kv_heads, int num_sms)
{
    int64_t longest = 1;
    for (int g = 0; g < x.count; ++g)
        longest = std::max(longest, x.keys(g));
    const int32_t most = (int32_t)((longest + fd::kSharedTile - 1) / fd::kSharedTile);
    const int slots = std::min(num_sms, kMaxSlots);
    int32_t best = most, last = -1;
    double best_time = -1;
    for (int waves = 1; waves <= 8; ++waves) {
        int32_t lo = 1, hi = most;   // in tiles; items fall as the chunk grows
        while (lo < hi) {
            const int32_t mid = lo + (hi - lo) / 2;
            if (size_of(x, num_qo_heads, num_kv_heads, mid * fd::kSharedTile).items <= (int64_t)waves * slots)
                hi = mid;
            else
                lo = mid + 1;
        }
        if (lo == last)
            continue;
        last = lo;
        // a chunk that leaves far more items than waves (long batches of
        // prefixes) is not simulated: one split each is all there is
        if (size_of(x, num_qo_heads, num_kv_heads, lo * fd::kSharedTile).items > 64LL * slots)
            continue;
        const double t = grid_time(x, num_qo_heads, num_kv_heads, lo * fd::kSharedTile, slots);
        if (best_time < 0 || t < best_time) {
            best_time = t;
            best = lo;
        }
    }
    return best * fd::kSharedTile;
}

// Chunk length of the suffixes' plan.  Suffixes are short and many: where the
// room's splits can be one wave of the split kernel's CTAs with chunks of at most
// kMostSuffixChunk keys, that is the plan (each CTA has one item and none is
// claimed: 32 requests x 256 keys, 8 KV heads 6.6 us for 12.9 us with the default
// chunk of 224, x 512 keys 9.5 for 15.7, 16 x 2048 keys 26.2 for 33.7); else the
// default, which balances long requests.
constexpr int64_t kMostSuffixChunk = 4096;

int suffix_chunk(int batch, int num_kv_heads, int64_t tokens, int num_sms)
{
    const int64_t slots = (int64_t)num_sms * fd::split_ctas_per_sm();
    const int64_t spare = slots / num_kv_heads - batch;   // splits beyond one a request
    if (spare <= 0 || tokens <= 0)
        return 0;
    const int64_t c = std::max<int64_t>(round_up(tokens / (spare + 1) + 1, FD_TILE_TOKENS), FD_MIN_CHUNK);
    return c <= kMostSuffixChunk ? (int)c : 0;
}

// Where the items' streams add up their O, when one has over kFlush steps (a
// step is a tile; with one row tile the streams take every other one).
int64_t flush_bytes(int64_t items, int32_t chunk)
{
    return chunk / fd::kSharedTile > fd::kFlush ? items * 2 * fd::kSharedQRows * kHeadDim * 4 : 0;
}

// Workspace of a plan: header | tickets | the suffix plan's scratch, laid out as in a
// workspace of its own (from kTicketBytes on) | partial LSE | partial O | sums of O.
int64_t suffix_bytes(const fd_plan_info &suffix)
{
    return fd::kTicketBytes + round_up(suffix.workspace_bytes, 256);
}

int64_t shared_bytes(const fd_plan_info &suffix, int64_t rows, int64_t items, int32_t chunk)
{
    return suffix_bytes(suffix) + round_up(rows * 4, 256) + rows * kHeadDim * 4 + flush_bytes(items, chunk);
}

// Whether a plan's workspace holds what its other fields say (a plan is the caller's
// memory, and the kernels write by those fields).
bool holds_its_parts(const fd_shared_plan &plan)
{
    const fd_plan_info &s = plan.suffix;
    const int64_t suffix = FD_WORKSPACE_HEADER_BYTES + round_up((int64_t)s.batch * s.num_kv_heads * 4, 256) +
                           round_up((int64_t)s.num_partial_rows * 4, 256) + (int64_t)s.num_partial_rows * kHeadDim * 4;
    return s.workspace_bytes >= suffix &&
           plan.workspace_bytes >= shared_bytes(s, plan.num_partial_rows, plan.num_items, plan.chunk);
}

int make_plan(int batch, int num_qo_heads, int num_kv_heads, int head_dim, const Prefixes &x,
              int64_t max_suffix_tokens, int num_sms, int chunk, fd_shared_plan *plan)
{
    if (!plan || batch <= 0 || x.count <= 0 || !x.req_indptr || !x.indptr || (x.page_size && !x.last_len))
        return FD_ERR_INVALID_ARG;
    if (max_suffix_tokens < 0 || max_suffix_tokens > INT32_MAX || num_sms < 0 || chunk < 0 ||
        chunk % fd::kSharedTile != 0 || chunk > (1 << 30))
        return FD_ERR_INVALID_ARG;
    fd_plan_info suffix;
    if (num_sms == 0) {
        const int rc = fd_num_sms(-1, &num_sms);
        if (rc != FD_OK)
            return rc;
    }
    try {   // the planner's host arrays
        const int at = num_kv_heads > 0 ? suffix_chunk(batch, num_kv_heads, max_suffix_tokens, num_sms) : 0;
        const int rc = fd_plan_graph(batch, num_qo_heads, num_kv_heads, head_dim, max_suffix_tokens, num_sms, at,
                                     &suffix);
        if (rc != FD_OK)
            return rc;
    } catch (...) {
        return FD_ERR_INVALID_ARG;
    }
    if (x.req_indptr[0] != 0 || x.indptr[0] != 0 || x.req_indptr[x.count] != batch)
        return FD_ERR_INVALID_ARG;
    for (int g = 0; g < x.count; ++g) {
        if (x.req_indptr[g + 1] < x.req_indptr[g] || x.indptr[g + 1] < x.indptr[g])
            return FD_ERR_INVALID_ARG;
        if (x.page_size && x.indptr[g + 1] > x.indptr[g] &&
            (x.last_len[g] < 1 || x.last_len[g] > x.page_size))
            return FD_ERR_INVALID_ARG;
        if (x.keys(g) > INT32_MAX - fd::kSharedTile)
            return FD_ERR_INVALID_ARG;
    }
    if (chunk == 0)
        chunk = choose_chunk(x, num_qo_heads, num_kv_heads, num_sms);
    const PlanSize z = size_of(x, num_qo_heads, num_kv_heads, chunk);
    if (z.items > INT32_MAX || z.rows > INT32_MAX / kHeadDim)
        return FD_ERR_INVALID_ARG;
    memset(plan, 0, sizeof *plan);
    plan->suffix = suffix;
    plan->num_prefixes = x.count;
    plan->chunk = chunk;
    plan->num_items = (int32_t)z.items;
    plan->num_partial_rows = (int32_t)z.rows;
    plan->page_size = x.page_size;
    plan->prefix_rows = x.indptr[x.count];
    plan->workspace_bytes = shared_bytes(suffix, z.rows, z.items, chunk);
    plan->timeout_ns = FD_DEFAULT_TIMEOUT_NS;
    return FD_OK;
}

}  // namespace

extern "C" int fd_plan_shared(int batch, int num_qo_heads, int num_kv_heads, int head_dim, int num_prefixes,
                              const int32_t *prefix_req_indptr_host, const int32_t *prefix_indptr_host,
                              int64_t max_suffix_tokens, int num_sms, int chunk, fd_shared_plan *plan)
{
    const Prefixes x{num_prefixes, prefix_req_indptr_host, prefix_indptr_host, nullptr, 0};
    return make_plan(batch, num_qo_heads, num_kv_heads, head_dim, x, max_suffix_tokens, num_sms, chunk, plan);
}

extern "C" int fd_plan_shared_paged(int batch, int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                                    int num_prefixes, const int32_t *prefix_req_indptr_host,
                                    const int32_t *prefix_page_indptr_host,
                                    const int32_t *prefix_last_page_len_host, int64_t max_suffix_tokens,
                                    int num_sms, int chunk, fd_shared_plan *plan)
{
    if (page_size <= 0 || page_size % 16 != 0)
        return FD_ERR_UNSUPPORTED;
    const Prefixes x{num_prefixes, prefix_req_indptr_host, prefix_page_indptr_host, prefix_last_page_len_host,
                     page_size};
    return make_plan(batch, num_qo_heads, num_kv_heads, head_dim, x, max_suffix_tokens, num_sms, chunk, plan);
}

namespace {

// Rows of a page that one box brings: the largest power of two that divides a
// page, up to a whole tile.
int page_box_rows(int page_size)
{
    int b = 16;
    while (b < fd::kSharedTile && page_size % (2 * b) == 0)
        b *= 2;
    return b;
}

// A page pool [rows, Hkv, 128] bf16 as a 4-D tensor: 64 columns, 8 rows, Hkv * 2
// blocks of 64 columns, groups of 8 rows (pages are whole groups).  One box (64,
// 8, 2, box_rows / 8) lands as [8-row group][half][8 rows][128 bytes], so boxes
// of any page size stack up to one operand tile with a single group stride.
int make_page_map(CUtensorMap *map, const void *base, int64_t rows, int num_kv_heads, int box_rows)
{
    auto encode = fd::tensor_map_encoder();
    if (!encode)
        return FD_ERR_CUDA;
    const cuuint64_t row = (cuuint64_t)num_kv_heads * kHeadDim * 2;
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)num_kv_heads * 2, (cuuint64_t)(rows / 8)};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, 2, (cuuint32_t)(box_rows / 8)};
    const cuuint32_t elem_strides[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides,
                              box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FD_OK : FD_ERR_INVALID_ARG;
}

struct SharedTables {
    const int32_t *req_indptr, *prefix_indptr, *prefix_last_len, *prefix_indices;
    const int32_t *kv_indptr, *kv_last_len, *kv_indices;
    int num_pages, num_page_entries;
};

int decode_shared(const fd_shared_plan *plan, const SharedTables &t, const void *q, const void *k_prefix,
                  const void *v_prefix, const void *k, const void *v, float scale, float *o, float *lse,
                  void *workspace, int64_t workspace_bytes, void *stream, const fd::QuantKV *quant)
{
    if (!plan)
        return FD_ERR_INVALID_ARG;
    const fd_plan_info &s = plan->suffix;
    int rc = fd::check_info(&s);
    if (rc != FD_OK)
        return rc;
    const bool paged = plan->page_size > 0;
    if (s.batch <= 0 || plan->num_prefixes <= 0 || plan->chunk <= 0 || plan->chunk % fd::kSharedTile != 0 ||
        plan->num_items < 0 || plan->num_partial_rows < 0 || plan->prefix_rows < 0 || plan->page_size < 0 ||
        plan->prefix_rows > INT32_MAX || !holds_its_parts(*plan))
        return FD_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < plan->workspace_bytes)
        return FD_ERR_WORKSPACE;
    const bool has_prefix = plan->num_items > 0, has_suffix = s.total_tokens > 0;
    if (!q || !o || !lse || !t.req_indptr || !t.prefix_indptr || (has_prefix && (!k_prefix || !v_prefix)) ||
        (has_suffix && (!k || !v || !t.kv_indptr)))
        return FD_ERR_INVALID_ARG;
    if (paged && (!t.prefix_last_len || (has_prefix && !t.prefix_indices) || t.num_pages <= 0 ||
                  (int64_t)t.num_pages * plan->page_size > INT32_MAX || t.num_page_entries < 0 ||
                  (has_suffix && !t.kv_last_len) || (t.num_page_entries > 0 && !t.kv_indices)))
        return FD_ERR_INVALID_ARG;
    const void *p16[] = {q, k_prefix, v_prefix, k, v, o, workspace};
    for (const void *x : p16)
        if (!aligned(x, 16))
            return FD_ERR_INVALID_ARG;
    const void *p4[] = {lse, t.req_indptr, t.prefix_indptr, t.prefix_last_len, t.prefix_indices, t.kv_indptr,
                        t.kv_last_len, t.kv_indices};
    for (const void *x : p4)
        if (!aligned(x, 4))
            return FD_ERR_INVALID_ARG;
    if (!isfinite(scale))
        return FD_ERR_INVALID_ARG;
    if (quant && (!quant->k_scale || !quant->v_scale || !aligned(quant->k_scale, 4) || !aligned(quant->v_scale, 4)))
        return FD_ERR_INVALID_ARG;

    fd::SharedMaps maps;
    memset(&maps, 0, sizeof maps);
    const int box_rows = paged ? page_box_rows(plan->page_size) : fd::kSharedTile;
    if (has_prefix) {
        const int64_t rows = paged ? (int64_t)t.num_pages * plan->page_size : plan->prefix_rows;
        const void *base[2] = {k_prefix, v_prefix};
        CUtensorMap *map[2] = {&maps.k, &maps.v};
        for (int i = 0; i < 2; ++i) {
            rc = quant ? fd::make_kv_map_fp8(map[i], base[i], rows, s.num_kv_heads, box_rows)
                 : paged ? make_page_map(map[i], base[i], rows, s.num_kv_heads, box_rows)
                         : fd::make_kv_map(map[i], base[i], rows, s.num_kv_heads, box_rows);
            if (rc != FD_OK)
                return rc;
        }
    }
    cudaStream_t cs = as_stream(stream);
    // The requests' own keys: the split kernel, planned on the device, its
    // merged states into o and lse.
    if (has_suffix) {
        const fd::WorkspaceLayout wl = fd::workspace_layout(static_cast<uint8_t *>(workspace) + fd::kTicketBytes, s.batch,
                                                            s.num_kv_heads, s.num_partial_rows);
        // The split kernel counts a request's splits up from zero and leaves zero.
        // More groups than the tickets' own place holds: other calls' scratch may have
        // been where they are, so the call clears them (2 us of a call of at least
        // 16385 groups).
        const int64_t ticket_bytes = (int64_t)s.batch * s.num_kv_heads * 4;
        int *tickets = reinterpret_cast<int *>(static_cast<uint8_t *>(workspace) + FD_WORKSPACE_HEADER_BYTES);
        if (ticket_bytes > fd::kTicketBytes) {
            tickets = wl.counters;
            if (cudaMemsetAsync(tickets, 0, (size_t)ticket_bytes, cs) != cudaSuccess)
                return FD_ERR_CUDA;
        }
        fd_plan_info info = s;
        info.timeout_ns = plan->timeout_ns;
        const fd::PagedKV pk{plan->page_size, t.num_pages, t.kv_last_len, nullptr, t.kv_indices, t.num_page_entries};
        rc = fd::launch_stage1(&info, q, k, v, t.kv_indptr, scale, wl.partial_o, wl.partial_lse, workspace, o, lse,
                               tickets, nullptr, cs, paged ? &pk : nullptr, quant, true, nullptr, has_prefix);
        if (rc != FD_OK)
            return rc;
    }
    uint8_t *part = static_cast<uint8_t *>(workspace) + suffix_bytes(s);
    fd::SharedParams p;
    memset(&p, 0, sizeof p);
    p.q = static_cast<const uint16_t *>(q);
    p.req_indptr = t.req_indptr;
    p.prefix_indptr = t.prefix_indptr;
    p.prefix_last_len = t.prefix_last_len;
    p.prefix_indices = t.prefix_indices;
    p.k_scale = quant ? quant->k_scale : nullptr;
    p.v_scale = quant ? quant->v_scale : nullptr;
    p.partial_lse = reinterpret_cast<float *>(part);
    p.partial_o = reinterpret_cast<float *>(part + round_up((int64_t)plan->num_partial_rows * 4, 256));
    p.flush = p.partial_o + (int64_t)plan->num_partial_rows * kHeadDim;
    p.o = o;
    p.lse = lse;
    p.status = static_cast<int *>(workspace);
    p.batch = s.batch;
    p.num_qo_heads = s.num_qo_heads;
    p.num_kv_heads = s.num_kv_heads;
    p.group = s.group_size;
    p.num_prefixes = plan->num_prefixes;
    p.chunk = plan->chunk;
    p.num_items = plan->num_items;
    p.num_partial_rows = plan->num_partial_rows;
    p.prefix_rows = (int32_t)plan->prefix_rows;
    p.page_size = plan->page_size;
    p.num_pages = t.num_pages;
    p.box_rows = box_rows;
    p.has_suffix = has_suffix;
    p.suffix_indptr = t.kv_indptr;
    p.suffix_last_len = t.kv_last_len;
    p.max_suffix_tokens = (int32_t)s.total_tokens;
    p.scale = scale;
    p.timeout_ns = plan->timeout_ns;
    const cudaError_t e = fd::launch_shared(maps, p, quant ? quant->type : fd::kKvTypeBf16, cs);
    return e == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

}  // namespace

extern "C" int fd_decode_shared(const fd_shared_plan *plan, const int32_t *prefix_req_indptr_dev,
                                const int32_t *prefix_indptr_dev, const int32_t *kv_indptr_dev, const void *q,
                                const void *k_prefix, const void *v_prefix, const void *k, const void *v,
                                float scale, float *o, float *lse, void *workspace, int64_t workspace_bytes,
                                void *stream)
{
    if (plan && plan->page_size != 0)
        return FD_ERR_INVALID_ARG;
    const SharedTables t{prefix_req_indptr_dev, prefix_indptr_dev, nullptr, nullptr, kv_indptr_dev, nullptr, nullptr, 0, 0};
    return decode_shared(plan, t, q, k_prefix, v_prefix, k, v, scale, o, lse, workspace, workspace_bytes, stream,
                         nullptr);
}

extern "C" int fd_decode_shared_paged(const fd_shared_plan *plan, int num_pages,
                                      const int32_t *prefix_req_indptr_dev, const int32_t *prefix_page_indptr_dev,
                                      const int32_t *prefix_last_page_len_dev,
                                      const int32_t *prefix_page_indices_dev, const int32_t *kv_page_indptr_dev,
                                      const int32_t *kv_last_page_len_dev, const int32_t *kv_page_indices_dev,
                                      int num_page_entries, const void *q, const void *k_pages,
                                      const void *v_pages, float scale, float *o, float *lse, void *workspace,
                                      int64_t workspace_bytes, void *stream)
{
    if (plan && plan->page_size <= 0)
        return FD_ERR_INVALID_ARG;
    const SharedTables t{prefix_req_indptr_dev, prefix_page_indptr_dev, prefix_last_page_len_dev,
                         prefix_page_indices_dev, kv_page_indptr_dev, kv_last_page_len_dev, kv_page_indices_dev,
                         num_pages, num_page_entries};
    return decode_shared(plan, t, q, k_pages, v_pages, k_pages, v_pages, scale, o, lse, workspace, workspace_bytes,
                         stream, nullptr);
}

extern "C" int fd_decode_shared_fp8(const fd_shared_plan *plan, const int32_t *prefix_req_indptr_dev,
                                const int32_t *prefix_indptr_dev, const int32_t *kv_indptr_dev, const void *q,
                                const void *k_prefix_fp8, const void *v_prefix_fp8, const void *k, const void *v,
                                const float *k_scale, const float *v_scale, float scale, float *o, float *lse, void *workspace, int64_t workspace_bytes,
                                void *stream)
{
    if (plan && plan->page_size != 0)
        return FD_ERR_INVALID_ARG;
    const SharedTables t{prefix_req_indptr_dev, prefix_indptr_dev, nullptr, nullptr, kv_indptr_dev, nullptr, nullptr, 0, 0};
    const fd::QuantKV f{fd::kKvTypeFp8, k_scale, v_scale};
    return decode_shared(plan, t, q, k_prefix_fp8, v_prefix_fp8, k, v, scale, o, lse, workspace, workspace_bytes, stream,
                         &f);
}

extern "C" int fd_decode_shared_paged_fp8(const fd_shared_plan *plan, int num_pages,
                                      const int32_t *prefix_req_indptr_dev, const int32_t *prefix_page_indptr_dev,
                                      const int32_t *prefix_last_page_len_dev,
                                      const int32_t *prefix_page_indices_dev, const int32_t *kv_page_indptr_dev,
                                      const int32_t *kv_last_page_len_dev, const int32_t *kv_page_indices_dev,
                                      int num_page_entries, const void *q, const void *k_pages_fp8,
                                      const void *v_pages_fp8, const float *k_scale, const float *v_scale, float scale, float *o, float *lse, void *workspace,
                                      int64_t workspace_bytes, void *stream)
{
    if (plan && plan->page_size <= 0)
        return FD_ERR_INVALID_ARG;
    const SharedTables t{prefix_req_indptr_dev, prefix_page_indptr_dev, prefix_last_page_len_dev,
                         prefix_page_indices_dev, kv_page_indptr_dev, kv_last_page_len_dev, kv_page_indices_dev,
                         num_pages, num_page_entries};
    const fd::QuantKV f{fd::kKvTypeFp8, k_scale, v_scale};
    return decode_shared(plan, t, q, k_pages_fp8, v_pages_fp8, k_pages_fp8, v_pages_fp8, scale, o, lse, workspace, workspace_bytes,
                         stream, &f);
}
