// shared_kernel.cuh -- decode attention over prefixes that many requests
// share, on sm_103a: each prefix's keys are read once for all of its requests.
//
// Mathematics: with R requests behind a prefix, the R * G queries of a KV head
// are the rows of one matrix, S = Q K^T, P = exp2(S c - m) by row with a
// running maximum, O += P V: the split-KV partial of `fd_decode`, with up to
// 256 query rows instead of 8.  Every (prefix, split, KV head, block of 256
// rows) is one CTA; the partials (normalised O, LSE) go to a workspace and a
// second kernel merges them with the state of the request's own keys by LSE.
//
// Bound: up to 128 rows a KV head the bytes of K and V (a 128-key tile of both
// is 64 KB in bf16; 32 requests of 32 heads behind 65536 keys 50-52 us, 5.3 TB/s),
// above that the tensor cores (a tile of two row tiles 1.9-2.1 us, 1.9 PFLOP/s
// with the products of both parts of P; 256 requests of 64 heads behind 32768
// keys 281-292 us).  The products run on tcgen05
// with their accumulators in tensor memory: S and O of one 128-row tile take
// 256 columns, so a CTA holds two such streams.  With more than 128 rows the
// streams are two row tiles that share each K and V tile; with fewer, both
// take the same rows and every other key tile, so that one stream's softmax
// runs under the other's products, and their states are merged at the end.
//
// P enters the second product as a sum of two 16-bit parts, hi + lo, which
// keeps 16 bits of each weight (one part alone would be off by 2^-9, and the
// output by more than its fp32 type says): three products of 128 x 128 x 128 a
// tile for the two that the definition has.
//
// FP8 K and V: the products are in f16 (every E4M3 value is an f16 value); four
// warps widen each raw tile into an operand tile in shared memory, and q
// rows are scaled into f16 by a power of two.  A tile of one row tile takes 1.1 us
// on contiguous keys (4.4 TB/s over the SMs) and 1.5 in 16-key pages (16 boxes a
// tile): the chain of its steps, in which each instruction of the widening counts
// (a select for each value past the last key made it 1.46).
//
// Warps: 0-15 the softmax -- two warpgroups a stream, one a half of the tile's
// keys; a thread owns a row and 64 of its scores (tcgen05.ld gives it the row's
// columns).  16 the producer (TMA), 17 issues the products of both streams in
// turn (a warp for each let the two streams' products run through one another:
// both then ended late, and the call took a fifth longer), 18-21 do the widening
// (FP8).
//
// The reference m of a row's weights only has to keep them in their type's
// range: the weights are floating-point numbers, their size costs no accuracy.
// So m is the maximum of the row's first tile, and the steps behind it turn
// scores into weights as they arrive, with no maximum and no exchange between
// the warps of a row on the way.  A row whose later scores are out of that
// range (its sum over 2^40; a weight over f16's with FP8 K/V) is seen at the
// end, and the CTA then does its item again with careful steps, which raise m
// and rescale O.  (One key deep in the prefix 28 nats above a row's first tile, or 6.2
// with FP8 K/V, does that to every request behind it: 45 requests behind 20001
// keys 52 us for 31, FP8 56 for 34.)  Careful steps alone took a quarter longer (310 us for 250 of
// the prefixes' grid, 256 x 64 heads behind 32768 keys): the tensor cores waited
// for the maximum, the vote of a row's two warps, and then for the weights.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "device_common.cuh"
#include "kernels.h"
#include "shared_kernels.h"
#include "tcgen05.cuh"

namespace fd {
namespace {

constexpr int kBufBytes = kSharedTile * kHeadDim * 2;   // a K, V or Q tile of 16-bit values: 32 KB
constexpr int kHalfBytes = kBufBytes / 2;
constexpr int kBuffers = 7;                             // Q tiles and rings together
constexpr int kWideBuffers = 4;                         // FP8: operand tiles; the rest of the ring is raw
constexpr int kRawBytes = kBufBytes / 2;                // FP8: a raw tile
constexpr int kMaxRing = 6;                             // at most 5 are used; room for 5 alone: calls 0.1 us longer
constexpr int kSoftmaxThreads = 512;
constexpr int kStreamWarps = 8;
constexpr int kProducerWarp = 16, kMmaWarp = 17, kWidenWarp = 18, kWidenWarps = 4;
template <int DT>
constexpr int kThreads = DT == kKvTypeFp8 ? 704 : 640;
constexpr int kTmemCols = 512;
constexpr int kStreamCols = 256;                        // S (and P over it) 128, O 128
// Careful steps: log2 of the growth of a row's maximum that raises m.
constexpr float kRaise = 8.f;
// The other steps: the most that a row's sum may be; beyond it the item is done
// again.  (FP8 K/V has weights in f16: one past their range is inf, its lo part
// -inf, and the row's O NaN, which tells without a look at each weight.)
constexpr float kMostSum = 1099511627776.f;
constexpr uint32_t kSleepNs = 100000;                    // a wait's sleep between looks at the timer
constexpr int kOutStride = kHeadDim + 4;                // floats between rows of the epilogue's staging

struct SharedSmem {
    uint64_t full[kMaxRing], empty[kMaxRing];           // operand tiles
    uint64_t raw_full[kMaxRing], raw_empty[kMaxRing];   // FP8: raw tiles
    uint64_t s_full[2], p_ready[2][2], o_done[2];
    uint64_t q_ready, tail, drain;
    uint32_t tmem;
    int abort;
    int redo;               // a row's weights left their type's range
    int issued;             // ring fills issued (for the drain after an error)
    int tail_issued;
    // the CTA's item
    int ok, req0, rows, kvh, row0, key0, keys, base, part_row, part_stride, q_tiles;
    union {
        float q_scale[kSharedBlockRows];      // FP8, before the first step: a row's factor of the scores
        float row_max[2][2][kSharedQRows];    // a stream's row maxima, by half of the keys
    };
};
// At the end, behind the staged rows: the streams' sums by half, stream 1's maxima.
struct SharedEnd {
    float row_sum[2][2][kSharedQRows];
    float row_ref[kSharedQRows];
};
constexpr int kEndOffset = kSharedBlockRows * kOutStride * 4;
static_assert(kEndOffset + (int)sizeof(SharedEnd) <= kBuffers * kBufBytes, "the epilogue works over the ring");
constexpr int kSharedAlloc = kBuffers * kBufBytes + (int)((sizeof(SharedSmem) + 15) / 16 * 16);
// the dynamic shared memory of a CTA starts 1024-byte aligned (the kernel checks)
static_assert(kSharedAlloc <= 232448, "shared memory of one CTA");

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats as a pair of 16-bit values (round to nearest), and back.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float2 a)
{
    if constexpr (DT == kKvTypeFp8) {
        const __half2 h = __floats2half2_rn(a.x, a.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if constexpr (DT == kKvTypeFp8)
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else
        return bf16x2_to_float2(w);
}

// Barrier of `threads` threads with the OR of a predicate over them.
__device__ __forceinline__ bool barrier_or(int id, int threads, bool x)
{
    int r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %3, 0;\n\t"
                 "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"(threads), "r"((int)x)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ void barrier(int id, int threads)
{
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The registers a tcgen05.ld wrote may be read from here on (an empty barrier
// for the compiler, behind tcgen05.wait::ld).
template <int N>
__device__ __forceinline__ void settle(uint32_t (&r)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                          "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// 16 values of O to memory that only this thread uses (four at a time, the
// stream's rows apart): added, or the first ones.
__device__ __forceinline__ void flush16(float *dst, const uint32_t (&o)[16], bool add)
{
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        if (add)
            asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst + j * kSharedQRows),
                         "f"(__uint_as_float(o[j])), "f"(__uint_as_float(o[j + 1])), "f"(__uint_as_float(o[j + 2])),
                         "f"(__uint_as_float(o[j + 3]))
                         : "memory");
        else
            __stcg(reinterpret_cast<uint4 *>(dst + j * kSharedQRows), make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]));
    }
}

__device__ __forceinline__ void add_flushed16(const float *src, uint32_t (&o)[16])
{
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + j * kSharedQRows));
        o[j] = __float_as_uint(__uint_as_float(o[j]) + v.x);
        o[j + 1] = __float_as_uint(__uint_as_float(o[j + 1]) + v.y);
        o[j + 2] = __float_as_uint(__uint_as_float(o[j + 2]) + v.z);
        o[j + 3] = __float_as_uint(__uint_as_float(o[j + 3]) + v.w);
    }
}

__device__ __forceinline__ void scale_flushed16(float *dst, float f)
{
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        float4 *d = reinterpret_cast<float4 *>(dst + j * kSharedQRows);
        const float4 v = __ldcg(d);
        __stcg(d, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
    }
}

// Wait for a phase; false (and the CTA's abort flag set) when the time limit
// passed or another warp gave up.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, const SharedParams &p, SharedSmem *sm)
{
    const uint32_t a = smem_addr(bar);
    if (p.timeout_ns > 0) {
        // These waits are the pipeline's hand-overs: a waiting warp sleeps until
        // the phase completes (polling takes issue slots from the warps at
        // work), and looks at the timer only when it woke for nothing.
        if (mbar_try_wait(a, parity))
            return true;
        const uint64_t t0 = global_timer_ns();
        while (!*reinterpret_cast<volatile int *>(&sm->abort)) {
            if (mbar_try_wait_for(a, parity, kSleepNs))
                return true;
            if ((int64_t)(global_timer_ns() - t0) > p.timeout_ns)
                break;
        }
    }
    if (!*reinterpret_cast<volatile int *>(&sm->abort)) {
        *reinterpret_cast<volatile int *>(&sm->abort) = 1;
        report(p.status, FD_ERR_TIMEOUT);
    }
    return false;
}

// --------------------------------------------------- where a CTA's work lies

struct PrefixCoord {
    int32_t g, req0, reqs;     // prefix, its first request and their number
    int32_t base, len;         // first key row or page-list entry, keys
    int32_t splits, blocks;    // splits of the keys, 256-row blocks of a KV head's rows
    int32_t item0, row0;       // items and partial rows of the prefixes before
};

// Whole warp: the prefix that holds item `j` (or request `j`).  False when
// there is none or the tables are outside what the plan was made for.
__device__ __forceinline__ bool locate_prefix(const SharedParams &p, int32_t j, bool by_request, PrefixCoord &out)
{
    const int lane = threadIdx.x & 31;
    int32_t item_carry = 0, row_carry = 0;
    for (int g0 = 0; g0 < p.num_prefixes; g0 += 32) {
        const int g = g0 + lane;
        int32_t r0 = 0, reqs = 0, base = 0, len = 0, splits = 0, blocks = 0;
        if (g < p.num_prefixes) {
            const int32_t r1 = __ldcg(p.req_indptr + g + 1), b1 = __ldcg(p.prefix_indptr + g + 1);
            r0 = __ldcg(p.req_indptr + g);
            base = __ldcg(p.prefix_indptr + g);
            const int32_t last = p.page_size ? __ldcg(p.prefix_last_len + g) : 1;
            // a prefix outside the batch or the rows is nobody's; no sum below
            // overflows for what is left
            if (r0 >= 0 && r0 <= r1 && r1 <= p.batch && base >= 0 && base <= b1 && b1 <= p.prefix_rows) {
                const int64_t keys = !p.page_size ? b1 - base
                                     : b1 == base ? 0 : (int64_t)(b1 - base - 1) * p.page_size + last;
                reqs = r1 - r0;
                if (reqs > 0 && keys > 0 && keys <= INT32_MAX - kSharedTile && last >= 1 &&
                    (!p.page_size || last <= p.page_size)) {
                    len = (int32_t)keys;
                    splits = shared_splits(len, p.chunk);
                    blocks = (int32_t)(((int64_t)reqs * p.group + kSharedBlockRows - 1) / kSharedBlockRows);
                } else if (keys != 0) {
                    reqs = 0;
                }
            }
        }
        const int64_t items64 = (int64_t)splits * blocks * p.num_kv_heads;
        const int64_t rows64 = (int64_t)splits * reqs * p.num_qo_heads;
        const bool fits = items64 <= p.num_items && rows64 <= p.num_partial_rows;
        if (!fits)
            reqs = 0;
        const int32_t items = fits ? (int32_t)items64 : 0, rows = fits ? (int32_t)rows64 : 0;
        int32_t item_incl = items, row_incl = rows;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t t = __shfl_up_sync(0xffffffffu, item_incl, o);
            const int32_t u = __shfl_up_sync(0xffffffffu, row_incl, o);
            if (lane >= o) {
                item_incl += t;
                row_incl += u;
            }
        }
        item_incl += item_carry;
        row_incl += row_carry;
        const bool hit = g < p.num_prefixes && (by_request ? j >= r0 && j < r0 + reqs
                                                           : j >= item_incl - items && j < item_incl);
        const unsigned mask = __ballot_sync(0xffffffffu, hit);
        if (mask) {
            const int src = __ffs(mask) - 1;
            out.g = g0 + src;
            out.req0 = __shfl_sync(0xffffffffu, r0, src);
            out.reqs = __shfl_sync(0xffffffffu, reqs, src);
            out.base = __shfl_sync(0xffffffffu, base, src);
            out.len = __shfl_sync(0xffffffffu, len, src);
            out.splits = __shfl_sync(0xffffffffu, splits, src);
            out.blocks = __shfl_sync(0xffffffffu, blocks, src);
            out.item0 = __shfl_sync(0xffffffffu, item_incl - items, src);
            out.row0 = __shfl_sync(0xffffffffu, row_incl - rows, src);
            // by int32 sums that may have wrapped: the prefix's items are among the grid's, each
            // of which one CTA computes, and its rows in range all the same
            return out.item0 >= 0 && out.row0 >= 0 &&
                   (int64_t)out.item0 + (int64_t)out.splits * out.blocks * p.num_kv_heads <= p.num_items &&
                   (int64_t)out.row0 + (int64_t)out.splits * out.reqs * p.num_qo_heads <= p.num_partial_rows;
        }
        item_carry = __shfl_sync(0xffffffffu, item_incl, 31);
        row_carry = __shfl_sync(0xffffffffu, row_incl, 31);
    }
    return false;
}

// The stream of K and V tiles of n tiles goes K0, K1, V0, K2, V1, ..., the order
// in which the products take them.  A place in it: its buffer and the parity
// of the buffer's use.
struct Place {
    int slot, size;
    uint32_t phase;

    __device__ __forceinline__ Place(int first, int size_) : slot(first), size(size_), phase(0) {}
    // by at most `size`
    __device__ __forceinline__ void advance(int by)
    {
        slot += by;
        if (slot >= size) {
            slot -= size;
            phase ^= 1;
        }
    }
};

// ------------------------------------------------------------------- kernel

// Layout of a 16-bit operand tile of 128 rows x 128 values, 128-byte swizzle.
//  [64-value half][128 rows][128 bytes]; bf16 pages: [8-row group][half][8
//  rows][128 bytes], which one box of a page's rows lands as.
template <bool GROUPED>
struct TileLayout {
    static constexpr uint32_t kHalf = GROUPED ? 1024 : kHalfBytes;   // between halves
    static constexpr uint32_t kGroup = GROUPED ? 2048 : 1024;        // between 8-row groups
};

template <bool PAGED, int DT>
__global__ void __launch_bounds__(kThreads<DT>, 1)
    shared_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ SharedParams p)
{
    constexpr bool kFp8 = DT == kKvTypeFp8;
    using TL = TileLayout<PAGED && !kFp8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    SharedSmem *sm = reinterpret_cast<SharedSmem *>(smem + kBuffers * kBufBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // One thread: all barriers before their first phase.
    auto init_barriers = [&](bool again) {
        auto init = [&](uint64_t *bar, uint32_t count) {
            if (again)
                mbar_inval(smem_addr(bar));
            mbar_init(smem_addr(bar), count);
        };
        for (int i = 0; i < kMaxRing; ++i) {
            init(&sm->full[i], kFp8 ? kWidenWarps : 1);
            init(&sm->empty[i], 1);
            init(&sm->raw_full[i], 1);
            init(&sm->raw_empty[i], kWidenWarps);
        }
        for (int s = 0; s < 2; ++s) {
            init(&sm->s_full[s], 1);
            init(&sm->p_ready[s][0], kStreamWarps);
            init(&sm->p_ready[s][1], kStreamWarps);
            init(&sm->o_done[s], 1);
        }
        init(&sm->q_ready, kSoftmaxThreads / 32);
        init(&sm->tail, 1);
        init(&sm->drain, 1);
        fence_mbar_init();
        sm->issued = 0;
        sm->tail_issued = 0;
    };
    if (warp == kMmaWarp)
        tmem_alloc(smem_addr(&sm->tmem), kTmemCols);
    // With suffixes, the grid before this one is theirs and lets this one start
    // once its own wait is over: what was written before the call is there then,
    // and nothing here depends on the suffixes' grid but its end, which this one
    // awaits at its own (the merge needs both).  Data of earlier grids are read
    // through L2, as no wait of this grid has come before.
    if (!p.has_suffix)
        griddep_wait();
    if (warp == kProducerWarp) {
        PrefixCoord c;
        const int w = blockIdx.x;
        // operand tiles of a 1024-byte swizzle pattern: the base must be aligned
        const bool found = locate_prefix(p, w, false, c) && (smem_addr(smem) & 1023) == 0;
        if (lane == 0) {
            sm->ok = found;
            sm->q_tiles = 1;
            if (found) {
                const int rest = w - c.item0;
                const int qb = rest % c.blocks, sk = rest / c.blocks;
                const int split = sk / p.num_kv_heads;
                const int len = shared_split_len(c.len, c.splits);
                sm->kvh = sk % p.num_kv_heads;
                sm->req0 = c.req0;
                sm->row0 = qb * kSharedBlockRows;
                sm->rows = min(c.reqs * p.group - sm->row0, kSharedBlockRows);
                sm->key0 = split * len;
                sm->keys = min(c.len - sm->key0, len);
                sm->base = c.base;
                sm->part_row = c.row0 + split;
                sm->part_stride = c.splits;
                sm->q_tiles = sm->rows > kSharedQRows ? 2 : 1;
            } else {
                report(p.status, FD_ERR_DEVICE_BOUNDS);
            }
            init_barriers(false);
            sm->abort = 0;
            sm->redo = 0;
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem = sm->tmem;
    const bool ok = sm->ok;
    const int q_tiles = sm->q_tiles;
    // The ring that TMA fills: raw tiles (FP8), or operand tiles.  Two tiles of K and
    // V on their way a CTA suffice on contiguous keys, and with more of them the
    // 152 CTAs slow one another at the memory (32 requests behind 131072 keys: 4
    // buffers 92.7 us, 6 98.9); pages, whose tiles are several boxes, take one more
    // (pages of 128 keys: 4 93.0, 5 92.3, 6 94.8; of 16: 96.4, 94.9, 94.4).
    const int nb = kFp8 ? 2 * (kBuffers - q_tiles - kWideBuffers) : PAGED ? 5 : 4;
    static_assert(kBuffers >= 2 + 5, "two Q tiles and the ring");
    const int nw = kFp8 ? kWideBuffers : nb;   // operand tiles
    const int n = ok ? (sm->keys + kSharedTile - 1) / kSharedTile : 0;
    // local steps of stream s: every tile (two row tiles) or every other one
    auto steps = [&](int s) { return q_tiles == 2 ? n : (n + 1 - s) / 2; };
    const uint32_t q_smem = smem_addr(smem), ring = q_smem + q_tiles * kBufBytes;
    uint8_t *ring_ptr = smem + q_tiles * kBufBytes;
    // Position pos of the stream (see Place) holds K of tile t, or V of tile t.
    auto at_pos = [&](int pos, bool &is_k) {
        is_k = pos == 0 || ((pos & 1) && pos < 2 * n - 1);
        return is_k ? (pos + 1) / 2 : pos == 2 * n - 1 ? n - 1 : (pos - 2) / 2;
    };

    // At most two passes over the item: the second with careful steps, when the
    // first left the weights' range.
    float c2 = 0.f;   // softmax warps: what a score is multiplied by
    for (int pass = 0; pass < 2; ++pass) {
        const bool careful = pass > 0;
        if (warp == kProducerWarp && ok) {
            // --------------------------------------------------------- producer
            const uint64_t pol = l2_evict_first_policy();
            const int box = PAGED ? p.box_rows : kSharedTile;
            const int boxes = kSharedTile / box;
            constexpr int kRow = kFp8 ? kHeadDim : 2 * kHeadDim, kTileBytes = kSharedTile * kRow;
            uint64_t *bar_full = kFp8 ? sm->raw_full : sm->full, *bar_empty = kFp8 ? sm->raw_empty : sm->empty;
            const uint32_t raw0 = ring + (kFp8 ? kWideBuffers * kBufBytes : 0);
            // Paged: the lane's box of the next tile is at row `off` of the request's
            // page `pg`; a tile on, that is a fixed number of pages and rows further.
            int pg = 0, off = 0, key = sm->keys;
            const int pages_on = PAGED ? kSharedTile / p.page_size : 0;
            const int rows_on = PAGED ? kSharedTile % p.page_size : 0;
            if (PAGED && lane < boxes) {
                key = lane * box;
                pg = (sm->key0 + key) / p.page_size;
                off = (sm->key0 + key) % p.page_size;
            }
            // The next tile's page is looked up a tile ahead and used when its turn
            // comes; -1: no box of this lane (past the last key).
            int id_next = -1, off_next = 0;
            auto look_up = [&]() {
                const bool has = key < sm->keys;
                id_next = has ? __ldcg(p.prefix_indices + sm->base + pg) : -1;
                off_next = has ? off : -1;
                key += lane < boxes ? kSharedTile : 0;
                pg += pages_on;
                off += rows_on;
                if (off >= p.page_size) {
                    off -= p.page_size;
                    ++pg;
                }
            };
            auto pool_row = [&]() -> int {
                if (off_next < 0)
                    return -1;
                if (id_next < 0 || id_next >= p.num_pages) {   // read page 0 in its place
                    report(p.status, FD_ERR_DEVICE_BOUNDS);
                    id_next = 0;
                }
                return id_next * p.page_size + off_next;
            };
            Place at(0, nb);
            auto load = [&](const CUtensorMap *map, int row, uint64_t *bar, uint32_t bytes) {
                const uint32_t dst = raw0 + at.slot * kTileBytes, b = smem_addr(bar);
                if (lane == 0)
                    mbar_arrive_expect_tx(b, bytes);
                __syncwarp();
                if constexpr (kFp8) {
                    if (PAGED ? row >= 0 : lane == 0)
                        tma_load_2d(dst + (PAGED ? lane * box * kRow : 0), map, sm->kvh * kHeadDim, row, b, pol);
                } else if constexpr (PAGED) {
                    if (row >= 0)
                        asm volatile(
                            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                            ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst + lane * box * kRow),
                            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(0), "r"(2 * sm->kvh), "r"(row >> 3),
                            "r"(b), "l"(pol)
                            : "memory");
                } else if (lane == 0) {
                    tma_load_3d(dst, map, 0, row, 2 * sm->kvh, b, pol);
                }
            };
            if (PAGED)
                look_up();
            int row_k = sm->base + sm->key0 - kSharedTile, row_v = 0;
            for (int pos = 0; pos < 2 * n; ++pos, at.advance(1)) {
                bool is_k;
                const int t = at_pos(pos, is_k);
                if (is_k) {
                    row_v = row_k;
                    if constexpr (PAGED) {
                        row_k = pool_row();
                        look_up();
                    } else {
                        row_k += kSharedTile;
                    }
                }
                if (pos >= nb && !__all_sync(0xffffffffu, wait_phase(&bar_empty[at.slot], at.phase ^ 1, p, sm)))
                    break;
                if (lane == 0)
                    sm->issued = pos + 1;
                const int valid = min(sm->keys - t * kSharedTile, kSharedTile);
                const uint32_t bytes = PAGED ? (valid + box - 1) / box * box * kRow : kTileBytes;
                if (is_k) {
                    load(&tm_k, row_k, &bar_full[at.slot], bytes);
                    continue;
                }
                const int row_t = t == n - 1 ? row_k : row_v;   // K of tile t + 1 has gone before, but for the last
                if (kFp8 || valid == kSharedTile) {
                    load(&tm_v, row_t, &bar_full[at.slot], bytes);
                } else {
                    // The rows past the last key (another prefix's, or nobody's) get
                    // weight 0, but 0 * NaN would still reach O: zero them before the
                    // products see the tile (FP8: the widening warps do).
                    load(&tm_v, row_t, &sm->tail, bytes);
                    if (lane == 0)
                        sm->tail_issued = 1;
                    if (!__all_sync(0xffffffffu, wait_phase(&sm->tail, 0, p, sm)))
                        break;
                    uint8_t *v = ring_ptr + at.slot * kBufBytes;
                    for (int i = lane; i < (kSharedTile - valid) * 16; i += 32) {
                        const int r = valid + i / 16, c = i % 16;
                        const uint32_t off = (c >> 3) * TL::kHalf + (r >> 3) * TL::kGroup + (r & 7) * 128 +
                                             (c & 7) * 16;
                        *reinterpret_cast<uint4 *>(v + off) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&bar_full[at.slot]));
                }
            }
        } else if (warp == kMmaWarp && ok) {
            // ------------------------------------------------------ the products
            // A wait that gave up is reported; the products then work on what there
            // is, so that no branch depends on it.
            constexpr uint32_t id_s = mma_idesc(128, kSharedTile, !kFp8, false);
            constexpr uint32_t id_o = mma_idesc(128, kHeadDim, !kFp8, true);
            const uint32_t leader = elect_one();
            const bool two = q_tiles == 2;
            const int steps0 = steps(0), steps1 = steps(1);
            const uint32_t q_lo = smem_desc_lo(q_smem, 16);
            const uint32_t k_lo = smem_desc_lo(ring, 16);
            const uint32_t v_lo = smem_desc_lo(ring, TL::kHalf);
            constexpr uint32_t q_hi = smem_desc_hi(1024), kv_hi = smem_desc_hi(TL::kGroup);
            constexpr uint32_t kBuf16 = kBufBytes / 16;
            Place k_at(0, nw), v_at(n > 1 ? 2 : 1, nw);
            int k_tile = 0, v_tile = 0;
            wait_phase(&sm->q_ready, 0, p, sm);
            // S of stream s's next step: K of its tile; frees the buffer after the
            // last stream that takes it.
            auto scores = [&](int s) {
                wait_phase(&sm->full[k_at.slot], k_at.phase, p, sm);
                tcgen05_fence_after();
                const uint32_t qa = q_lo + (two ? s : 0) * kBuf16, ka = k_lo + k_at.slot * kBuf16;
#pragma unroll
                for (int k = 0; k < 8; ++k)   // 16 head dimensions a step
                    mma_ss(tmem + s * kStreamCols, qa + ((k >> 2) * kHalfBytes + (k & 3) * 32) / 16, q_hi,
                           ka + ((k >> 2) * TL::kHalf + (k & 3) * 32) / 16, kv_hi, id_s, k > 0, leader);
                tcgen05_commit(smem_addr(&sm->s_full[s]), leader);
                if (!two || s == 1) {
                    tcgen05_commit(smem_addr(&sm->empty[k_at.slot]), leader);
                    k_at.advance(k_tile == 0 ? 1 : 2);
                    ++k_tile;
                }
            };
            // O += P V of stream s's step i, in two parts: each half of the keys is
            // ready in two parts of 32.
            const int run0 = shared_run(steps0), run1 = shared_run(steps1);
            int anew[2] = {0, 0};   // the step at which O of a stream next starts anew
            auto values = [&](int s, int i, bool last) {
                const bool fresh = i == anew[s];
                if (fresh)
                    anew[s] += s ? run1 : run0;
                wait_phase(&sm->full[v_at.slot], v_at.phase, p, sm);
                const uint32_t pa = tmem + s * kStreamCols, va = v_lo + v_at.slot * kBuf16;
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    wait_phase(&sm->p_ready[s][part], i & 1, p, sm);
                    tcgen05_fence_after();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {   // 16 keys a step, hi then lo
                        const int k = (j >> 1) * 4 + part * 2 + (j & 1);
                        const uint32_t vk = va + k * 2 * TL::kGroup / 16;
                        mma_ts(pa + 128, pa + 16 * k, vk, kv_hi, id_o, !fresh || part > 0 || j > 0, leader);
                        mma_ts(pa + 128, pa + 16 * k + 8, vk, kv_hi, id_o, 1, leader);
                    }
                }
                if (!two || s == 1) {
                    tcgen05_commit(smem_addr(&sm->empty[v_at.slot]), leader);
                    v_at.advance(v_tile == n - 2 ? 1 : 2);
                    ++v_tile;
                }
                if (last)
                    tcgen05_commit(smem_addr(&sm->o_done[s]), leader);
            };
            scores(0);
            if (steps1 > 0)
                scores(1);
            for (int i = 0; i < steps0; ++i) {
                values(0, i, i == steps0 - 1);
                if (i + 1 < steps0)
                    scores(0);
                if (i < steps1)
                    values(1, i, i == steps1 - 1);
                if (i + 1 < steps1)
                    scores(1);
            }
            // whatever the others saw, the products in flight end before tensor
            // memory is freed
            tcgen05_commit(smem_addr(&sm->drain), leader);
            mbar_wait(smem_addr(&sm->drain), 0, kDrainTimeoutNs);
            __syncwarp();
        } else if (kFp8 && warp >= kWidenWarp && warp < kWidenWarp + kWidenWarps && ok) {
            // ------------------------------------- FP8: raw tiles to f16 operands
            // A unit of work is 8 rows of one half of the head, 16 values a lane: a raw
            // row is 8 chunks of 16 bytes, chunk c at c ^ (row % 8), and becomes two
            // chunks of the operand's half c / 4.  The lanes of a quarter warp are two
            // rows r and r ^ 5 and four chunks, which meet no bank twice on either side.
            // All of a warp's units of a tile are loaded before the first is stored.
            constexpr int kMine = 2 * kSharedTile / 8 / kWidenWarps;
            constexpr uint32_t kStep = kWidenWarps / 2 * 1024;   // bytes between a warp's units, raw and widened
            static_assert(kWidenWarps % 2 == 0 && kMine * kWidenWarps * 4 == kSharedTile, "whole units a warp");
            const uint8_t *raw0 = ring_ptr + kWideBuffers * kBufBytes;
            const int me = warp - kWidenWarp;   // first unit: rows 8 (me / 2) .., half me % 2
            const int r8 = (lane >> 3) ^ (((lane >> 2) & 1) * 5), cc = lane & 3;
            const int row = (me >> 1) * 8 + r8;
            // the lane's chunk of the first unit: raw, and the first of its two of the operand
            const uint32_t lane_src = (me >> 1) * 1024 + r8 * 128 + ((((me & 1) * 4 + cc) ^ r8) << 4);
            const uint32_t lane_dst = (me >> 1) * 1024 + (me & 1) * kHalfBytes + r8 * 128 + (((2 * cc) ^ r8) << 4);
            Place from(0, nb), to(0, kWideBuffers);
            for (int pos = 0; pos < 2 * n; ++pos, from.advance(1), to.advance(1)) {
                bool is_k;
                const int t = at_pos(pos, is_k);
                const int valid = sm->keys - t * kSharedTile;
                bool go = wait_phase(&sm->raw_full[from.slot], from.phase, p, sm);
                if (go && pos >= kWideBuffers)
                    go = wait_phase(&sm->empty[to.slot], to.phase ^ 1, p, sm);
                if (!__all_sync(0xffffffffu, go))
                    break;
                const uint8_t *src = raw0 + from.slot * kRawBytes + lane_src;
                uint8_t *dst = ring_ptr + to.slot * kBufBytes;
                uint8_t *dst0 = dst + lane_dst, *dst1 = dst + (lane_dst ^ 16);
                uint4 x[kMine];
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    x[j] = *reinterpret_cast<const uint4 *>(src + j * kStep);
                if (!is_k && valid < kSharedTile) {   // V rows past the last key
#pragma unroll
                    for (int j = 0; j < kMine; ++j)
                        if (row + j * (kWidenWarps * 4) >= valid)
                            x[j] = make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                    uint32_t f[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
                            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
                            : "=r"(f[2 * q]), "=r"(f[2 * q + 1])
                            : "r"(w[q]));
                    *reinterpret_cast<uint4 *>(dst0 + j * kStep) = make_uint4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<uint4 *>(dst1 + j * kStep) = make_uint4(f[4], f[5], f[6], f[7]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_addr(&sm->raw_empty[from.slot]));
                    mbar_arrive(smem_addr(&sm->full[to.slot]));
                }
            }
        } else if (warp < kProducerWarp) {
            // -------------------------------------------------------- the softmax
            const int s = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;
            const int trow = quad * 32 + lane;   // row of the stream's tile: lane of tensor memory
            const uint32_t s_col = tmem + ((uint32_t)quad << 21) + s * kStreamCols + half * 64, o_col = s_col + 128;
            const int pair_bar = 2 + s * 4 + quad;   // barrier of the two warps that share rows
            const bool two = q_tiles == 2;
            float factor = p.scale, v_scale = 1.f;
            if constexpr (kFp8) {
                factor *= ok ? __ldcg(p.k_scale + sm->kvh) : 1.f;
                v_scale = ok ? __ldcg(p.v_scale + sm->kvh) : 1.f;
            }
            if (ok && !careful) {
                // Q rows into shared memory, [half][128 rows][128 bytes] a tile; a
                // negative factor of the scores turns q around.
                const uint32_t flip = factor < 0.f ? 0x80008000u : 0u;
                for (int i = tid; i < q_tiles * kSharedQRows * 16; i += kSoftmaxThreads) {
                    const int r = i >> 4, ch = i & 15;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (r < sm->rows) {
                        const int gr = sm->row0 + r;
                        const int64_t row = (int64_t)(sm->req0 + gr / p.group) * p.num_qo_heads + sm->kvh * p.group +
                                            gr % p.group;
                        v = __ldcg(reinterpret_cast<const uint4 *>(p.q + row * kHeadDim) + ch);
                    }
                    v.x ^= flip;
                    v.y ^= flip;
                    v.z ^= flip;
                    v.w ^= flip;
                    if constexpr (kFp8) {
                        // to f16, times the power of two that puts the row's largest
                        // magnitude in [2^8, 2^9): exact down to 2^-22 of it
                        uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        float amax = 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 a = bf16x2_to_float2(w[j]);
                            amax = fmaxf(amax, fmaxf(fabsf(a.x), fabsf(a.y)));
                        }
#pragma unroll
                        for (int o = 1; o < 16; o <<= 1)
                            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                        int sh = 0;
                        if (amax > 0.f) {
                            int e;
                            frexpf(amax, &e);
                            sh = min(max(9 - e, -100), 100);
                        }
                        const float up = __int_as_float((127 + sh) << 23);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 a = bf16x2_to_float2(w[j]);
                            w[j] = pack2<DT>(make_float2(a.x * up, a.y * up));
                        }
                        v = make_uint4(w[0], w[1], w[2], w[3]);
                        if (ch == 0)
                            sm->q_scale[r] = __int_as_float((127 - sh) << 23);
                    }
                    const int rr = r & 127;
                    *reinterpret_cast<uint4 *>(smem + (r >> 7) * kBufBytes + (ch >> 3) * kHalfBytes + rr * 128 +
                                               (((ch & 7) ^ (rr & 7)) << 4)) = v;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            __syncwarp();
            if (lane == 0 && ok)
                mbar_arrive(smem_addr(&sm->q_ready));
            // log2 e times the factor of the scores; never 0, so that a masked score
            // (-inf) stays -inf
            if (!careful) {
                c2 = fabsf(factor) * kLog2e;
                if constexpr (kFp8) {
                    barrier(1, kSoftmaxThreads);   // q_scale is written
                    c2 *= sm->q_scale[(two ? s * kSharedQRows : 0) + trow];
                    barrier(1, kSoftmaxThreads);   // row_max takes its place
                }
                c2 = c2 == 0.f ? 1.17549435e-38f : c2;
            }
            // FP8: weights are 2^7 times larger, which keeps seven more bits of the
            // small ones in f16; it cancels in O
            constexpr float kBias = kFp8 ? 7.f : 0.f;
            // Where the thread adds up its 64 values of O (see kFlush): 16 bytes of each
            // of the stream's rows side by side, so that a warp writes whole lines.
            const bool flushed = steps(s) > kFlush;
            const int run = shared_run(steps(s));
            int next_flush = run;
            float *my_flush = p.flush + (((int64_t)blockIdx.x * 2 + s) * 32 + half * 16) * (4 * kSharedQRows) +
                              4 * trow;
            auto flush = [&](int i) {   // O of the steps before step i: their products are done
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[16];
                    tmem_ld16(o_col + 16 * c, o);
                    tmem_wait_ld();
                    settle(o);
                    flush16(my_flush + c * (16 * kSharedQRows), o, i > run);
                }
                next_flush += run;
            };
            float m_ref = -INFINITY, l = 0.f;   // what the weights refer to (a raw score), their sum
            bool go = ok;
            // 16 scores to weights, over their columns: hi in the first 8, lo in the others
            auto weights = [&](const uint32_t (&r)[16], int j16, float off, float2 &sum) {
                const float2 c22 = make_float2(c2, c2), off2 = make_float2(off, off);
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 score = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                    const float2 x = fma2(score, c22, off2);
                    const float2 w = make_float2(ex2(x.x), ex2(x.y));
                    sum = add2(sum, w);
                    hi[j] = pack2<DT>(w);
                    const float2 h = unpack2<DT>(hi[j]);
                    lo[j] = pack2<DT>(fma2(h, make_float2(-1.f, -1.f), w));
                }
                tmem_st8(s_col + 16 * j16, hi);
                tmem_st8(s_col + 16 * j16 + 8, lo);
            };
            auto publish = [&](int part) {
                tmem_wait_st();
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&sm->p_ready[s][part]));
            };
            auto load = [&](uint32_t (&r)[16], int j16) { tmem_ld16(s_col + 16 * j16, r); };
            auto ready = [&](uint32_t (&r)[16], int valid) {   // loaded, scores past the last key masked
                tmem_wait_ld();
                settle(r);
                if (valid < 16) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j >= valid)
                            r[j] = 0xff800000u;
                }
            };
            // All 64 scores to weights, the next 16 on their way meanwhile.
            auto step = [&](uint32_t (&r0)[16], uint32_t (&r1)[16], int valid, float off) {   // r0: loaded
                float2 sum = make_float2(0.f, 0.f);
                ready(r0, valid);
                load(r1, 1);
                weights(r0, 0, off, sum);
                ready(r1, valid - 16);
                load(r0, 2);
                weights(r1, 1, off, sum);
                publish(0);
                ready(r0, valid - 32);
                load(r1, 3);
                weights(r0, 2, off, sum);
                ready(r1, valid - 48);
                weights(r1, 3, off, sum);
                publish(1);
                l += sum.x + sum.y;
            };
            for (int i = 0; i < steps(s); ++i) {
                // After an error the steps go on without work, so that the barriers
                // of a row's two warps always meet.
                if (go)
                    go = __all_sync(0xffffffffu, wait_phase(&sm->s_full[s], i & 1, p, sm));
                const int t = two ? i : 2 * i + s;
                const int valid = sm->keys - t * kSharedTile - half * 64;
                uint32_t r0[16], r1[16];
                if (i > 0 && !careful) {
                    if (go) {
                        tcgen05_fence_after();
                        if (i == next_flush)
                            flush(i);
                        load(r0, 0);
                        step(r0, r1, valid, kBias - m_ref * c2);
                    }
                    continue;
                }
                // The first step, and every careful one: a row's maximum is that of
                // both halves of its keys.
                float mt = -INFINITY;
                bool raise = false;
                if (go) {
                    tcgen05_fence_after();
                    if (i == next_flush)
                        flush(i);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        load(r0, c);
                        ready(r0, valid - 16 * c);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            mt = fmaxf(mt, __uint_as_float(r0[j]));
                    }
                    raise = mt > m_ref && (m_ref == -INFINITY || (mt - m_ref) * c2 > kRaise);
                }
                if (barrier_or(pair_bar, 64, raise)) {
                    sm->row_max[s][half][trow] = mt;
                    barrier(pair_bar, 64);
                    const float both = fmaxf(mt, sm->row_max[s][half ^ 1][trow]);
                    const bool up = both > m_ref && (m_ref == -INFINITY || (both - m_ref) * c2 > kRaise);
                    const float m_new = up ? both : m_ref;
                    const float f = m_ref == -INFINITY ? 0.f : ex2((m_ref - m_new) * c2);
                    l *= f;
                    m_ref = m_new;
                    if (i > 0 && go) {   // the products up to the last step are done: s_full followed them
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t o[16];
                            tmem_ld16(o_col + 16 * c, o);
                            tmem_wait_ld();
                            settle(o);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st16(o_col + 16 * c, o);
                            if (i >= run)
                                scale_flushed16(my_flush + c * (16 * kSharedQRows), f);
                        }
                    }
                    barrier(pair_bar, 64);   // row_max is read before the next step writes it
                }
                if (!go)
                    continue;
                load(r0, 0);
                // a row whose scores are all -inf so far keeps weights of 0
                step(r0, r1, valid, (m_ref == -INFINITY ? 0.f : -m_ref * c2) + kBias);
            }
            // ----------------------------------------------------- the partial
            for (int x = 0; x < 2; ++x)   // both streams' products are done with the ring
                if (go && steps(x) > 0)
                    go = __all_sync(0xffffffffu, wait_phase(&sm->o_done[x], 0, p, sm));
            tcgen05_fence_after();
            // Out of range: a weight too large for its type, or no score to refer to
            // in the first tile.
            if (go && !careful && steps(s) > 0) {
                bool again = m_ref == -INFINITY || l > kMostSum;
                if constexpr (kFp8) {
                    uint32_t o[16];
                    tmem_ld16(o_col, o);
                    tmem_wait_ld();
                    settle(o);
                    const float sum = __uint_as_float(o[0]) + (flushed ? __ldcg(my_flush) : 0.f);
                    again |= sum != sum;
                }
                if (again)
                    sm->redo = 1;
            }
            barrier(1, kSoftmaxThreads);
            if (careful || !sm->redo) {
                float *stage = reinterpret_cast<float *>(smem);   // [q_tiles * 128][kOutStride]
                SharedEnd *end = reinterpret_cast<SharedEnd *>(smem + kEndOffset);
                float *mine = stage + ((two ? s * kSharedQRows : 0) + trow) * kOutStride + half * 64;
                if (go)
                    end->row_sum[s][half][trow] = l;
                if (!two && s == 1) {
                    // one row tile: stream 1 hands its state to stream 0
                    if (go && half == 0)
                        end->row_ref[trow] = m_ref;
                    if (go && steps(1) > 0) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t o[16];
                            tmem_ld16(o_col + 16 * c, o);
                            tmem_wait_ld();
                            settle(o);
                            if (flushed)
                                add_flushed16(my_flush + c * (16 * kSharedQRows), o);
#pragma unroll
                            for (int j = 0; j < 16; j += 4)
                                *reinterpret_cast<uint4 *>(mine + 16 * c + j) =
                                    make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                        }
                    }
                }
                barrier(1, kSoftmaxThreads);
                if (go && (two || s == 0)) {
                    float f0 = 1.f, f1 = 0.f, m = m_ref, den = end->row_sum[s][0][trow] + end->row_sum[s][1][trow];
                    const bool join = !two && steps(1) > 0;
                    if (join) {
                        const float m1 = end->row_ref[trow], l1 = end->row_sum[1][0][trow] + end->row_sum[1][1][trow];
                        m = fmaxf(m_ref, m1);
                        f0 = m_ref == -INFINITY ? 0.f : ex2((m_ref - m) * c2);
                        f1 = m1 == -INFINITY ? 0.f : ex2((m1 - m) * c2);
                        den = den * f0 + l1 * f1;
                    }
                    const float inv = v_scale / den;
                    f0 *= inv;
                    f1 *= inv;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[16];
                        tmem_ld16(o_col + 16 * c, o);
                        tmem_wait_ld();
                        settle(o);
                        if (flushed)
                            add_flushed16(my_flush + c * (16 * kSharedQRows), o);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            float4 v = make_float4(__uint_as_float(o[j]) * f0, __uint_as_float(o[j + 1]) * f0,
                                                   __uint_as_float(o[j + 2]) * f0, __uint_as_float(o[j + 3]) * f0);
                            float4 *d = reinterpret_cast<float4 *>(mine + 16 * c + j);
                            if (join) {
                                const float4 w = *d;
                                v.x = fmaf(w.x, f1, v.x);
                                v.y = fmaf(w.y, f1, v.y);
                                v.z = fmaf(w.z, f1, v.z);
                                v.w = fmaf(w.w, f1, v.w);
                            }
                            *d = v;
                        }
                    }
                    const int r = (two ? s * kSharedQRows : 0) + trow;
                    if (half == 0 && r < sm->rows) {
                        const int gr = sm->row0 + r;
                        const int64_t out = (int64_t)(gr / p.group) * p.num_qo_heads + sm->kvh * p.group + gr % p.group;
                        p.partial_lse[sm->part_row + out * sm->part_stride] =
                            den == 0.f ? -INFINITY : (m * c2 + log2f(den) - kBias) * kLn2;
                    }
                }
                barrier(1, kSoftmaxThreads);
                if (go) {   // whole rows, a warp at a time
                    for (int r = warp; r < sm->rows; r += kSoftmaxThreads / 32) {
                        const int gr = sm->row0 + r;
                        const int64_t out = (int64_t)(gr / p.group) * p.num_qo_heads + sm->kvh * p.group + gr % p.group;
                        const float4 v = *reinterpret_cast<const float4 *>(stage + r * kOutStride + 4 * lane);
                        float *dst = p.partial_o + (sm->part_row + out * sm->part_stride) * kHeadDim;
                        reinterpret_cast<float4 *>(dst)[lane] = v;
                    }
                }
            }
        }
        tcgen05_fence_before();
        __syncthreads();
        if (careful || !sm->redo || sm->abort)
            break;
        if (warp == kProducerWarp && lane == 0)
            init_barriers(true);   // every phase of the first pass has completed
        __syncthreads();
        tcgen05_fence_after();
    }
    griddep_launch_dependents();
    if (p.has_suffix)
        griddep_wait();
    if (warp == kMmaWarp) {
        tcgen05_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    // After an error nobody waited for the copies in flight: do so before the
    // CTA ends and its shared memory may be handed on.
    if (warp == kProducerWarp && lane == 0 && ok && sm->abort) {
        uint64_t *bar_full = kFp8 ? sm->raw_full : sm->full;
        for (int i = 0; i < nb; ++i) {
            const int last = sm->issued - 1 - i;   // the newest fill of each buffer
            if (last >= 0 && !(sm->tail_issued && last == 2 * n - 1))
                mbar_wait(smem_addr(&bar_full[last % nb]), (last / nb) & 1, kDrainTimeoutNs);
        }
        if (sm->tail_issued)
            mbar_wait(smem_addr(&sm->tail), 0, kDrainTimeoutNs);
    }
}

// Stage 2: for each (request, query head) the merge of its prefix's partials
// and, where there is one, the state of its own keys (in o, lse).  A row is
// WARPS warps', lane = 4 output columns, kMergeBatch partials of loads in flight
// a warp; with several warps each takes every WARPS-th batch and the first one
// adds their states up.  Bound: a chain of loads (tables, partials, a batch at a
// time), 4-5 us behind the prefixes' grid.
constexpr int kMergeWarps = 4;
constexpr int kMergeBatch = 8;

struct MergeState {
    float m, den;   // maximum of the LSEs, sum of the weights that refer to it
    float4 acc;
};

template <int WARPS>
__global__ void __launch_bounds__(kMergeWarps * 32) shared_merge_kernel(const __grid_constant__ SharedParams p)
{
    __shared__ MergeState s_state[kMergeWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WARPS;
    const int row = blockIdx.x * (kMergeWarps / WARPS) + warp / WARPS;
    const bool has_row = row < p.batch * p.num_qo_heads;
    // The tables were there before the prefixes' grid (or the suffixes'), which this
    // one's start follows: they are read before the wait for its partials.  With no
    // keys at all this grid is the call's first, and what it follows may still be
    // writing them.
    if (p.num_items == 0 && !p.has_suffix)
        griddep_wait();
    const int b = row / p.num_qo_heads;
    PrefixCoord c;
    int n = 0;
    int64_t first = 0;
    const bool found = has_row && locate_prefix(p, b, true, c);
    if (found) {
        n = c.splits;
        first = c.row0 + (int64_t)(row - c.req0 * p.num_qo_heads) * n;
    }
    griddep_wait();
    griddep_launch_dependents();
    // More own keys than the plan has room for (or any, where it has none): some were
    // not attended.
    if (row == 0 && part == 0 && p.suffix_indptr) {
        int64_t keys = 0;
        for (int i = lane; i < p.batch; i += 32) {
            const int64_t d = (int64_t)__ldcg(p.suffix_indptr + i + 1) - __ldcg(p.suffix_indptr + i);
            if (d > 0)
                keys += p.page_size && p.suffix_last_len ? (d - 1) * p.page_size + __ldcg(p.suffix_last_len + i) : d;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            keys += __shfl_xor_sync(0xffffffffu, keys, o);
        if (lane == 0 && keys > p.max_suffix_tokens)
            report(p.status, FD_ERR_DEVICE_BOUNDS);
    }
    if (has_row && !found && lane == 0)
        report(p.status, FD_ERR_DEVICE_BOUNDS);
    float4 *o_row = reinterpret_cast<float4 *>(p.o + (int64_t)row * kHeadDim) + lane;
    float m = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.has_suffix && has_row && part == 0) {
        m = p.lse[row];
        acc = *o_row;
        if (m != -INFINITY)
            den = 1.f;
        else
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float *lse_in = p.partial_lse + first;
    const float4 *o_in = reinterpret_cast<const float4 *>(p.partial_o + first * kHeadDim) + lane;
    for (int i0 = part * kMergeBatch; i0 < n; i0 += WARPS * kMergeBatch) {
        float l[kMergeBatch];
        float4 v[kMergeBatch];
#pragma unroll
        for (int u = 0; u < kMergeBatch; ++u) {
            l[u] = -INFINITY;
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + u < n) {
                l[u] = __ldcg(lse_in + i0 + u);
                v[u] = __ldcg(o_in + (int64_t)(i0 + u) * (kHeadDim / 4));
            }
        }
        float m_new = m;
        bool nan = false;
#pragma unroll
        for (int u = 0; u < kMergeBatch; ++u) {
            m_new = fmaxf(m_new, l[u]);
            nan |= l[u] != l[u];
        }
        if (m_new == -INFINITY && !nan)
            continue;
        const float f = expf(m - m_new);
        den *= f;
        acc.x *= f;
        acc.y *= f;
        acc.z *= f;
        acc.w *= f;
#pragma unroll
        for (int u = 0; u < kMergeBatch; ++u) {
            const float w = expf(l[u] - m_new);
            if (w == 0.f)   // no keys, or none that counts: its O may be anything
                continue;
            den += w;
            acc.x = fmaf(w, v[u].x, acc.x);
            acc.y = fmaf(w, v[u].y, acc.y);
            acc.z = fmaf(w, v[u].z, acc.z);
            acc.w = fmaf(w, v[u].w, acc.w);
        }
        m = m_new;
    }
    if constexpr (WARPS > 1) {
        s_state[warp][lane] = MergeState{m, den, acc};
        __syncthreads();
        if (part > 0)
            return;
        float m_all = m;
#pragma unroll
        for (int w = 1; w < WARPS; ++w)
            m_all = fmaxf(m_all, s_state[warp + w][lane].m);
        const float f = den == 0.f ? 0.f : expf(m - m_all);
        den *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
            const MergeState x = s_state[warp + w][lane];
            if (x.den == 0.f)   // no partials, or no keys
                continue;
            const float g = expf(x.m - m_all);
            den = fmaf(g, x.den, den);
            acc.x = fmaf(g, x.acc.x, acc.x);
            acc.y = fmaf(g, x.acc.y, acc.y);
            acc.z = fmaf(g, x.acc.z, acc.z);
            acc.w = fmaf(g, x.acc.w, acc.w);
        }
        m = m_all;
    }
    if (!has_row)
        return;
    const float inv = den == 0.f ? 0.f : 1.f / den;   // no keys at all: O = 0, LSE = -inf
    *o_row = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    __syncwarp();
    if (lane == 0)
        p.lse[row] = den == 0.f ? -INFINITY : m + logf(den);
}

}  // namespace
}  // namespace fd
