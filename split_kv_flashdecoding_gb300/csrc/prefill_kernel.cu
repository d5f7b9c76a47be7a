// prefill_kernel.cu -- attention of one to many query tokens a request over an INT8
// paged cache with a scale per page and KV head, on sm_103a: prompts, chunks of them
// behind cached keys, checks of drafted tokens (causal), cross attention (all keys).
//
// Mathematics: the T * G queries of a request and KV head are the rows of one
// matrix; with integer codes C and page scales k, v of a key's page,
//     e_j = c k <q, C_K,j> + log2 v,  P_j = exp2(e_j - E),  O = (sum_j P_j C_V,j) / l,
//     l = sum_j P_j / v,
// c = scale log2 e and E near the row's largest e.  So both scales are numbers of a
// 16-key group of a tile (pages are whole groups): the K scale goes into the factor
// of the score, the V scale into the addend of the exponent, and the codes go into
// the products as they are.  V scales count from the largest of the split's first tile
// (v_ref).  Where others are 2^20 of it or more, or 2^-40 or less, the CTA does its item a
// second time with l summed by itself, over the row's largest score: O and l then have
// references of their own, and no range of scales that one of them cannot hold.
//
// Every (request, block of 256 rows, split of the keys, KV head) is one CTA.  The
// products run on tcgen05 in f16 with their accumulators in tensor memory: two
// streams of S (P over it) and O, 256 columns each: two row tiles that share each K
// and V tile, or, with up to 128 rows, alternate key tiles of one row tile.  A
// weight enters the second product as one f16 value (2^-12 of it on the average;
// the output is bf16), so a tile costs the two products of the definition.
//
// Four warps copy the codes into shared memory and widen them into operand tiles.
//
// Bound: the tensor cores at many rows (2048 cycles for the products of two row tiles
// with 128 keys), one chain of scores, weights and products a stream beside it: 3100
// cycles.  32 heads, 8192 queries and keys 414 us, 1.33 PFLOP/s, of which an item's start
// and end (queries 3.7 us, first weights 3.6, output 2.6, with nothing beside them) are
// a sixth; 32768 queries and keys 5.8 ms, 1.50 PFLOP/s; 64 heads, a chunk of 2047 behind
// 30001 cached keys, 1.53 ms, 1.36 PFLOP/s.  The roles' loops together are near
// what the SM holds of instructions: the same steps in other code ran up to 8 % slower
// (stalls for instructions 1.1 an issue for 0.6).  At few rows the bytes: 2400 cycles
// a tile of 32 KB of codes, 3.3 TB/s; the widening's chain (copies, loads, stores,
// hand-over), the weights' and the copies' latency each take a part of it, and leaving
// any one out saves 3 to 15 %.
//
// Warps: 0-7 the softmax, a warpgroup a stream; a thread owns a row and all of its
// scores, 128 in registers.  (Two threads a row, 64 scores each, took 3600 cycles a
// tile of two row tiles, this form 3300 in its place and 3100 with the steps since: the
// streams wait for the chain scores -> weights -> products, and a thread that needs no
// other one shortens it.)  8-11 load and widen, 12 issues the products of both streams
// in turn, 13 looks up the tiles' scales.
//
// A row's reference E comes from the tiles up to the last one (the first tile's from
// its own largest e): of each the log of its sum of weights, which costs no
// comparisons; it is up to log2 128 above the largest e, but then the row's sum is that
// much larger, too, and what f16 loses of weights near the others is as little of it.  E is
// raised, with O rescaled, when that is over 2^kRaise above it: so no step waits for
// its own maximum.  A score so far above all before it that its weight is over
// f16's range is seen at the end, and the CTA then does its item again with the
// maximum of every step before its weights.
//
// E goes down, too, when the tiles since the largest have stayed far below it: a key
// that takes nearly all of a row's weight, its V near 0, would otherwise push the
// others' weights below f16's smallest number, of which O consists (a first key with 99 %
// of 131072 keys' weight: O off by 9 % of its norm, so 0.3 %).  It waits for some tiles
// (kFade), and does not go all the way (kDeep), because a score over f16's range costs a
// second pass, and with E at each tile's own level many items of wide-spread scores
// would have one: 64 heads, a chunk of 2047 tokens behind 30001 keys, 1532 us with E at
// the largest, 1549 so, 1753 without waiting, and 2003 for 1571 in an older form whose E
// was at the largest and whose weights were 2^5 times larger.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "device_common.cuh"
#include "int8_widen.cuh"
#include "prefill_kernels.h"
#include "tc_stream.cuh"
#include "tcgen05.cuh"

namespace fd {
namespace {

constexpr int kTileRows = 128;                              // query rows of a tensor-core tile
constexpr int kBufBytes = kPrefillTile * kHeadDim * 2;      // an f16 tile: 32 KB
constexpr int kHalfBytes = kBufBytes / 2;
constexpr int kBuffers = 7;                                 // Q tiles and the ring together
constexpr int kRing = 4;                                    // operand tiles of K and V
constexpr int kRawBytes = kBufBytes / 2;                    // a tile of codes: those on their way take the rest
constexpr int kScaleSlots = 4;
constexpr int kSoftmaxThreads = 256;
constexpr int kStreamWarps = 4;
constexpr int kLoadWarp = 8, kLoadWarps = 4, kMmaWarp = 12, kScaleWarp = 13;   // (and two warps without work)
constexpr int kThreads = 512;
// Registers a thread: at the launch, and after the warpgroups have shared them out,
// two of the softmax, the loads, the products.
constexpr int kRegs = 128, kSoftmaxRegs = 184, kLoadRegs = 80, kMmaRegs = 56;
static_assert(2 * kSoftmaxRegs + kLoadRegs + kMmaRegs <= kThreads / 128 * kRegs, "no more than the launch has");
static_assert(kThreads * kRegs <= 65536, "registers of an SM");
constexpr int kTmemCols = 512;
constexpr int kStreamCols = 256;                            // S (and P over it) 128, O 128
// In log2.  The tiles' level is that of the last one, or of one before it less kFade a
// tile since then, and less what the last one is under it, beyond kGap and up to kFall.
// E follows it, down to kDeep below the largest, when it is more than kRaise above or
// kLower below E.
constexpr float kRaise = 3.f, kLower = 6.f, kDeep = 7.f;
constexpr float kFade = 0.125f, kGap = 6.f, kFall = 8.f;
// Weights are 2^kBias larger than over E: of small ones' bits.  Careful steps, whose
// weights over E are at most 2^kRaise, have as much as f16 takes.
constexpr float kBias = 1.f, kCarefulBias = 12.f;
static_assert(kBias + kDeep + kRaise < 16 && kCarefulBias + kRaise < 16, "a weight of the largest so far is in range");
constexpr int kOutStride = kHeadDim + 4;                    // floats between rows of the epilogue's staging
constexpr int kGroups = kPrefillTile / 16;
// log2 of a V scale over v_ref in a first pass, and what one of 2^-126, that of a page of
// zeros, counts as at the least.  A row's sum is of weights over E, divided by the
// scales: with 128 keys of the largest scale and score E is 2^(kMostV + 7), a key of a page
// of zeros and the same score 2^-87 of that, and one of 2^-39 of its weight still a number.
constexpr float kLeastV = -40.f, kMostV = 20.f, kZeroV = -60.f;
constexpr float kSmallestScale = 1.17549435e-38f;

struct PrefillSmem {
    uint64_t full[kRing], empty[kRing];
    uint64_t scales_ready[kScaleSlots], scales_free[kScaleSlots];
    uint64_t s_full[2], p_ready[2][2], o_done[2];
    uint64_t q_ready, drain;
    uint32_t tmem;
    int abort, redo, wide;
    // the CTA's item
    int ok, q0, tokens, len, base, kvh, row0, rows, key0, keys, splits, part_row, q_tiles;
    float v_ref, ref_log;                 // a V scale, and its log2
    float4 scale[kScaleSlots][kGroups];   // a tile's groups: K scale, log2 (V scale / v_ref), v_ref / V scale
    float q_scale[kPrefillRows];          // a row's factor
};
struct PrefillEnd {   // at the end, behind the staged rows: stream 1's state, one row tile
    float row_sum[kTileRows], row_ref[kTileRows], row_top[kTileRows];
};
// One row tile: stream 1's O [128][kOutStride], the rest of its state, staged rows.
constexpr int kEndOffset = kTileRows * kOutStride * 4;
constexpr int kStageOffset = kEndOffset + (int)sizeof(PrefillEnd);
constexpr int kRowStage = kHeadDim * 4 + 16;            // bytes between staged rows
static_assert(kStageOffset % 16 == 0 && kStageOffset + kTileRows * kRowStage <= kBuffers * kBufBytes &&
                  kPrefillRows * kRowStage <= kBuffers * kBufBytes,
              "the epilogue works over the ring");
constexpr int kPrefillAlloc = kBuffers * kBufBytes + (int)((sizeof(PrefillSmem) + 15) / 16 * 16);
static_assert(kPrefillAlloc <= 232448, "shared memory of one CTA");

__device__ __forceinline__ uint32_t pack_f16x2(float2 a)
{
    const __half2 h = __floats2half2_rn(a.x, a.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

struct RequestCoord {
    int32_t q0, tokens;        // first token and their number
    int32_t base, len;         // first page-list entry, keys
    int32_t splits, blocks;
    int32_t item0, row0, merge0;   // items, partial rows and merged rows of the requests before
};

// One request's numbers; one outside the tokens or the list has none of them (false).
__device__ __forceinline__ bool size_request(const PrefillParams &p, int b, int32_t &q0, int32_t &tokens,
                                             int32_t &base, int32_t &len, int32_t &splits, int32_t &blocks)
{
    q0 = __ldcg(p.q_indptr + b);
    base = __ldcg(p.page_indptr + b);
    tokens = len = splits = blocks = 0;
    const int32_t q1 = __ldcg(p.q_indptr + b + 1), e1 = __ldcg(p.page_indptr + b + 1);
    const int32_t last = __ldcg(p.last_len + b);
    const int64_t keys = e1 == base ? 0 : (int64_t)(e1 - base - 1) * p.page_size + last;
    if (q0 < 0 || q0 > q1 || q1 > p.num_tokens || base < 0 || base > e1 || e1 > p.page_entries ||
        (e1 != base && (last < 1 || last > p.page_size)) || keys > INT32_MAX - kPrefillTile)
        return false;
    tokens = q1 - q0;
    len = (int32_t)keys;
    splits = prefill_splits(len, p.chunk);
    blocks = (int32_t)(((int64_t)tokens * p.group + kPrefillRows - 1) / kPrefillRows);
    return true;
}

// Whole warp: reports tables that need other items or rows than the plan has.
__device__ __forceinline__ void check_tables(const PrefillParams &p)
{
    int64_t items = 0, rows = 0;
    bool good = true;
    for (int b = threadIdx.x & 31; b < p.batch; b += 32) {
        int32_t q0, tokens, base, len, splits, blocks;
        good &= size_request(p, b, q0, tokens, base, len, splits, blocks);
        items += (int64_t)splits * blocks * p.num_kv_heads;
        rows += splits > 1 ? (int64_t)splits * tokens * p.num_qo_heads : 0;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        items += __shfl_xor_sync(0xffffffffu, items, o);
        rows += __shfl_xor_sync(0xffffffffu, rows, o);
    }
    if (!good || items != p.num_items || rows != p.num_partial_rows)
        report(p.status, FD_ERR_DEVICE_BOUNDS);
}

// Whole warp: the request that holds item `j` (or, by_row, merged row `j`).  False
// when there is none or the tables are outside what the plan was made for.
__device__ __forceinline__ bool locate_request(const PrefillParams &p, int32_t j, bool by_row, RequestCoord &out)
{
    const int lane = threadIdx.x & 31;
    int32_t item_carry = 0, row_carry = 0, merge_carry = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int b = b0 + lane;
        int32_t q0 = 0, tokens = 0, base = 0, len = 0, splits = 0, blocks = 0;
        if (b < p.batch)
            size_request(p, b, q0, tokens, base, len, splits, blocks);
        const int64_t items64 = (int64_t)splits * blocks * p.num_kv_heads;
        const int64_t merge64 = splits > 1 ? (int64_t)tokens * p.num_qo_heads : 0;
        const int64_t rows64 = merge64 * splits;
        const bool fits = items64 <= p.num_items && rows64 <= p.num_partial_rows && merge64 <= p.merge_rows;
        const int32_t items = fits ? (int32_t)items64 : 0, rows = fits ? (int32_t)rows64 : 0;
        const int32_t merge = fits ? (int32_t)merge64 : 0;
        int32_t item_incl = items, row_incl = rows, merge_incl = merge;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t t = __shfl_up_sync(0xffffffffu, item_incl, o);
            const int32_t u = __shfl_up_sync(0xffffffffu, row_incl, o);
            const int32_t w = __shfl_up_sync(0xffffffffu, merge_incl, o);
            if (lane >= o) {
                item_incl += t;
                row_incl += u;
                merge_incl += w;
            }
        }
        item_incl += item_carry;
        row_incl += row_carry;
        merge_incl += merge_carry;
        const bool hit = by_row ? j >= merge_incl - merge && j < merge_incl : j >= item_incl - items && j < item_incl;
        const unsigned mask = __ballot_sync(0xffffffffu, hit);
        if (mask) {
            const int src = __ffs(mask) - 1;
            out.q0 = __shfl_sync(0xffffffffu, q0, src);
            out.tokens = __shfl_sync(0xffffffffu, tokens, src);
            out.base = __shfl_sync(0xffffffffu, base, src);
            out.len = __shfl_sync(0xffffffffu, len, src);
            out.splits = __shfl_sync(0xffffffffu, splits, src);
            out.blocks = __shfl_sync(0xffffffffu, blocks, src);
            out.item0 = __shfl_sync(0xffffffffu, item_incl - items, src);
            out.row0 = __shfl_sync(0xffffffffu, row_incl - rows, src);
            out.merge0 = __shfl_sync(0xffffffffu, merge_incl - merge, src);
            // by int32 sums that may have wrapped: in range all the same
            const int64_t m = out.splits > 1 ? (int64_t)out.tokens * p.num_qo_heads : 0;
            return out.item0 >= 0 && out.row0 >= 0 && out.merge0 >= 0 &&
                   (int64_t)out.item0 + (int64_t)out.splits * out.blocks * p.num_kv_heads <= p.num_items &&
                   (int64_t)out.row0 + m * out.splits <= p.num_partial_rows && out.merge0 + m <= p.merge_rows;
        }
        item_carry = __shfl_sync(0xffffffffu, item_incl, 31);
        row_carry = __shfl_sync(0xffffffffu, row_incl, 31);
        merge_carry = __shfl_sync(0xffffffffu, merge_incl, 31);
    }
    return false;
}

// Where the 16-key groups of an item's tiles are, tile by tile: a lane follows group
// lane % 8.
struct GroupPages {
    struct Spot {
        int id, off;   // page and row in it; off -1: past the last key
    };
    const PrefillParams &p;
    int pg, off, left, base, pages_on, rows_on;

    __device__ __forceinline__ GroupPages(const PrefillParams &p_, int key0, int keys, int base_) : p(p_), base(base_)
    {
        const int at = 16 * (threadIdx.x & 7);
        pg = (key0 + at) / p.page_size;
        off = (key0 + at) % p.page_size;
        left = keys - at;
        pages_on = kPrefillTile / p.page_size;
        rows_on = kPrefillTile % p.page_size;
    }
    __device__ __forceinline__ Spot next()
    {
        const Spot x{left > 0 ? __ldcg(p.page_indices + base + pg) : 0, left > 0 ? off : -1};
        left -= kPrefillTile;
        pg += pages_on;
        off += rows_on;
        if (off >= p.page_size) {
            off -= p.page_size;
            ++pg;
        }
        return x;
    }
    __device__ __forceinline__ int page_of(const Spot &x) const   // page 0 for what is not there
    {
        const bool in = x.id >= 0 && x.id < p.num_pages;
        if (!in)
            report(p.status, FD_ERR_DEVICE_BOUNDS);
        return in ? x.id : 0;
    }
};

// Operand tiles: 128 rows x 128 f16 values, [64-value half][128 rows][128 bytes],
// 128-byte swizzle.
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    PrefillSmem *sm = reinterpret_cast<PrefillSmem *>(smem + kBuffers * kBufBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // One thread: all barriers before their first phase.
    auto init_barriers = [&](bool again) {
        auto init = [&](uint64_t *bar, uint32_t count) {
            if (again)
                mbar_inval(smem_addr(bar));
            mbar_init(smem_addr(bar), count);
        };
        for (int i = 0; i < kRing; ++i) {
            init(&sm->full[i], kLoadWarps);
            init(&sm->empty[i], 1);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            init(&sm->scales_ready[i], 1);
            init(&sm->scales_free[i], 2 * kStreamWarps);   // both streams', or twice the one's
        }
        for (int s = 0; s < 2; ++s) {
            init(&sm->s_full[s], 1);
            init(&sm->p_ready[s][0], kStreamWarps);
            init(&sm->p_ready[s][1], kStreamWarps);
            init(&sm->o_done[s], 1);
        }
        init(&sm->q_ready, kSoftmaxThreads / 32);
        init(&sm->drain, 1);
        fence_mbar_init();
    };
    if (warp == kMmaWarp)
        tmem_alloc(smem_addr(&sm->tmem), kTmemCols);
    griddep_wait();
    if (warp == kLoadWarp) {
        RequestCoord c;
        const int w = blockIdx.x;
        // operand tiles of a 1024-byte swizzle pattern: the base must be aligned
        const bool found = locate_request(p, w, false, c) && (smem_addr(smem) & 1023) == 0;
        if (lane == 0) {
            sm->ok = found;
            sm->q_tiles = 1;
            sm->keys = 0;
            if (found) {
                // a request's last blocks first: with a causal mask they have the most keys
                const int rest = w - c.item0, sb = rest / p.num_kv_heads;
                const int split = sb % c.splits, block = c.blocks - 1 - sb / c.splits;
                const int len = prefill_split_len(c.len, c.splits);
                sm->kvh = rest % p.num_kv_heads;
                sm->q0 = c.q0;
                sm->tokens = c.tokens;
                sm->len = c.len;
                sm->base = c.base;
                sm->row0 = block * kPrefillRows;
                sm->rows = min(c.tokens * p.group - sm->row0, kPrefillRows);
                sm->key0 = split * len;
                const int last_token = (sm->row0 + sm->rows - 1) >> p.group_log2;
                const int end = p.causal ? min(c.len, c.len - c.tokens + last_token + 1) : c.len;
                sm->keys = max(0, min(end - sm->key0, len));
                sm->splits = c.splits;
                sm->part_row = c.row0 + split;
                sm->q_tiles = sm->rows > kTileRows ? 2 : 1;
            } else {
                report(p.status, FD_ERR_DEVICE_BOUNDS);
            }
        }
    }
    if (warp == kScaleWarp && lane == 0) {
        init_barriers(false);
        sm->abort = 0;
        sm->redo = 0;
        sm->wide = 0;
        sm->v_ref = 1.f;
        sm->ref_log = 0.f;
    }
    if (warp == kLoadWarp + 1 && blockIdx.x == 0)
        check_tables(p);
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem = sm->tmem;
    const bool ok = sm->ok;
    const int q_tiles = sm->q_tiles;
    const bool two = q_tiles == 2;
    const int n = (sm->keys + kPrefillTile - 1) / kPrefillTile;
    // local steps of stream s: every tile (two row tiles) or every other one
    auto steps = [&](int s) { return two ? n : (n + 1 - s) / 2; };
    const uint32_t q_smem = smem_addr(smem), ring = q_smem + q_tiles * kBufBytes;
    uint8_t *ring_ptr = smem + q_tiles * kBufBytes;
    // Position pos of the stream (see Place) holds K of tile t, or V of tile t.
    auto at_pos = [&](int pos, bool &is_k) {
        is_k = pos == 0 || ((pos & 1) && pos < 2 * n - 1);
        return is_k ? (pos + 1) / 2 : pos == 2 * n - 1 ? n - 1 : (pos - 2) / 2;
    };

    // At most two passes over the item: the second with careful steps, when the
    // first left f16's range or met V scales far from its reference.  The whole CTA, at
    // the first one's end: whether the second follows.
    auto another_pass = [&] {
        tcgen05_fence_before();
        __syncthreads();
        if (!sm->redo || sm->abort)
            return false;
        if (warp == kLoadWarp && lane == 0)
            init_barriers(true);   // every phase of the first pass has completed
        __syncthreads();
        tcgen05_fence_after();
        return true;
    };
    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
        int pass = 0;
        do {
            if (warp == kScaleWarp && n > 0) {
                // ------------------------------------------------ the tiles' scales
                // lanes 0-7 the groups' K scales, 8-15 their V scales
                GroupPages pages(p, sm->key0, sm->keys, sm->base);
                auto scale_of = [&](const GroupPages::Spot &x) {
                    const float *from = (lane < 8 ? p.k_scale : p.v_scale) + sm->kvh;
                    return lane < 16 && x.off >= 0 ? __ldcg(from + (int64_t)pages.page_of(x) * p.scale_heads)
                                                   : kSmallestScale;
                };
                const bool wide = pass > 0 && sm->wide;
                float scale = scale_of(pages.next()), ref_log = 0.f;
                GroupPages::Spot ahead = pages.next();
#pragma unroll 1
                for (int t = 0; t < n; ++t) {
                    if (t == 0) {
                        // pages of zeros have the smallest scale: no reference (1 where all have)
                        float m = lane >= 8 && scale > kSmallestScale && scale < INFINITY ? scale : 0.f;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1)
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        const float ref = m > 0.f ? m : 1.f;
                        ref_log = log2f(ref);
                        if (lane == 0) {
                            sm->v_ref = ref;
                            sm->ref_log = ref_log;
                        }
                    }
                    float lv = log2f(scale) - ref_log;
                    if (!wide) {
                        // far from the reference: in a second pass (its results do not count)
                        const bool zero = scale == kSmallestScale;
                        const bool out = lane >= 8 && !zero && scale >= 0.f && scale < INFINITY &&
                                         !(lv >= kLeastV && lv <= kMostV);
                        if (out)
                            sm->redo = sm->wide = 1;
                        lv = zero ? fmaxf(lv, kZeroV) : fminf(fmaxf(lv, kLeastV), kMostV);
                    }
                    if (!(scale >= 0.f && scale < INFINITY))
                        lv = __int_as_float(0x7fffffff);
                    const float v = __shfl_sync(0xffffffffu, lv, (lane & 7) + 8);
                    if (t >= kScaleSlots &&
                        !__all_sync(0xffffffffu, wait_phase(&sm->scales_free[t % kScaleSlots],
                                                            (t / kScaleSlots - 1) & 1, p, sm)))
                        break;
                    // (no number, an infinity or below 0, which would take -inf or the least
                    // score for the largest: what sees the group is NaN by its weights; what
                    // does not see it adds 0 times a number)
                    const float k = scale >= 0.f && scale < INFINITY ? scale : __int_as_float(0x7fffffff);
                    if (lane < 8)
                        sm->scale[t % kScaleSlots][lane] = make_float4(k, v, v == v ? exp2f(-v) : 1.f, 0.f);
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&sm->scales_ready[t % kScaleSlots]));
                    scale = scale_of(ahead);
                    ahead = pages.next();
                }
            }
            if (warp != kMmaWarp || n == 0)
                continue;
            // ------------------------------------------------------ the products
            // A wait that gave up is reported; the products then work on what there
            // is, so that no branch depends on it.
            constexpr uint32_t id_s = mma_idesc(128, kPrefillTile, false, false);
            constexpr uint32_t id_o = mma_idesc(128, kHeadDim, false, true);
            const uint32_t leader = elect_one();
            const int steps0 = steps(0), steps1 = steps(1);
            const uint32_t q_lo = smem_desc_lo(q_smem, 16);
            const uint32_t k_lo = smem_desc_lo(ring, 16);
            const uint32_t v_lo = smem_desc_lo(ring, kHalfBytes);
            constexpr uint32_t hi = smem_desc_hi(1024);
            constexpr uint32_t kBuf16 = kBufBytes / 16;
            Place k_at(0, kRing), v_at(n > 1 ? 2 : 1, kRing);
            int k_tile = 0, v_tile = 0;
            wait_phase(&sm->q_ready, 0, p, sm);
            // S of stream s's next step: K of its tile; frees the buffer after the
            // last stream that takes it.
            auto scores = [&](int s) {
                wait_phase(&sm->full[k_at.slot], k_at.phase, p, sm);
                tcgen05_fence_after();
                const uint32_t qa = q_lo + (two ? s : 0) * kBuf16, ka = k_lo + k_at.slot * kBuf16;
#pragma unroll
                for (int k = 0; k < 8; ++k) {   // 16 head dimensions a step
                    const uint32_t off = ((k >> 2) * kHalfBytes + (k & 3) * 32) / 16;
                    mma_ss(tmem + s * kStreamCols, qa + off, hi, ka + off, hi, id_s, k > 0, leader);
                }
                tcgen05_commit(smem_addr(&sm->s_full[s]), leader);
                if (!two || s == 1) {
                    tcgen05_commit(smem_addr(&sm->empty[k_at.slot]), leader);
                    k_at.advance(k_tile == 0 ? 1 : 2);
                    ++k_tile;
                }
            };
            // O += P V of stream s's step i, as each half of the weights is ready.
            auto values = [&](int s, int i, bool last) {
                wait_phase(&sm->full[v_at.slot], v_at.phase, p, sm);
                const uint32_t pa = tmem + s * kStreamCols, va = v_lo + v_at.slot * kBuf16;
#pragma unroll
                for (int k = 0; k < 8; ++k) {   // 16 keys a step
                    if (k % 4 == 0) {
                        wait_phase(&sm->p_ready[s][k / 4], i & 1, p, sm);
                        tcgen05_fence_after();
                    }
                    mma_ts(pa + 128, pa + 8 * k, va + k * 2 * 1024 / 16, hi, id_o, i > 0 || k > 0, leader);
                }
                if (!two || s == 1) {
                    tcgen05_commit(smem_addr(&sm->empty[v_at.slot]), leader);
                    v_at.advance(v_tile == n - 2 ? 1 : 2);
                    ++v_tile;
                }
                if (last)
                    tcgen05_commit(smem_addr(&sm->o_done[s]), leader);
            };
            // One copy of each for both streams: with two the roles' loops waited for
            // instructions (a prompt of 32768 tokens 5930 us for 5880).
#pragma unroll 1
            for (int i = -1; i < steps0; ++i)
#pragma unroll 1
                for (int s = 0; s < 2; ++s) {
                    const int last = (s == 0 ? steps0 : steps1) - 1;
                    if (i >= 0 && i <= last)
                        values(s, i, i == last);
                    if (i < last)
                        scores(s);
                }
            // whatever the others saw, the products in flight end before tensor
            // memory is freed
            tcgen05_commit(smem_addr(&sm->drain), leader);
            mbar_wait(smem_addr(&sm->drain), 0, kDrainTimeoutNs);
            __syncwarp();
        } while (pass++ == 0 && another_pass());
    } else if (warp >= kLoadWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
        int pass = 0;
        do {
            if (n == 0)
                continue;
            // --------------------------------------- codes to f16 operand tiles
            // A warp has two 16-key groups of each tile; its unit of work is 8 rows of one
            // half of the head, 16 values a lane: the lanes of a quarter warp are two rows
            // r and r ^ 5 and four chunks of 16 bytes, whose 32 bytes of f16 meet no bank
            // twice.  (A unit of each of the eight groups, eight page rows to ask the other
            // lanes for: 443 us of 438 for 8192 queries and keys of 32 heads.)  The codes
            // come by 16-byte asynchronous copies, two or four tiles ahead, each to a place
            // of its lane's own: a lane waits for its own copies alone.  (Loads into
            // registers a tile ahead: 2.9 us a tile of one row tile; their latency showed.)
            const int me = warp - kLoadWarp;
            const int r8 = (lane >> 3) ^ (((lane >> 2) & 1) * 5), cc = lane & 3;
            const uint32_t lane_dst = me * 4096 + r8 * 128 + (((2 * cc) ^ r8) << 4);
            const int64_t row_bytes = (int64_t)p.num_kv_heads * kHeadDim;
            const int lane_off = sm->kvh * kHeadDim + cc * 16;
            // The lane's group (lane % 8) of a tile: its page id a tile ahead.
            GroupPages pages(p, sm->key0, sm->keys, sm->base);
            GroupPages::Spot here = pages.next();
            int row_k = 0, row_v = 0;   // pool rows of the lane's group: newest K tile, the one before
            const uint32_t raw = ring + kRing * kBufBytes + me * (kRawBytes / kLoadWarps) + lane * 16;
            uint8_t *raw_ptr = ring_ptr + kRing * kBufBytes + me * (kRawBytes / kLoadWarps) + lane * 16;
            auto issue = [&](int pos, int place) {
                bool is_k;
                const int t = at_pos(pos, is_k);
                if (is_k) {
                    row_v = row_k;
                    row_k = pages.page_of(here) * p.page_size + max(here.off, 0);
                    here = pages.next();
                }
                const int8_t *from = (is_k ? p.k : p.v) + lane_off;
                const int row = is_k || t == n - 1 ? row_k : row_v;   // (K of tile t + 1 has gone before V of t)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int rows_of = __shfl_sync(0xffffffffu, row, 2 * me + g);
                    const int8_t *at = from + (int64_t)(rows_of + r8) * row_bytes;
#pragma unroll
                    for (int j = 0; j < 4; ++j)   // rows 8 (j / 2) of the group, half j % 2
                        cp_async_16(raw + place * kRawBytes + (4 * g + j) * 512,
                                    at + (j >> 1) * 8 * row_bytes + (j & 1) * 64);
                }
            };
            // `Ahead` tiles of codes on their way: two beside two Q tiles, else four.  (Three
            // operand tiles and four of codes made the products wait for each V tile.)
            auto stream = [&](auto ahead) {
                constexpr int kAhead = decltype(ahead)::value;
                Place to(0, kRing);
                for (int pos = 0; pos < kAhead; ++pos) {
                    if (pos < 2 * n)
                        issue(pos, pos);
                    cp_async_commit();
                }
#pragma unroll 1
                for (int pos = 0; pos < 2 * n; ++pos) {
                    cp_async_wait_group<kAhead - 1>();
                    bool go = true;
                    if (pos >= kRing)
                        go = wait_phase(&sm->empty[to.slot], to.phase ^ 1, p, sm);
                    if (!__all_sync(0xffffffffu, go))
                        break;
                    const uint8_t *src = raw_ptr + (pos % kAhead) * kRawBytes;
                    uint8_t *dst0 = ring_ptr + to.slot * kBufBytes + lane_dst;
                    uint8_t *dst1 = ring_ptr + to.slot * kBufBytes + (lane_dst ^ 16);
#pragma unroll
                    for (int h = 0; h < 8; h += 4) {   // the units of a group
                        uint4 x[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[j] = *reinterpret_cast<const uint4 *>(src + (h + j) * 512);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                            const int unit = h / 4 * 2048 + (j >> 1) * 1024 + (j & 1) * kHalfBytes;
                            uint32_t f[8];
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                int8x4_to_f16x2x2<0, 1, 2, 3>(w[q], f[2 * q], f[2 * q + 1]);
                            *reinterpret_cast<uint4 *>(dst0 + unit) = make_uint4(f[0], f[1], f[2], f[3]);
                            *reinterpret_cast<uint4 *>(dst1 + unit) = make_uint4(f[4], f[5], f[6], f[7]);
                        }
                    }
                    // the place's codes have gone into the operand tile
                    if (pos + kAhead < 2 * n)
                        issue(pos + kAhead, pos % kAhead);
                    cp_async_commit();
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&sm->full[to.slot]));
                    to.advance(1);
                }
                cp_async_wait_group<0>();
            };
            if (two)
                stream(std::integral_constant<int, 2>{});
            else
                stream(std::integral_constant<int, 4>{});
        } while (pass++ == 0 && another_pass());
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // -------------------------------------------------------- the softmax
        const int s = warp >> 2, quad = warp & 3;
        const int trow = quad * 32 + lane;   // row of the stream's tile: lane of tensor memory
        const uint32_t s_col = tmem + ((uint32_t)quad << 21) + s * kStreamCols, o_col = s_col + 128;
        if (ok) {
            // Q rows as f16 into shared memory, a tile [half][128 rows][128 bytes]; a
            // negative factor of the scores turns q around.  Each row times the
            // power of two that puts its largest magnitude in [2^8, 2^9): exact down
            // to 2^-22 of it.
            const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
            // a thread: chunk tid % 16 of every 16th row, all its loads in flight at once
            // (four at a time, with divisions by the group: 12 us)
            constexpr int kRowsOnce = kSoftmaxThreads / 16, kOfTile = kTileRows / kRowsOnce;
            const int ch = tid & 15;
            uint4 v[2][kOfTile];
#pragma unroll
            for (int k = 0; k < 2 * kOfTile; ++k) {
                const int r = k * kRowsOnce + (tid >> 4), gr = sm->row0 + r;
                v[k / kOfTile][k % kOfTile] = make_uint4(0u, 0u, 0u, 0u);
                if (r < sm->rows) {
                    const uint16_t *from = p.q + (sm->q0 + (gr >> p.group_log2)) * p.q_stride +
                                           ((sm->kvh << p.group_log2) + (gr & (p.group - 1))) * kHeadDim;
                    v[k / kOfTile][k % kOfTile] = __ldcg(reinterpret_cast<const uint4 *>(from) + ch);
                }
            }
            auto to_tile = [&](uint4 (&x)[kOfTile], int tile) {
                uint32_t w[kOfTile][4], most[kOfTile];
#pragma unroll
                for (int k = 0; k < kOfTile; ++k) {
                    w[k][0] = x[k].x ^ flip;
                    w[k][1] = x[k].y ^ flip;
                    w[k][2] = x[k].z ^ flip;
                    w[k][3] = x[k].w ^ flip;
                    const uint32_t m = __vmaxu2(__vmaxu2(w[k][0] & 0x7fff7fffu, w[k][1] & 0x7fff7fffu),
                                                __vmaxu2(w[k][2] & 0x7fff7fffu, w[k][3] & 0x7fff7fffu));
                    most[k] = max(m << 16, m & 0xffff0000u);   // of the bits of magnitudes
                }
#pragma unroll
                for (int o = 1; o < 16; o <<= 1)
#pragma unroll
                    for (int k = 0; k < kOfTile; ++k)
                        most[k] = max(most[k], __shfl_xor_sync(0xffffffffu, most[k], o));
#pragma unroll
                for (int k = 0; k < kOfTile; ++k) {
                    const int rr = k * kRowsOnce + (tid >> 4);
                    const int sh = min(max(9 + 126 - (int)(most[k] >> 23), -119), 126);   // 2^-sh, too, is normal
                    const float up = __int_as_float((127 + sh) << 23);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 a = bf16x2_to_float2(w[k][j]);
                        w[k][j] = pack_f16x2(make_float2(a.x * up, a.y * up));
                    }
                    if (ch == 0)
                        sm->q_scale[tile * kTileRows + rr] = __int_as_float((127 - sh) << 23);
                    *reinterpret_cast<uint4 *>(smem + tile * kBufBytes + (ch >> 3) * kHalfBytes + rr * 128 +
                                               (((ch & 7) ^ (rr & 7)) << 4)) =
                        make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
                }
            };
            to_tile(v[0], 0);
            if (two)
                to_tile(v[1], 1);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
        if (lane == 0 && ok)
            mbar_arrive(smem_addr(&sm->q_ready));
        const int r_mine = (two ? s * kTileRows : 0) + trow;
        barrier(1, kSoftmaxThreads);   // q_scale is written
        // what a score of codes is multiplied by
        const float c2 = fabsf(p.scale) * kLog2e * (ok ? sm->q_scale[r_mine] : 0.f);
        // keys of the item that the row sees
        const int token = min((sm->row0 + r_mine) >> p.group_log2, sm->tokens - 1);
        const int sees = ok && p.causal ? min(sm->keys, sm->len - sm->tokens + token + 1 - sm->key0) : sm->keys;
        float ref, l;   // E, and the row's sum
        // What the sum counts from: E less the bias or, for V scales of any size, the row's
        // largest score.
        float top;
        bool go = ok;
        // All of the row's tiles; careful: a maximum of every step before its weights.
        auto all_steps = [&](auto careful_t) {
            constexpr bool careful = decltype(careful_t)::value;
            float most = -INFINITY, level = -INFINITY;   // what E follows: the largest, the tiles' level
            constexpr float bias = careful ? kCarefulBias : kBias;
            const bool wide = careful && sm->wide;
            ref = top = -INFINITY;
            l = 0.f;
            // E to the tiles' level, when it is far from there, and O with it.
            auto follow = [&](bool first) {
                const float to = careful ? most : fmaxf(level, most - kDeep);
                const bool far = to > ref + kRaise || to < ref - kLower;
                if (!__any_sync(0xffffffffu, far))
                    return;
                const float f = !far ? 1.f : ref == -INFINITY ? 0.f : ex2(ref - to);
                ref = far ? to : ref;
                if (!wide)
                    l *= f;
                if (first)
                    return;
                // the products up to the last step are done: s_full followed them
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t o[16];
                    tmem_ld16(o_col + 16 * c, o);
                    tmem_wait_ld();
                    settle(o);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                    tmem_st16(o_col + 16 * c, o);
                }
            };
            for (int i = 0; i < steps(s) && go; ++i) {
                const int t = two ? i : 2 * i + s;
                go = __all_sync(0xffffffffu,
                                wait_phase(&sm->s_full[s], i & 1, p, sm) &&
                                    wait_phase(&sm->scales_ready[t % kScaleSlots], (t / kScaleSlots) & 1, p, sm));
                if (!go)
                    break;
                const float4 *group = sm->scale[t % kScaleSlots];
                const int valid = sees - t * kPrefillTile;
                tcgen05_fence_after();
                float here_top = -INFINITY;
                if (i == 0 || careful) {   // E from this tile's own scores
                    const bool all = __all_sync(0xffffffffu, valid >= kPrefillTile);
#pragma unroll 1
                    for (int c0 = 0; c0 < kGroups; c0 += 4) {
                        uint32_t x[64];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            tmem_ld16(s_col + 16 * (c0 + c), x + 16 * c);
                        tmem_wait_ld();
                        settle(x);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            float mt = -INFINITY;
                            if (all) {
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    mt = fmaxf(mt, __uint_as_float(x[16 * c + j]));
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    mt = fmaxf(mt, 16 * (c0 + c) + j < valid ? __uint_as_float(x[16 * c + j]) : -INFINITY);
                            }
                            const float4 g = group[c0 + c];
                            most = fmaxf(most, fmaf(mt, c2 * g.x, g.y));
                            here_top = fmaxf(here_top, mt * (c2 * g.x));
                        }
                    }
                }
                if (wide && here_top > top) {
                    l *= ex2(top - here_top);
                    top = here_top;
                }
                follow(i == 0);
                const float base = bias - (ref == -INFINITY ? 0.f : ref);
                float sum_tile = 0.f;
                auto publish = [&](int part) {
                    tmem_wait_st();
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&sm->p_ready[s][part]));
                };
                if (careful && wide) {
                    // 16 scores at a time, rarely run and short: two exponentials each, over E and
                    // over `top`
                    const float from = top == -INFINITY ? 0.f : top;
#pragma unroll 1
                    for (int c = 0; c < kGroups; ++c) {
                        const float4 g = group[c];
                        uint32_t x[16];
                        tmem_ld16(s_col + 16 * c, x);
                        tmem_wait_ld();
                        settle(x);
                        const float less = g.y == g.y ? from : g.y;   // (no number: neither is the sum)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            l += 16 * c + j < valid ? ex2(fmaf(__uint_as_float(x[j]), c2 * g.x, -less)) : 0.f;
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            float e[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                e[k] = fmaf(__uint_as_float(x[j + k]), c2 * g.x, g.y + base);
                                e[k] = 16 * c + j + k < valid ? ex2(e[k]) : 0.f;
                            }
                            x[j / 2] = pack_f16x2(make_float2(e[0], e[1]));
                        }
                        tmem_st8(s_col + 8 * c, x);   // (over the first half of the scores, as below)
                        if (c == 3)
                            publish(0);
                    }
                } else {
                    uint32_t r[kPrefillTile];   // the row's scores, then its weights
#pragma unroll
                    for (int c = 0; c < kGroups; ++c)
                        tmem_ld16(s_col + 16 * c, r + 16 * c);
                    tmem_wait_ld();
                    settle(r);
                    // 16 scores to weights; the weights of 16 keys are 8 columns, over those of
                    // the first half of the scores
                    auto weights = [&](int c, auto cut) {
                        const float4 g = group[c];
                        const float2 f = make_float2(c2 * g.x, c2 * g.x), off = make_float2(g.y + base, g.y + base);
                        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int at = 16 * c + 2 * j;
                            float2 x = fma2(make_float2(__uint_as_float(r[at]), __uint_as_float(r[at + 1])), f, off);
                            if constexpr (decltype(cut)::value) {
                                x.x = at < valid ? x.x : -INFINITY;
                                x.y = at + 1 < valid ? x.y : -INFINITY;
                            }
                            const float2 e = make_float2(ex2(x.x), ex2(x.y));
                            sum = add2(sum, e);
                            r[8 * c + j] = pack_f16x2(e);
                        }
                        const float part = sum.x + sum.y;
                        sum_tile += part;
                        l = fmaf(part, g.z, l);
                    };
                    auto tile = [&](auto cut) {
#pragma unroll
                        for (int c = 0; c < kGroups; c += 2) {
                            weights(c, cut);
                            weights(c + 1, cut);
                            tmem_st16(s_col + 8 * c, r + 8 * c);
                            if (c == 2)
                                publish(0);
                        }
                    };
                    // (compares and selects for each score of every tile took 13 % of a prompt)
                    if (__any_sync(0xffffffffu, valid < kPrefillTile))
                        tile(std::true_type{});
                    else
                        tile(std::false_type{});
                }
                publish(1);
                if (lane == 0 || (lane == 1 && !two))
                    mbar_arrive(smem_addr(&sm->scales_free[t % kScaleSlots]));
                if constexpr (!careful) {
                    const float here = __log2f(sum_tile) - base;
                    level = fmaxf(here, level - kFade - fminf(fmaxf(level - here - kGap, 0.f), kFall));
                    most = fmaxf(most, here);
                }
            }
            if (!wide)
                top = ref - bias;
            // both streams' products are done with the ring
            for (int x = 0; x < 2; ++x)
                if (go && steps(x) > 0)
                    go = __all_sync(0xffffffffu, wait_phase(&sm->o_done[x], 0, p, sm));
            tcgen05_fence_after();
        };
        all_steps(std::false_type{});
        if (go && steps(s) > 0) {   // a weight over f16's range
            uint32_t o[16];
            tmem_ld16(o_col, o);
            tmem_wait_ld();
            settle(o);
            if (!(fabsf(__uint_as_float(o[0])) < INFINITY))
                sm->redo = 1;
        }
        if (another_pass()) {
            if (lane == 0 && ok)
                mbar_arrive(smem_addr(&sm->q_ready));
            all_steps(std::true_type{});
        } else if (sm->redo) {
            go = false;
        }
        // ------------------------------------------------------- the output
        barrier(1, kSoftmaxThreads);   // in place of the ring
        float *stage = reinterpret_cast<float *>(smem);   // [q_tiles * 128][kOutStride]
        PrefillEnd *end = reinterpret_cast<PrefillEnd *>(smem + kEndOffset);
        float *mine = stage + r_mine * kOutStride;
        if (!two && s == 1 && go) {
            // one row tile: stream 1 hands its state to stream 0
            end->row_sum[trow] = l;
            end->row_ref[trow] = ref;
            end->row_top[trow] = top;
            if (steps(1) > 0) {
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t o[16];
                    tmem_ld16(o_col + 16 * c, o);
                    tmem_wait_ld();
                    settle(o);
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<uint4 *>(mine + 16 * c + j) =
                            make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
            }
        }
        if (!two)
            barrier(1, kSoftmaxThreads);
        if (go && (two || s == 0)) {
            float f0 = 1.f, f1 = 0.f, m = ref, den = l;
            const bool join = !two && steps(1) > 0;
            if (join) {
                const float m1 = end->row_ref[trow], top1 = end->row_top[trow], my_top = top;
                m = fmaxf(ref, m1);
                top = fmaxf(my_top, top1);
                f0 = ref == -INFINITY ? 0.f : ex2(ref - m);
                f1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
                den = l * (my_top == -INFINITY ? 0.f : ex2(my_top - top)) +
                      end->row_sum[trow] * (top1 == -INFINITY ? 0.f : ex2(top1 - top));
            }
            // a row that sees no key: O = 0, LSE = -inf
            const float inv = den == 0.f ? 0.f : 1.f / den;
            // O = (O over E) 2^(E - bias - top) v_ref / den, the powers in two halves
            // where these are numbers of any size
            float up = inv, last = sm->v_ref;
            if (sm->wide) {
                last = ex2(0.5f * (m - kCarefulBias - top + sm->ref_log));
                up *= last;
            }
            f0 *= up;
            f1 *= up;
            // The warp's 32 rows through shared memory, so that whole rows are written
            // (by its threads, a row each: 4 us of the store unit).
            const int first = r_mine - lane;
            const bool partial = sm->splits > 1;
            uint8_t *rows = smem + (two ? 0 : kStageOffset) + first * kRowStage;
            auto row_of = [&](int r) {   // of the request's rows [token][head]
                const int gr = sm->row0 + r;
                return (int64_t)(gr >> p.group_log2) * p.num_qo_heads + (sm->kvh << p.group_log2) +
                       (gr & (p.group - 1));
            };
#pragma unroll 2
            for (int c = 0; c < 8; ++c) {
                uint32_t o[16];
                float v[16];
                if (n > 0) {
                    tmem_ld16(o_col + 16 * c, o);
                    tmem_wait_ld();
                    settle(o);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] = inv == 0.f ? 0.f : __uint_as_float(o[j]) * f0;
                if (join && inv != 0.f) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[j] = fmaf(mine[16 * c + j], f1, v[j]);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] *= last;
                if (partial) {
                    float4 *to = reinterpret_cast<float4 *>(rows + lane * kRowStage) + 4 * c;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        to[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                } else {
                    uint4 *to = reinterpret_cast<uint4 *>(rows + lane * kRowStage) + 2 * c;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        to[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]),
                                           pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                                           pack_bf16x2(v[8 * j + 4], v[8 * j + 5]),
                                           pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
                }
            }
            if (r_mine < sm->rows) {
                const float lse = den == 0.f ? -INFINITY : (top + log2f(den)) * kLn2;
                if (partial)
                    p.partial_lse[sm->part_row + row_of(r_mine) * sm->splits] = lse;
                else if (p.lse)
                    p.lse[(int64_t)sm->q0 * p.num_qo_heads + row_of(r_mine)] = lse;
            }
            __syncwarp();
            const int count = min(sm->rows - first, 32);
            if (partial) {
#pragma unroll 4
                for (int r = 0; r < count; ++r)
                    reinterpret_cast<uint4 *>(p.partial_o + (sm->part_row + row_of(first + r) * sm->splits) *
                                                                kHeadDim)[lane] =
                        reinterpret_cast<const uint4 *>(rows + r * kRowStage)[lane];
            } else {   // two rows at once
#pragma unroll 4
                for (int r = lane >> 4; r < count; r += 2)
                    reinterpret_cast<uint4 *>(p.o + ((int64_t)sm->q0 * p.num_qo_heads + row_of(first + r)) *
                                                        kHeadDim)[lane & 15] =
                        reinterpret_cast<const uint4 *>(rows + r * kRowStage)[lane & 15];
            }
        }
    }
    tcgen05_fence_before();
    __syncthreads();   // the output has been read from tensor memory
    griddep_launch_dependents();
    if (warp == kMmaWarp) {
        tcgen05_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Stage 2, a warp a row: the merge by LSE of the partials of the requests with
// several splits, lane = 4 output columns, kMergeBatch partials of loads in flight.
constexpr int kMergeWarps = 4;
constexpr int kMergeBatch = 8;

__global__ void __launch_bounds__(kMergeWarps * 32) prefill_merge_kernel(const __grid_constant__ PrefillParams p)
{
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    griddep_wait();
    griddep_launch_dependents();
    if (row >= p.merge_rows)
        return;
    RequestCoord c;
    if (!locate_request(p, row, true, c)) {
        if (lane == 0)
            report(p.status, FD_ERR_DEVICE_BOUNDS);
        return;
    }
    const int64_t first = c.row0 + (int64_t)(row - c.merge0) * c.splits;
    const int64_t out = (int64_t)c.q0 * p.num_qo_heads + (row - c.merge0);
    const float *lse_in = p.partial_lse + first;
    const float4 *o_in = reinterpret_cast<const float4 *>(p.partial_o + first * kHeadDim) + lane;
    float m = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < c.splits; i0 += kMergeBatch) {
        float l[kMergeBatch];
        float4 v[kMergeBatch];
#pragma unroll
        for (int u = 0; u < kMergeBatch; ++u) {
            l[u] = -INFINITY;
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + u < c.splits) {
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
            if (w == 0.f)   // a split without a key that the row sees
                continue;
            den += w;
            acc.x = fmaf(w, v[u].x, acc.x);
            acc.y = fmaf(w, v[u].y, acc.y);
            acc.z = fmaf(w, v[u].z, acc.z);
            acc.w = fmaf(w, v[u].w, acc.w);
        }
        m = m_new;
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    reinterpret_cast<uint2 *>(p.o + out * kHeadDim)[lane] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && p.lse)
        p.lse[out] = den == 0.f ? -INFINITY : m + logf(den);
}

}  // namespace

cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t stream)
{
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrefillAlloc);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            configured[dev] = true;
    }
    e = launch_dependent(prefill_kernel, dim3((unsigned)p.num_items), kThreads, kPrefillAlloc, stream, p);
    if (e != cudaSuccess || p.merge_rows == 0)
        return e;
    return launch_dependent(prefill_merge_kernel, dim3((unsigned)((p.merge_rows + kMergeWarps - 1) / kMergeWarps)),
                            kMergeWarps * 32, 0, stream, p);
}

}  // namespace fd
