// pages_kernel.cu -- copying, forking, freeing and compacting the pages of a
// paged cache, on the device's own page tables and reference counts.
//
// All table arithmetic is on whole numbers and its results do not depend on
// the order of the threads: a fresh page is the free page of a given rank, a
// rank is a count of what comes before (counts per block of pages, then a scan
// in the block), and reference counts are only added to.
//
// Bound: the copies move each page once in and once out (HBM); the table
// kernels read and write a few words per page and table entry, so their time
// is that of short dependent launches, two for a fork and two or three for a
// compaction: 6.6-8.1 and 5.5-7.5 us a call up to 65536 pages and 51200 entries.  A
// fork in three launches, with the fresh pages listed by one of its own, took 7.4-7.9
// us (for 6.7-7.9 then) and 1.9 us more of the host; one launch of an 8-CTA cluster with its barrier
// between the steps 7.5-10 us at 1000-4096 pages, 22-28 us at 65536.
#include <cuda_runtime.h>

#include "api_util.h"
#include "cache_kernels.h"
#include "device_common.cuh"

namespace fd {
namespace {

// Words of PagesScratch::info.
enum Info { kFail, kNeeded, kInfoWords };

constexpr int kScanThreads = kPagesPerBlock / 4;
constexpr int kBlockWords = kPagesPerBlock / 32;
static_assert(kBlockWords == 32, "a block's bits are a word of each lane");
static_assert(kScanThreads % 32 == 0, "whole warps");

constexpr int kChildThreads = 1024;
constexpr int kTableThreads = 256;
constexpr int kCopyThreads = 256;

// Exclusive prefix sum of one value per thread over the CTA; `total` gets the
// sum.  `scratch`: one int per warp and one more, free after the call returns
// to all threads.
__device__ __forceinline__ int cta_exclusive_scan(int v, int *scratch, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += t;
    }
    __syncthreads();
    if (lane == 31)
        scratch[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int w = lane < warps ? scratch[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o)
                w += t;
        }
        scratch[lane] = w;   // inclusive over the warps
    }
    __syncthreads();
    total = scratch[warps - 1];
    return incl - v + (warp ? scratch[warp - 1] : 0);
}

// Sum over the CTA of one value per thread.
__device__ __forceinline__ int cta_sum(int v, int *scratch)
{
    int total;
    cta_exclusive_scan(v, scratch, total);
    return total;
}

// The four reference counts of this thread's pages in block `blk` (pages past
// the end count as in use, -1).
__device__ __forceinline__ int4 load_refs(const int32_t *refs, int num_pages, int blk)
{
    const int i = blk * kPagesPerBlock + 4 * (int)threadIdx.x;
    int4 r = make_int4(-1, -1, -1, -1);
    if (i + 3 < num_pages) {
        r.x = refs[i], r.y = refs[i + 1], r.z = refs[i + 2], r.w = refs[i + 3];
    } else {
        if (i < num_pages) r.x = refs[i];
        if (i + 1 < num_pages) r.y = refs[i + 1];
        if (i + 2 < num_pages) r.z = refs[i + 2];
    }
    return r;
}

// ------------------------------------------------------------------- copies

// One CTA copies one segment of one page of one pool, 16 bytes a thread and
// load, all of a thread's loads in flight before its first store.  488 pages of 8
// pools of 32 KB: 6.4 TB/s, 95 % of a plain copy.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyPagesParams p)
{
    constexpr int kLoads = kCopySegment / 16 / kCopyThreads;
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x / p.segments, seg = blockIdx.x - c * p.segments;
    // plain loads: the grid before may have written these while this one already ran
    const int src = p.src[c], dst = p.dst[c];
    if (src < 0)
        return;
    if (src >= p.num_pages || dst < 0 || dst >= p.num_pages) {
        if (p.status && threadIdx.x == 0)
            report(p.status, FD_ERR_DEVICE_BOUNDS);
        return;
    }
    const int64_t bytes = p.page_bytes[blockIdx.y];
    const int64_t at = (int64_t)seg * kCopySegment;
    if (at >= bytes || src == dst)
        return;
    const int n = (int)(min(bytes - at, (int64_t)kCopySegment) / 16);
    const uint4 *s = reinterpret_cast<const uint4 *>(p.pool[blockIdx.y] + src * bytes + at);
    uint4 *d = reinterpret_cast<uint4 *>(p.pool[blockIdx.y] + dst * bytes + at);
    uint4 v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int j = (int)threadIdx.x + i * kCopyThreads;
        if (j < n)
            v[i] = s[j];
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int j = (int)threadIdx.x + i * kCopyThreads;
        if (j < n)
            d[j] = v[i];
    }
}

// --------------------------------------------------------------------- fork

// What child i takes from its parent; ok = false: outside the tables.
struct Child {
    int have, next, last, tail;   // parent's pages, own pages, keys of the last page, its id (-1: none)
    bool ok;
};

__device__ __forceinline__ Child read_child(const ForkParams &p, int i)
{
    Child c{0, 0, 0, -1, true};
    const int par = p.parent[i], a = p.new_indptr[i], e = p.new_indptr[i + 1];
    c.next = e - a;
    c.ok = par >= -1 && par < p.old_batch && a >= 0 && e >= a && e <= p.new_entries;
    if (c.ok && par >= 0) {
        const int b = p.page_indptr[par], f = p.page_indptr[par + 1];
        c.have = f - b;
        c.ok = b >= 0 && f >= b && f <= p.old_entries && c.have <= c.next;
        if (c.ok && c.have > 0) {
            c.last = p.last_len[par];
            c.tail = p.indices[f - 1];
            c.ok = c.last >= 1 && c.last <= p.page_size && c.tail >= 0 && c.tail < p.num_pages;
        }
    }
    return c;
}

// Launch 1.  CTA 0: every child's fresh pages and their first rank, whether
// its last page is a copy.  CTAs 1..: free pages of each block, refs_out =
// refs_in, and -1 in the entries that are no child's (in front of the first table
// and behind the last; here, as these CTAs end long before CTA 0: 0.3 us more of a
// fork in the next launch).
__global__ void __launch_bounds__(kChildThreads) fork_count_kernel(const __grid_constant__ ForkParams p)
{
    extern __shared__ int s_first[];   // [old_batch] lowest child of each request (CTA 0)
    __shared__ int s_scan[33];
    __shared__ int s_fail;
    const int tid = threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x > 0) {
        const int blk = blockIdx.x - 1;
        const int used0 = p.new_batch > 0 ? p.new_indptr[0] : 0;
        const int used1 = p.new_batch > 0 ? max(p.new_indptr[p.new_batch], 0) : 0;   // in range if the call is
        int n = 0;
        if (tid < kScanThreads) {
            const int4 r = load_refs(p.refs_in, p.num_pages, blk);
            n = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
            const int i = blk * kPagesPerBlock + 4 * tid;
            if (i < p.num_pages) p.refs_out[i] = r.x;
            if (i + 1 < p.num_pages) p.refs_out[i + 1] = r.y;
            if (i + 2 < p.num_pages) p.refs_out[i + 2] = r.z;
            if (i + 3 < p.num_pages) p.refs_out[i + 3] = r.w;
            // which of the block's pages are free, a bit each: the next launch
            // looks for them while it changes the counts
            unsigned bits = (unsigned)((r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3)
                            << (4 * (tid & 7));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                bits |= __shfl_xor_sync(0xffffffffu, bits, o);
            if ((tid & 7) == 0)
                p.s.list[blk * kBlockWords + tid / 8] = (int)bits;
        }
        n = cta_sum(n, s_scan);
        if (tid == 0)
            p.s.block_count[blk] = n;
        const int64_t at = (int64_t)blk * kChildThreads + tid, step = (int64_t)p.blocks * kChildThreads;
        for (int64_t i = at; i < min(used0, p.new_entries); i += step)
            p.new_indices[i] = -1;
        for (int64_t i = used1 + at; i < p.new_entries; i += step)
            p.new_indices[i] = -1;
        return;
    }
    if (tid == 0)
        s_fail = 0;
    // Every old table is within its array, the ended requests' too: the next
    // launch, which takes their references away, starts only on tables that are.
    // (The first of a thread's tables is on its way while the parents are read.)
    const bool has_table = tid < p.old_batch;
    const int first_a = has_table ? p.page_indptr[tid] : 0, first_e = has_table ? p.page_indptr[tid + 1] : 0;
    auto inside = [&](int a, int e) { return a >= 0 && e >= a && e <= p.old_entries; };
    for (int i = tid; i < p.old_batch; i += kChildThreads)
        s_first[i] = p.new_batch;
    __syncthreads();
    bool torn = has_table && !inside(first_a, first_e);
    for (int i = tid + kChildThreads; i < p.old_batch; i += kChildThreads)
        torn |= !inside(p.page_indptr[i], p.page_indptr[i + 1]);
    if (torn)
        s_fail = 1;
    for (int i = tid; i < p.new_batch; i += kChildThreads) {
        const int par = p.parent[i];
        if (par >= 0 && par < p.old_batch)
            atomicMin(&s_first[par], i);
    }
    __syncthreads();
    int base = 0;
    for (int i0 = 0; i0 < p.new_batch; i0 += kChildThreads) {
        const int i = i0 + tid;
        int fresh = 0;
        if (i < p.new_batch) {
            const Child c = read_child(p, i);
            int copy = 0;
            if (!c.ok) {
                s_fail = 1;
            } else {
                // a partly filled last page goes on in the request's first
                // child, where no other request has it, and is copied for the rest
                if (c.have > 0 && c.last < p.page_size)
                    copy = !(s_first[p.parent[i]] == i && p.refs_in[c.tail] == 1);
                fresh = c.next - c.have + copy;
            }
            p.s.child_copy[i] = copy;
        }
        int total;
        const int at = cta_exclusive_scan(fresh, s_scan, total);
        if (i < p.new_batch)
            p.s.child_rank[i] = base + at;
        base += total;
    }
    __syncthreads();
    if (tid == 0) {
        p.s.info[kFail] = s_fail;
        p.s.info[kNeeded] = base;
    }
}

// Launch 2.  CTAs 0..new_batch-1 write a child's table, its copy and its
// references; the others take an old request's references away.  The fresh
// page of rank r is the r-th free one: a block's share from the blocks' counts,
// its place there from the bits, a word a lane.
__global__ void __launch_bounds__(kTableThreads) fork_table_kernel(const __grid_constant__ ForkParams p)
{
    __shared__ int s_scan[33];
    __shared__ int s_before[kTableThreads];   // free pages before each of 256 blocks
    const int tid = threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    int free_pages = 0, count = 0;
    for (int b0 = 0; b0 < p.blocks; b0 += kTableThreads) {
        int total;
        count = b0 + tid < p.blocks ? p.s.block_count[b0 + tid] : 0;
        s_before[tid] = free_pages + cta_exclusive_scan(count, s_scan, total);
        free_pages += total;
    }
    const bool outside = p.s.info[kFail] != 0;
    const bool fail = outside || p.s.info[kNeeded] > free_pages;   // nothing changes then
    if (fail) {
        if (blockIdx.x == 0) {
            if (tid == 0)
                report(p.status, outside ? FD_ERR_DEVICE_BOUNDS : FD_ERR_NO_PAGES);
            for (int i = tid; i < p.new_entries; i += kTableThreads)
                p.new_indices[i] = -1;
            for (int i = tid; i < p.new_batch; i += kTableThreads)
                p.copy_src[i] = p.copy_dst[i] = -1;
        }
        return;
    }
    if ((int)blockIdx.x >= p.new_batch) {
        const int b = blockIdx.x - p.new_batch;
        const int a = p.page_indptr[b], e = p.page_indptr[b + 1];   // within the array, or the call had failed
        for (int i = a + tid; i < e; i += kTableThreads) {
            const int page = p.indices[i];
            if (page >= 0 && page < p.num_pages)
                atomicSub(p.refs_out + page, 1);
            else
                report(p.status, FD_ERR_DEVICE_BOUNDS);
        }
        return;
    }
    const int i = blockIdx.x;
    const Child c = read_child(p, i);
    const int copy = p.s.child_copy[i], rank = p.s.child_rank[i], a = p.new_indptr[i];
    const int *old = c.have > 0 ? p.indices + p.page_indptr[p.parent[i]] : nullptr;
    const int kept = c.have - copy, fresh = c.next - kept;   // entries that are the parent's own, and not
    auto enter = [&](int j, int page) {
        if (page >= 0 && page < p.num_pages) {
            atomicAdd(p.refs_out + page, 1);
        } else {
            page = -1;
            report(p.status, FD_ERR_DEVICE_BOUNDS);
        }
        p.new_indices[a + j] = page;
    };
    for (int j = tid; j < kept; j += kTableThreads)
        enter(j, old[j]);
    if (tid == 0) {
        p.copy_src[i] = copy ? c.tail : -1;
        if (!copy)
            p.copy_dst[i] = -1;
    }
    if (fresh == 0)
        return;
    const int warp = tid >> 5, lane = tid & 31;
    int before = 0;
    for (int b0 = 0; b0 < p.blocks; b0 += kTableThreads) {
        if (p.blocks > kTableThreads) {   // else they are there
            int total;
            count = b0 + tid < p.blocks ? p.s.block_count[b0 + tid] : 0;
            __syncthreads();
            s_before[tid] = before + cta_exclusive_scan(count, s_scan, total);
            before += total;
        }
        __syncthreads();
        const int n = min(p.blocks - b0, kTableThreads);
        for (int b = warp; b < n; b += kTableThreads / 32) {
            const int first = s_before[b];
            if (first >= rank + fresh || first + kPagesPerBlock <= rank)
                continue;
            unsigned bits = (unsigned)p.s.list[(b0 + b) * kBlockWords + lane];
            int r = __popc(bits);
            const int mine = r;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, r, o);
                if (lane >= o)
                    r += t;
            }
            r += first - mine;   // rank of the lane's first free page
            if (r + mine <= rank || r >= rank + fresh)
                bits = 0;
            for (; bits; bits &= bits - 1, ++r) {
                if (r < rank || r >= rank + fresh)
                    continue;
                const int page = (b0 + b) * kPagesPerBlock + 32 * lane + __ffs(bits) - 1;
                enter(kept + r - rank, page);
                if (copy && r == rank)
                    p.copy_dst[i] = page;
            }
        }
    }
}

// ------------------------------------------------------------------ compact

// Up to so many blocks of pages every CTA of the next launch counts them all
// itself: 1000 pages 5.6 us for 6.4, 4096 7.1 for 7.2, 8192 would be 8.6 for 7.3.
constexpr int kFewBlocks = 4;

// Launch 1.  Pages in use in each block.
__global__ void __launch_bounds__(kScanThreads) compact_count_kernel(const __grid_constant__ CompactParams p)
{
    __shared__ int s_scan[33];
    griddep_wait();
    griddep_launch_dependents();
    const int4 r = load_refs(p.refs_in, p.num_pages, blockIdx.x);
    const int n = cta_sum((r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0), s_scan);
    if (threadIdx.x == 0)
        p.s.block_count[blockIdx.x] = n;
}

// How the call divides the pages: those in use at or behind `limit` move (in
// order) to the free ones before it (in order).
struct Division {
    int limit, below, moves, fail;   // below: pages in use before the limit
};

// All threads of a CTA; `before` gets the pages in use before block blk.
__device__ __forceinline__ Division divide_pages(const CompactParams &p, int blk, int *scratch, int &before)
{
    const bool few = p.blocks <= kFewBlocks;   // counted here, else by the launch before
    int all = 0, ahead = 0;
    if (few) {
        for (int i = 0; i < p.blocks; ++i) {
            const int4 r = load_refs(p.refs_in, p.num_pages, i);
            const int n = (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
            all += n;
            ahead += i < blk ? n : 0;
        }
    } else {
        for (int i = threadIdx.x; i < p.blocks; i += blockDim.x) {
            const int n = p.s.block_count[i];
            all += n;
            ahead += i < blk ? n : 0;
        }
    }
    before = cta_sum(ahead, scratch);
    const int live = cta_sum(all, scratch);
    Division d;
    d.limit = p.limit > 0 ? min(p.limit, p.num_pages) : live;
    const int lb = few ? 0 : d.limit / kPagesPerBlock;   // the limit's block
    int n = 0;
    for (int i = threadIdx.x; i < min(lb, p.blocks); i += blockDim.x)
        n += p.s.block_count[i];
    for (int i = lb * kPagesPerBlock + threadIdx.x; i < d.limit; i += blockDim.x)
        n += p.refs_in[i] > 0;
    d.below = cta_sum(n, scratch);
    d.moves = live - d.below;
    d.fail = d.moves > d.limit - d.below || d.moves > p.max_moves;
    return d;
}

// Launch 2.  Ranks: the r-th moving page goes to the r-th free page before the
// limit.  Counts of pages that stay are copied through; a moving page's and
// its place's are set by the next launch, so refs_out may be refs_in.
__global__ void __launch_bounds__(kScanThreads) compact_rank_kernel(const __grid_constant__ CompactParams p)
{
    __shared__ int s_scan[33];
    const int tid = threadIdx.x, blk = blockIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    int before;
    const Division d = divide_pages(p, blk, s_scan, before);
    if (blk == 0 && tid == 0) {
        p.s.info[kFail] = d.fail;
        p.s.info[kNeeded] = d.fail ? 0 : d.moves;
        if (d.fail)
            report(p.status, FD_ERR_NO_PAGES);
    }
    for (int i = blk * kScanThreads + tid; i < p.max_moves; i += p.blocks * kScanThreads)
        if (d.fail || i >= d.moves)
            p.copy_src[i] = p.copy_dst[i] = -1;
    const int4 r = load_refs(p.refs_in, p.num_pages, blk);
    const int v[4] = {r.x, r.y, r.z, r.w};
    int total;
    int rank = before + cta_exclusive_scan((v[0] > 0) + (v[1] > 0) + (v[2] > 0) + (v[3] > 0), s_scan, total);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int page = blk * kPagesPerBlock + 4 * tid + j;
        if (page >= p.num_pages)
            break;
        if (!d.fail && v[j] > 0 && page >= d.limit) {
            p.copy_src[rank - d.below] = page;
            p.s.list[page] = rank - d.below;
        } else {
            const int slot = page - rank;   // rank among the free pages
            if (!d.fail && v[j] <= 0 && page < d.limit && slot < d.moves)
                p.copy_dst[slot] = page;
            else
                p.refs_out[page] = v[j];
            p.s.list[page] = -1;
        }
        rank += v[j] > 0;
    }
}

// Launch 3.  The tables' entries, and the counts of the pages that move.
__global__ void __launch_bounds__(kTableThreads) compact_table_kernel(const __grid_constant__ CompactParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int i = blockIdx.x * kTableThreads + threadIdx.x;
    const int moves = p.s.info[kNeeded];
    if (i < moves) {
        const int src = p.copy_src[i], refs = p.refs_in[src];
        p.refs_out[p.copy_dst[i]] = refs;
        p.refs_out[src] = 0;
    }
    if (i < p.entries) {
        int page = p.indices[i];
        if (page < -1 || page >= p.num_pages) {   // -1: no page
            report(p.status, FD_ERR_DEVICE_BOUNDS);
        } else if (page >= 0) {
            const int rank = p.s.list[page];
            if (rank >= 0)
                page = p.copy_dst[rank];
        }
        p.new_indices[i] = page;
    }
}

}  // namespace

cudaError_t launch_copy_pages(const CopyPagesParams &p, int num_pools, cudaStream_t stream)
{
    return launch_dependent(copy_pages_kernel, dim3((unsigned)(p.num_copies * p.segments), (unsigned)num_pools),
                            kCopyThreads, 0, stream, p);
}

cudaError_t launch_fork(const ForkParams &p, cudaStream_t stream)
{
    const int smem = p.old_batch * (int)sizeof(int);
    cudaError_t e = cudaSuccess;
    // The limit is the kernel's, not the call's: always the most that a fork may
    // need, so that no call lowers it between another thread's setting and launch.
    if (smem > 40 * 1024)
        e = cudaFuncSetAttribute(fork_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMaxTableBatch * (int)sizeof(int));
    if (e == cudaSuccess)
        e = launch_dependent(fork_count_kernel, dim3((unsigned)(1 + p.blocks)), kChildThreads, smem, stream, p);
    if (e == cudaSuccess && p.new_batch + p.old_batch > 0)
        e = launch_dependent(fork_table_kernel, dim3((unsigned)(p.new_batch + p.old_batch)), kTableThreads, 0,
                             stream, p);
    return e;
}

cudaError_t launch_compact(const CompactParams &p, cudaStream_t stream)
{
    cudaError_t e = cudaSuccess;
    if (p.blocks > kFewBlocks)
        e = launch_dependent(compact_count_kernel, dim3((unsigned)p.blocks), kScanThreads, 0, stream, p);
    if (e == cudaSuccess)
        e = launch_dependent(compact_rank_kernel, dim3((unsigned)p.blocks), kScanThreads, 0, stream, p);
    const int n = p.entries > p.max_moves ? p.entries : p.max_moves;
    if (e == cudaSuccess && n > 0)
        e = launch_dependent(compact_table_kernel, dim3((unsigned)((n + kTableThreads - 1) / kTableThreads)),
                             kTableThreads, 0, stream, p);
    return e;
}

}  // namespace fd
