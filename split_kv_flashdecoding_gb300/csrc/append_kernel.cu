// append_kernel.cu -- rotary positions on new queries and keys, and the write
// of the new keys and values into a paged cache (bf16, FP8 E4M3, INT4 or INT8).
//
// Mathematics: pair i of a head's first rotary_dim values is turned by the
// angle position * f_i: (a, b) -> gain (a cos - b sin, b cos + a sin).  The
// angle is kept in turns as a 64-bit fixed-point fraction: step_i = f_i / 2 pi
// * 2^64, and position * step_i modulo 2^64 is the exact fraction of a turn of
// that step (the plan's rounding of f_i, 2^-53 of it, is all that a far
// position loses), so one integer product replaces a long range reduction.
// The fraction is rounded to fp32 for its sine and cosine (the angle by 2^-25 of a half
// turn, 9e-8, at most, as much as these are rounded by themselves).  The arithmetic is
// fp32; each output is rounded once.
//
// Bound: bytes of q (in and out), k, v and the cache rows.  A CTA takes one
// token (short calls, whose time is the chain token -> request -> page -> row)
// or several (long calls); the tokens' angles are computed once in shared
// memory for all of the token's heads.  A thread's unit is two 8-value chunks
// that hold both halves of 8 pairs, read and written 16 bytes at a time.
// Measured: 32768 tokens of 32 + 8 + 8 heads 126 us in bf16, 6.4 TB/s, 94 % of a
// plain copy's rate; 12345 tokens into FP8 51 us, 5.5 TB/s, of which some 8 us
// are the first CTAs' look-ups and the last ones' end; into INT4 58 us, 4.6 TB/s,
// with a division a code; 64 tokens 3.8 us, the chain.
//
// INT8 with a scale per page and KV head: the scale of a page needs the largest
// magnitude of all of its new keys, so a CTA takes the new keys of one page for its
// heads (append_int8_kernel below); the queries go as above, in CTAs of their own
// behind those of the same launch.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "api_util.h"
#include "cache_kernels.h"
#include "device_common.cuh"
#include "kernels.h"

namespace fd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;      // tokens of one CTA
constexpr int kUnits = kHeadDim / 16;   // two-chunk units of a head
constexpr int kHeadLanes = kThreads / kUnits;

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_to_float2(u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Four quotients as E4M3 bytes, round to nearest even, saturated to +-448.
__device__ __forceinline__ uint32_t pack4_fp8(float2 a, float2 b)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Bit 7 of each byte of w that is a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w)
{
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Four values over a scale as E4M3 bytes, the rounded quotients to nearest even,
// saturated (NaN stays NaN): the negative ones, as inv = -1 / mag keeps the signs of
// zeros.  The product x inv is up to two units off, which lands beside some of
// E4M3's ties (15 of the bf16 values over 0.03); one step of Newton's method on its
// exact remainder (Markstein's) mends it.  An infinite product has no remainder and
// becomes NaN.
__device__ __forceinline__ uint32_t pack4_over(const float *x, float mag, float inv)
{
    float2 y[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float2 v = make_float2(x[2 * j], x[2 * j + 1]), inv2 = make_float2(inv, inv);
        y[j] = mul2(v, inv2);
        y[j] = fma2(fma2(y[j], make_float2(mag, mag), v), inv2, y[j]);
    }
    return pack4_fp8(y[0], y[1]);
}

// Sixteen values over a scale as E4M3 bytes.
__device__ __forceinline__ void pack16_fp8(const float (&a)[8], const float (&b)[8], float scale, uint32_t (&u)[4])
{
    const float mag = fabsf(scale), inv = -1.f / mag;
    const uint32_t flip = scale < 0.f ? 0u : 0x80808080u;
    u[0] = pack4_over(a, mag, inv);
    u[1] = pack4_over(a + 4, mag, inv);
    u[2] = pack4_over(b, mag, inv);
    u[3] = pack4_over(b + 4, mag, inv);
    // Rare: infinite products (or NaN), or a scale whose products and remainders do
    // not stay well inside fp32's range.  Divisions; for all values they took 5 to 9 %
    // more of a call, this way 0 to 1.6 %.
    if ((nan_codes(u[0]) | nan_codes(u[1]) | nan_codes(u[2]) | nan_codes(u[3])) != 0 ||
        !(mag > 1e-15f && mag < 1e15f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float *x = i < 2 ? a + 4 * i : b + 4 * (i - 2);
            u[i] = pack4_fp8(make_float2(__fdiv_rn(x[0], -mag), __fdiv_rn(x[1], -mag)),
                             make_float2(__fdiv_rn(x[2], -mag), __fdiv_rn(x[3], -mag)));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] ^= flip;
}

// Eight values as four-bit codes round(x / scale) in -8..7, value j in nibble j.
__device__ __forceinline__ uint32_t pack8_int4(const float (&x)[8], float scale)
{
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = min(max(__float2int_rn(__fdiv_rn(x[i], scale)), -8), 7);
        w |= (uint32_t)(c & 0xF) << (4 * i);
    }
    return w;
}

// Where two pairs' (cos, sin) are in a token's row of 32 such: the lanes of a
// head read every 2nd (interleaved) or every 4th of them at once, here from
// different banks (32768 tokens: 131 us for 135 in order).
__device__ __forceinline__ int place(int x)
{
    return x ^ ((x >> 3) & 3);
}

// (a, b) turned by the angle of (c, s).
__device__ __forceinline__ void turn(float &a, float &b, float c, float s)
{
    const float x = a, y = b;
    a = x * c - y * s;
    b = y * c + x * s;
}

// A unit's two chunks turned, the first one's start below rotary_dim: `row` has the
// token's (cos, sin), of each chunk's 4 pairs or of the unit's 8.
__device__ __forceinline__ void turn_unit(float (&a)[8], float (&b)[8], const float2 *row, int c0, int c1,
                                          bool turns1, bool interleaved)
{
    const float4 *cs = reinterpret_cast<const float4 *>(row);
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 f = cs[place(c0 / 4 + j)];
            turn(a[4 * j], a[4 * j + 1], f.x, f.y);
            turn(a[4 * j + 2], a[4 * j + 3], f.z, f.w);
        }
        if (turns1) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 f = cs[place(c1 / 4 + j)];
                turn(b[4 * j], b[4 * j + 1], f.x, f.y);
                turn(b[4 * j + 2], b[4 * j + 3], f.z, f.w);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 f = cs[place(c0 / 2 + j)];
            turn(a[2 * j], b[2 * j], f.x, f.y);
            turn(a[2 * j + 1], b[2 * j + 1], f.z, f.w);
        }
    }
}

// (cos, sin) of pair j of a token at position pos, into its row of them.
__device__ __forceinline__ void put_angle(const fd_rope_info &rope, int pos, int j, float2 *row)
{
    const uint64_t turns = (uint64_t)(int64_t)pos * rope.step[j];
    float s, c;
    sincospif((float)(int64_t)turns * 1.0842021724855044e-19f, &s, &c);   // turns / 2^63: half turns
    row[2 * place(j >> 1) + (j & 1)] = make_float2(c * rope.gain, s * rope.gain);
}

// Where the two chunks of unit u of a head start: they run on over the 8 lanes; pairs
// of an interleaved layout lie within a chunk, those of the other one in the two
// chunks of a unit.
__device__ __forceinline__ void unit_chunks(const fd_rope_info &rope, int u, int &c0, int &c1)
{
    const int rot = rope.rotary_dim, rot_units = rot / 16;
    c0 = 8 * u, c1 = kHeadDim / 2 + 8 * u;
    if (!rope.interleaved) {
        c0 = u < rot_units ? 8 * u : rot + 8 * (u - rot_units);
        c1 = c0 + (u < rot_units ? rot : kHeadDim - rot) / 2;
    }
}

// The tokens of block `block`.  INT8: their queries alone.
template <int KVT>
__device__ __forceinline__ void append_tokens(const AppendParams &p, int block)
{
    __shared__ __align__(16) float2 s_cs[kMaxTokens][kHeadDim / 2];
    __shared__ int64_t s_row[kMaxTokens];    // cache row of the token, -1: none
    __shared__ int s_pos[kMaxTokens], s_ok[kMaxTokens], s_count[kMaxTokens];

    const int tid = threadIdx.x;
    const int t0 = block * p.tokens_per_cta;
    const int nt = min(p.tokens_per_cta, p.num_tokens - t0);
    if (tid < kMaxTokens)
        s_count[tid] = 0;
    // Thread (head lane, unit u): the same unit of every 32nd head of the CTA's
    // tokens, one after another, so that nothing is divided and all lanes are at
    // work.  The 8 lanes of a head stay together, which the INT4 scale's reduction
    // relies on.
    const int heads = p.num_qo_heads + (KVT == kKvTypeInt8 ? 0 : 2 * p.num_kv_heads);
    const int u = tid % kUnits, lane_head = tid / kUnits;
    const int rot = p.rope.rotary_dim;
    int c0, c1;
    unit_chunks(p.rope, u, c0, c1);
    const bool turns0 = c0 < rot, turns1 = c1 < rot;
    int tt = 0, head = lane_head;   // of the unit to load next
    auto settle = [&]() {           // into a token's heads
        while (head >= heads) {
            head -= heads;
            ++tt;
        }
    };
    settle();
    // Two units are loaded ahead of the one that is worked on, the first two while
    // the tables are looked up (one ahead: 32768 tokens 131 us, two 126, with four
    // CTAs an SM either way).
    struct Unit {
        int tt, head;
        uint4 a, b;
    };
    Unit u0, u1;
    auto load_unit = [&](Unit &x) {
        x.tt = tt;
        x.head = head;
        if (tt < nt) {
            const int kv = head - p.num_qo_heads;
            const int64_t t = t0 + tt;
            const uint16_t *src = kv < 0                ? p.q + t * p.q_stride + head * kHeadDim
                                  : kv < p.num_kv_heads ? p.k + t * p.k_stride + kv * kHeadDim
                                                        : p.v + t * p.v_stride + (kv - p.num_kv_heads) * kHeadDim;
            x.a = *reinterpret_cast<const uint4 *>(src + c0);
            x.b = *reinterpret_cast<const uint4 *>(src + c1);
        }
        head += kHeadLanes;
        settle();
    };
    // The grid before this one may write the tables, positions and scales (a fork, a
    // page copy) while this one already runs, so they are read by plain loads behind
    // the wait, here and below: __ldg is for what nobody writes meanwhile.  (Loads
    // past L1, __ldcg, took 1 to 3 % longer.)
    griddep_wait();
    griddep_launch_dependents();
    load_unit(u0);
    load_unit(u1);
    __syncthreads();

    // request of each token: how many of append_indptr[1..B] are at or below it
    {
        int cnt[kMaxTokens];
#pragma unroll
        for (int i = 0; i < kMaxTokens; ++i)
            cnt[i] = 0;
        for (int b = tid; b < p.batch; b += kThreads) {
            const int e = p.append_indptr[b + 1];
#pragma unroll
            for (int i = 0; i < kMaxTokens; ++i)
                cnt[i] += e <= t0 + i;
        }
#pragma unroll
        for (int i = 0; i < kMaxTokens; ++i) {
            if (i < nt) {
                const int c = __reduce_add_sync(0xffffffffu, cnt[i]);
                if ((tid & 31) == 0 && c)
                    atomicAdd(&s_count[i], c);
            }
        }
    }
    __syncthreads();
    if (tid < nt) {
        const int t = t0 + tid, b = s_count[tid];
        int64_t row = -1;
        int pos = 0, ok = 0;
        if (b < p.batch) {   // else: a padded row behind the last request, left as it is
            const int a0 = p.append_indptr[b], a1 = p.append_indptr[b + 1];
            const int e0 = p.kv_page_indptr[b], e1 = p.kv_page_indptr[b + 1];
            const int last = p.kv_last_page_len[b];
            if (p.positions)
                pos = p.positions[t];
            const int64_t len = (int64_t)(e1 - e0 - 1) * p.page_size + last;
            const int64_t key = len - (a1 - t);
            ok = t >= a0 && t < a1 && e0 >= 0 && e1 > e0 && e1 <= p.num_page_entries && last >= 1 &&
                 last <= p.page_size && key >= 0;
            if (ok) {
                const int page = p.kv_page_indices[e0 + (int)(key / p.page_size)];
                ok = page >= 0 && page < p.num_pages;
                row = (int64_t)page * p.page_size + key % p.page_size;
                if (!p.positions)
                    pos = (int)key;
            }
            if (!ok)
                report(p.status, FD_ERR_DEVICE_BOUNDS);
        }
        s_row[tid] = row;
        s_pos[tid] = pos;
        s_ok[tid] = ok;
    }
    __syncthreads();
    for (int i = tid; i < nt * (p.rope.rotary_dim / 2); i += kThreads) {
        const int tt = i / (p.rope.rotary_dim / 2), j = i % (p.rope.rotary_dim / 2);
        put_angle(p.rope, s_pos[tt], j, s_cs[tt]);
    }
    __syncthreads();

    auto body = [&](Unit &x) {
        const int token = x.tt, head = x.head, kv = head - p.num_qo_heads;
        const bool is_v = kv >= p.num_kv_heads;
        float a[8], b[8];
        unpack8(x.a, a);
        unpack8(x.b, b);
        load_unit(x);
        if (!s_ok[token])
            return;
        const int64_t t = t0 + token, row = s_row[token];
        if (!is_v && turns0)
            turn_unit(a, b, s_cs[token], c0, c1, turns1, p.rope.interleaved);
        if (kv < 0) {
            uint16_t *dst = p.q_out + t * p.q_out_stride + head * kHeadDim;
            *reinterpret_cast<uint4 *>(dst + c0) = pack8(a);
            *reinterpret_cast<uint4 *>(dst + c1) = pack8(b);
            return;
        }
        if constexpr (KVT == kKvTypeInt8)
            return;   // the page blocks'
        const int kvh = is_v ? kv - p.num_kv_heads : kv;
        const int64_t at = (row * p.num_kv_heads + kvh) * kHeadDim;   // values before this head's row
        uint8_t *pool = static_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages);
        if constexpr (KVT == kKvTypeBf16) {
            *reinterpret_cast<uint4 *>(pool + 2 * (at + c0)) = pack8(a);
            *reinterpret_cast<uint4 *>(pool + 2 * (at + c1)) = pack8(b);
        } else if constexpr (KVT == kKvTypeFp8) {
            uint32_t w[4];
            pack16_fp8(a, b, (is_v ? p.v_scale : p.k_scale)[kvh], w);
            *reinterpret_cast<uint2 *>(pool + at + c0) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2 *>(pool + at + c1) = make_uint2(w[2], w[3]);
        } else {
            // one scale per (row, head): largest magnitude / 7 over the head's
            // 8 lanes (1 for a row of zeros; NaN when the row holds one)
            float m = 0.f;
            bool nan = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m = fmaxf(m, fmaxf(fabsf(a[j]), fabsf(b[j])));
                nan |= a[j] != a[j] || b[j] != b[j];
            }
            if (nan)
                m = __int_as_float(0x7fffffff);
            const unsigned lanes = 0xffu << (tid & 24);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                const float n = __shfl_xor_sync(lanes, m, o);
                m = (m != m || n != n) ? __int_as_float(0x7fffffff) : fmaxf(m, n);
            }
            float scale = __fdiv_rn(m, 7.f);
            if (scale == 0.f)
                scale = 1.f;
            *reinterpret_cast<uint32_t *>(pool + (at + c0) / 2) = pack8_int4(a, scale);
            *reinterpret_cast<uint32_t *>(pool + (at + c1) / 2) = pack8_int4(b, scale);
            if (u == 0)
                (is_v ? p.v_scale_out : p.k_scale_out)[(int64_t)kvh * p.num_pages * p.page_size + row] = scale;
        }
    };
    while (u0.tt < nt) {
        body(u0);
        if (u1.tt >= nt)
            break;
        body(u1);
    }
}

template <int KVT>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const __grid_constant__ AppendParams p)
{
    append_tokens<KVT>(p, blockIdx.x);
}

// ------------------------------------------------- INT8: the new keys of a page
//
// Mathematics, for a page and KV head with f keys from before under scale s0 (0
// where f = 0): m = max |x| over the new keys' values (K rotated),
//     s = max(s0, m / 127, 2^-126),  code = rint(x / s),
// and where s > s0 the codes from before become rint(c s0 / s).  A scale only
// grows while its page fills, so a code is carried over at most as often as a key
// with a new largest value arrives (about 1/(f + 1) of single-token steps).
//
// Bound: bytes, as above.  A warp holds 16 or 4 rows of a head (8 lanes a row, 16 values
// each) in registers, from the maximum to the codes, when the page has no more new
// keys than its warps hold; else it reads them a second time, out of L2.  A kernel a
// rotary layout, and no divisions beside the quotients of pack8_int8: with both in one the
// warps waited for instructions (12345 tokens 64.0 us for 62.2, then 58.8).  Measured:
// 32768 tokens of 32 + 8 + 8 heads 139.8 us, 5.3 TB/s, of which the page blocks alone take
// 74; 64 tokens 4.4 us, the chain.
constexpr int kPageWarps = kThreads / 32;
constexpr int kAngleRows = 64;     // tokens of a page whose angles are in shared memory at once
constexpr int kFewRows = 4, kManyRows = 16;   // rows that a warp holds
constexpr float kSmallestScale = 1.17549435e-38f;

struct PageWork {
    int32_t token, place, rows;   // first new token, its place in the page, new tokens in it
    int32_t entry;                // page-list entry
    int32_t key;                  // first new token's key index
    int32_t page;                 // -1: none
};

// The whole CTA: the work of page `t` of the call's new keys, counted over the
// requests.  page -1: there is none.
__device__ __forceinline__ void find_page(const AppendParams &p, int t, PageWork &out, int (&scan)[kPageWarps])
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0)
        out.page = -1;
    int carry = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
        const int b = b0 + tid;
        int n = 0, a0 = 0, a1 = 0, e0 = 0;
        uint32_t len = 0, first = 0;   // keys of the table, the first new one
        const uint32_t page_size = (uint32_t)p.page_size;
        if (b < p.batch) {
            a0 = p.append_indptr[b];
            a1 = p.append_indptr[b + 1];
            e0 = p.kv_page_indptr[b];
            const int e1 = p.kv_page_indptr[b + 1], last = p.kv_last_page_len[b];
            if (a1 > a0) {
                const int64_t keys = (int64_t)(e1 - e0 - 1) * p.page_size + last;
                const bool ok = a0 >= 0 && a1 <= p.num_tokens && e0 >= 0 && e1 > e0 && e1 <= p.num_page_entries &&
                                last >= 1 && last <= p.page_size && keys <= INT32_MAX;
                if (!ok || keys < a1 - a0)   // tokens outside the table are skipped
                    report(p.status, FD_ERR_DEVICE_BOUNDS);
                if (ok) {
                    len = (uint32_t)keys;
                    first = keys < a1 - a0 ? 0 : len - (uint32_t)(a1 - a0);
                    n = (int)((len - 1) / page_size - first / page_size) + 1;
                }
            }
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += x;
        }
        __syncthreads();
        if (lane == 31)
            scan[warp] = incl;
        __syncthreads();
        int before = carry, total = 0;
#pragma unroll
        for (int w = 0; w < kPageWarps; ++w) {
            before += w < warp ? scan[w] : 0;
            total += scan[w];
        }
        incl += before;
        if (n > 0 && t >= incl - n && t < incl) {
            const uint32_t pg = first / page_size + (uint32_t)(t - (incl - n)), start = pg * page_size;
            const uint32_t lo = max(first, start), hi = min(len, start + page_size);
            out.key = (int)lo;
            out.token = a1 - (int)(len - lo);
            out.place = (int)(lo - start);
            out.rows = (int)(hi - lo);
            out.entry = e0 + (int)pg;
            const int page = p.kv_page_indices[out.entry];
            const bool in = page >= 0 && page < p.num_pages;
            if (!in)
                report(p.status, FD_ERR_DEVICE_BOUNDS);
            out.page = in ? page : -1;
        }
        carry += total;
        if (t > 0 && t < carry)
            break;
    }
    if (t == 0 && carry > p.page_ctas && tid == 0)   // requests whose tokens are not apart
        report(p.status, FD_ERR_DEVICE_BOUNDS);
    __syncthreads();
}

// Magnitudes compare as the bits of their floats do; a NaN's are above all others'.
__device__ __forceinline__ uint32_t magnitude(const float (&x)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
    return m;
}

// The same of eight bf16 values, two at a time.
__device__ __forceinline__ uint32_t magnitude(const uint4 &w)
{
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
}

__device__ __forceinline__ float max_or_nan(float a, float b)
{
    return a != a || b != b ? __int_as_float(0x7fffffff) : fmaxf(a, b);
}

// Eight values over a scale (quotients of at most 127 in magnitude), rounded to whole
// numbers, as bytes.  The quotient is rounded to fp32 as a division would (a step of
// Markstein's, as in pack4_over: many values of a page are half-way between codes, its
// largest being 127), then 1.5 * 2^23 + y has rint(y) in its low bits.  up: 1, or for a
// scale near the ends of fp32's range the power of two that the caller has put into
// `scale` (a value that it takes below fp32's range has the code 0 either way).
__device__ __forceinline__ uint2 pack8_int8(const float (&x)[8], float scale, float inv, float up)
{
    const float2 inv2 = make_float2(inv, inv), minus = make_float2(-scale, -scale);
    const float2 magic = make_float2(12582912.f, 12582912.f);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float2 y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float2 v = make_float2(x[4 * i + 2 * j], x[4 * i + 2 * j + 1]);
            if (up != 1.f)
                v = mul2(v, make_float2(up, up));
            y[j] = mul2(v, inv2);
            y[j] = fma2(fma2(y[j], minus, v), inv2, y[j]);
            y[j] = add2(y[j], magic);
        }
        w[i] = __byte_perm(__byte_perm(__float_as_uint(y[0].x), __float_as_uint(y[0].y), 0x0040),
                           __byte_perm(__float_as_uint(y[1].x), __float_as_uint(y[1].y), 0x0040), 0x5410);
    }
    return make_uint2(w[0], w[1]);
}

// Four codes times r, rounded, within -127 .. 127.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r)
{
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = (int)(int8_t)(w >> (8 * i));
        const int d = min(max(__float2int_rn((float)c * r), -127), 127);
        out |= (uint32_t)(d & 0xff) << (8 * i);
    }
    return out;
}

// Warps a head: as many as hold a page's new rows in registers, and for few heads as
// many as there are; no more than hold the rows that have their angles in shared
// memory at once.
__host__ __device__ __forceinline__ int warps_per_head(int64_t rows, int num_kv_heads)
{
    const int group = rows <= kFewRows ? kFewRows : kManyRows;
    const int most = kAngleRows / group < kPageWarps ? kAngleRows / group : kPageWarps;
    int wph = 1;
    while (wph < most && (wph * group < rows || kPageWarps / wph / 2 >= num_kv_heads))
        wph *= 2;
    return wph;
}

struct PageSmem {
    float2 cs[kAngleRows][kHeadDim / 2];   // (cos, sin) of the rows' angles
    PageWork work;
    int scan[kPageWarps];
    uint32_t most[2][kPageWarps];
};

// The new keys of one page, for part `at` of its heads, K's then V's: a step is a head
// for every `wph` warps, which share its rows, kGroupRows a warp at once.
template <bool kInterleaved, int kGroupRows>
__device__ __forceinline__ void append_page(const AppendParams &p, PageSmem &sm, const PageWork work, int wph, int at)
{
    constexpr int kAngleGroups = kAngleRows / kGroupRows;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = warp % wph;
    const int steps = (p.num_kv_heads * wph + kPageWarps - 1) / kPageWarps;   // of K, and of V
    const int u = lane & 7, row4 = lane >> 3;
    const int rot = p.rope.rotary_dim, pairs = rot / 2;
    int c0, c1;
    unit_chunks(p.rope, u, c0, c1);
    const bool turns0 = c0 < rot, turns1 = c1 < rot;
    const int n = work.rows;
    const int groups = (n + kGroupRows - 1) / kGroupRows;
    const bool held = groups <= wph;   // every warp has its rows in registers
    const int64_t row_bytes = (int64_t)p.num_kv_heads * kHeadDim;

    auto angles = [&](int from) {   // of the tokens from row `from` on
        const int j = tid & (kHeadDim / 2 - 1);
        if (j < pairs)
            for (int r = from + tid / (kHeadDim / 2); r < min(n, from + kAngleRows); r += kThreads / (kHeadDim / 2))
                put_angle(p.rope, p.positions ? p.positions[work.token + r] : work.key + r, j, sm.cs[r - from]);
    };
    int have_angles = -1;   // the first row of those in shared memory
    const int first = 2 * steps * at / p.blocks_per_page, last = 2 * steps * (at + 1) / p.blocks_per_page;
#pragma unroll 1
    for (int it = first; it < last; ++it) {
        const bool is_v = it >= steps;
        const int head = ((is_v ? it - steps : it) * kPageWarps + warp) / wph;
        const bool mine = head < p.num_kv_heads;
        const int64_t stride = is_v ? p.v_stride : p.k_stride;
        const uint16_t *src = (is_v ? p.v : p.k) + work.token * stride + (mine ? head : 0) * kHeadDim;
        float *const scales = (is_v ? p.v_scale_out : p.k_scale_out) + (int64_t)work.page * p.scale_heads + (mine ? head : 0);
        const bool rotate = !is_v && rot > 0;
        uint4 raw[kGroupRows / 4][2];   // rows 4 i + row4 of a group
        auto load = [&](int g) {
#pragma unroll
            for (int i = 0; i < kGroupRows / 4; ++i) {
                const int r = g * kGroupRows + 4 * i + row4;
                raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
                if (mine && r < n) {
                    raw[i][0] = *reinterpret_cast<const uint4 *>(src + r * stride + c0);
                    raw[i][1] = *reinterpret_cast<const uint4 *>(src + r * stride + c1);
                }
            }
        };
        // Groups part, part + wph, ..; K's angles are there for 64 rows at a time.
        auto each_group = [&](auto &&work_on) {
#pragma unroll 1
            for (int g0 = 0; g0 < groups; g0 += kAngleGroups) {
                const int from = g0 * kGroupRows;
                if (rotate && have_angles != from) {
                    __syncthreads();   // the others are done with those before
                    angles(from);
                    __syncthreads();
                    have_angles = from;
                }
#pragma unroll 1
                for (int g = g0 + part; g < min(groups, g0 + kAngleGroups); g += wph) {
                    if (!held)
                        load(g);
                    work_on(g, from);
                }
            }
        };
        auto unit = [&](int i, int r, int from, float (&a)[8], float (&b)[8]) {   // row r of the new ones
            unpack8(raw[i][0], a);
            unpack8(raw[i][1], b);
            if (rotate && turns0 && r < n)
                turn_unit(a, b, sm.cs[r - from], c0, c1, turns1, kInterleaved);
        };
        if (held)
            load(part);
        const float s0 = work.place > 0 && mine ? *scales : 0.f;
        uint32_t bits = 0;
        each_group([&](int g, int from) {
#pragma unroll
            for (int i = 0; i < kGroupRows / 4; ++i) {
                if (g * kGroupRows + 4 * i >= n)   // (a step's page has one row)
                    break;
                if (is_v) {
                    bits = max(bits, max(magnitude(raw[i][0]), magnitude(raw[i][1])));
                } else {
                    float a[8], b[8];
                    unit(i, g * kGroupRows + 4 * i + row4, from, a, b);
                    bits = max(bits, max(magnitude(a), magnitude(b)));
                }
            }
        });
        bits = __reduce_max_sync(0xffffffffu, bits);
        if (wph > 1) {
            if (lane == 0)
                sm.most[it & 1][warp] = bits;
            __syncthreads();
            for (int w = 0; w < wph; ++w)
                bits = max(bits, sm.most[it & 1][warp - part + w]);
        }
        const float s = max_or_nan(s0, max_or_nan(__fdiv_rn(__uint_as_float(bits), 127.f), kSmallestScale));
        // a page whose scale is no number has the codes 0: its values are NaN
        const bool number = s < INFINITY;
        const float up = s > 1e-15f && s < 1e15f ? 1.f : s < 1.f ? 0x1p100f : 0x1p-100f;
        const float s_up = s * up, inv = __fdiv_rn(1.f, s_up);
        if (mine && part == 0 && lane == 0)
            *scales = s;   // (all have read s0: the exchange of the maxima)
        uint8_t *const rows = static_cast<uint8_t *>(is_v ? p.v_pages : p.k_pages) +
                              ((int64_t)work.page * p.page_size * p.num_kv_heads + (mine ? head : 0)) * kHeadDim;
        if (mine && work.place > 0 && s != s0) {
            const float r = number ? __fdiv_rn(s0, s) : 0.f;
#pragma unroll 1
            for (int i = part * 4 + row4; i < work.place; i += 4 * wph) {
                uint4 *to = reinterpret_cast<uint4 *>(rows + i * row_bytes) + u;
                const uint4 c = *to;
                *to = make_uint4(rescale4(c.x, r), rescale4(c.y, r), rescale4(c.z, r), rescale4(c.w, r));
            }
        }
        each_group([&](int g, int from) {
#pragma unroll
            for (int i = 0; i < kGroupRows / 4; ++i) {
                if (g * kGroupRows + 4 * i >= n)
                    break;
                const int r = g * kGroupRows + 4 * i + row4;
                float a[8], b[8];
                unit(i, r, from, a, b);
                uint2 x = pack8_int8(a, s_up, inv, up), y = pack8_int8(b, s_up, inv, up);
                if (!number)
                    x = y = make_uint2(0u, 0u);
                if (mine && r < n) {
                    uint8_t *dst = rows + (work.place + r) * row_bytes;
                    *reinterpret_cast<uint2 *>(dst + c0) = x;
                    *reinterpret_cast<uint2 *>(dst + c1) = y;
                }
            }
        });
    }
}

// Blocks: blocks_per_page for each page with new keys, then the queries'.
template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 3) append_int8_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ __align__(16) PageSmem sm;
    const int block = blockIdx.x, page_blocks = p.page_ctas * p.blocks_per_page;
    if (block >= page_blocks) {
        append_tokens<kKvTypeInt8>(p, block - page_blocks);
        return;
    }
    griddep_wait();
    griddep_launch_dependents();
    find_page(p, block / p.blocks_per_page, sm.work, sm.scan);
    if (sm.work.page < 0)
        return;
    // Up to four rows (a step's, drafted tokens'): code and registers for no more, 64
    // tokens 4.4 us for 4.95 and 256 of 64 + 8 + 8 heads 7.0 for 7.9.
    const PageWork work = sm.work;
    const int at = block % p.blocks_per_page;
    if (work.rows <= kFewRows)
        append_page<kInterleaved, kFewRows>(p, sm, work, warps_per_head(work.rows, p.num_kv_heads), at);
    else
        append_page<kInterleaved, kManyRows>(p, sm, work, warps_per_head(work.rows, p.num_kv_heads), at);
}

}  // namespace

cudaError_t launch_append_int8(const AppendParams &params, cudaStream_t stream)
{
    AppendParams p = params;
    // Requests of n new keys reach into at most (n + 2 page_size - 2) / page_size
    // pages, and no more than n.
    const int64_t some = p.batch < p.num_tokens ? p.batch : p.num_tokens;
    const int64_t pages = p.num_tokens / p.page_size + 2 * some;
    p.page_ctas = (int32_t)(pages < p.num_tokens ? pages : p.num_tokens);
    const int64_t rows = (p.num_tokens + p.page_ctas - 1) / p.page_ctas;
    const int steps = 2 * ((p.num_kv_heads * warps_per_head(rows, p.num_kv_heads) + kPageWarps - 1) / kPageWarps);
    // Blocks a page: one (its angles are computed once) where that fills the SMs
    // twice, more for fewer pages and for those whose rows are read twice.
    const int64_t fill = 152 * 2, want = rows > kAngleRows ? 4 * fill : fill;
    const int64_t share = want / p.page_ctas > 1 ? want / p.page_ctas : 1;
    p.blocks_per_page = (int32_t)(share < steps ? share : steps);
    constexpr int kWave = 152 * 3;
    const int waves = (p.num_tokens + kWave * kMaxTokens - 1) / (kWave * kMaxTokens);
    p.tokens_per_cta = (p.num_tokens + kWave * waves - 1) / (kWave * waves);
    const int64_t q_ctas = p.num_qo_heads > 0 ? (p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta : 0;
    const int64_t grid = (int64_t)p.page_ctas * p.blocks_per_page + q_ctas;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    const auto kernel = p.rope.interleaved ? append_int8_kernel<true> : append_int8_kernel<false>;
    return launch_dependent(kernel, dim3((unsigned)grid), kThreads, 0, stream, p);
}

cudaError_t launch_append(const AppendParams &params, int kv_type, cudaStream_t stream)
{
    AppendParams p = params;
    // One token a CTA up to one wave of resident CTAs (a short call is a chain of
    // dependent loads: more CTAs, shorter chains), then as few whole waves as
    // kMaxTokens tokens a CTA allow, equal CTAs (12345 tokens of 48 heads in FP8: 7
    // a CTA took 0.6 us less than 8).
    constexpr int kWave = 152 * 4;
    const int waves = (p.num_tokens + kWave * kMaxTokens - 1) / (kWave * kMaxTokens);
    p.tokens_per_cta = (p.num_tokens + kWave * waves - 1) / (kWave * waves);
    const dim3 grid((unsigned)((p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta));
    switch (kv_type) {
    case kKvTypeBf16: return launch_dependent(append_kernel<kKvTypeBf16>, grid, kThreads, 0, stream, p);
    case kKvTypeFp8: return launch_dependent(append_kernel<kKvTypeFp8>, grid, kThreads, 0, stream, p);
    case kKvTypeInt8: return launch_append_int8(params, stream);
    default: return launch_dependent(append_kernel<kKvTypeInt4>, grid, kThreads, 0, stream, p);
    }
}

}  // namespace fd
