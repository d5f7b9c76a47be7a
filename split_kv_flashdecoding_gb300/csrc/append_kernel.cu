// append_kernel.cu -- rotary positions on new queries and keys, and the write
// of the new keys and values into a paged cache (bf16, FP8 E4M3 or INT4).
//
// Mathematics: pair i of a head's first rotary_dim values is turned by the
// angle position * f_i: (a, b) -> gain (a cos - b sin, b cos + a sin).  The
// angle is kept in turns as a 64-bit fixed-point fraction: step_i = f_i / 2 pi
// * 2^64, and position * step_i modulo 2^64 is the exact fraction of a turn of
// that step (the plan's rounding of f_i, 2^-53 of it, is all that a far
// position loses), so one integer product replaces a long range reduction.
// The arithmetic is fp32; each output is rounded once.
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

template <int KVT>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ __align__(16) float2 s_cs[kMaxTokens][kHeadDim / 2];
    __shared__ int64_t s_row[kMaxTokens];    // cache row of the token, -1: none
    __shared__ int s_pos[kMaxTokens], s_ok[kMaxTokens], s_count[kMaxTokens];

    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * p.tokens_per_cta;
    const int nt = min(p.tokens_per_cta, p.num_tokens - t0);
    if (tid < kMaxTokens)
        s_count[tid] = 0;
    // Thread (head lane, unit u): the same unit of every 32nd head of the CTA's
    // tokens, one after another, so that nothing is divided and all lanes are at
    // work.  The 8 lanes of a head stay together, which the INT4 scale's reduction
    // relies on.
    const int heads = p.num_qo_heads + 2 * p.num_kv_heads;
    const int u = tid % kUnits, lane_head = tid / kUnits;
    // The unit's two chunks start at c0 and c1, which run on over the 8 lanes;
    // pairs of an interleaved layout lie within a chunk, those of the other one in
    // the two chunks of a unit.
    const int rot = p.rope.rotary_dim, rot_units = rot / 16;
    int c0 = 8 * u, c1 = kHeadDim / 2 + 8 * u;
    if (!p.rope.interleaved) {
        c0 = u < rot_units ? 8 * u : rot + 8 * (u - rot_units);
        c1 = c0 + (u < rot_units ? rot : kHeadDim - rot) / 2;
    }
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
        const uint64_t turns = (uint64_t)(int64_t)s_pos[tt] * p.rope.step[j];
        float s, c;
        sincospif((float)(int64_t)turns * 1.0842021724855044e-19f, &s, &c);   // turns / 2^63: half turns
        s_cs[tt][2 * place(j >> 1) + (j & 1)] = make_float2(c * p.rope.gain, s * p.rope.gain);
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
        if (!is_v && turns0) {
            // the pairs' (cos, sin): of each chunk's 4 pairs, or of the unit's 8
            const float4 *cs = reinterpret_cast<const float4 *>(s_cs[token]);
            if (p.rope.interleaved) {
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
        if (kv < 0) {
            uint16_t *dst = p.q_out + t * p.q_out_stride + head * kHeadDim;
            *reinterpret_cast<uint4 *>(dst + c0) = pack8(a);
            *reinterpret_cast<uint4 *>(dst + c1) = pack8(b);
            return;
        }
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

}  // namespace

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
    default: return launch_dependent(append_kernel<kKvTypeInt4>, grid, kThreads, 0, stream, p);
    }
}

}  // namespace fd
