// tcgen05.cuh -- sm_103a tensor-memory and fifth-generation tensor-core
// wrappers in inline PTX.
#pragma once

#include <stdint.h>

namespace fd {

// Whole warp: allocate `cols` columns (a power of two, 32..512) of tensor
// memory; the base address is written to shared address `dst`.
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void tcgen05_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tcgen05_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// One lane of a converged warp: nonzero there.  The instructions below are run
// by the whole warp and issued by that lane (`leader`), so that their operands
// are computed once for the warp.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t x;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
    return x;
}

// One arrival on `bar` once every tcgen05.mma the leader issued has completed.
__device__ __forceinline__ void tcgen05_commit(uint32_t bar, uint32_t leader)
{
    asm volatile("{\n\t.reg .pred l;\n\tsetp.ne.u32 l, %1, 0;\n\t"
                 "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
                 "r"(leader)
                 : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading
// and stride byte offsets (all multiples of 16).
//  K-major operand: 8-row groups of 128-byte rows `sbo` apart (lbo unused).
//  MN-major operand: 128-byte rows of 64 MN elements, one row per K index;
//    8-row groups of K `sbo` apart, blocks of 64 MN elements `lbo` apart.
// In two words: the first counts 16 bytes in its low bits, so that an operand
// further on is the first word plus a constant.
__device__ __forceinline__ uint32_t smem_desc_lo(uint32_t addr, uint32_t lbo)
{
    return ((addr & 0x3FFFF) >> 4) | ((lbo >> 4) << 16);
}

__host__ __device__ constexpr uint32_t smem_desc_hi(uint32_t sbo)
{
    return (sbo >> 4) | (1u << 14) | (2u << 29);
}

// Instruction descriptor of kind::f16 with fp32 accumulation, M x N tile.
// bf16: element type of both operands (else f16); b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t mma_idesc(int m, int n, bool bf16, bool b_mn)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D (+)= A B, A and B in shared memory (descriptor words); accumulate: 0
// overwrites D.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate, uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred p, l;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\tsetp.ne.u32 l, %7, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}

// D (+)= A B, A in tensor memory (two 16-bit elements a column), B in shared.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t accumulate, uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred p, l;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 l, %6, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}

#define FD_R4(b) "=r"(r[b]), "=r"(r[b + 1]), "=r"(r[b + 2]), "=r"(r[b + 3])
#define FD_W4(b) "r"(r[b]), "r"(r[b + 1]), "r"(r[b + 2]), "r"(r[b + 3])

// 16 columns of the warp's 32 lanes: register j of thread t is column j of lane t.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : FD_R4(0), FD_R4(4), FD_R4(8), FD_R4(12)
        : "r"(addr));
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
                 FD_W4(0), FD_W4(4)
                 : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        FD_W4(0), FD_W4(4), FD_W4(8), FD_W4(12)
        : "memory");
}

#undef FD_R4
#undef FD_W4

__device__ __forceinline__ void tmem_wait_ld()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

}  // namespace fd
