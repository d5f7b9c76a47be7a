// int8_widen.cuh -- two's-complement bytes as f16 values, exactly.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fd {

// Two's-complement bytes of x -> f16x2: lo = bytes A and B, hi = bytes C and D
// (the first of each in the low half).  A byte with its sign bit flipped is
// u = n + 128; under the exponent byte of 1024 it is the f16 1024 + u, and
// subtracting 1152 leaves n, exactly.
template <int A, int B, int C, int D>
__device__ __forceinline__ void int8x4_to_f16x2x2(uint32_t x, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = x ^ 0x80808080u;
    constexpr uint32_t k1024 = 0x64646464u, k1152 = 0x64806480u;
    lo = __byte_perm(u, k1024, 0x4040u | A | (B << 8));
    hi = __byte_perm(u, k1024, 0x4040u | C | (D << 8));
    asm("sub.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(k1152));
    asm("sub.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(k1152));
}

}  // namespace fd
