// tc_stream.cuh -- what the tensor-core attention kernels share: waits of their
// pipelines, barriers of some of a CTA's warps, the order of a stream's tiles.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"

namespace fd {

constexpr uint32_t kSleepNs = 100000;   // a wait's sleep between looks at the timer

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// Wait for a phase; false (and the CTA's abort flag set) when the time limit
// passed or another warp gave up.
template <typename Params, typename Smem>
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, const Params &p, Smem *sm)
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

}  // namespace fd
