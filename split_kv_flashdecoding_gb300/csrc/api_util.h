// api_util.h -- small host helpers shared by the files that hold C entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fd {

// The first bytes behind a workspace's header, which the calls over prefixes, forks
// and compactions keep for merge tickets: zero between calls, wherever the rest
// of a plan's or a page operation's scratch begins, so that one workspace serves
// calls of different plans and operators.  Room for 16384 (request, KV head) groups.
constexpr int64_t kTicketBytes = 64 * 1024;

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline int64_t round_up(int64_t x, int64_t m)
{
    return (x + m - 1) / m * m;
}

inline cudaStream_t as_stream(void *s)
{
    return reinterpret_cast<cudaStream_t>(s);
}

// Launch as a programmatic dependent of the preceding grid in the stream (the
// kernel waits for that grid before it touches global memory).
template <typename Kernel, typename... Args>
cudaError_t launch_dependent(Kernel kern, dim3 grid, int threads, int smem_bytes, cudaStream_t stream,
                             Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Whether rows of `na` values, `sa` apart, from a on share a value with rows of `nb`
// values, `sb` apart, from b on: n rows each, 16-bit values.  Rows that lie between
// one another at different distances count as if they did.
inline bool rows_overlap(const void *a, int64_t na, int64_t sa, const void *b, int64_t nb, int64_t sb, int64_t n)
{
    const int64_t x = (int64_t)(reinterpret_cast<uintptr_t>(a) / 2), y = (int64_t)(reinterpret_cast<uintptr_t>(b) / 2);
    if (x + (n - 1) * sa + na <= y || y + (n - 1) * sb + nb <= x)
        return false;
    if (n == 1 || sa != sb)
        return true;
    const int64_t d = ((x - y) % sa + sa) % sa;   // where a's rows begin behind b's, up to whole rows
    return d < nb || d + na > sa;
}

}  // namespace fd
