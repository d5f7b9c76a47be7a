// shared_kernel.cu -- launch of shared-prefix decode attention (see
// shared_kernel.cuh).
#include "shared_kernel.cuh"

namespace fd {
namespace {

template <typename Kernel>
cudaError_t launch_prefixes(Kernel kern, bool (&configured)[64], const SharedMaps &maps, const SharedParams &p,
                            cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedAlloc);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            configured[dev] = true;
    }
    return launch_dependent(kern, dim3((unsigned)p.num_items), kThreads, kSharedAlloc, stream, maps.k, maps.v, p);
}

}  // namespace

cudaError_t launch_shared(const SharedMaps &maps, const SharedParams &p, int kv_type, cudaStream_t stream)
{
    (void)kv_type;
    if (p.num_items > 0) {
        static bool configured[2][64] = {};
        const cudaError_t e = p.page_size ? launch_prefixes(shared_kernel<true>, configured[1], maps, p, stream)
                                          : launch_prefixes(shared_kernel<false>, configured[0], maps, p, stream);
        if (e != cudaSuccess)
            return e;
    }
    const int64_t rows = (int64_t)p.batch * p.num_qo_heads;
    return launch_dependent(shared_merge_kernel, dim3((unsigned)((rows + kMergeWarps - 1) / kMergeWarps)),
                            kMergeWarps * 32, 0, stream, p);
}

}  // namespace fd
