// shared_kernel.cu -- launch of shared-prefix decode attention (see
// shared_kernel.cuh).
#include "shared_kernel.cuh"

namespace fd {
namespace {

template <bool PAGED, int DT>
cudaError_t launch_prefixes(const SharedMaps &maps, const SharedParams &p, cudaStream_t stream)
{
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(shared_kernel<PAGED, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedAlloc);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            configured[dev] = true;
    }
    return launch_dependent(shared_kernel<PAGED, DT>, dim3((unsigned)p.num_items), kThreads<DT>, kSharedAlloc, stream,
                            maps.k, maps.v, p);
}

}  // namespace

cudaError_t launch_shared(const SharedMaps &maps, const SharedParams &p, int kv_type, cudaStream_t stream)
{
    if (p.num_items > 0) {
        cudaError_t e;
        if (kv_type == kKvTypeFp8)
            e = p.page_size ? launch_prefixes<true, kKvTypeFp8>(maps, p, stream)
                            : launch_prefixes<false, kKvTypeFp8>(maps, p, stream);
        else
            e = p.page_size ? launch_prefixes<true, kKvTypeBf16>(maps, p, stream)
                            : launch_prefixes<false, kKvTypeBf16>(maps, p, stream);
        if (e != cudaSuccess)
            return e;
    }
    const int64_t rows = (int64_t)p.batch * p.num_qo_heads;
    return launch_dependent(shared_merge_kernel, dim3((unsigned)((rows + kMergeWarps - 1) / kMergeWarps)),
                            kMergeWarps * 32, 0, stream, p);
}

}  // namespace fd
