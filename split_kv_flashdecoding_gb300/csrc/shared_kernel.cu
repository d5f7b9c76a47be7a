// shared_kernel.cu -- launch of shared-prefix decode attention (see
// shared_kernel.cuh).
#include "shared_kernel.cuh"

namespace fd {
namespace {

constexpr int kFewRows = 256;

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
    // A warp a row, or four where a row has more partials than a warp loads at
    // once and the rows are few: 64 rows of 19 partials 13.7 us for 14.6 (the whole
    // call), 128 of 16 15.7 for 17.1, 256 of 19 as good, 1024 of 19 19.9 for 17.7.
    const int64_t rows = (int64_t)p.batch * p.num_qo_heads;
    if (rows <= kFewRows && p.num_partial_rows > kMergeBatch * rows)
        return launch_dependent(shared_merge_kernel<kMergeWarps>, dim3((unsigned)rows), kMergeWarps * 32, 0, stream, p);
    return launch_dependent(shared_merge_kernel<1>, dim3((unsigned)((rows + kMergeWarps - 1) / kMergeWarps)),
                            kMergeWarps * 32, 0, stream, p);
}

}  // namespace fd
