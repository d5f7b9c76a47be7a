// split_kernel_int8.cu -- stage 1 for INT8 K/V with a scale per page and KV head:
// the split kernels of split_kernel.cuh with the codes widened to f16 in registers.
//
// S = s_K[page] Q C_K^T and O = (P s_V[page]) C_V with integer codes C: a page is a
// whole number of 16-key halves of a tile, so the K scale multiplies a half's logits
// and the V scale its weights, and the codes go into the products as they are (a
// byte with its sign bit flipped under the exponent of 1024, less 1152: exact, 1.25
// instructions a code).  Tiles come as the FP8 path's, in boxes of the pages' rows;
// a lane each of the producer warp copies the four scales of a tile beside them.
#include "split_kernel.cuh"

namespace fd {

cudaError_t launch_split_int8(const KvMaps &maps, const SplitParams &p, int group, int num_ctas,
                              cudaStream_t stream)
{
    return launch_split_dt<kKvInt8>(maps, p, group, num_ctas, stream);
}

}  // namespace fd
