// split_kernel_int8.cu -- stage 1 for INT8 K/V with a scale per page and KV head:
// the split kernels of split_kernel.cuh with the codes widened to f16 in registers.
//
// S = s_K[page] Q C_K^T and O = (P s_V[page]) C_V with integer codes C: a page is a
// whole number of 16-key halves of a tile, so the K scale multiplies a half's logits
// and the V scale its weights, and the codes go into the products as they are (a
// byte with its sign bit flipped under the exponent of 1024, less 1152: exact, 1.25
// instructions a code).  Tiles come as the FP8 path's, in boxes of the pages' rows;
// the consumer warps look their tiles' scales up themselves (PageScaleFeed).
//
// Bound: with pages of 16 keys the copy engine's rate a box, as for FP8; else the
// consumers' arithmetic beside the copies.  32 query heads over 65536 keys of 8 KV
// heads take 37.3 us in pages of 16 (FP8 36.1) and 31 in pages of 64 (28.3); 64
// requests of up to 16384 keys in pages of 64 202 us, 5.2 TB/s (197); 16 of 64 heads
// over 32768 keys in pages of 32 222 us, 4.8 TB/s (204).
#include "split_kernel.cuh"

namespace fd {

cudaError_t launch_split_int8(const KvMaps &maps, const SplitParams &p, int group, int num_ctas,
                              cudaStream_t stream)
{
    return launch_split_dt<kKvInt8>(maps, p, group, num_ctas, stream);
}

}  // namespace fd
