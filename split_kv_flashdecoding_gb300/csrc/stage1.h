// stage1.h -- the split kernel's host launch, shared by the files that hold C
// entry points (internal).
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fd.h"

namespace fd {

// Quantised K/V: the element type (kKvTypeFp8, kKvTypeInt4 or kKvTypeInt8) and
// the device scales -- FP8: [Hkv] each; INT4: [Hkv][rows] each; INT8:
// [num_pages][scale_heads(Hkv)] each.
struct QuantKV {
    int type;
    const float *k_scale;
    const float *v_scale;
};

// Floats of a page's row of INT8 scales: whole 16-byte pieces, as page copies take.
constexpr int scale_heads(int num_kv_heads)
{
    return (num_kv_heads + 3) / 4 * 4;
}

// The page-pool description of a paged KV cache (see fd_decode_paged).
struct PagedKV {
    int32_t page_size;
    int32_t num_pages;
    const int32_t *last_len_dev;
    const int32_t *last_len_host;
    const int32_t *page_indices_dev;
    int32_t num_page_entries;   // kv_page_indptr[batch]
};

// Where a fused decode keeps its scratch in a workspace of a plan:
// status header | tickets [B * Hkv] | partial LSE | partial O | flags [num_work].
struct WorkspaceLayout {
    int *counters;
    float *partial_lse;
    float *partial_o;
    int *flags;
};

WorkspaceLayout workspace_layout(void *workspace, int64_t batch, int64_t num_kv_heads,
                                 int64_t num_partial_rows);

// cuTensorMapEncodeTiled, or null when the driver has none.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// K or V [rows, Hkv, 128] bf16 as a tensor map of one head's box_rows rows.
int make_kv_map(CUtensorMap *map, const void *base, int64_t rows, int num_kv_heads, int box_rows);

// FP8 or INT8 K or V [rows, Hkv, 128], one byte a value, likewise.
int make_kv_map_fp8(CUtensorMap *map, const void *base, int64_t rows, int num_kv_heads, int box_rows);

// Argument checks and the split kernel's launch (see fd_api.cu).  early_next: see
// SplitParams (device_plan only).
int check_info(const fd_plan_info *info);
int launch_stage1(const fd_plan_info *info, const void *q, const void *k, const void *v,
                  const int32_t *kv_indptr_dev, float scale, float *partial_o, float *partial_lse,
                  void *workspace, float *o, float *lse, int *counters,
                  const int32_t *kv_indptr_host, cudaStream_t stream,
                  const PagedKV *paged = nullptr, const QuantKV *quant = nullptr,
                  bool device_plan = false, int *flags = nullptr, bool early_next = false);

}  // namespace fd
