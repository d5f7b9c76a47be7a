/*
 * fd.h -- C ABI of libfd: split-KV ("flash-decoding") decode attention for
 * NVIDIA GB300 (sm_103a).
 *
 * Method: "FlashDecoding++: sequence-dimension KV split parallelism for LLM
 * serving" (techknowgenie.com).  §2 adds the sequence axis to the grid so a
 * batch-1 decode step fills every SM; §3 computes a partial softmax per chunk
 * (stage 1) and merges the partials by their log-sum-exp (stage 2); §6 (chunk
 * size tuning guide) sizes the chunks from the SM count.
 *
 * What one decode step computes (for each request b and query head hq, with
 * G = Hq / Hkv and KV head kvh = hq / G):
 *     s_j   = scale * <q[b,hq,:], K[j,kvh,:]>      j in [kv_indptr[b], kv_indptr[b+1])
 *     O     = sum_j softmax(s)_j * V[j,kvh,:]
 *     LSE   = ln sum_j exp(s_j)
 *
 * Tensor layouts (all row-major, contiguous, device memory unless noted):
 *     q          bf16  [B, Hq, D]
 *     k, v       bf16  [T, Hkv, D]   ragged "packed" KV cache, T = kv_indptr[B]
 *     kv_indptr  int32 [B+1]         0 = kv_indptr[0] <= ... <= kv_indptr[B] = T
 *     o          fp32  [B, Hq, D]
 *     lse        fp32  [B, Hq]       natural log; -inf for a request with no keys
 *     partial_o  fp32  [num_partial_rows, D]
 *     partial_lse fp32 [num_partial_rows]
 * Partial row of (request b, query head hq, split s):
 *     split_prefix[b] * Hq + hq * splits_b + s
 * where splits_b is request b's split count and split_prefix[b] is the sum of
 * splits_b' over b' < b.
 *
 * Supported: D = 128; G = Hq / Hkv in {1, 2, 4, 8}.  Others return
 * FD_ERR_UNSUPPORTED.  q, k, v, o, partial_o must be 16-byte aligned.
 *
 * Ownership: the caller owns every buffer.  The library allocates no device
 * memory and keeps no state between calls besides a cached SM count per device,
 * with one exception: fd_decode_static_workspace keeps its scratch in a fixed
 * device array of FD_STATIC_WORKSPACE_BYTES inside the library (present on
 * every GPU that loads it, holding the last such call's contents) and caches
 * that array's device address per device.
 * All device work is asynchronous on the given stream (a cudaStream_t passed as
 * void*; NULL = legacy default stream).
 *
 * Errors: every entry point returns an fd_status (0 = FD_OK, negative =
 * error) and never throws.  Arguments are validated on the host before any
 * launch; launch failures return FD_ERR_CUDA.  Errors the kernels detect
 * (a bounded wait that ran out, a derived index outside the plan) are written
 * to a status word in the workspace and read by fd_get_device_status().
 *
 * Workspace: a caller-owned device buffer, zero-filled before its first use.
 * Its first FD_WORKSPACE_HEADER_BYTES hold the device status word and the
 * work counter of the split kernel (used when a plan has more split items than
 * one wave of resident CTAs: the kernel then runs persistent CTAs that claim
 * items from the counter); fd_decode also keeps in it one merge ticket per
 * (request, KV head) and the split partials (size:
 * fd_plan_info.workspace_bytes).  The counter and the tickets return to zero
 * at the end of every successful call; after a call that reported an error
 * status, zero the workspace again before reusing it.  Calls that share one
 * workspace must be ordered on one stream.
 *   Which calls may share one: fd_decode and its forms (paged, FP8, INT4, graph)
 * lay their tickets and partials out by batch and KV heads, so a workspace of theirs
 * serves calls of one batch and head count (with fd_append_paged* and
 * fd_copy_pages, which use the header alone); zero it again before another use.
 * fd_decode_shared* of any plans, fd_fork_pages, fd_compact_pages, fd_append_paged*
 * and fd_copy_pages may all share one that is large enough for each.
 *
 * Launches: the kernels are launched with programmatic stream serialisation:
 * each may begin launching while the previous grid in the stream finishes,
 * and waits for that grid to complete before it reads or writes global
 * memory, so stream order is kept.  Two exceptions change no result.  Before
 * that wait, the split kernel of a long split may prefetch the split's
 * first K/V rows into L2 (a hint), and the paged one reads the page list
 * through L2 to aim those prefetches; every value it computes is read after the
 * wait.  And within a call of fd_decode_shared*, the prefixes' kernel starts once
 * the suffixes' kernel is past its wait, so that all that was written before the
 * call is there: it reads its inputs and writes its own partials while that kernel
 * runs, and ends after it.  The merge kernel behind it reads the prefixes' tables
 * before its wait.
 */
#ifndef FD_H
#define FD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fd_status {
    FD_OK = 0,
    FD_ERR_INVALID_ARG = -1,   /* bad pointer, size, layout or indptr */
    FD_ERR_UNSUPPORTED = -2,   /* head_dim or group size not built */
    FD_ERR_WORKSPACE = -3,     /* workspace missing or too small */
    FD_ERR_CUDA = -4,          /* a CUDA runtime call or launch failed */
    FD_ERR_TIMEOUT = -5,       /* an in-kernel wait ran past its limit */
    FD_ERR_DEVICE_BOUNDS = -6, /* a kernel derived an index outside the plan */
    FD_ERR_NO_PAGES = -7       /* a page operation found too few free pages */
} fd_status;

/* Keys per pipeline stage; every chunk length is a multiple of it. */
#define FD_TILE_TOKENS 32
/* Bytes at the start of every workspace reserved for the device status. */
#define FD_WORKSPACE_HEADER_BYTES 256
/* Default bound on each in-kernel wait, in nanoseconds. */
#define FD_DEFAULT_TIMEOUT_NS 1000000000LL

/*
 * A decode plan (plain data; fill it with fd_plan).
 *
 * The plan fixes one chunk length C for the step.  Request b (L_b keys) is cut
 * into splits_b = ceil(L_b / C) splits of equal length rounded up to a
 * multiple of FD_TILE_TOKENS (the last one ragged); each (split, KV head) is
 * one CTA of the split kernel.  The kernels re-derive each CTA's key range
 * from kv_indptr on the device with this same rule, so no per-step work list
 * is copied to the GPU.
 */
typedef struct fd_plan_info {
    int32_t batch;
    int32_t num_qo_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t group_size;        /* num_qo_heads / num_kv_heads */
    int32_t chunk;             /* max keys per split, multiple of FD_TILE_TOKENS */
    int32_t total_splits;      /* sum over requests of splits_b */
    int32_t max_splits;        /* max over requests of splits_b */
    int32_t num_work;          /* split-kernel CTAs = total_splits * num_kv_heads */
    int32_t num_partial_rows;  /* total_splits * num_qo_heads */
    int32_t num_sms;           /* SM count the chunk was chosen for */
    int32_t ctas_per_sm;       /* target CTAs per SM the chunk was chosen for */
    int64_t total_tokens;      /* kv_indptr[batch] */
    int64_t workspace_bytes;   /* workspace fd_decode needs for this plan */
    int64_t timeout_ns;        /* limit on each in-kernel wait; 0 makes every
                                  wait give up at once (a test hook: the call
                                  then reports FD_ERR_TIMEOUT) */
} fd_plan_info;

/* Human-readable name of a status code (static string). */
const char *fd_status_string(int status);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
int fd_version(void);

/* SM count of a CUDA device (cached after the first query). */
int fd_num_sms(int device, int *num_sms);

/*
 * fd_plan -- choose the chunk length and size the split grid (host only, no
 * CUDA call unless num_sms == 0).
 *
 * Article §2 (split grid = batch x heads x chunks) and §6 (chunk size tuning
 * guide: enough CTAs to fill the SMs, chunks not so small that the stage-2
 * reduction dominates, adapted to the load).  With chunk == 0 the plan tries
 *     C_w = max(FD_MIN_CHUNK, roundup(ceil(T * Hkv / (w * num_sms * ctas_per_sm)), FD_TILE_TOKENS))
 * for w = 1, 2, 4, 8 waves of resident CTAs, simulates how the hardware would
 * dispatch each grid in launch order onto num_sms * ctas_per_sm slots (per-CTA
 * cost = its 32-key tiles + a fixed overhead), and keeps the shortest.  Even
 * batches get one wave; ragged ones get smaller chunks that balance the
 * slots.  chunk > 0 forces C (must be a positive multiple of FD_TILE_TOKENS).
 *
 * kv_indptr_host: host int32 [batch+1].  num_sms: 0 = query the current
 * device.  ctas_per_sm: resident CTAs per SM; 0 = what the split kernel's
 * launch shape fits (2).  Writes *info; returns
 * FD_ERR_INVALID_ARG for a malformed indptr or head counts,
 * FD_ERR_UNSUPPORTED for an unsupported head_dim or group size.
 */
#define FD_MIN_CHUNK 128
int fd_plan(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
            const int32_t *kv_indptr_host, int num_sms, int ctas_per_sm, int chunk,
            fd_plan_info *info);

/*
 * fd_plan_work_items -- list the plan's CTAs in launch order (host only).
 * items: caller-owned host int32 [num_work][5] = (b, kv_head, split,
 * tok_begin, tok_end) with absolute key rows [tok_begin, tok_end).
 * capacity: rows available in items; FD_ERR_INVALID_ARG if too small.
 */
int fd_plan_work_items(const fd_plan_info *info, const int32_t *kv_indptr_host,
                       int32_t *items, int64_t capacity);

/*
 * fd_decode_split -- stage 1 (article §3, "local chunk computation"): one CTA
 * per (split, KV head) streams its keys once through shared memory (TMA,
 * multi-stage mbarrier pipeline), and for each of the G query heads that share
 * the KV head computes the local max, the local exp-sum and the local
 * probability-weighted sum of V.  It stores the partial in normalised form,
 *     partial_o   = (sum_j exp(s_j - m) V_j) / (sum_j exp(s_j - m))
 *     partial_lse = m + ln(sum_j exp(s_j - m)),
 * which carries the same information as the article's (output, max, sum).
 *
 * info: from fd_plan for this kv_indptr.  kv_indptr_dev: device copy of the
 * same indptr.  scale: softmax scale (applied to q.k).  workspace: device,
 * >= FD_WORKSPACE_HEADER_BYTES (status word, work counter).
 */
int fd_decode_split(const fd_plan_info *info, const void *q, const void *k,
                    const void *v, const int32_t *kv_indptr_dev, float scale,
                    float *partial_o, float *partial_lse, void *workspace,
                    int64_t workspace_bytes, void *stream);

/*
 * fd_merge -- stage 2 (article §3, "global reduction"): for each (b, hq) take
 * M = max_i partial_lse_i, weights w_i = exp(partial_lse_i - M), and write
 *     o = sum_i w_i partial_o_i / sum_i w_i,   lse = M + ln sum_i w_i.
 * A request with no keys gets o = 0, lse = -inf.
 */
int fd_merge(const fd_plan_info *info, const int32_t *kv_indptr_dev,
             const float *partial_o, const float *partial_lse, float *o, float *lse,
             void *workspace, int64_t workspace_bytes, void *stream);

/*
 * fd_decode -- plan (default chunking for the current device), stage 1 and
 * stage 2 in one call.  Stage 2 is fused into the split kernel: the CTA that
 * finishes a (request, KV head) group last (a ticket in the workspace) merges
 * the group's partials with the same arithmetic as fd_merge, and a request
 * with a single split writes O and LSE directly.  The partials live in the
 * workspace, which must hold fd_plan_info.workspace_bytes (FD_ERR_WORKSPACE
 * otherwise; query it with fd_plan for the same arguments).  Needs kv_indptr
 * on the host (for the plan) and on the device (for the kernels); the two must
 * hold the same values.
 */
int fd_decode(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
              const int32_t *kv_indptr_host, const int32_t *kv_indptr_dev,
              const void *q, const void *k, const void *v, float scale,
              float *o, float *lse, void *workspace, int64_t workspace_bytes,
              void *stream);

/*
 * Paged KV cache -- FD++ §6 ("vLLM and TensorRT-LLM integration"): the engine
 * keeps K/V in fixed-size physical pages from a page table, and each split
 * chunk streams the pages its keys fall in.
 *
 * Layout:
 *     k_pages, v_pages      bf16  [num_pages, page_size, Hkv, D]   page pools
 *     kv_page_indptr        int32 [B+1]   request b owns page-list entries
 *                                          kv_page_indptr[b] .. kv_page_indptr[b+1]-1
 *     kv_page_indices       int32 [kv_page_indptr[B]]   physical page of each entry
 *     kv_last_page_len      int32 [B]     keys in request b's last page, 1..page_size
 * Request b's keys are, in order, rows 0..page_size-1 of its pages, the last
 * page filled to kv_last_page_len[b]; it has (pages_b - 1) * page_size +
 * kv_last_page_len[b] keys (0 with no pages).  page_size must be a positive
 * multiple of 16 (FD_ERR_UNSUPPORTED otherwise).  A page index outside
 * [0, num_pages) sets FD_ERR_DEVICE_BOUNDS in the status word (the page is not
 * read).
 */

/*
 * fd_plan_paged -- fd_plan for a paged layout: the same chunking on the
 * requests' key counts (host only).  Sizes the fd_decode_paged workspace.
 */
int fd_plan_paged(int batch, int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                  const int32_t *kv_page_indptr_host, const int32_t *kv_last_page_len_host,
                  int num_sms, int ctas_per_sm, int chunk, fd_plan_info *info);

/*
 * fd_decode_paged -- fd_decode over a paged KV cache: plan, stage 1 with each
 * 32-key tile copied from the page it lies in (TMA boxes never cross a page),
 * stage 2 fused.  kv_page_indptr and kv_last_page_len are given on the host
 * (for the plan) and on the device (for the kernels) with the same values;
 * kv_page_indices on the device.  Workspace as fd_decode, sized by
 * fd_plan_paged.
 */
int fd_decode_paged(int batch, int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                    int num_pages, const int32_t *kv_page_indptr_host,
                    const int32_t *kv_last_page_len_host, const int32_t *kv_page_indptr_dev,
                    const int32_t *kv_last_page_len_dev, const int32_t *kv_page_indices_dev,
                    const void *q, const void *k_pages, const void *v_pages, float scale,
                    float *o, float *lse, void *workspace, int64_t workspace_bytes,
                    void *stream);

/*
 * FP8 (E4M3) KV cache -- FD++ §4 ("quantisation-friendly kernel fusion"): the
 * quantised K and V are read from HBM as they are and dequantised on chip, in
 * registers, straight into the tensor-core operands, so the stream moves half
 * the bytes of bf16.
 *
 * Layout: K and V hold one OCP FP8 E4M3 byte per value (1 sign, 4 exponent
 * bits with bias 7, 3 mantissa bits; no infinities) in the same shapes as the
 * bf16 entry points ([T, Hkv, D] ragged, [num_pages, page_size, Hkv, D]
 * paged).  k_scale and v_scale (device, fp32 [Hkv]) give each KV head's
 * scale: the value of a K byte is E4M3(byte) * k_scale[head], and likewise
 * for V.  q stays bf16 and O, LSE fp32.  The arithmetic matches the bf16 path
 * (every E4M3 value is exact in f16, the products accumulate in fp32); the
 * result is attention over the dequantised K and V.  Byte 0x7F / 0xFF (NaN)
 * propagates as NaN.  Workspace and plan as for fd_decode / fd_decode_paged.
 */
int fd_decode_fp8(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                  const int32_t *kv_indptr_host, const int32_t *kv_indptr_dev,
                  const void *q, const void *k_fp8, const void *v_fp8,
                  const float *k_scale, const float *v_scale, float scale,
                  float *o, float *lse, void *workspace, int64_t workspace_bytes,
                  void *stream);

int fd_decode_paged_fp8(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                        int page_size, int num_pages, const int32_t *kv_page_indptr_host,
                        const int32_t *kv_last_page_len_host, const int32_t *kv_page_indptr_dev,
                        const int32_t *kv_last_page_len_dev, const int32_t *kv_page_indices_dev,
                        const void *q, const void *k_pages_fp8, const void *v_pages_fp8,
                        const float *k_scale, const float *v_scale, float scale,
                        float *o, float *lse, void *workspace, int64_t workspace_bytes,
                        void *stream);

/*
 * INT4 KV cache -- FD++ §4 names INT4 beside FP8: the packed codes are read
 * from HBM as they are and widened on chip, in registers, into the
 * tensor-core operands, so the stream moves about a quarter of the bytes of
 * bf16.  The page fixes no INT4 format; this is the plainest one that keeps a
 * head's values on a common scale per key: symmetric codes, one scale per
 * (key row, KV head).
 *
 * Layout: K and V hold head_dim / 2 bytes per (row, KV head): [T, Hkv, D/2]
 * ragged, [num_pages, page_size, Hkv, D/2] paged.  Byte j of a row holds
 * element 2j in its low nibble and element 2j + 1 in its high nibble, each a
 * four-bit two's-complement code c in -8..7.  k_scale and v_scale (device,
 * fp32) are head-major: [Hkv][rows], rows = T (ragged) or
 * num_pages * page_size (paged; entry h * rows + p * page_size + r belongs to
 * row r of page p).  The value of a K element is c * k_scale[h][row], and
 * likewise for V.  q stays bf16 and O, LSE fp32; the result is attention over
 * the dequantised K and V (the codes widen to f16 exactly and each q row is
 * scaled into f16 by a power of two, as for FP8; each row's K scale multiplies
 * its logit in fp32, and its V scale its softmax weight, which enters P V as
 * an f16 hi + lo pair after division by a power of two that bounds the V
 * scales seen so far, so scales of any finite magnitude keep the path's
 * relative accuracy).  A scale of +-inf or NaN propagates (as NaN); the scales
 * of rows past a request's last key (the rest of its last page) are never
 * used.  Workspace and plan as for fd_decode / fd_decode_paged.
 */
int fd_decode_int4(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                   const int32_t *kv_indptr_host, const int32_t *kv_indptr_dev,
                   const void *q, const void *k_int4, const void *v_int4,
                   const float *k_scale, const float *v_scale, float scale,
                   float *o, float *lse, void *workspace, int64_t workspace_bytes,
                   void *stream);

int fd_decode_paged_int4(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                         int page_size, int num_pages, const int32_t *kv_page_indptr_host,
                         const int32_t *kv_last_page_len_host, const int32_t *kv_page_indptr_dev,
                         const int32_t *kv_last_page_len_dev, const int32_t *kv_page_indices_dev,
                         const void *q, const void *k_pages_int4, const void *v_pages_int4,
                         const float *k_scale, const float *v_scale, float scale,
                         float *o, float *lse, void *workspace, int64_t workspace_bytes,
                         void *stream);

/*
 * Graph-capturable decode -- for engines that run decode steps as CUDA graphs
 * with a fixed batch (FD++ §6 integration).  fd_decode plans on the host from
 * the host copy of kv_indptr on every call, which a graph replay cannot
 * repeat.  Here the plan is made once for a capacity, and each call takes
 * device data only, so it can be captured in a CUDA graph and replayed with
 * new lengths written to the device indptr between replays.
 *
 * fd_plan_graph -- host only.  Fixes the chunk length (`chunk`, or 0 for the
 * planner's choice for max_total_tokens keys spread evenly over the batch) and
 * sizes the plan for any kv_indptr with kv_indptr[batch] <= max_total_tokens:
 * at most floor(max_total_tokens / chunk) + batch splits.  info->workspace_bytes
 * is the workspace fd_decode_graph needs.
 *
 * fd_decode_graph -- plan + stage 1 with stage 2 fused, the split of every
 * request derived on the device from kv_indptr_dev (same split rule as
 * fd_plan for that chunk; an empty request gives O = 0, LSE = -inf).  Reads no
 * host memory and makes no host-synchronising call, so it may be captured.
 * K and V must hold at least max_total_tokens rows.  A device indptr beyond the
 * capacity sets FD_ERR_DEVICE_BOUNDS in the status word.  Workspace as
 * fd_decode (zero-filled once, reused across replays on one stream).
 */
int fd_plan_graph(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                  int64_t max_total_tokens, int num_sms, int chunk, fd_plan_info *info);

int fd_decode_graph(const fd_plan_info *info, const int32_t *kv_indptr_dev,
                    const void *q, const void *k, const void *v, float scale,
                    float *o, float *lse, void *workspace, int64_t workspace_bytes,
                    void *stream);

/*
 * fd_merge_states -- the merge of attention states computed over disjoint
 * parts of the same keys: the exchange step of sequence sharding (one
 * request's keys cut into contiguous shards on several GPUs, each running
 * fd_decode on its shard; the per-shard O and LSE are gathered and merged
 * here).  FD++ §3 stage 2: the same global reduction, now across shards.
 *
 * For each row r: M = max_s lse_states[s][r], w_s = exp(lse_states[s][r] - M),
 * o[r] = sum_s w_s o_states[s][r] / sum_s w_s, lse[r] = M + ln sum_s w_s; a
 * row whose states are all -inf (no keys in any shard) gets o = 0, lse = -inf.
 * o_states fp32 [num_states, rows, head_dim], lse_states fp32 [num_states,
 * rows], o [rows, head_dim], lse [rows], all on the device; rows = B * Hq.
 */
int fd_merge_states(int num_states, int rows, int head_dim, const float *o_states,
                    const float *lse_states, float *o, float *lse, void *stream);

/*
 * fd_decode_static_workspace -- fd_decode for callers that cannot allocate.
 *
 * The article has no counterpart: this is a library convenience.  Some
 * callers run decode attention where they must not allocate device memory:
 * the enqueue step of an inference-engine plugin, a runtime whose memory is
 * planned up front and owned by someone else, code that may not grow the
 * process's footprint.  This entry point needs only the inputs and outputs.
 * Its scratch (status word, merge tickets, split partials) is a fixed device
 * array of FD_STATIC_WORKSPACE_BYTES inside the library, which every GPU that
 * loads the library holds until the process exits; it calls no cudaMalloc,
 * cudaFree or other allocating routine.
 *
 * Arguments and results as fd_decode, without the workspace.  Returns
 * FD_ERR_WORKSPACE, before touching the GPU, when the plan for these
 * arguments needs more than FD_STATIC_WORKSPACE_BYTES (fd_plan reports the
 * need in fd_plan_info.workspace_bytes); use fd_decode with a workspace then.
 * The first call on a device looks up the array's device address with that
 * device current and caches it for the life of the process; make that first
 * call before any stream capture.  The cached address does not survive
 * cudaDeviceReset (or any other teardown of the device's primary context):
 * after one, this entry point must not be called again in the process.  Each call
 * clears the workspace header and the merge tickets on its stream before it runs.
 * All calls share the one array, which keeps the last call's contents: calls
 * that can overlap on the GPU (other streams, other host threads, without
 * ordering between them) race and give wrong results.  The status word is
 * not reachable from outside the library, so errors the kernels detect are
 * not reported by this entry point.
 */
#define FD_STATIC_WORKSPACE_BYTES (16 << 20)
int fd_decode_static_workspace(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                               const int32_t *kv_indptr_host, const int32_t *kv_indptr_dev,
                               const void *q, const void *k, const void *v, float scale,
                               float *o, float *lse, void *stream);

/*
 * ---- Decode attention over shared prefixes ----
 *
 * For a batch whose requests share long prefixes (a system prompt, a document,
 * samples of one prompt): each prefix's keys are read and attended once for all
 * of its requests, each request's own keys (its suffix) as in fd_decode, and
 * the two states are merged by LSE.  The result is fd_decode's over the prefix
 * followed by the suffix.
 *
 * Layout: consecutive requests share a prefix.  prefix_req_indptr int32 [P+1]:
 * prefix g's requests are prefix_req_indptr[g] .. prefix_req_indptr[g+1]-1; it
 * starts at 0 and ends at the batch, so a request without a prefix sits under
 * one of no keys.
 *   ragged  k_prefix, v_prefix bf16 [Tp, Hkv, D], prefix g's keys are rows
 *           prefix_indptr[g] .. prefix_indptr[g+1]-1; k, v and kv_indptr hold the
 *           suffixes, as for fd_decode
 *   paged   prefix g's pages are prefix_page_indices[prefix_page_indptr[g] ..],
 *           the last one filled to prefix_last_page_len[g]; the suffixes' tables
 *           kv_page_indptr, kv_last_page_len, kv_page_indices, as for
 *           fd_decode_paged; all in the same page pools
 *
 * The plan is made once on the host for the prefixes and a room for suffix
 * keys; a call takes device data only, makes no host-synchronising call and may
 * be captured in a CUDA graph.  Replays see the suffixes' current lengths; the
 * prefixes' tables must hold what the plan was made for.
 */
typedef struct fd_shared_plan {
    fd_plan_info suffix;       /* the requests' own keys (as fd_plan_graph) */
    int32_t num_prefixes;
    int32_t chunk;             /* max prefix keys per split, a multiple of 128 */
    int32_t num_items;         /* CTAs over the prefixes */
    int32_t num_partial_rows;  /* partial (O, LSE) rows over the prefixes */
    int32_t page_size;         /* 0: ragged */
    int32_t reserved;
    int64_t prefix_rows;       /* prefix_indptr[P]: key rows or page-list entries */
    int64_t workspace_bytes;   /* workspace a call needs (zero-filled once) */
    int64_t timeout_ns;        /* as in fd_plan_info */
} fd_shared_plan;

/*
 * fd_plan_shared, fd_plan_shared_paged -- host only (no CUDA call unless
 * num_sms == 0).  max_suffix_tokens: room for the requests' own keys, all
 * together; 0: there are none (k, v and the suffix tables may then be NULL).
 * chunk: 0, or the chunk length to use (a multiple of 128).
 */
int fd_plan_shared(int batch, int num_qo_heads, int num_kv_heads, int head_dim, int num_prefixes,
                   const int32_t *prefix_req_indptr_host, const int32_t *prefix_indptr_host,
                   int64_t max_suffix_tokens, int num_sms, int chunk, fd_shared_plan *plan);

int fd_plan_shared_paged(int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                         int page_size, int num_prefixes, const int32_t *prefix_req_indptr_host,
                         const int32_t *prefix_page_indptr_host,
                         const int32_t *prefix_last_page_len_host, int64_t max_suffix_tokens,
                         int num_sms, int chunk, fd_shared_plan *plan);

/*
 * fd_decode_shared, fd_decode_shared_paged -- one decode step.  Ragged: k and v
 * must hold max_suffix_tokens rows.  scale must be finite.  A request without any
 * key gets O = 0, LSE = -inf.  More suffix keys than the plan's room (any, in
 * suffix tables that are given to a plan without room), prefix tables beyond it, or a page outside [0, num_pages) set FD_ERR_DEVICE_BOUNDS
 * (the outputs are then not valid).  num_page_entries: entries of
 * kv_page_indices.  O adds up in fp32 with weights of up to 2^40: V of up to 2^80
 * in magnitude.  The weights enter the product with V as two 16-bit parts, as in
 * fd_decode, which leaves 2e-6 of O in the 2-norm, up to 6e-6 with long prefixes.  Workspace: zeroed once, calls that share it in the order of one
 * stream; calls of other plans and the page operators below may be among them.
 */
int fd_decode_shared(const fd_shared_plan *plan, const int32_t *prefix_req_indptr_dev,
                     const int32_t *prefix_indptr_dev, const int32_t *kv_indptr_dev, const void *q,
                     const void *k_prefix, const void *v_prefix, const void *k, const void *v,
                     float scale, float *o, float *lse, void *workspace, int64_t workspace_bytes,
                     void *stream);

int fd_decode_shared_paged(const fd_shared_plan *plan, int num_pages,
                           const int32_t *prefix_req_indptr_dev,
                           const int32_t *prefix_page_indptr_dev,
                           const int32_t *prefix_last_page_len_dev,
                           const int32_t *prefix_page_indices_dev,
                           const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
                           const int32_t *kv_page_indices_dev, int num_page_entries, const void *q,
                           const void *k_pages, const void *v_pages, float scale, float *o,
                           float *lse, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * fd_decode_shared_fp8, fd_decode_shared_paged_fp8 -- the same over E4M3 K/V
 * (prefixes and suffixes), with the scales of fd_decode_fp8.  The bytes widen to
 * f16 exactly; byte 0x7F / 0xFF (NaN) propagates as NaN.
 */
int fd_decode_shared_fp8(const fd_shared_plan *plan, const int32_t *prefix_req_indptr_dev,
                     const int32_t *prefix_indptr_dev, const int32_t *kv_indptr_dev, const void *q,
                     const void *k_prefix_fp8, const void *v_prefix_fp8, const void *k, const void *v,
                     const float *k_scale, const float *v_scale, float scale, float *o, float *lse,
                     void *workspace, int64_t workspace_bytes, void *stream);

int fd_decode_shared_paged_fp8(const fd_shared_plan *plan, int num_pages,
                           const int32_t *prefix_req_indptr_dev,
                           const int32_t *prefix_page_indptr_dev,
                           const int32_t *prefix_last_page_len_dev,
                           const int32_t *prefix_page_indices_dev,
                           const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
                           const int32_t *kv_page_indices_dev, int num_page_entries, const void *q,
                           const void *k_pages_fp8, const void *v_pages_fp8, const float *k_scale,
                           const float *v_scale, float scale, float *o,
                           float *lse, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * ---- Writing and rearranging a paged cache ----
 *
 * What a serving step does to the cache around fd_decode_paged: it writes the
 * new keys and values (with their rotary positions), makes the next step's
 * page tables, and from time to time moves the pages together.  All of these
 * take device data and host sizes only, launch on the given stream, make no
 * host-synchronising call and may be captured in a CUDA graph.  Their errors on
 * the device go to the status word of the workspace (fd_get_device_status).
 */

/* How fd_plan_rope scales the frequencies f_i = base^(-2 i / rotary_dim). */
#define FD_ROPE_PLAIN 0
#define FD_ROPE_LINEAR 1   /* f / factor */
#define FD_ROPE_BANDS 2    /* f where it makes more than `high` turns over trained_len
                              positions, f / factor below `low` turns, a linear
                              ramp in the number of turns between */
#define FD_ROPE_YARN 3     /* YaRN: f up to the pair that makes `high` turns over
                              trained_len, f / factor from the one that makes `low`
                              (both rounded outwards), a linear ramp in the pair
                              index between; cos and sin times 0.1 ln(factor) + 1 */

typedef struct fd_rope_config {
    double base;               /* >= 1 */
    double factor;             /* >= 1; not read for FD_ROPE_PLAIN */
    double trained_len;        /* FD_ROPE_BANDS and FD_ROPE_YARN, as are: */
    double low, high;          /* turns, low < high (YaRN's usual ones are 1 and 32) */
    int32_t scaling;           /* FD_ROPE_* */
    int32_t interleaved;       /* pairs (2i, 2i + 1); else (i, i + rotary_dim / 2) */
} fd_rope_config;

/*
 * Rotary positions of a model (plain data; fill it with fd_plan_rope).  Pair i
 * of a head's first rotary_dim values turns by position * f_i; step[i] is f_i
 * in turns, times 2^64, so that the angle of any 32-bit position is exact to
 * the rounding of f_i in 64 bits.
 */
typedef struct fd_rope_info {
    int32_t head_dim;
    int32_t rotary_dim;        /* values of a head that turn, from its start */
    int32_t interleaved;       /* as in the config */
    float gain;                /* factor of cos and sin */
    uint64_t step[64];
} fd_rope_info;

/*
 * fd_plan_rope -- the rotary frequencies (host only, no CUDA call).
 * rotary_dim: a multiple of 16 up to head_dim (128).
 */
int fd_plan_rope(int head_dim, int rotary_dim, const fd_rope_config *config, fd_rope_info *info);

/*
 * fd_append_paged -- one call per step and layer before decode: rotate the new
 * queries and keys and write the new keys and values into the paged cache.
 *
 *     q, k, v        bf16 [num_tokens, heads, D], heads contiguous, any token
 *                    stride (elements, a multiple of 8, at least heads * D), so
 *                    they may be parts of one fused projection
 *     q_out          bf16, the rotated queries; q itself is allowed (with its
 *                    stride), and rows between those of q, k and v (with theirs);
 *                    other memory within theirs is not
 *     append_indptr  int32 [B+1]  request b's new tokens are rows
 *                    append_indptr[b] .. append_indptr[b+1]-1
 *     kv_page_indptr, kv_last_page_len, kv_page_indices   the page tables with
 *                    the new keys counted in: request b's new keys are the
 *                    last ones of its table
 *     positions      int32 [num_tokens] position of each token, or NULL: the
 *                    token's key index in its table (keys behind a shared prefix
 *                    that is not in the table need positions)
 * rope: NULL for no rotation.  num_qo_heads may be 0 (no queries).
 * num_page_entries: entries of kv_page_indices.  Tokens from append_indptr[B]
 * on (a padded batch) are left alone, in q_out and in the cache.  A token whose
 * key or page lies outside the tables or the pool is skipped and sets
 * FD_ERR_DEVICE_BOUNDS.  Rotation is in fp32; each output is rounded once.
 * Two tokens of a call must not have the same key.  workspace: at least
 * FD_WORKSPACE_HEADER_BYTES.
 *
 * fd_append_paged_fp8: E4M3(value / scale[head]), nearest even, saturated at
 * +-448 (k_scale, v_scale as in fd_decode_paged_fp8, read).
 * fd_append_paged_int4: codes round(value / scale) in -8..7 with scale = the
 * row's largest magnitude / 7 (1 for a row of zeros, NaN for a row with one),
 * stored in k_scale, v_scale [Hkv][num_pages * page_size] (written).
 */
int fd_append_paged(int batch, int num_tokens, int num_qo_heads, int num_kv_heads, int head_dim,
                    int page_size, int num_pages, const fd_rope_info *rope, const void *q,
                    int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                    int64_t v_stride, const int32_t *append_indptr_dev,
                    const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
                    const int32_t *kv_page_indices_dev, int num_page_entries,
                    const int32_t *positions_dev, void *q_out, int64_t q_out_stride, void *k_pages,
                    void *v_pages, void *workspace, int64_t workspace_bytes, void *stream);

int fd_append_paged_fp8(int batch, int num_tokens, int num_qo_heads, int num_kv_heads, int head_dim,
                        int page_size, int num_pages, const fd_rope_info *rope, const void *q,
                        int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                        int64_t v_stride, const int32_t *append_indptr_dev,
                        const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
                        const int32_t *kv_page_indices_dev, int num_page_entries,
                        const int32_t *positions_dev, void *q_out, int64_t q_out_stride,
                        void *k_pages_fp8, void *v_pages_fp8, const float *k_scale,
                        const float *v_scale, void *workspace, int64_t workspace_bytes,
                        void *stream);

int fd_append_paged_int4(int batch, int num_tokens, int num_qo_heads, int num_kv_heads,
                         int head_dim, int page_size, int num_pages, const fd_rope_info *rope,
                         const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, const int32_t *append_indptr_dev,
                         const int32_t *kv_page_indptr_dev, const int32_t *kv_last_page_len_dev,
                         const int32_t *kv_page_indices_dev, int num_page_entries,
                         const int32_t *positions_dev, void *q_out, int64_t q_out_stride,
                         void *k_pages_int4, void *v_pages_int4, float *k_scale, float *v_scale,
                         void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Page tables on the device.  page_refs int32 [num_pages] counts how many
 * table entries (of these tables, or of others the program keeps, such as a
 * shared prefix's) hold each page; 0 is a free page.  fd_fork_pages and
 * fd_compact_pages make the next tables and counts and list the page copies
 * they need; fd_copy_pages makes those copies in every pool (K and V of every
 * layer) at once.  new_page_refs may be page_refs itself; otherwise they share no
 * memory.  num_pages is at most (2^31 - 1) / 16.
 *
 * fd_pages_workspace_bytes -- the workspace of a fork or compaction (host
 * only).  new_batch: the fork's, 0 for a compaction.  For these calls alone the
 * workspace need not be zeroed beyond its header; one that is shared with
 * fd_decode_shared* is zeroed whole, once.
 */
int fd_pages_workspace_bytes(int num_pages, int new_batch, int64_t *bytes);

/*
 * fd_fork_pages -- the page tables of the next step: requests that fork (beams,
 * several samples of a prompt), go on, start or end.
 *
 * Request i of the new batch goes on from request parent[i] of the old one (-1:
 * a new request); an old request that is nobody's parent ends.
 * new_page_indptr [new_batch+1] gives the new tables' sizes: each child has at
 * least its parent's pages.  Its first entries are its parent's, the rest are
 * fresh pages.  A partly filled last page of the parent (kv_last_page_len <
 * page_size) goes on in the lowest child of that parent if its count is 1; every
 * other child gets a fresh page in its place and copy_src[i] -> copy_dst[i] is
 * the copy it needs (-1, -1: none).  Fresh pages are the lowest free ones, in
 * the order of the new tables' entries; pages that this call sets free are not
 * among them.  new_page_refs = page_refs minus the old entries plus the new.
 * Entries of new_page_indices that no table has (new_page_entries may be more
 * than new_page_indptr[new_batch], as in a captured call) become -1.
 *
 * With too few free pages (FD_ERR_NO_PAGES), or a parent, table or tail page
 * outside the arguments' ranges (FD_ERR_DEVICE_BOUNDS), nothing changes:
 * new_page_refs = page_refs, and the new indices and copies are -1.  Other page
 * ids outside the pool set FD_ERR_DEVICE_BOUNDS and become -1.
 * old_batch and new_batch up to 32768 (FD_ERR_UNSUPPORTED above).
 * kv_page_indices and new_page_indices must not share memory.
 */
int fd_fork_pages(int old_batch, int new_batch, int page_size, int num_pages,
                  const int32_t *parent_dev, const int32_t *kv_page_indptr_dev,
                  const int32_t *kv_last_page_len_dev, const int32_t *kv_page_indices_dev,
                  int num_page_entries, const int32_t *new_page_indptr_dev, int new_page_entries,
                  const int32_t *page_refs_dev, int32_t *new_page_indices_dev,
                  int32_t *new_page_refs_dev, int32_t *copy_src_dev, int32_t *copy_dst_dev,
                  void *workspace, int64_t workspace_bytes, void *stream);

/*
 * fd_compact_pages -- move the pages in use to the front of the pool.
 *
 * The pages in use at or behind `limit` (0: the number of pages in use, a full
 * compaction) move, in order, to the free pages before it, in order.
 * copy_src[r] -> copy_dst[r] is the r-th move (-1, -1 past the last), of at most
 * max_moves; the number of pages in use and that of free ones both bound it.
 * new_page_indices is kv_page_indices (every table of the pool, concatenated)
 * with the moved pages renamed; it may be the same array (in part: refused).
 * Entries of -1 (no page) stay; other ids outside the pool stay too and set
 * FD_ERR_DEVICE_BOUNDS.  With more moves than free pages before the limit or
 * than max_moves, nothing changes (FD_ERR_NO_PAGES) and the copies are -1.
 */
int fd_compact_pages(int num_pages, const int32_t *page_refs_dev,
                     const int32_t *kv_page_indices_dev, int num_page_entries, int limit,
                     int max_moves, int32_t *new_page_indices_dev, int32_t *new_page_refs_dev,
                     int32_t *copy_src_dev, int32_t *copy_dst_dev, void *workspace,
                     int64_t workspace_bytes, void *stream);

/*
 * fd_copy_pages -- copy page src[i] to page dst[i] (i < num_copies, device
 * lists; src[i] < 0: none) within each of num_pools pools.  pools (host array of
 * device pointers, 16-byte aligned): pool j holds num_pages pages of
 * page_bytes[j] bytes (a multiple of 16).  An INT4 cache's scales are
 * num_kv_heads pools each, of page_size * 4 bytes a page.  num_copies times the
 * 16 KB segments of a page is at most 2^31 - 1.  No page may be both a
 * source and a destination, nor a destination twice (the lists of fork and
 * compact never hold such a pair); what lands in one that is, is undefined.  Ids
 * outside the pool are skipped and set FD_ERR_DEVICE_BOUNDS (workspace may be
 * NULL: then only skipped).
 */
int fd_copy_pages(int num_pools, void *const *pools, const int64_t *page_bytes, int num_pages,
                  int num_copies, const int32_t *src_dev, const int32_t *dst_dev, void *workspace,
                  int64_t workspace_bytes, void *stream);

/*
 * fd_get_device_status -- synchronise the stream, read and clear the status
 * word the kernels write into the workspace.  Returns FD_OK,
 * FD_ERR_TIMEOUT, FD_ERR_DEVICE_BOUNDS, FD_ERR_NO_PAGES, or FD_ERR_CUDA if the
 * read failed.
 */
int fd_get_device_status(void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FD_H */
