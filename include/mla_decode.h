/*
 * mla_decode.h -- C ABI of the Blackwell (sm_100a) MLA decoding library.
 *
 * Multi-head latent attention (MLA) decoding over a paged latent KV cache, in
 * the "MQA mode" of the upstream FlashMLA documentation ("MLA Mode" footnote to
 * the support matrix): every query head attends one shared latent KV head whose
 * cached rows are d_qk = 576 wide (512 latent columns, then 64 RoPE columns) or
 * d_qk = 512 wide (no RoPE part); V is the leading d_v = 512 columns of the same
 * rows.  Cached tokens sit in 64-token pages found through a block table.
 *
 * The call sequence is the one the "FlashMLA" usage page (deepep.org) shows:
 * mla_get_metadata once per decoding step (its result is reused by every
 * layer), then mla_decode_with_kvcache once per layer, which returns (o, lse).
 *
 * Conventions for every entry point:
 *   - Pointers named "device" are CUDA device pointers; "host" ones are host memory.
 *   - The caller allocates and owns every buffer.  The library allocates no
 *     memory and keeps no state between calls (apart from a per-process cache
 *     of one CUDA driver entry point and per-device kernel attributes set on
 *     first use).
 *   - Calls taking a stream enqueue work on it and return without
 *     synchronising; results are ready when the stream reaches that point.
 *     A stream of NULL means the legacy default stream.
 *   - Invalid arguments are rejected on the host before anything is enqueued;
 *     the return value says why (mla_status_string gives a message).
 *   - Errors that only the device can see (a block-table entry outside the
 *     cache, a pipeline wait that ran out of time) are recorded in a status
 *     word at the start of the workspace; mla_read_device_status reads it.
 *     The outputs of a call that recorded one are unspecified: rows may hold
 *     anything, including what they held before (a cluster that gave up, or a
 *     combine that stopped waiting once the status word was set, writes nothing).
 *
 * Array layouts (all row-major / C order):
 *   q             [batch, s_q, h_q, d_qk]             bf16 or fp16
 *   kvcache       [num_blocks, 64, h_kv, d_qk]        same dtype as q, or, with
 *                 [num_blocks, 64, h_kv, 656] bytes   dtype MLA_BF16_FP8KV, "FP8 with scale"
 *                                                     rows (see mla_dtype)
 *   block_table   [batch, max_blocks_per_seq] int32   physical page ids; only the
 *                                                     first ceil(L_b / 64) entries
 *                                                     of row b are read
 *   cache_seqlens [batch] int32                       L_b >= 0
 *   o             [batch, s_q, h_q, 512]              same dtype as q
 *   lse           [batch, s_q, h_q] float32           natural log
 *   tile_md       [num_parts, 8] int32                scheduler output (opaque)
 *   num_splits    [batch * row_groups + 1] int32      scheduler output, prefix sums
 */
#ifndef MLA_DECODE_H_
#define MLA_DECODE_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MLA_API __attribute__((visibility("default")))
#else
#define MLA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_PAGE_SIZE 64       /* tokens per KV-cache page ("block size of 64") */
#define MLA_HEAD_DIM_V 512     /* d_v: the latent width */
#define MLA_MD_INTS 8          /* int32 entries per row of tile_md */
#define MLA_ROWS_PER_GROUP 128 /* query rows (s_q * h_q) handled per row group */

typedef enum {
    MLA_OK = 0,
    MLA_ERR_INVALID_ARG = 1,  /* null pointer, negative size, misaligned buffer, ... */
    MLA_ERR_UNSUPPORTED = 2,  /* valid request this build does not implement */
    MLA_ERR_WORKSPACE = 3,    /* workspace smaller than mla_decode_workspace_bytes */
    MLA_ERR_CUDA = 4,         /* a CUDA runtime / driver call failed */
    MLA_ERR_TIMEOUT = 5,      /* device: a pipeline wait gave up (kernel returned early) */
    MLA_ERR_DEVICE_CHECK = 6  /* device: a needed block-table entry was outside [0, num_blocks),
                                 or a sequence needs more than max_blocks_per_seq pages */
} mla_status;

/*
 * Data types of a call.  MLA_BF16 / MLA_FP16: q, kvcache and o all of that type.
 * MLA_BF16_FP8KV: q and o bfloat16, kvcache in the "FP8 with scale" format of the
 * upstream FlashMLA documentation ("FP8 KV Cache" section): each token row is 656
 * bytes, 512 float8_e4m3 latent values, then 4 little-endian float32 scales (the
 * k-th for latent values [128k, 128k + 128)), then the 64 bfloat16 RoPE values
 * (not quantized); d_qk must be 576.  The kernel dequantizes each latent value to
 * bfloat16 as bf16(e4m3 * scale), the product in float32 rounded to nearest even,
 * and computes in bfloat16 as for a bfloat16 cache.
 */
typedef enum { MLA_BF16 = 0, MLA_FP16 = 1, MLA_BF16_FP8KV = 2 } mla_dtype;

/* Message for a status code; never NULL. */
MLA_API const char* mla_status_string(int status);

/*
 * Number of scheduler partitions for a device: one per pair of SMs (the
 * decode kernel runs one two-CTA cluster per partition).  On success writes
 * *num_parts (> 0).  Errors: MLA_ERR_INVALID_ARG (null), MLA_ERR_CUDA (no such
 * device).
 */
MLA_API mla_status mla_num_sm_parts(int device, int* num_parts);

/*
 * Sizes of the scheduler outputs for a problem: *tile_md_ints = num_parts * 8,
 * *num_splits_ints = batch * ceil(heads_per_kv / 128) + 1.
 * heads_per_kv = s_q * h_q / h_kv, as in get_mla_metadata's second argument.
 */
MLA_API mla_status mla_metadata_sizes(int batch, int heads_per_kv, int h_kv, int num_parts,
                              size_t* tile_md_ints, size_t* num_splits_ints);

/*
 * Tile scheduler ("FlashMLA" usage page: get_mla_metadata(cache_seqlens,
 * s_q * h_q // h_kv, h_kv) returns tile_scheduler_metadata and num_splits; the
 * page's Tile Scheduler "distributes work across GPU resources"; the upstream
 * FlashMLA documentation's "Usage / MLA Decoding" call also takes is_fp8).
 *
 * Splits the work -- for each request b and row group of 128 query rows, the
 * ceil(L_b / 64) pages of its cache plus a fixed per-chunk overhead -- into
 * num_parts contiguous ranges of nearly equal cost.  A (request, row group)
 * whose pages fall into more than one range is split; num_splits holds the
 * prefix sums of the split counts, and the decode call merges split results.
 *
 *   cache_seqlens    device [batch] int32
 *   heads_per_kv     s_q * h_q / h_kv (> 0)
 *   h_kv             number of KV heads (must be 1: MQA mode)
 *   num_parts        from mla_num_sm_parts (the same value must be passed to decode)
 *   is_fp8_kvcache   nonzero when the decode calls read an "FP8 with scale" cache:
 *                    its pages take longer, so a chunk's fixed overhead counts for
 *                    fewer pages (any schedule is valid for either cache; this one
 *                    balances the work better)
 *   tile_md          device [num_parts, 8] int32, written
 *   num_splits       device [batch * row_groups + 1] int32, written
 * Runs one small kernel on `stream`; no host synchronisation.
 */
MLA_API mla_status mla_get_metadata(const int32_t* cache_seqlens, int batch, int heads_per_kv, int h_kv,
                                    int num_parts, int is_fp8_kvcache, int32_t* tile_md, int32_t* num_splits,
                                    void* stream);

/* Same schedule computed on the host: every pointer is host memory. */
MLA_API mla_status mla_get_metadata_host(const int32_t* cache_seqlens, int batch, int heads_per_kv, int h_kv,
                                         int num_parts, int is_fp8_kvcache, int32_t* tile_md, int32_t* num_splits);

/*
 * Bytes of device workspace mla_decode_with_kvcache needs: a control block of
 * fixed size (the status word and two int32 counters for each of up to
 * MLA_MAX_VIRTUAL_BATCHES (request, row group) pairs), then float32 partial
 * outputs and LSEs for up to batch * row_groups + num_parts splits of 128 rows
 * each.  Returns 0 for invalid sizes, and for batch * row_groups above
 * MLA_MAX_VIRTUAL_BATCHES.
 *
 * mla_decode_workspace_zero_bytes returns the size of the control block (the
 * same for every problem).  It must be zero before a workspace is first used;
 * every call leaves its counters zero again, for every later call of any size:
 * the control block does not depend on the problem, so the partial results of
 * one call never land on the counters of another.  The status word keeps the
 * first device error until it is read with mla_read_device_status's clear flag;
 * meanwhile the workspace serves further calls.  (The two stages of a call:
 * the combine stage clears the counters.)
 *
 * Device errors.  MLA_ERR_DEVICE_CHECK: requests whose lengths and block-table
 * entries are in order get their results, in this call too; what the others get
 * is unspecified.  MLA_ERR_TIMEOUT: the rows that a cluster whose wait gave up
 * had still to do are unspecified (where they were split, not written); all
 * others are right.
 */
#define MLA_MAX_VIRTUAL_BATCHES 16384
MLA_API size_t mla_decode_workspace_bytes(int batch, int s_q, int h_q, int h_kv, int num_parts);
MLA_API size_t mla_decode_workspace_zero_bytes(int batch, int s_q, int h_q, int h_kv);

/*
 * Dense MLA decoding with a paged KV cache ("FlashMLA" usage page:
 * flash_mla_with_kvcache(q, kvcache, block_table, cache_seqlens, dv,
 * tile_scheduler_metadata, num_splits, causal) -> (o, lse); upstream FlashMLA
 * documentation, "Usage / MLA Decoding": lse is the log-sum-exp of the
 * attention scores per query head).
 *
 * For request b, query token s and head h (kv head 0):
 *   n      = causal ? clamp(L_b - s_q + 1 + s, 0, L_b) : L_b   (bottom-right mask)
 *   x_j    = softmax_scale * <q[b,s,h,:], k_j>,  k_j = cached row j (j < n)
 *   lse    = log(sum_j exp(x_j))                 (-inf when n = 0)
 *   o      = sum_j exp(x_j - lse) * k_j[0:512]   (0 when n = 0)
 *
 *   q, kvcache      device, dtype `dtype` (see mla_dtype), 16-byte aligned
 *   d_qk            576 or 512 (576 for MLA_BF16_FP8KV);  dv must be 512;  h_kv must be 1;
 *                   page_size must be 64
 *   block_table     device int32 [batch, max_blocks_per_seq]
 *   cache_seqlens   device int32 [batch]  (the same array given to mla_get_metadata)
 *   tile_md, num_splits, num_parts   from mla_get_metadata for this batch
 *   causal          0 or 1
 *   softmax_scale   > 0, or <= 0 for 1/sqrt(d_qk)
 *   active_heads    heads [0, active_heads) are real, heads [active_heads, h_q) are
 *                   padding ("FlashMLA vLLM Optimization" page, active-head switch: a
 *                   tensor-parallel rank's query is padded to h_q heads of which it
 *                   consumes only a few).  Padding heads are still computed inside the
 *                   MMA tiles, but their o and lse are left as they were and the
 *                   combine skips them.  A value that is not a multiple of 8 in
 *                   (0, h_q] (0 included), or an h_q that is not a multiple of 8,
 *                   means every head is real.
 *   o               device [batch, s_q, h_q, 512], dtype of q, 16-byte aligned, written
 *                   (real heads)
 *   lse             device float32 [batch, s_q, h_q], written (real heads)
 *   workspace       device, >= mla_decode_workspace_bytes(...), 256-byte aligned
 * Enqueues the split-KV kernel and the combine kernel on `stream`.  Calls
 * sharing one workspace must not run concurrently.
 */
MLA_API mla_status mla_decode_with_kvcache(const void* q, int batch, int s_q, int h_q, int d_qk,
                                   const void* kvcache, int num_blocks, int page_size, int h_kv,
                                   const int32_t* block_table, int max_blocks_per_seq,
                                   const int32_t* cache_seqlens, int dv, int dtype,
                                   const int32_t* tile_md, int num_parts,
                                   const int32_t* num_splits, int causal, float softmax_scale,
                                   int active_heads, void* o, float* lse, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * The same, with the call's device errors recorded in *device_status (device int32; the first error if it
 * holds 0) instead of the workspace's status word; null: as mla_decode_with_kvcache.
 */
MLA_API mla_status mla_decode_with_kvcache_status(const void* q, int batch, int s_q, int h_q, int d_qk,
                                   const void* kvcache, int num_blocks, int page_size, int h_kv,
                                   const int32_t* block_table, int max_blocks_per_seq,
                                   const int32_t* cache_seqlens, int dv, int dtype,
                                   const int32_t* tile_md, int num_parts,
                                   const int32_t* num_splits, int causal, float softmax_scale,
                                   int active_heads, void* o, float* lse, void* workspace,
                                   size_t workspace_bytes, int32_t* device_status, void* stream);

/*
 * The two stages of mla_decode_with_kvcache, for callers that schedule or time
 * them separately (the split-KV / combine kernel pair named on the "FlashMLA
 * vLLM Optimization" page, background section).  Calling mla_decode_splitkv
 * and then mla_decode_combine on one stream with the same arguments is exactly
 * mla_decode_with_kvcache.
 *
 * mla_decode_splitkv: same arguments and checks as mla_decode_with_kvcache.
 *   Each (request, row group) processed by one partition is written to o / lse
 *   directly; one spread over several partitions leaves float32 partial results
 *   in the workspace.
 * mla_decode_combine: merges those partial results into o / lse
 *   (lse = log sum_k exp(lse_k), o = sum_k exp(lse_k - lse) o_k); batch, s_q,
 *   h_q, h_kv, dv, dtype, num_splits, num_parts, active_heads, o, lse and
 *   workspace must be the ones given to mla_decode_splitkv.
 */
MLA_API mla_status mla_decode_splitkv(const void* q, int batch, int s_q, int h_q, int d_qk,
                                      const void* kvcache, int num_blocks, int page_size, int h_kv,
                                      const int32_t* block_table, int max_blocks_per_seq,
                                      const int32_t* cache_seqlens, int dv, int dtype,
                                      const int32_t* tile_md, int num_parts,
                                      const int32_t* num_splits, int causal, float softmax_scale,
                                      int active_heads, void* o, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream);

MLA_API mla_status mla_decode_combine(int batch, int s_q, int h_q, int h_kv, int dv, int dtype,
                                      const int32_t* num_splits, int num_parts, int active_heads,
                                      void* o, float* lse, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * Token-level sparse decoding over an "FP8 with scale" cache (upstream FlashMLA
 * documentation, "Sparse Attention (indices tensor)": indices [batch, s_q, topk],
 * indices[i][j][k] = page * page_size + offset of the k-th row query token j of
 * request i attends, -1 invalid, no block table; the support matrix lists sparse
 * decoding with the FP8 cache only).
 *
 * For request b, query token s and head h (kv head 0):
 *   E      = { k < topk : 0 <= indices[b][s][k] < num_blocks * 64 }   (other entries are invalid)
 *   x_k    = softmax_scale * <q[b,s,h,:], row(indices[b][s][k])>,  k in E   (a row listed twice
 *            counts twice)
 *   lse    = log(sum_{k in E} exp(x_k))                   (-inf when E is empty)
 *   o      = sum_{k in E} exp(x_k - lse) * row(...)[0:512] (0 when E is empty)
 * with rows dequantized as for MLA_BF16_FP8KV.  No causal mask (the list is what the
 * token sees).
 *
 * mla_get_metadata_sparse: the tile scheduler for num_tokens = batch * s_q query tokens of
 *   topk entries each, h_q heads (h_q / h_kv rows per token); tile_md as for
 *   mla_get_metadata with num_parts rows, num_splits [num_tokens * ceil(h_q / h_kv / 128) + 1].
 * mla_decode_sparse:
 *   q            device [batch, s_q, h_q, 576] bfloat16, 16-byte aligned
 *   kvcache      device [num_blocks, 64, 1, 656] bytes ("FP8 with scale" rows) for MLA_BF16_FP8KV,
 *                or [num_blocks, 64, 1, 576] bf16 / fp16 rows for MLA_BF16 / MLA_FP16 (a
 *                16-bit cache: not on the pages, whose sparse decode reads FP8; same definition);
 *                16-byte aligned
 *   indices      device int32 [batch, s_q, topk]
 *   dtype        MLA_BF16_FP8KV, MLA_BF16 or MLA_FP16; d_qk 576 (MLA_ERR_UNSUPPORTED otherwise), dv 512,
 *                h_kv 1, page_size 64
 *   tile_md, num_splits, num_parts   from mla_get_metadata_sparse for this batch * s_q and topk
 *   active_heads, softmax_scale, o, lse  as for mla_decode_with_kvcache
 *   workspace    >= mla_decode_workspace_bytes(batch * s_q, 1, h_q, 1, num_parts)
 * Enqueues the split-KV kernel and the combine kernel on `stream`.
 * mla_decode_sparse_splitkv: its first stage alone; mla_decode_combine with batch * s_q,
 *   s_q = 1 is the second (as for mla_decode_splitkv).
 */
MLA_API mla_status mla_get_metadata_sparse(int num_tokens, int topk, int h_q, int h_kv, int num_parts,
                                           int32_t* tile_md, int32_t* num_splits, void* stream);
/* The same schedule computed on the host into host arrays (synchronous; for tests and tools). */
MLA_API mla_status mla_get_metadata_sparse_host(int num_tokens, int topk, int h_q, int h_kv, int num_parts,
                                                int32_t* tile_md, int32_t* num_splits);
MLA_API mla_status mla_decode_sparse(const void* q, int batch, int s_q, int h_q, int d_qk, const void* kvcache,
                                     int num_blocks, int page_size, int h_kv, const int32_t* indices, int topk,
                                     int dv, int dtype, const int32_t* tile_md, int num_parts,
                                     const int32_t* num_splits, float softmax_scale, int active_heads, void* o,
                                     float* lse, void* workspace, size_t workspace_bytes, void* stream);
MLA_API mla_status mla_decode_sparse_splitkv(const void* q, int batch, int s_q, int h_q, int d_qk,
                                             const void* kvcache, int num_blocks, int page_size, int h_kv,
                                             const int32_t* indices, int topk, int dv, int dtype,
                                             const int32_t* tile_md, int num_parts, const int32_t* num_splits,
                                             float softmax_scale, int active_heads, void* o, float* lse,
                                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * Sparse MLA prefill (upstream FlashMLA documentation, "Sparse MLA Prefill": flash_mla_sparse_fwd(q,
 * kv, indices, sm_scale) returns (out, max_logits, lse), equivalent to the documentation's PyTorch
 * code).  No batch dimension and no pages: query token i attends the rows indices[i][0][k] of kv.
 *
 * For query token i and head h (kv head 0), over the valid entries E = { k < topk :
 * 0 <= indices[i][0][k] < s_kv } (-1 or any index >= s_kv is invalid):
 *   P_k        = <q[i,h,:], kv[idx_k,0,:]> * sm_scale * log2(e)
 *   max_logits = max_{k in E} P_k                      (-inf when E is empty)
 *   lse        = log2(sum_{k in E} 2^{P_k})             (base 2; -inf when E is empty)
 *   out        = sum_{k in E} 2^{P_k - lse} kv[idx_k,0,0:512]   (0 when E is empty)
 * (The documentation's equivalent code multiplies by the whole focused row; as everywhere in
 * the MQA mode, V is the leading dv = 512 columns.)
 *
 *   q            device [s_q, h_q, 576] bf16 or fp16, 16-byte aligned
 *   kv           device [s_kv, 1, 576], the dtype of q, 16-byte aligned
 *   indices      device int32 [s_q, 1, topk]
 *   dtype        MLA_BF16 or MLA_FP16;  dv 512;  h_kv 1
 *   sm_scale     > 0, or <= 0 for 1/sqrt(576)
 *   tile_md, num_splits, num_parts   from mla_get_metadata_sparse(s_q, topk, h_q, 1, num_parts, ...)
 *   out          device [s_q, h_q, 512], the dtype of q, written
 *   max_logits   device float32 [s_q, h_q], written
 *   lse          device float32 [s_q, h_q], written (base 2)
 *   workspace    >= mla_decode_workspace_bytes(s_q, 1, h_q, 1, num_parts), zero control block
 * Enqueues the split-KV kernel and the combine kernel on `stream`.  Errors: as for
 * mla_decode_with_kvcache; MLA_ERR_UNSUPPORTED for an FP8 dtype.
 */
MLA_API mla_status mla_sparse_prefill(const void* q, int s_q, int h_q, int d_qk, const void* kv, int s_kv, int h_kv,
                                      const int32_t* indices, int topk, int dv, int dtype, float sm_scale,
                                      const int32_t* tile_md, int num_parts, const int32_t* num_splits, void* out,
                                      float* max_logits, float* lse, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * Attention of ragged runs of new tokens over the paged cache: chunks of prompts and decode steps of
 * any length in one call.  Run b is the query tokens [cu_seqlens_q[b], cu_seqlens_q[b + 1]) of the
 * call's total_q; its keys are the first L_b = cache_seqlens[b] cached rows of its pages, the run's own
 * tokens among them (append them first).
 *
 * For token i of run b (0 <= i < n_b, n_b its tokens) and head h:
 *   n    = causal ? clamp(L_b - n_b + 1 + i, 0, L_b) : L_b        (bottom-right mask)
 *   x_j  = softmax_scale * <q[t,h,:], k_j>  (j < n),  lse = log(sum_j exp(x_j))   (-inf when n = 0)
 *   o    = sum_j exp(x_j - lse) * k_j[0:512]                                       (0 when n = 0)
 * Cached rows past the last one that a group of 128 query rows (tokens x heads) sees are not read into its
 * result, whatever they hold; rows that only some of the group's tokens see have weight zero for the others,
 * so that infinities or NaN in them reach the whole group.  Rows of q, o and lse past cu_seqlens_q[batch] are left as they were.
 *
 * mla_get_metadata_varlen: the tile scheduler, once per step for every layer.  Each run's rows are cut
 *   into groups of 128; a group's work is the pages that its last token sees.
 *   cu_seqlens_q   device int32 [batch + 1], ascending within [0, total_q]
 *   cache_seqlens  device int32 [batch]
 *   total_q        query tokens of the call (rows of q); batch <= 16384, total_q * h_q < 2^30
 *   plan           device int32 [mla_varlen_plan_ints(...)], 16-byte aligned, written (opaque)
 *   One small kernel on `stream`.  Runs that are not an ascending split of the tokens give a plan
 *   without work; the decode call with it records MLA_ERR_DEVICE_CHECK and writes nothing.
 * mla_get_metadata_varlen_host: the same schedule into host memory (8-byte aligned).
 * mla_decode_varlen:
 *   q              device [total_q, h_q, d_qk], dtype `dtype`, 16-byte aligned
 *   kvcache, block_table, dv, dtype, softmax_scale   as for mla_decode_with_kvcache
 *   cache_seqlens  the array given to mla_get_metadata_varlen
 *   plan, num_parts   from mla_get_metadata_varlen for the same batch, total_q and h_q
 *   o              device [total_q, h_q, 512], 16-byte aligned;  lse device float32 [total_q, h_q]
 *   workspace      >= mla_decode_varlen_workspace_bytes(num_parts), control block zero as for
 *                  mla_decode_with_kvcache (one workspace serves both)
 *   scratch        device, >= mla_decode_varlen_scratch_bytes(...), 256-byte aligned, any contents, or
 *                  null.  Over an FP8 cache, runs of several groups read each page several times: with
 *                  scratch their pages are dequantized once into it (the same values); without, at
 *                  every read.  mla_decode_varlen_scratch_bytes is 0 where it would not pay (16-bit
 *                  caches, fewer than three groups per run on average) or would exceed 8 GiB.  (The
 *                  schedule balances for the dequantized pages then; it is valid without scratch too.)
 *   Enqueues the split-KV and the combine kernel on `stream` (and, with scratch, one before them).
 * mla_decode_varlen_status: the same, with the call's device errors recorded in *device_status (device int32; the
 *   first error if it holds 0) instead of the workspace's status word; null: as mla_decode_varlen.
 */
MLA_API size_t mla_varlen_plan_ints(int batch, int total_q, int h_q, int h_kv, int num_parts);
MLA_API mla_status mla_get_metadata_varlen(const int32_t* cu_seqlens_q, const int32_t* cache_seqlens, int batch, int total_q,
                                           int h_q, int h_kv, int causal, int num_parts, int is_fp8_kvcache, int32_t* plan,
                                           void* stream);
MLA_API mla_status mla_get_metadata_varlen_host(const int32_t* cu_seqlens_q, const int32_t* cache_seqlens, int batch,
                                                int total_q, int h_q, int h_kv, int causal, int num_parts,
                                                int is_fp8_kvcache, int32_t* plan);
MLA_API size_t mla_decode_varlen_workspace_bytes(int num_parts);
MLA_API size_t mla_decode_varlen_scratch_bytes(int batch, int total_q, int h_q, int max_blocks_per_seq, int dtype);
MLA_API mla_status mla_decode_varlen(const void* q, int total_q, int h_q, int d_qk, const void* kvcache, int num_blocks,
                                     int page_size, int h_kv, const int32_t* block_table, int batch,
                                     int max_blocks_per_seq, const int32_t* cache_seqlens, int dv, int dtype,
                                     const int32_t* plan, int num_parts, float softmax_scale, void* o, float* lse,
                                     void* workspace, size_t workspace_bytes, void* scratch, size_t scratch_bytes,
                                     void* stream);
MLA_API mla_status mla_decode_varlen_status(const void* q, int total_q, int h_q, int d_qk, const void* kvcache,
                                            int num_blocks, int page_size, int h_kv, const int32_t* block_table,
                                            int batch, int max_blocks_per_seq, const int32_t* cache_seqlens, int dv,
                                            int dtype, const int32_t* plan, int num_parts, float softmax_scale, void* o,
                                            float* lse, void* workspace, size_t workspace_bytes, void* scratch,
                                            size_t scratch_bytes, int32_t* device_status, void* stream);

/*
 * Appending new tokens to the paged cache.  One pass over a step's new tokens: the latent is
 * normalised (optionally), the position columns of keys and queries are rotated, and each token's
 * row goes to the cache row that its slot names.
 *
 * For token t with latent x [512], key position columns e [64] and position n:
 *   y    = norm_weight ? x * rsqrt(mean(x^2) + norm_eps) * norm_weight : x        (float32)
 *   R(n) = rotation of pair i by the angle whose cosine and sine are cos_sin[n][i] and
 *          cos_sin[n][32 + i]:  (a, b) -> (a cos - b sin, b cos + a sin); pair i is columns
 *          (2 i, 2 i + 1) when interleaved, else (i, i + 32)                       (float32)
 *   16-bit cache:  row slots[t] = [ y | R(n) e ], each rounded once to the cache's type
 *   MLA_BF16_FP8KV: row slots[t] = e4m3(y_i / s_k), s_k, bf16(R(n) e), where for k = 0..3
 *          s_k = max(max_{i in block k} |y_i| * (1/448), 2^-126) in float32 (block k: latent columns
 *          [128 k, 128 k + 128)) and the quotient is rounded to float32, then to the nearest e4m3
 *          value.  y is quantized from float32: it is not rounded to bfloat16 before.
 *   queries (q_pe not null):  q[t][h][512:576] = R(n) q_pe[t][h], rounded once; other columns of q
 *          are left as they were.  q_pe may be those columns of q themselves.
 *
 *   latent         device [num_tokens] rows of 512, latent_stride values apart
 *   k_pe           device [num_tokens] rows of 64, k_pe_stride values apart; null with d_qk 512
 *   norm_weight    device [512] or null;  norm_eps >= 0
 *   positions      device int32 [num_tokens] (not read with d_qk 512)
 *   cos_sin        device float32 [max_position, 64]
 *   slots          device int32 [num_tokens]: flat cache rows (page * 64 + offset).  A negative slot
 *                  is padding: no row is written (the token's query columns are rotated all the
 *                  same).  Slots of one call are distinct; of two tokens with one slot the row
 *                  holds parts of either.
 *   kvcache        device [num_blocks, 64, 1, d_qk] or [num_blocks, 64, 1, 656] bytes; d_qk 576, or
 *                  512 (16-bit only: rows without position columns, no queries)
 *   q_pe, q        device; element (t, h, j) at t * token_stride + h * head_stride + j; both or
 *                  neither null; rows of q (576 wide) must not overlap
 *   dtype          type of latent, k_pe, norm_weight, q_pe, q and a 16-bit cache (bfloat16 for
 *                  MLA_BF16_FP8KV)
 *   device_status  device int32 or null: a slot outside the cache or a position outside the table
 *                  leaves the token's row (and for a position its query columns) as it was and
 *                  records MLA_ERR_DEVICE_CHECK there if it holds 0
 * Every pointer but positions and slots is 16-byte aligned and every stride a multiple of 8 values,
 * at least 0.  Enqueues one kernel on `stream`.
 */
MLA_API mla_status mla_append_kvcache(const void* latent, long long latent_stride, const void* k_pe,
                                      long long k_pe_stride, const void* norm_weight, float norm_eps,
                                      const int32_t* positions, const float* cos_sin, int max_position,
                                      const int32_t* slots, int num_tokens, void* kvcache, int num_blocks, int page_size,
                                      int h_kv, int d_qk, int dtype, int interleaved, const void* q_pe,
                                      long long q_pe_token_stride, long long q_pe_head_stride, void* q,
                                      long long q_token_stride, long long q_head_stride, int h_q, int32_t* device_status,
                                      void* stream);

/*
 * Page keys: one 8-bit summary per cache page, which page selection scores.
 *
 * For every page j of request b with prev_seqlens[b] / 64 <= j < cache_seqlens[b] / 64 (whole
 * divisions: the pages that the tokens between the two lengths completed; a page that is not full
 * has no key), with rows r_0 .. r_63 at physical page P = block_table[b][j]:
 *   m              = (r_0 + ... + r_63) / 64          (float32: rounded once from a sum within 2^-40 of
 *                                                      sum |r_i| / 64; no order of finite rows overflows)
 *   page_scales[P] = max(max_i |m_i| * (1/127), 2^-126)                     (float32)
 *   page_keys[P]   = m_i / page_scales[P], rounded to float32 and then to the nearest whole number
 * An FP8 cache's latents are bf16(e4m3 * scale), as for attention.  Other pages' keys are left as
 * they were.  A page with infinities or NaN gets an unspecified key.
 *
 *   kvcache, dtype, d_qk   as for mla_append_kvcache
 *   block_table    device int32 [batch, max_blocks_per_seq], fewer than 2^31 entries; batch <= 2^30
 *   prev_seqlens, cache_seqlens   device int32 [batch]
 *   page_keys      device int8 [num_blocks, d_qk], 16-byte aligned;  page_scales float32 [num_blocks]
 *   device_status  device int32 or null: an entry outside the cache (skipped), or a length beyond the
 *                  table (its pages past the table are skipped), records MLA_ERR_DEVICE_CHECK
 * Enqueues one kernel on `stream`.
 */
MLA_API mla_status mla_summarize_pages(const void* kvcache, int num_blocks, int page_size, int h_kv, int d_qk, int dtype,
                                       const int32_t* block_table, int max_blocks_per_seq, const int32_t* prev_seqlens,
                                       const int32_t* cache_seqlens, int batch, int8_t* page_keys, float* page_scales,
                                       int32_t* device_status, void* stream);

/*
 * Page selection for block-sparse decoding: the pages whose keys (mla_summarize_pages) score best for
 * each query token, as a block table of its own that mla_decode_with_kvcache reads with one request
 * per token.
 *
 * Token t = b * s_q + s sees n = clamp(L_b - s_q + 1 + s, 0, L_b) cached rows (causal; L_b otherwise) in
 * N = ceil(n / 64) pages.  For page j of them, P = block_table[b][j]:
 *   s_h    = max(max_i |q[b,s,h,i]| * (1/127), 2^-126),  q8_h = q / s_h, rounded to float32, then to
 *            the nearest whole number
 *   score  = max over heads h of (s_h * <q8_h, page_keys[P]>), times page_scales[P]
 *            (the inner product is a whole number, each product rounded once to float32: every
 *            implementation gets the same bits; NaN counts as the least)
 * The first n_first and the last n_last pages are always in (the last one may be partly filled and need
 * have no key); the others fill topn places by score, the lower page first where scores are equal.
 *   page_table[t]   the chosen pages' physical ids in ascending order of j, then -1   (all N when N <= topn)
 *   page_seqlens[t] cached rows in them: 64 for each but the last, which holds n - 64 (N - 1)   (0 when n = 0)
 *
 *   q              device [batch, s_q, h_q, d_qk] bf16 or fp16 (dtype), 16-byte aligned; d_qk 576 or
 *                  512, h_q <= 128
 *   page_keys      device int8 [num_blocks, d_qk], 16-byte aligned;  page_scales device float32 [num_blocks]
 *   block_table    device int32 [batch, max_blocks_per_seq];  cache_seqlens device int32 [batch]
 *   topn >= n_first + n_last, n_first >= 0, n_last >= 1, topn < 2^25
 *   page_table     device int32 [batch * s_q, topn], written;  page_seqlens device int32 [batch * s_q], written
 *   workspace      device, >= mla_select_workspace_bytes(...), 16-byte aligned, any contents
 *   device_status  device int32 or null: records MLA_ERR_DEVICE_CHECK for a block-table entry outside
 *                  the cache (scored as page 0) or a length beyond the table (cut to it), MLA_ERR_TIMEOUT
 * Enqueues three kernels on `stream`.  Then mla_get_metadata(page_seqlens, batch * s_q, h_q, 1, ...) and
 * mla_decode_with_kvcache(q, batch * s_q, 1, h_q, ..., page_table, topn, page_seqlens, ..., causal 0).
 */
MLA_API size_t mla_select_workspace_bytes(int batch, int s_q, int h_q, int d_qk, int max_blocks_per_seq);
MLA_API mla_status mla_select_pages(const void* q, int batch, int s_q, int h_q, int d_qk, int dtype,
                                    const int8_t* page_keys, const float* page_scales, int num_blocks,
                                    const int32_t* block_table, int max_blocks_per_seq, const int32_t* cache_seqlens,
                                    int causal, int topn, int n_first, int n_last, int32_t* page_table,
                                    int32_t* page_seqlens, void* workspace, size_t workspace_bytes,
                                    int32_t* device_status, void* stream);

/*
 * Reads the device status word of a workspace (synchronises `stream`).
 * *device_status receives MLA_OK or the first device-side error recorded by a
 * decode call that used this workspace; clear != 0 then zeroes the workspace's
 * whole control block (the status word back to MLA_OK; the split / combine
 * counters are zero already after a whole call, but not after its first stage
 * alone).
 */
MLA_API mla_status mla_read_device_status(void* workspace, int clear, int* device_status, void* stream);

/*
 * Allocation-free variant of mla_decode_with_kvcache (the pages describe no
 * counterpart: it exists for callers that cannot allocate device memory).
 *
 * Some callers cannot call cudaMalloc or any allocator at decode time: runtimes
 * that plan all device memory ahead and forbid later allocations, plugins that
 * are handed only tensor pointers by a host framework that owns every buffer,
 * and latency-critical paths where an allocation could block.  This entry point
 * takes the same arguments as mla_decode_with_kvcache minus the workspace; it
 * uses instead a fixed scratch array of MLA_NOALLOC_SCRATCH_BYTES compiled into
 * the library, which every GPU that loads the library holds until the process
 * exits.  The caller still provides q, kvcache, block_table, cache_seqlens, the
 * scheduler outputs, o and lse.
 *
 *   - Problems needing more than MLA_NOALLOC_SCRATCH_BYTES of workspace
 *     (mla_decode_workspace_bytes) are rejected with MLA_ERR_WORKSPACE.
 *   - The first call on a device looks up the device address of the scratch
 *     array (once per device, with that device current); make that first call
 *     before capturing any stream on that device.
 *   - No memory is allocated or freed; each call clears the scratch's status
 *     word and its own split / combine counters with an asynchronous memset on
 *     `stream` and then enqueues the same kernels as mla_decode_with_kvcache.
 *     Device-side errors of a call are read with mla_read_noalloc_status.
 *   - All calls on a device share one scratch array, which keeps the last
 *     call's contents: calls whose execution overlaps on the GPU (different
 *     streams without ordering between them) race on it and give wrong results.
 */
#define MLA_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)

MLA_API mla_status mla_decode_with_kvcache_noalloc(const void* q, int batch, int s_q, int h_q, int d_qk,
                                                   const void* kvcache, int num_blocks, int page_size,
                                                   int h_kv, const int32_t* block_table,
                                                   int max_blocks_per_seq, const int32_t* cache_seqlens,
                                                   int dv, int dtype, const int32_t* tile_md,
                                                   int num_parts, const int32_t* num_splits, int causal,
                                                   float softmax_scale, int active_heads, void* o, float* lse,
                                                   void* stream);

/*
 * Device status of the allocation-free entry point's scratch on the current
 * device (synchronises `stream`): MLA_OK, or the device-side error
 * (MLA_ERR_DEVICE_CHECK, MLA_ERR_TIMEOUT) recorded by the last
 * mla_decode_with_kvcache_noalloc call on this device, whose o / lse are then
 * not to be trusted.  Read it after a call and before the next one: every
 * call clears it when it starts.  clear != 0 resets it to MLA_OK.  Errors:
 * MLA_ERR_INVALID_ARG (null), MLA_ERR_CUDA.
 */
MLA_API mla_status mla_read_noalloc_status(int clear, int* device_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_DECODE_H_ */
