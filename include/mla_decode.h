/*
 * mla_decode.h -- C ABI of libmla: split-KV absorbed-MLA decode over a paged
 * fp8 e4m3fn KV cache on GB300 (sm_103a).
 *
 * The operation (moonmath-ai/amd-kernels README, "MLA absorbed decode",
 * "Use / MLA decode" and "Constraints / MLA decode"):
 *   one fused fp8 row per cached token is both K (all d_v + d_rope columns) and
 *   V (the first d_v columns), dequantized by ONE per-tensor kv_scale; queries
 *   come split into a latent part q_lat and a RoPE part q_pe; the pool is paged
 *   with page_size 1, so kv_indices is a flat per-token slot list in which any
 *   permutation or subset of the pool is legal; a call serves plain decode
 *   (q_len 1) and speculative verify (q_len > 1: draft position t of a request of
 *   S keys attends KV positions [0, S - q_len + t], inclusive); the output is
 *   written in place and an optional base-2 log-sum-exp is returned.
 *
 * For query row r = b*q_len + t and head h, with k_j the dequantized rows of
 * request b's visible positions:
 *   s_j  = scale * (q_lat[r,h,:] . k_j[0:d_v] + q_pe[r,h,:] . k_j[d_v:d_v+d_rope])
 *   o    = sum_j softmax(s)_j k_j[0:d_v]                    (bf16, round to nearest)
 *   lse  = log2 sum_j 2^(s_j * log2 e)                        (fp32, base 2)
 * A row that sees no key gets o = 0 and lse = -inf.
 *
 * Split-KV ("flash-decoding"): the planner splits each request's positions into
 * num_splits contiguous ranges (hip_mha_decoding_num_partitions: wave-aligned
 * split-K target, MLA-style branch); each (request, head block, split) CTA
 * writes a normalized fp32 partial and its base-2 LSE to the workspace and a
 * split-K reduce merges them in increasing split order, a fixed association
 * (README, "Numerics": the merge sums in a fixed association, so results are
 * deterministic run to run).
 *
 * Conventions shared by every entry point:
 *   - Pointers named q_*, pool, *indices, *indptr, seq_lens, o*, lse*, workspace
 *     are DEVICE pointers owned by the caller; the library never allocates,
 *     frees or keeps them past the call.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls only
 *     enqueue work on it: no host synchronisation, no allocation, so a call
 *     can be captured into a CUDA graph (the plan depends on shapes alone).
 *   - Return value: MLA_OK (0) or a negative MLA_ERR_* status; nothing is
 *     enqueued when a status other than MLA_OK or MLA_ERR_LAUNCH_FAILED is
 *     returned.  mla_status_string() names each status.
 *   - Faults found on the device (a slot outside [0, pool_rows), a bounded wait
 *     that ran out) are never raised as GPU faults: the kernel skips the bad
 *     access, ORs an MLA_DEVERR_* bit into the workspace's error word and
 *     finishes; outputs of the affected rows are then unspecified.  The word
 *     is sticky: clear it with mla_workspace_reset() and read it with
 *     mla_read_device_error().
 */
#ifndef MLA_DECODE_H
#define MLA_DECODE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------------- */
#define MLA_OK 0
#define MLA_ERR_INVALID_ARG (-1)         /* null pointer, negative size, plan/shape mismatch */
#define MLA_ERR_UNSUPPORTED_SHAPE (-2)   /* d_v/d_rope not (512,64) dense or (448,64) sparse,
                                            heads outside [1,128], too many splits,
                                            more than 65535 requests or tokens */
#define MLA_ERR_MISALIGNED (-3)          /* a buffer is not 16-byte aligned */
#define MLA_ERR_WORKSPACE_TOO_SMALL (-4) /* workspace_bytes < plan->workspace_bytes */
#define MLA_ERR_UNSUPPORTED_DEVICE (-5)  /* current device is not compute capability 10.3 */
#define MLA_ERR_LAUNCH_FAILED (-6)       /* a kernel launch returned a CUDA error */
#define MLA_ERR_CUDA (-7)                /* another CUDA runtime/driver call failed */

/* ---- device error bits (workspace error word) ------------------------------- */
#define MLA_DEVERR_BAD_SLOT 1u       /* a dense slot outside [0, pool_rows): key skipped */
#define MLA_DEVERR_TIMEOUT 2u        /* a bounded pipeline wait ran out: CTA gave up */
#define MLA_DEVERR_BAD_LENGTH 4u     /* seq_lens[b] outside [0, kv_indptr[b+1]-kv_indptr[b]];
                                        a fork's child longer than its parent */
#define MLA_DEVERR_BAD_POSITION 8u   /* mla_cache_append: a position outside the table */
#define MLA_DEVERR_BAD_TABLE 16u     /* mla_cache_fork: a parent outside [0, num_parents), or
                                        table offsets outside their lists */

/* Element types of the DCP share buffers (mla_decode_dcp, mla_dcp_lse_merge_ranks). */
#define MLA_DTYPE_BF16 0
#define MLA_DTYPE_F32 1

/* Largest split count the reducer accepts (hip_mha_decoding_num_partitions: the
 * reducer's 256-partition specialization caps the MLA-style split count). */
#define MLA_MAX_SPLITS 256
/* Bytes at the start of every workspace that hold the device error word and
 * the fused merge's arrival tickets; zero them before a workspace's first use
 * (mla_workspace_reset does). */
#define MLA_WORKSPACE_HEADER_BYTES 65536

/*
 * A launch plan: a pure function of shapes and the SM count (README, "MLA
 * absorbed decode": the op plans from tensor shapes alone, so it is CUDA-graph
 * capturable with no host synchronisation).  Plain data: copy it, store it,
 * recompute it; it holds no pointer.  Fields after `variant` echo the shape the
 * plan was made for; the decode entry points reject a plan whose echo differs
 * from their arguments.
 */
typedef struct {
    int32_t num_splits;      /* KV ranges per request (1..MLA_MAX_SPLITS) */
    int32_t rows_per_cta;    /* query rows (draft position x head) per CTA: 16, or 32
                                when a request has more than 16 rows; above 16 the
                                planners take 16 where a CTA's work is short (a
                                32-row CTA starts later), else 32; results agree
                                with the oracle either way */
    int32_t block_n;         /* keys per pipeline block */
    int32_t head_blocks;     /* CTAs sharing one (request, split) */
    int32_t grid_x, grid_y, grid_z;  /* head_blocks, num_splits, batch (or tokens) */
    int32_t variant;         /* kernel variant: 2 = tcgen05 split kernel, then the
                                split-K reduce kernel when num_splits > 1;
                                other values are rejected (MLA_ERR_INVALID_ARG) */
    int64_t workspace_bytes; /* bytes of device workspace the call needs */
    int32_t batch, q_len, num_heads, d_v, d_rope, sm_count;
    int64_t total_keys;      /* dense: kv_indices length; sparse: tokens * (topk + extra_topk) */
    int32_t kv_share;        /* 1: every CTA gathers its own KV rows (a request's
                                head blocks read the same rows, the repeats
                                served from L2); other values are rejected */
    int32_t extra_topk;      /* sparse: candidates per token in the second
                                (compressed) cache, 0 without one; dense: 0 */
    int32_t long_first;      /* dense, 1: grid slice z serves the z-th longest
                                request (ties by index), so the longest work is
                                scheduled first; set when the grid outlasts one
                                wave and batch <= 256; results do not depend on it */
    int32_t merge_cluster;   /* 1: the split-K merge is a second kernel (the split-K
                                reduce); 2 or 4: it is fused into the split kernel,
                                whose CTAs form clusters of that many consecutive
                                splits (num_splits a multiple of it) that merge
                                their partials through each other's shared memory,
                                the last cluster of a tile to finish merging the
                                clusters' results; results do not depend on the
                                timing.  The planner sets 1 (measured on GB300
                                the fused merge never beat the reduce kernel);
                                a caller may opt in by setting a size that fits */
} mla_plan_t;

/*
 * Dense plan.  total_keys = number of entries of kv_indices (a shape, not a
 * value); sm_count = the device's multiProcessorCount.  d_v must be 512 and
 * d_rope 64 (README, "Constraints / MLA decode": kv_lora_rank 512,
 * qk_rope_head_dim 64); num_heads in [1, 128] (same passage: H 1..128); any
 * q_len >= 1 with q_len * num_heads <= 2^20; batch <= 65535 (the requests are
 * the split grid's third dimension).  Writes *out and returns MLA_OK, or a
 * status.
 */
int mla_decode_plan(int32_t batch, int32_t q_len, int32_t num_heads, int64_t total_keys,
                    int32_t d_v, int32_t d_rope, int32_t sm_count, mla_plan_t* out);

/*
 * Sparse top-k plan (flashinfer.mla.cake_sparse_mla_sm120_dsv4_nvfp4_plan_splits:
 * one decode call's (num_splits, chunks per CTA) from tokens, heads, top-k, the
 * second cache's extra_topk and the SM count; "[Perf] pa_decode_sparse ..."
 * issue: 64 heads, 448 NoPE + 64 RoPE columns, top-k 2048).  d_v must be 448
 * and d_rope 64.  extra_topk = candidates per token in a second (compressed)
 * cache, 0 without one (mla_sparse_decode_extra).  max_splits caps num_splits
 * (0 = MLA_MAX_SPLITS).  Every split count from 1 up is valid for this kernel
 * (a split may even be empty), so a small cap costs speed only and is never an
 * error.  num_tokens <= 65535 (the tokens are the split grid's third dimension).
 */
int mla_sparse_decode_plan(int32_t num_tokens, int32_t num_heads, int32_t topk,
                           int32_t extra_topk, int32_t d_v, int32_t d_rope, int32_t sm_count,
                           int32_t max_splits, mla_plan_t* out);

/*
 * Dense decode: enqueues the split kernel and, when plan->num_splits > 1, the
 * split-K reduce (launched as a programmatic dependent of the split kernel, so
 * it is scheduled while the split kernel drains).  Layouts (row-major,
 * contiguous):
 *   q_lat    bf16 [batch*q_len, num_heads, 512]   row r = b*q_len + t
 *   q_pe     bf16 [batch*q_len, num_heads, 64]
 *   pool     e4m3fn bytes [pool_rows, 576] (a [pool_rows, 1, 576] tensor), 16-byte aligned
 *   seq_lens int32 [batch]; kv_indptr int32 [batch+1]; kv_indices int32 [kv_indptr[batch]]
 *            request b's position j lives in slot kv_indices[kv_indptr[b] + j],
 *            j < seq_lens[b] <= kv_indptr[b+1] - kv_indptr[b]
 *   o_lat    bf16 [batch*q_len, num_heads, 512], written
 *   lse      fp32 [batch*q_len, num_heads] base 2, written when non-NULL
 *   workspace >= plan->workspace_bytes bytes, 256-byte aligned; its first
 *            MLA_WORKSPACE_HEADER_BYTES hold the error word, the rest is
 *            scratch for the fp32 partials.  Calls that share a workspace must
 *            not overlap on the GPU.
 * scale multiplies the raw q.k dot product of dequantized rows (typically
 * (512+64)^-0.5); kv_scale dequantizes the pool.  Rows are copied in 128-key
 * blocks: the keys of a block that a call masks (past a request's length, or
 * invalid sparse entries) become zero rows without reading the pool, so only
 * the rows the page table names matter.  A NaN code in one of those, or a NaN or
 * infinite query, makes NaN of o and lse in the rows that see it and leaves every
 * other row as it is.
 */
int mla_decode(const mla_plan_t* plan, const void* q_lat, const void* q_pe,
               const void* pool, int64_t pool_rows, const int32_t* seq_lens,
               const int32_t* kv_indices, const int32_t* kv_indptr, int32_t batch,
               int32_t q_len, int32_t num_heads, float scale, float kv_scale,
               void* o_lat, float* lse, void* workspace, int64_t workspace_bytes,
               void* stream);

/*
 * Sparse top-k decode: token t attends the pool rows indices[t, 0:topk]
 * (a negative entry is invalid and skipped, the has_invalid case of the
 * pa_decode_sparse issue; a token with no valid entry gets o = 0, lse = -inf).
 *   q_nope bf16 [num_tokens, num_heads, 448]; q_pe bf16 [num_tokens, num_heads, 64]
 *   pool   e4m3fn bytes [pool_rows, 512]; indices int32 [num_tokens, topk]
 *   o      bf16 [num_tokens, num_heads, 448]; lse fp32 [num_tokens, num_heads] or NULL
 * Other arguments as for mla_decode.
 */
int mla_sparse_decode(const mla_plan_t* plan, const void* q_nope, const void* q_pe,
                      const void* pool, int64_t pool_rows, const int32_t* indices,
                      int32_t num_tokens, int32_t num_heads, int32_t topk, float scale,
                      float kv_scale, void* o, float* lse, void* workspace,
                      int64_t workspace_bytes, void* stream);

/*
 * Dense decode of one rank's share under decode context parallelism (DCP;
 * moonmath-ai/amd-kernels README, "MLA absorbed decode" and "Use / MLA decode":
 * one op serves plain decode, speculative verify and DCP; under DCP seq_lens
 * counts this rank's positions, glen gives the global lengths, and the op
 * returns a base-2 LSE for the cross-rank merge; "Constraints / MLA decode":
 * DCP needs glen whenever cp_world > 1).
 *   Rank cp_rank of cp_world holds the positions p of every request with
 *   p % cp_world == cp_rank, in increasing order: its kv_indices/kv_indptr/
 *   seq_lens list those positions' slots, so local key j is the global
 *   position j * cp_world + cp_rank.
 *   glen  int32 [batch] device: global lengths.  Draft row t of request b sees
 *         the local keys j < seq_lens[b] with j * cp_world + cp_rank <=
 *         glen[b] - q_len + t (the draft window of mla_decode in global
 *         positions); a row that sees none gets o = 0, lse = -inf.
 *   o     [batch*q_len, num_heads, 512]: the share's normalised output
 *         (softmax over the rank's visible keys, times kv_scale), bf16 when
 *         o_dtype is MLA_DTYPE_BF16 (the op's own output type, as in the
 *         pages) or fp32 when MLA_DTYPE_F32 (no rounding before the merge, at
 *         twice the exchange bytes); 16-byte aligned;
 *   lse   fp32 [batch*q_len, num_heads] base 2 of the share, required when
 *         cp_world > 1.
 * cp_world in [1, MLA_MAX_SPLITS], cp_rank in [0, cp_world); glen and lse are
 * required when cp_world > 1 (else MLA_ERR_INVALID_ARG), as is a known
 * o_dtype.  With cp_world == 1, glen == NULL and MLA_DTYPE_BF16 the call is
 * mla_decode.  The plan is mla_decode_plan's for the rank's own kv_indices
 * length.  Other arguments as for mla_decode.
 */
int mla_decode_dcp(const mla_plan_t* plan, const void* q_lat, const void* q_pe,
                   const void* pool, int64_t pool_rows, const int32_t* seq_lens,
                   const int32_t* kv_indices, const int32_t* kv_indptr, int32_t batch,
                   int32_t q_len, int32_t num_heads, float scale, float kv_scale,
                   const int32_t* glen, int32_t cp_rank, int32_t cp_world, int32_t o_dtype,
                   void* o, float* lse, void* workspace, int64_t workspace_bytes,
                   void* stream);

/*
 * The split kernel of mla_decode_dcp alone (as mla_decode_splits is to
 * mla_decode): with plan->num_splits == 1 it writes the share o / lse; with
 * more it leaves the fp32 partials in the workspace for mla_splitk_reduce.
 * Arguments as for mla_decode_dcp.
 */
int mla_decode_dcp_splits(const mla_plan_t* plan, const void* q_lat, const void* q_pe,
                          const void* pool, int64_t pool_rows, const int32_t* seq_lens,
                          const int32_t* kv_indices, const int32_t* kv_indptr, int32_t batch,
                          int32_t q_len, int32_t num_heads, float scale, float kv_scale,
                          const int32_t* glen, int32_t cp_rank, int32_t cp_world,
                          int32_t o_dtype, void* o, float* lse, void* workspace,
                          int64_t workspace_bytes, void* stream);

/*
 * Cross-rank merge of DCP shares (README, "Use / MLA decode":
 * mla_dcp_lse_merge_ranks combines the ranks' outputs and base-2 LSEs after
 * the all-to-all).  For each of `rows` rows, with k over the cp_world ranks:
 *   M = max_k lse_in[k, row];  w_k = 2^(lse_in[k, row] - M)
 *   out[row, :] = bf16(sum_k w_k parts_in[k, row, :] / sum_k w_k)
 *   lse_out[row] = M + log2 sum_k w_k           (when lse_out is non-NULL)
 * in a fixed association (each column sums its terms in increasing k).  A row whose
 * shares are all -inf gets out = 0 and lse_out = -inf.
 *   parts_in [cp_world, rows, d_v] (rank-major, as an all-gather leaves it),
 *            bf16 or fp32 as parts_dtype (MLA_DTYPE_BF16 / MLA_DTYPE_F32) says
 *   lse_in   fp32 [cp_world, rows] base 2
 *   out      bf16 [rows, d_v], written; lse_out fp32 [rows] or NULL
 * d_v a multiple of 8 up to 512; cp_world in [1, MLA_MAX_SPLITS]; parts_in and
 * out 16-byte aligned.  Device pointers; enqueued on `stream`.
 */
int mla_dcp_lse_merge_ranks(const void* parts_in, int32_t parts_dtype, const float* lse_in,
                            int32_t cp_world, int64_t rows, int32_t d_v, void* out,
                            float* lse_out, void* stream);

/*
 * Sparse top-k decode over two caches in one call (flashinfer
 * cake_sparse_mla_sm120_dsv4_nvfp4_plan_splits: extra_topk candidate slots per
 * token in the second (compressed) cache).  Token t attends, in one softmax,
 * the valid entries of indices[t, 0:topk] (rows of pool) together with the
 * valid entries of extra_indices[t, 0:extra_topk] (rows of extra_pool); a
 * negative entry in either table is invalid and skipped, and a token with no
 * valid entry gets o = 0, lse = -inf.
 *   extra_pool    e4m3fn bytes [extra_rows, 512], the main pool's row format
 *                 (448 NoPE + 64 RoPE columns) and kv_scale; 16-byte aligned
 *   extra_indices int32 [num_tokens, extra_topk]
 * The plan is mla_sparse_decode_plan's with the same topk and extra_topk.
 * With extra_topk == 0 the call is mla_sparse_decode (extra_pool and
 * extra_indices may be NULL).  Other arguments as for mla_sparse_decode.
 */
int mla_sparse_decode_extra(const mla_plan_t* plan, const void* q_nope, const void* q_pe,
                            const void* pool, int64_t pool_rows, const int32_t* indices,
                            const void* extra_pool, int64_t extra_rows,
                            const int32_t* extra_indices, int32_t num_tokens, int32_t num_heads,
                            int32_t topk, int32_t extra_topk, float scale, float kv_scale,
                            void* o, float* lse, void* workspace, int64_t workspace_bytes,
                            void* stream);
/* The split kernel of mla_sparse_decode_extra alone (see mla_decode_splits). */
int mla_sparse_decode_extra_splits(const mla_plan_t* plan, const void* q_nope,
                                   const void* q_pe, const void* pool, int64_t pool_rows,
                                   const int32_t* indices, const void* extra_pool,
                                   int64_t extra_rows, const int32_t* extra_indices,
                                   int32_t num_tokens, int32_t num_heads, int32_t topk,
                                   int32_t extra_topk, float scale, float kv_scale, void* o,
                                   float* lse, void* workspace, int64_t workspace_bytes,
                                   void* stream);

/*
 * The two halves of mla_decode / mla_sparse_decode, for callers that keep the
 * per-split partials (for example to merge them with another rank's) or time
 * the kernels one by one.  mla_decode_splits enqueues only the split kernel:
 * with plan->num_splits == 1 it writes o_lat / lse exactly as mla_decode does;
 * otherwise it leaves the normalized fp32 partials and their base-2 LSEs in the
 * workspace, where mla_workspace_partials() finds them, and
 * mla_splitk_reduce(o_part, lse_part, rows, num_splits, d_v, kv_scale, ...)
 * finishes the call.  Arguments as for mla_decode / mla_sparse_decode.
 */
int mla_decode_splits(const mla_plan_t* plan, const void* q_lat, const void* q_pe,
                      const void* pool, int64_t pool_rows, const int32_t* seq_lens,
                      const int32_t* kv_indices, const int32_t* kv_indptr, int32_t batch,
                      int32_t q_len, int32_t num_heads, float scale, float kv_scale,
                      void* o_lat, float* lse, void* workspace, int64_t workspace_bytes,
                      void* stream);
int mla_sparse_decode_splits(const mla_plan_t* plan, const void* q_nope, const void* q_pe,
                             const void* pool, int64_t pool_rows, const int32_t* indices,
                             int32_t num_tokens, int32_t num_heads, int32_t topk, float scale,
                             float kv_scale, void* o, float* lse, void* workspace,
                             int64_t workspace_bytes, void* stream);

/*
 * Device addresses, inside `workspace`, of the partials a plan's split kernel
 * writes: o_part fp32 [rows, num_splits, d_v] and lse_part fp32
 * [rows, num_splits], rows = batch * q_len * num_heads.  Host arithmetic only;
 * both are NULL when plan->num_splits == 1.
 */
int mla_workspace_partials(const mla_plan_t* plan, void* workspace, float** o_part,
                           float** lse_part);

/*
 * Split-K reduce on its own (hip_mha_decoding_num_partitions: the split-K
 * reducer that merges up to 256 partitions).  For each of `rows` rows:
 *   M = max_s lse_part[row, s];  w_s = 2^(lse_part[row, s] - M)
 *   o[row, :]  = bf16(out_scale * sum_s w_s o_part[row, s, :] / sum_s w_s)
 *   lse[row]   = M + log2 sum_s w_s            (when lse is non-NULL)
 * in a fixed association (sum_s w_s is 32 lane-strided partial sums joined by a
 * butterfly; each column sums its terms in increasing s, or, above 16 splits
 * and above 8 splits when rows <= 128, as four interleaved sums, s = g, g + 4,
 * ... for g = 0..3, each in increasing s, added in increasing g), so the result
 * does not vary from call to call; a row whose partials are all -inf gets o = 0 and
 * lse = -inf.  o_part fp32 [rows, num_splits, d_v] (normalized partials),
 * lse_part fp32 [rows, num_splits] base 2, o bf16 [rows, d_v]; d_v a multiple
 * of 8, num_splits in [1, MLA_MAX_SPLITS]; all 16-byte aligned.
 */
int mla_splitk_reduce(const float* o_part, const float* lse_part, int64_t rows,
                      int32_t num_splits, int32_t d_v, float out_scale, void* o,
                      float* lse, void* stream);

/*
 * Re-target a plan to a forced split count (1..MLA_MAX_SPLITS), updating its
 * grid, its merge cluster size (1, as the planner sets it) and its workspace
 * size.  For split sweeps
 * (moonmath-ai/amd-kernels README, "Results -- MLA decode": num_kv_splits swept
 * per shape) and tests; the planner's own choice needs no call to it.  A
 * caller may set merge_cluster to 1 afterwards (the separate reduce) or to
 * another size that fits; the decode calls reject one that does not.
 */
int mla_plan_force_splits(mla_plan_t* plan, int32_t num_splits);

/* Zero the workspace header, which holds the error word (enqueued on `stream`). */
int mla_workspace_reset(void* workspace, void* stream);

/*
 * Read the error word (MLA_DEVERR_* bits) into *code.  Synchronises `stream`;
 * not for the hot path.
 */
int mla_read_device_error(const void* workspace, int32_t* code, void* stream);

/*
 * Dense decode for callers that cannot allocate device memory: code running
 * where cudaMalloc is unavailable or not allowed (a no-allocation region of a
 * serving loop with a fixed memory budget, or a host framework that hands over
 * only its input and output buffers).  It is mla_decode with the workspace
 * replaced by a static scratch array inside the library, so the caller passes
 * inputs and outputs only and the call itself allocates nothing.  The pages
 * have no counterpart of this entry point.
 *   - Scratch: a file-scope __device__ array of MLA_NOALLOC_SCRATCH_BYTES; every
 *     GPU that loads the library holds it until the process exits.  A plan with
 *     plan->workspace_bytes above that size is rejected with
 *     MLA_ERR_WORKSPACE_TOO_SMALL and nothing is enqueued.
 *   - Set-up: the first call on a device (with that device current) looks up
 *     the array's device address once; make that first call before any stream
 *     capture on the device.  The address is kept for the life of the process,
 *     so do not use this entry point on a device after cudaDeviceReset.
 *   - Every call shares the one array and it keeps the last call's contents, so
 *     calls that overlap on the GPU (on different streams, or from different
 *     threads) race and must be serialised by the caller.
 *   - Device-side error bits (MLA_DEVERR_*) are not reported by this entry
 *     point: bad slots are still skipped safely, but there is no workspace to
 *     read them from.
 * Other arguments, layouts and status codes as for mla_decode.
 */
#define MLA_NOALLOC_SCRATCH_BYTES (32 * 1024 * 1024)
int mla_decode_noalloc(const mla_plan_t* plan, const void* q_lat, const void* q_pe,
                       const void* pool, int64_t pool_rows, const int32_t* seq_lens,
                       const int32_t* kv_indices, const int32_t* kv_indptr, int32_t batch,
                       int32_t q_len, int32_t num_heads, float scale, float kv_scale,
                       void* o_lat, float* lse, void* stream);

/*
 * A plan of mla_prefix_decode, from shapes alone; plain data like mla_plan_t.
 */
typedef struct {
    int32_t tiles;           /* 64-row tiles of the batch * q_len * num_heads query rows */
    int32_t ctas;            /* CTAs of the prefix kernel; 0 when prefix_cap is 0 */
    int32_t splits;          /* CTAs per tile, each an equal part of its 128-key blocks;
                                or 0: the sequence of all tiles' blocks is cut into
                                equal runs, one per CTA (at most MLA_MAX_SPLITS) */
    int32_t joined;          /* 1: a tile's blocks are the prefix's and then its requests'
                                own; 0: the requests' own keys go through the kernel of
                                mla_decode.  Results agree with the oracle either way */
    int32_t sm_count;
    int32_t reserved;        /* 0 */
    int64_t workspace_bytes; /* bytes of device workspace the call needs */
    int64_t prefix_cap;      /* entries of prefix_indices */
    mla_plan_t own;          /* the plan of the requests' own keys (mla_decode_plan) */
} mla_prefix_plan_t;

/*
 * Plan of a decode over a shared prefix of up to prefix_cap positions and
 * total_keys entries of the requests' own page tables.  Other arguments and
 * limits as for mla_decode_plan (d_v 512, d_rope 64); prefix_cap <= 2^30.
 */
int mla_prefix_decode_plan(int32_t batch, int32_t q_len, int32_t num_heads, int64_t prefix_cap,
                           int64_t total_keys, int32_t sm_count, mla_prefix_plan_t* out);

/*
 * Dense decode of a batch whose requests share a prefix: request b's keys are
 * the prefix's P slots followed by its own seq_lens[b] slots, and the call gives
 * what mla_decode gives on the joined page tables (S = P + seq_lens[b]; draft
 * position t attends positions [0, S - q_len + t]), but the prefix's rows are
 * fetched and multiplied once for the query rows of the whole batch.
 *   prefix_indices int32 [prefix_cap]: the prefix's slots, in any order of the pool
 *   prefix_len     int32 [1] device: P, the entries in use; NULL: all of them.
 *                  Outside [0, prefix_cap] it is clamped and sets
 *                  MLA_DEVERR_BAD_LENGTH.
 *   seq_lens, kv_indices, kv_indptr: the requests' own keys, as for mla_decode
 *                  (a request may have none; kv_indices has the plan's total_keys
 *                  entries and may be NULL when that is 0)
 *   workspace >= plan->workspace_bytes bytes, 256-byte aligned, zeroed header;
 *                  calls that share it must not overlap on the GPU
 * Other arguments, layouts and device errors as for mla_decode.  A NaN (or an
 * infinite query) makes NaN of the output rows that see it, not of the batch's
 * others.  The merge joins partials in a fixed order, so results do not vary from
 * call to call.
 */
int mla_prefix_decode(const mla_prefix_plan_t* plan, const void* q_lat, const void* q_pe,
                      const void* pool, int64_t pool_rows, const int32_t* prefix_indices,
                      const int32_t* prefix_len, const int32_t* seq_lens,
                      const int32_t* kv_indices, const int32_t* kv_indptr, int32_t batch,
                      int32_t q_len, int32_t num_heads, float scale, float kv_scale, void* o,
                      float* lse, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Cache append: one pass from the projections' outputs to what the decode
 * reads.  For each of num_tokens tokens, with p = positions[t] and, for
 * i in [0, 32), c_i = cos_sin[p, i], s_i = cos_sin[p, 32 + i]:
 *   kv row   the token's latent row x (row_bytes columns: d_v latent, then 64
 *            RoPE; row_bytes 576 for mla_decode's rows, 512 for
 *            mla_sparse_decode's).  The first kv_norm_cols columns (0, d_v or
 *            all of them) are RMS-normed, x_j * (mean x^2 + eps)^-1/2 *
 *            kv_weight[j] (weight 1 where kv_weight is NULL); the last 64 are
 *            then rotated; pool[slots[t]] = e4m3(y * (1 / kv_scale)), to
 *            nearest even, saturating at +-448 (NaN stays NaN).  A negative
 *            slot skips the row (a padding token).
 *   queries  the token's num_heads rows of q_cols columns, RMS-normed over all
 *            of them when q_norm is nonzero (times q_weight where non-NULL),
 *            the last 64 rotated, written as bf16 to q_nope (the first
 *            q_cols - 64) and q_pe (the last 64).
 * Rotation of (a, b) by (c, s): (a c - b s, b c + a s); the pairs are columns
 * (2 i, 2 i + 1), or (i, i + 32) when half_split is nonzero.  Everything is
 * computed in fp32 and rounded once.
 *   kv        bf16, token t's row at kv + t * kv_stride (elements); NULL: no
 *             rows are appended (slots and pool may then be NULL)
 *   kv_weight bf16 [kv_norm_cols] or NULL
 *   slots     int32 [num_tokens], each in [0, pool_rows) or negative; the slots
 *             of a call are distinct (of two tokens with one slot either may
 *             be found there, in part or whole).  A slot past the pool sets
 *             MLA_DEVERR_BAD_SLOT and its row is skipped.
 *   q         bf16, head h of token t at q + t * q_token_stride +
 *             h * q_head_stride; NULL (with num_heads 0): no queries
 *   q_weight  bf16 [q_cols] or NULL; q_cols a multiple of 64 in [64, 576]
 *   q_nope    bf16 [num_tokens, num_heads, q_cols - 64] (unused, may be NULL,
 *             when q_cols is 64); q_pe bf16 [num_tokens, num_heads, 64];
 *             neither overlaps q
 *   positions int32 [num_tokens]; cos_sin fp32 [max_positions, 64].  A position
 *             outside [0, max_positions) sets MLA_DEVERR_BAD_POSITION and
 *             nothing of that token is written.
 *   workspace at least MLA_WORKSPACE_HEADER_BYTES, 256-byte aligned: the error
 *             word.  Calls may share it, also when they overlap.
 * kv, weights, q, q_nope, q_pe, pool and cos_sin are 16-byte aligned and the
 * strides multiples of 8 elements (else MLA_ERR_MISALIGNED); num_heads <= 128;
 * eps >= 0 and finite; kv_scale finite and not zero.  num_tokens 0 is a no-op.
 */
int mla_cache_append(const void* kv, int64_t kv_stride, const void* kv_weight,
                     int32_t kv_norm_cols, const int32_t* slots, void* pool, int64_t pool_rows,
                     int32_t row_bytes, float kv_scale, const void* q, int64_t q_token_stride,
                     int64_t q_head_stride, const void* q_weight, int32_t q_norm, int32_t q_cols,
                     void* q_nope, void* q_pe, const int32_t* positions, const float* cos_sin,
                     int64_t max_positions, int32_t half_split, float eps, int32_t num_tokens,
                     int32_t num_heads, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Cache fork: the page tables of num_children requests that continue
 * num_parents requests, and copies of the rows that they do not share.  Child f
 * takes the first n_f = child_indptr[f+1] - child_indptr[f] positions of parent
 * p = parents[f] (n_f at most the parent's length, kv_indptr[p+1] -
 * kv_indptr[p]).  Its positions j < keep[f] name the parent's own slots; the
 * others take fresh slots in order, and the rows are copied there:
 *   table[child_indptr[f] + j] = kv_indices[kv_indptr[p] + j]         j < keep[f]
 *                              = fresh[fresh_indptr[f] + j - keep[f]]  otherwise,
 *   pool[table[...]] = pool[kv_indices[kv_indptr[p] + j]]              (bytes)
 * keep[f] <= 0 copies every row, keep[f] >= n_f none.  The fresh slots of a
 * call are distinct and none is a slot that the call copies from; table overlaps
 * no other argument.
 *   pool [pool_rows, row_bytes], row_bytes 576 or 512, 16-byte aligned
 *   kv_indices int32 [num_indices]; kv_indptr int32 [num_parents + 1]
 *   parents, keep int32 [num_children]; child_indptr, fresh_indptr int32
 *   [num_children + 1]; fresh int32 [num_fresh]
 *   table int32 [total], written; total = child_indptr[num_children] (a shape:
 *   entries of table past the last child's are not touched)
 * Found on the device: a slot outside the pool (MLA_DEVERR_BAD_SLOT: its row is
 * not copied, the table entry names it all the same), a child longer than its
 * parent (MLA_DEVERR_BAD_LENGTH) and a parent, offset or fresh entry outside
 * its list (MLA_DEVERR_BAD_TABLE): the entry becomes -1 and no row is copied.
 * workspace as for mla_cache_append.
 */
int mla_cache_fork(void* pool, int64_t pool_rows, int32_t row_bytes, const int32_t* kv_indices,
                   int64_t num_indices, const int32_t* kv_indptr, int32_t num_parents,
                   const int32_t* parents, const int32_t* keep, const int32_t* child_indptr,
                   int32_t num_children, const int32_t* fresh, int64_t num_fresh,
                   const int32_t* fresh_indptr, int32_t* table, int64_t total, void* workspace,
                   int64_t workspace_bytes, void* stream);

/*
 * Cache compaction: gathers the live rows at the front of the pool and rewrites
 * the page tables.  A row is live when an entry of kv_indices names it (any
 * number of times: shared prefixes stay shared).  With L live rows, the k-th
 * live row at or past L, in slot order, moves into the k-th free slot below L,
 * so only rows that have to move do, and the free slots are then [L, pool_rows):
 *   new_indices[i] = the slot of the row that kv_indices[i] named
 *   live[0]        = L
 * A negative entry stays as it is; one past the pool does too, and sets
 * MLA_DEVERR_BAD_SLOT.  Rows at or past L keep their old bytes.  The result
 * does not depend on timing.
 *   pool [pool_rows, row_bytes], row_bytes 576 or 512, 16-byte aligned, in place
 *   kv_indices int32 [num_indices]; new_indices int32 [num_indices], which may
 *   be kv_indices itself (else they do not overlap); live int32 [1], all device
 *   workspace of mla_cache_compact_workspace_bytes(pool_rows) bytes, 256-byte
 *   aligned, zeroed header (calls that overlap do not share it)
 * pool_rows < 2^31.
 */
int mla_cache_compact(void* pool, int64_t pool_rows, int32_t row_bytes,
                      const int32_t* kv_indices, int64_t num_indices, int32_t* new_indices,
                      int32_t* live, void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of mla_cache_compact for a pool of pool_rows rows; 0 for an
 * unsupported count. */
int64_t mla_cache_compact_workspace_bytes(int64_t pool_rows);

/* Static text for a status code. */
const char* mla_status_string(int status);

/*
 * Gather probe, for tests of the page-table gather (step a2): copies
 * out[i, :] = pool[indices[i], :] for i < n, byte for byte, through the split
 * kernel's own gather path (TMA tile::gather4 into the swizzled shared-memory
 * stage layout, then read back de-swizzled).  row_bytes is 576 (dense rows:
 * four 128-byte chunks and a 64-byte RoPE chunk) or 512 (sparse rows).  An
 * index outside [0, pool_rows) is not read; its output row is zero.  pool and
 * out 16-byte aligned; workspace (>= MLA_WORKSPACE_HEADER_BYTES, 256-byte
 * aligned) receives MLA_DEVERR_TIMEOUT if a bounded wait ran out.  Not on the
 * decode path.
 */
int mla_debug_gather(const void* pool, int64_t pool_rows, int32_t row_bytes,
                     const int32_t* indices, int64_t n, void* out, void* workspace,
                     void* stream);

/*
 * Sets the bound, in SM clock cycles, of the split kernel's pipeline waits
 * for launches enqueued after the call (process-wide; every device), and
 * returns the previous bound; cycles <= 0 restores the default, about one
 * second at GB300 clocks.  A wait that runs out ends its CTA's work: the CTA
 * stops issuing copies and MMAs, waits (with the full bound) for those it
 * already issued, writes what it has (its output rows are then unspecified),
 * sets MLA_DEVERR_TIMEOUT in the workspace error word and exits; the call
 * completes normally and the device stays usable.  For tests of that path:
 * while a bound other than the default is set, every CTA also starts with a
 * wait on a barrier that nothing completes, so at least that wait runs out
 * while the CTA's first copies are in flight.  Not on the decode path; not
 * thread-safe against concurrent decode calls that expect the default.
 */
int64_t mla_debug_wait_limit(int64_t cycles);

/*
 * The split count that the wave-fill rule of hip_mha_decoding_num_partitions
 * (MLA-style branch) gives for the given constants: ctas = ceil(heads/bm) *
 * batch; one_wave = sm/ctas; two_wave = 2*sm/ctas; pages = ceil(keys/page);
 * work_floor = ceil(pages/max_pages_per_split); np = clamp(work_floor,
 * one_wave, two_wave) rounded up to a power of two, capped by two_wave, by
 * max_splits and by pages; heads <= small_heads uses min(two_wave, pages).
 * The dense planner calls it with GB300 constants; it is exported so the
 * constants of the page it comes from can be checked against that page's
 * printed sweep.
 */
int32_t mla_wave_fill_splits(int32_t batch, int64_t keys_per_request, int32_t heads,
                             int32_t sm_count, int32_t bm, int32_t page,
                             int32_t max_pages_per_split, int32_t max_splits,
                             int32_t small_heads);

#ifdef __cplusplus
}
#endif
#endif /* MLA_DECODE_H */
