/*
 * moe_layout.h -- C ABI of the GB300 MoE dispatch-layout library
 * (libmoe_layout.so): token dispatch as a counting sort / bucketization,
 * and its inverse combine, on one GPU.
 *
 * The method is the one described on the page
 *   "07 DeepEP Counting Sort / Bucketization 深度校验：博客第一性原理 vs 源码实现"
 * cited as [CS] with its section numbers: count tokens per expert and per
 * logical rank (§4.2), prefix-sum the aligned counts (§5.2-§5.5, §7.2),
 * scatter every (token, expert) copy of a row into an expert-major buffer
 * (§6.4, §8.2) with zero rows in the alignment gaps (§7.3).  Combine is the
 * inverse gather with a top-k weighted sum.
 *
 * Conventions shared by every entry point
 *  - All array pointers are DEVICE pointers owned by the caller.  The library
 *    allocates no memory; scratch lives in a caller-provided workspace whose
 *    size moe_layout_workspace_bytes() returns.
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL means the
 *    legacy default stream) and returns before the GPU work finishes, except
 *    moe_layout_get_error(), which synchronises the stream.
 *  - Return value: MOE_OK, or an error found on the host before anything was
 *    launched (MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED), or MOE_ERR_CUDA if a
 *    launch failed.  Errors found by the kernels (bad expert id, capacity,
 *    timeout, an inverse-map entry out of range) are recorded in the
 *    workspace's sticky error word and read with moe_layout_get_error().
 *  - Notation: N tokens, K top-k slots, E experts, R logical ranks,
 *    L = E / R experts per rank, A alignment.  Logical rank r owns experts
 *    [r*L, (r+1)*L); ranks are partitions of one GPU buffer, not devices.
 *  - topk_idx is int64 [N, K] row-major; a negative entry is a masked slot;
 *    an entry >= E is an error (MOE_ERR_BAD_EXPERT_ID) and the slot is then
 *    treated as masked.
 *  - Slots and row indices are int32: N*K + E*(A-1) must be < 2^31.
 *  - Results are deterministic: the slot of a (token, k) pair inside its
 *    expert's segment is its rank in (token, k) order among that expert's
 *    pairs, independent of scheduling.  ([CS] §6.2/§6.4 hand out slots with
 *    atomics instead, so their order varies from run to run.)
 *  - Kernels are launched with programmatic dependent launch, and some of
 *    them start reading their inputs topk_idx, x and sf before the kernel in
 *    front of them on the stream has finished: the dispatch permutes prefetch
 *    token rows, the rank kernels stage ids.  This is safe after copies, after
 *    this library's own kernels (the gate, the norm and the quantisers, which write
 *    those inputs, do not release their dependents early) and after any other
 *    kernel that does not release its dependents early.  The kernel
 *    launched on the stream directly before one of these calls must not write
 *    the call's topk_idx, x or sf and also release its dependents before it
 *    ends (griddepcontrol.launch_dependents /
 *    cudaTriggerProgrammaticLaunchCompletion): put an event record or any
 *    ordinary kernel between them.
 *
 * Kernels are compiled for sm_103a only.
 */
#ifndef MOE_LAYOUT_H_
#define MOE_LAYOUT_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes.  0 is success. */
enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,   /* host check failed: null pointer, bad size or alignment;
                                device (moe_dispatch_sf_col_major): map entry out of range;
                                device (moe_gate_forward, moe_gate_forward_grouped): a NaN
                                or +inf key;
                                device (moe_quantize_cols, moe_expert_wgrad_fp8): a
                                segment that starts inside a block of 128 rows       */
  MOE_ERR_CUDA = 2,          /* a CUDA launch or copy failed                           */
  MOE_ERR_BAD_EXPERT_ID = 3, /* device: some topk_idx entry was >= E                   */
  MOE_ERR_CAPACITY = 4,      /* device: the layout needs more rows than capacity_rows  */
  MOE_ERR_TIMEOUT = 5,       /* device: a bounded wait inside a kernel ran out         */
  MOE_ERR_UNSUPPORTED = 6    /* host: sizes beyond what this build supports            */
};

/* Limits of this build.  Rows (token rows, scale rows, combine rows of
 * 2 * hidden bytes) longer than MOE_MAX_ROW_BYTES are refused with
 * MOE_ERR_UNSUPPORTED, which keeps every byte offset well inside int64. */
#define MOE_MAX_TOPK 32
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_ROW_BYTES (1 << 30)

/* Problem description.  Plain values, copied by every call. */
typedef struct moe_layout_desc {
  int64_t num_tokens;  /* N >= 0                                  */
  int32_t topk;        /* K, 1 <= K <= MOE_MAX_TOPK ([CS] §4.2)  */
  int32_t num_experts; /* E, 1 <= E <= MOE_MAX_EXPERTS           */
  int32_t num_ranks;   /* R >= 1, R divides E                     */
  int32_t alignment;   /* A >= 1 ([CS] §7.1-§7.2)                */
} moe_layout_desc;

/*
 * Bytes of device workspace the other calls need for this description
 * (sticky error word, grid-barrier words, the permute's work counter,
 * per-tile expert and rank histograms).  The workspace must
 * be zero-filled once before its first use (e.g. cudaMemsetAsync);
 * afterwards every call leaves it ready for the next.  One workspace serves
 * one stream at a time: calls that overlap on the GPU must not share it.
 * After MOE_ERR_TIMEOUT, zero-fill it again.
 */
MOE_API int moe_layout_workspace_bytes(const moe_layout_desc* desc, size_t* bytes);

/*
 * Count ([CS] §4.2).  Reads topk_idx [N*K]; writes
 *   expert_count[E]: number of (t, k) with topk_idx[t*K+k] == e;
 *   rank_count[R]:   number of tokens with at least one valid id in rank r,
 *                    each token counted once per rank (deduplicated);
 * and the per-tile histograms in `workspace` that moe_layout_scan needs.
 * Bad ids set MOE_ERR_BAD_EXPERT_ID in the workspace error word.
 */
MOE_API int moe_layout_count(const moe_layout_desc* desc, const int64_t* topk_idx,
                     int32_t* expert_count, int32_t* rank_count,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * Prefix sums and slot maps ([CS] §5.2-§5.5, §7.2, §6.4).  Must follow
 * moe_layout_count on the same topk_idx, counts and workspace.  Writes
 *   expert_offset[E+1]: exclusive sum of align(expert_count[e], A); expert
 *                       e's segment is rows [expert_offset[e], expert_offset[e+1]);
 *                       rank r's block starts at expert_offset[r*L];
 *   rank_psum[R]:       inclusive sum of rank_count;
 *   dst_slot[N*K]:      row of (t, k) in the receive buffer, -1 if masked;
 *   src_idx[rows]:      token of each row, -1 for the alignment-gap rows;
 *   total_rows[1]:      expert_offset[E] (device scalar).
 * capacity_rows is the length of src_idx (and of the receive buffers).  If
 * the layout needs more rows, MOE_ERR_CAPACITY is recorded, src_idx is not
 * written and every dst_slot entry is -1.  A bound that never fails is
 * N*K + E*(A-1).
 */
MOE_API int moe_layout_scan(const moe_layout_desc* desc, const int64_t* topk_idx,
                    const int32_t* expert_count, const int32_t* rank_count,
                    void* workspace, size_t workspace_bytes,
                    int32_t* expert_offset, int32_t* rank_psum,
                    int32_t* dst_slot, int32_t* src_idx, int64_t capacity_rows,
                    int32_t* total_rows, void* stream);

/*
 * moe_layout_count followed by moe_layout_scan, in one call, with the same
 * arguments and results.  For the largest batches (about a million pairs and
 * up), when every tile of the problem fits on the GPU at once, it runs as a
 * single cooperative kernel (count, per-expert scan over tiles, rank) with
 * two grid-wide barriers whose waits are bounded (MOE_ERR_TIMEOUT, after
 * which the workspace must be zero-filled again); otherwise it runs the two
 * calls' kernels.
 */
MOE_API int moe_layout_build(const moe_layout_desc* desc, const int64_t* topk_idx,
                             int32_t* expert_count, int32_t* rank_count,
                             void* workspace, size_t workspace_bytes,
                             int32_t* expert_offset, int32_t* rank_psum,
                             int32_t* dst_slot, int32_t* src_idx, int64_t capacity_rows,
                             int32_t* total_rows, void* stream);

/*
 * moe_layout_build with int32 routing ids (topk_idx int32 [N*K]); same
 * results.  Frameworks that keep top-k ids as int32 avoid a widening copy.
 */
MOE_API int moe_layout_build_i32(const moe_layout_desc* desc, const int32_t* topk_idx,
                                 int32_t* expert_count, int32_t* rank_count,
                                 void* workspace, size_t workspace_bytes,
                                 int32_t* expert_offset, int32_t* rank_psum,
                                 int32_t* dst_slot, int32_t* src_idx, int64_t capacity_rows,
                                 int32_t* total_rows, void* stream);

/*
 * Expand-mode dispatch permute ([CS] §6.3-§6.4, §8.2) with zero padding
 * ([CS] §7.3).  For every valid (t, k): recv_x row dst_slot[t*K+k] = x row t,
 * copied byte for byte (any row dtype: bf16, fp8, ...).  If sf is non-NULL
 * the scale-factor row sf[t] moves the same way into recv_sf.  With
 * zero_pad != 0, rows [expert_offset[e] + expert_count[e], expert_offset[e+1])
 * of recv_x (and recv_sf) are set to zero bytes.
 *   x [N, row_bytes], recv_x [capacity_rows, row_bytes]: row_bytes a positive
 *     multiple of 16, both base pointers 16-byte aligned;
 *   sf [N, sf_row_bytes], recv_sf [capacity_rows, sf_row_bytes]: sf_row_bytes
 *     a positive multiple of 4, pointers 4-byte aligned (NULL sf: no scale factors);
 *   dst_slot, expert_offset, expert_count: as written by the calls above.
 * Slots >= capacity_rows are not written and record MOE_ERR_CAPACITY.
 */
MOE_API int moe_dispatch_permute(const moe_layout_desc* desc, const void* x,
                         int64_t row_bytes, const void* sf, int64_t sf_row_bytes,
                         const int32_t* dst_slot, const int32_t* expert_offset,
                         const int32_t* expert_count, void* recv_x, void* recv_sf,
                         int64_t capacity_rows, int zero_pad, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * Non-expand (rank-contiguous) slot map: the page's first scatter
 * ([CS] §6.2, §8.1-§8.2), where each token goes once to every logical rank
 * it reaches, whatever the number of that rank's experts it picked.  Must
 * follow moe_layout_build (or moe_layout_count + moe_layout_scan) on the same
 * topk_idx and workspace; rank_count is that call's output.  Writes
 *   rank_slot[N*K]: for each token and rank it reaches, the highest k among
 *                   the token's slots reaching that rank (the page's master
 *                   lane) gets the row index; every other slot gets -1;
 *   rank_src[rows]: token of each row.
 * Rank r's rows are [rank_psum[r] - rank_count[r], rank_psum[r]); tokens are
 * in ascending order inside it.  rows = rank_psum[R-1].  If rows exceed
 * capacity_rows, MOE_ERR_CAPACITY is recorded, every rank_slot is -1 and
 * rank_src is not written.  N*R rows always suffice.
 */
MOE_API int moe_layout_rank_rows(const moe_layout_desc* desc, const int64_t* topk_idx,
                                 const int32_t* rank_count, void* workspace, size_t workspace_bytes,
                                 int32_t* rank_slot, int32_t* rank_src, int64_t capacity_rows,
                                 void* stream);

/*
 * Non-expand dispatch permute ([CS] §6.3, §8.2 "non-expand"): recv row
 * rank_slot[t*K+k] = x row t for every slot that has a row; scale-factor
 * rows move alongside when sf is non-NULL.  No padding.  Argument rules as
 * for moe_dispatch_permute; rank_psum (from the layout) gives the row total
 * checked against capacity_rows.
 */
MOE_API int moe_dispatch_permute_ranks(const moe_layout_desc* desc, const void* x,
                                       int64_t row_bytes, const void* sf, int64_t sf_row_bytes,
                                       const int32_t* rank_slot, const int32_t* rank_psum,
                                       void* recv, void* recv_sf, int64_t capacity_rows,
                                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Scale factors of a receive buffer in column-major, TMA-aligned form.  The
 * page "00 DeepEP Engram Architecture Deep-Dive" (§1.1 Python API, §1.2 C++
 * runtime) names the option use_tma_aligned_col_major_sf and does not define
 * it.  Reading taken: the [rows, sf_cols] matrix of 4-byte scale words (fp32
 * scales, or packed exponents: moved verbatim) is stored column after
 * column, column j at recv_sf_cm + j*ld words, and ld is a multiple of 4 so
 * that every column starts on a 16-byte boundary (a TMA global stride must
 * be a multiple of 16 bytes).  Rows follow the layout's inverse map:
 *   recv_sf_cm[j*ld + i] = sf[src[i]*sf_cols + j]   for i < rows, src[i] >= 0;
 * rows with src[i] = -1 (the alignment gaps of the expand layout, [CS] §7.3)
 * are zero in every column when zero_pad != 0 and are not written
 * otherwise; rows >= rows are never written.
 *   sf [N, sf_cols] 4-byte words, 4-byte aligned; sf_cols >= 1;
 *   src: src_idx of moe_layout_build (expand layout) or rank_src of
 *        moe_layout_rank_rows (non-expand layout), entries in [-1, N);
 *   total_rows: device int32[1] holding rows: the total_rows output of
 *        moe_layout_build, or rank_psum + R - 1;
 *   recv_sf_cm [sf_cols, ld] words, 16-byte aligned, ld >= capacity_rows,
 *        ld a multiple of 4.
 * sf_cols above MOE_MAX_ROW_BYTES / 4 or ld above 2^32 return
 * MOE_ERR_UNSUPPORTED.
 * rows > capacity_rows records MOE_ERR_CAPACITY and nothing is written; a
 * src entry outside [-1, N) is skipped and records MOE_ERR_INVALID_ARG.
 * Independent of moe_dispatch_permute: call it instead of passing sf there,
 * on the same stream, after the layout.
 */
MOE_API int moe_dispatch_sf_col_major(const moe_layout_desc* desc, const void* sf, int64_t sf_cols,
                                      const int32_t* src, const int32_t* total_rows, void* recv_sf_cm,
                                      int64_t ld, int64_t capacity_rows, int zero_pad, void* workspace,
                                      size_t workspace_bytes, void* stream);

/*
 * Combine: the inverse of the dispatch.  The pages keep the slot map for it
 * ([CS] §6.2) but print no arithmetic; this is the plain definition
 *   out[t, h] = bf16( sum over k = 0..K-1 with dst_slot[t*K+k] >= 0 of
 *                     weights[t*K+k] * float(expert_out[dst_slot[t*K+k], h]) )
 * accumulated in fp32 from 0 in ascending k with one fused multiply-add per
 * term, rounded once to bf16 (nearest, ties to even).  A token with no valid
 * slot gets zeros.
 *   expert_out bf16 [expert_out_rows, hidden]; out bf16 [N, hidden];
 *   weights fp32 [N*K]; hidden a positive multiple of 8; expert_out and out
 *   16-byte aligned.  Slots >= expert_out_rows are skipped and record
 *   MOE_ERR_CAPACITY.
 */
MOE_API int moe_combine_unpermute(const moe_layout_desc* desc, const void* expert_out,
                          int64_t expert_out_rows, int64_t hidden,
                          const int32_t* dst_slot, const float* weights,
                          void* out, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * moe_layout_build without a caller workspace, for callers that cannot
 * allocate device memory when they build the layout: for example an engine
 * that reserves all of HBM for its own allocator at start-up and forbids
 * cudaMalloc afterwards, a plugin that must not touch its host's memory
 * pool, or a latency-critical loop that cannot afford cudaMalloc's implicit
 * device synchronisation.  The pages have no counterpart to this call; it
 * exists only for such callers.
 *
 * Inputs and outputs are the caller's, exactly as for moe_layout_build.  The
 * scratch is a fixed array of MOE_NOALLOC_SCRATCH_BYTES inside the library,
 * which every GPU that loads the library holds until the process exits.
 *  - Problems whose workspace (moe_layout_workspace_bytes) is larger than
 *    that are rejected with MOE_ERR_UNSUPPORTED before anything is launched.
 *  - The first call on a device looks up the array's device address (with
 *    that device current) and caches it for that device's CUDA context; make
 *    that first call before any stream capture.  After a device reset the
 *    device has a new context and the array may sit at a new address: the
 *    first call in the new context looks it up again (again outside capture).
 *  - Every call on a device shares the array.  Each call clears the parts
 *    that must start at zero, but calls that overlap on the GPU (different
 *    streams, no ordering between them) race on it and give wrong results.
 *  - device_error: device int32 [1] that receives this call's device-side
 *    status (MOE_OK, MOE_ERR_BAD_EXPERT_ID, MOE_ERR_CAPACITY, MOE_ERR_TIMEOUT),
 *    written on `stream` after the layout.
 * Allocates nothing: no cudaMalloc, cudaFree or allocating library routine.
 */
#define MOE_NOALLOC_SCRATCH_BYTES (1u << 20)
MOE_API int moe_layout_build_noalloc(const moe_layout_desc* desc, const int64_t* topk_idx,
                                     int32_t* expert_count, int32_t* rank_count,
                                     int32_t* expert_offset, int32_t* rank_psum,
                                     int32_t* dst_slot, int32_t* src_idx, int64_t capacity_rows,
                                     int32_t* total_rows, int32_t* device_error, void* stream);

/*
 * Running receive statistics ([CS] §7.2 keeps per-expert totals across
 * calls next to the alignment step): cumulative[e] += expert_count[e] for
 * every e, on `stream`, after a layout call.  cumulative is a caller-owned
 * device int64 [E] the caller zeroes once.
 */
MOE_API int moe_layout_accumulate_stats(const moe_layout_desc* desc, const int32_t* expert_count,
                                        int64_t* cumulative, void* stream);

/*
 * Dispatch straight from host memory: the ids (and, if given, the top-k
 * weights and fp8 scale factors) are copied to the caller's device staging
 * buffers, the layout is built (moe_layout_build), and the token rows are
 * copied in chunks of chunk_tokens tokens (0 = one chunk) on copy_stream
 * while the permute (moe_dispatch_permute, zero padding on the first chunk)
 * of each chunk runs on `stream` as soon as its rows have landed.  Results
 * and errors are those of the two calls; on return everything is enqueued
 * on `stream` (copy_stream is joined into it).  Host buffers must be
 * page-locked for the copies to overlap.  A pipeline around the method's
 * steps; the pages have no counterpart to it.
 *   topk_idx_host [N*K] int64, x_host [N, row_bytes], sf_host [N, sf_row_bytes]
 *   or NULL, weights_host [N*K] fp32 or NULL (with weights NULL too);
 *   topk_idx, x, sf, weights: device buffers of the same sizes.
 */
MOE_API int moe_dispatch_from_host(const moe_layout_desc* desc, const int64_t* topk_idx_host,
                                   const void* x_host, int64_t row_bytes, const void* sf_host,
                                   int64_t sf_row_bytes, const float* weights_host,
                                   int64_t* topk_idx, void* x, void* sf, float* weights,
                                   int32_t* expert_count, int32_t* rank_count,
                                   int32_t* expert_offset, int32_t* rank_psum,
                                   int32_t* dst_slot, int32_t* src_idx, int32_t* total_rows,
                                   void* recv_x, void* recv_sf, int64_t capacity_rows,
                                   void* workspace, size_t workspace_bytes,
                                   int64_t chunk_tokens, void* stream, void* copy_stream);

/*
 * Combine straight to host memory: moe_combine_unpermute runs in chunks of
 * chunk_tokens tokens (0 = one chunk) on `stream` into the device buffer
 * `out` [N, hidden] bf16, and each chunk is copied to out_host on
 * copy_stream while the next chunk is combined; copy_stream is joined into
 * `stream` at the end, so synchronising `stream` covers the copies.
 * out_host must be page-locked for the copies to overlap.  A pipeline
 * around the method's steps; the pages have no counterpart to it.
 */
MOE_API int moe_combine_to_host(const moe_layout_desc* desc, const void* expert_out,
                                int64_t expert_out_rows, int64_t hidden,
                                const int32_t* dst_slot, const float* weights, void* out,
                                void* out_host, void* workspace, size_t workspace_bytes,
                                int64_t chunk_tokens, void* stream, void* copy_stream);

/* ------------------------------------------------------------------------
 * Around the layout: the gate that makes topk_idx and the weights, the 8-bit
 * rows the dispatch moves, and the expert products on the receive buffer.
 * The pages leave all of these to the caller; the formulas below are plain
 * definitions.  None of these kernels releases its dependents early, so their
 * outputs may be passed to the layout and dispatch calls directly.
 */

/* Gate settings.  Plain values, copied by every call. */
typedef struct moe_gate_desc {
  int32_t logits_bf16;   /* 0: fp32 logits (and gradient), 1: bf16                    */
  int32_t sigmoid;       /* scores: 0 softmax over the experts, 1 sigmoid             */
  int32_t normalize;     /* 1: a token's weights sum to scale                         */
  float scale;           /* factor of the weights                                     */
  float balance_coef;    /* factor of the balance loss                                */
} moe_gate_desc;

/* Bytes of the gate's workspace: its error word (read with
 * moe_layout_get_error) and the partial sums of the forward call.  Zero-fill
 * once; one stream at a time. */
MOE_API int moe_gate_workspace_bytes(const moe_layout_desc* desc, size_t* bytes);

/*
 * Top-k gate with per-expert counts and balance loss.  For token t with logits
 * l (row t at logits + t * logits_stride elements; columns contiguous):
 *   key_e = l_e + bias_e in fp32 (bias may be NULL: 0); the K largest keys, in
 *     descending order, equal keys by ascending id; a key of -inf is never
 *     taken, so l_e = -inf closes expert e for the token;
 *   the bias counts for this choice alone.  It is not a bias of the score: gates that
 *     choose by sigmoid(l_e) + b_e or softmax(l)_e + b_e choose other experts;
 *   s = softmax(l) or sigmoid(l) (without the bias), q = s / sum_e s;
 *   topk_idx[t*K+k] = id (int64), weights[t*K+k] = scale * s_id / D with
 *     D = the sum of the token's picked s if normalize, else 1; slots without
 *     an expert get id -1 and weight 0.
 * Tokens without a key above -inf are not routed (ids -1, weights 0).  Tokens
 * with a NaN or +inf key are treated the same and record MOE_ERR_INVALID_ARG
 * in the workspace.  Over the T routed tokens:
 *   expert_count[E], routed_tokens[1] = T,
 *   prob_mean[E] = (1/T) sum_t q, balance_loss[1] =
 *     balance_coef * E * sum_e (expert_count[e] / (K*T)) * prob_mean[e]
 * (zeros if T = 0).  Everything is fp32 and does not change from run to run; what is
 * below 2^-126 may come out as zero.
 * alignment and num_ranks of desc are not used.
 */
MOE_API int moe_gate_forward(const moe_layout_desc* desc, const moe_gate_desc* gate, const void* logits,
                             int64_t logits_stride, const float* bias, int64_t* topk_idx, float* weights,
                             int32_t* expert_count, float* prob_mean, int32_t* routed_tokens,
                             float* balance_loss, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of weights and balance_loss with respect to the logits, from the
 * forward call's logits, topk_idx, expert_count and routed_tokens.
 * dweights [N*K] and dloss [1] are fp32 and may each be NULL (zero).  The counts
 * and the choice of experts carry no gradient; the bias gets none.  dlogits
 * [N, dlogits_stride] has the logits' type; tokens that were not routed get 0.
 * dlogits may be the logits themselves (same base and stride).  Otherwise no row of
 * one may touch a row of the other (MOE_ERR_INVALID_ARG; ranges that interleave
 * need equal strides).
 */
MOE_API int moe_gate_backward(const moe_layout_desc* desc, const moe_gate_desc* gate, const void* logits,
                              int64_t logits_stride, const int64_t* topk_idx, const int32_t* expert_count,
                              const int32_t* routed_tokens, const float* dweights, const float* dloss,
                              void* dlogits, int64_t dlogits_stride, void* workspace, size_t workspace_bytes, void* stream);

/* Groups of experts: E / num_groups side by side.  Plain values, copied by every call. */
typedef struct moe_gate_groups {
  int32_t num_groups;    /* G, 1 <= G <= MOE_MAX_GROUPS, divides E                         */
  int32_t topk_groups;   /* groups a token's experts come from, 1 .. G                     */
  int32_t group_sum;     /* a group's score: the sum of its 1 or 2 largest keys            */
} moe_gate_groups;
#define MOE_MAX_GROUPS 32

/*
 * moe_gate_forward with experts chosen by score and limited to the best groups
 * (same arguments, outputs, workspace and errors otherwise; the gradient is
 * moe_gate_backward):
 *   key_e = s_e + bias_e, s = softmax(l) or sigmoid(l) (bias may be NULL: 0); an expert
 *     with l_e or bias_e = -inf is closed: its key is -inf and never taken;
 *   a group's score is the sum of its group_sum largest keys above -inf (of one, if it
 *     has no other); the topk_groups groups of the largest scores stay, equal scores by
 *     ascending group; a group whose experts are all closed never does;
 *   the K largest keys of those groups, in descending order, equal keys by ascending id;
 *   ids, weights (of s, without the bias), counts and balance loss as in moe_gate_forward.
 * Keys are compared as numbers, not as what 32 bits make of them: what fp32 leaves open is
 * settled to about 2^-46 (scores below 2^-124 may count as zeros there).  Where all biases
 * are equal the order of experts, and of groups with group_sum 1, is that of the logits;
 * sums of two are compared as sums of such keys: two that lie closer together than
 * that, saturated sigmoids for instance, may count as equal, and equal ones of different
 * scores (s(x) + s(-x) is 1 for every x) as different.
 * Tokens with a NaN or +inf among their logits or keys are not routed and record
 * MOE_ERR_INVALID_ARG.
 */
MOE_API int moe_gate_forward_grouped(const moe_layout_desc* desc, const moe_gate_desc* gate,
                                     const moe_gate_groups* groups, const void* logits, int64_t logits_stride,
                                     const float* bias, int64_t* topk_idx, float* weights, int32_t* expert_count,
                                     float* prob_mean, int32_t* routed_tokens, float* balance_loss,
                                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of moe_combine_unpermute's sum: for every valid (t, k)
 *   dy[dst_slot[t*K+k], h] = bf16(weights[t*K+k] * float(dout[t, h]))
 *   dweights[t*K+k] = sum_h float(dout[t, h]) * float(expert_out[dst_slot[t*K+k], h])
 * in fp32, in an order that does not change from run to run; dweights of a masked
 * slot is 0.  dweights may be NULL, and expert_out with it.  With zero_pad != 0 the
 * alignment-gap rows of dy are set to zero (expert_offset and expert_count as written by
 * the layout; NULL allowed otherwise) unless expert_offset[E] > capacity_rows, a layout
 * that did not fit; rows past the last segment are not written.
 *   dout bf16 [N, hidden], expert_out and dy bf16 [capacity_rows, hidden]; hidden a
 *   positive multiple of 8; 16-byte aligned.  dy may be expert_out itself (written in
 *   place); other overlaps are refused.  Slots >= capacity_rows are skipped (their
 *   dweights are 0) and record MOE_ERR_CAPACITY.
 */
MOE_API int moe_combine_backward(const moe_layout_desc* desc, const void* dout, int64_t hidden,
                                 const int32_t* dst_slot, const float* weights, const void* expert_out,
                                 void* dy, int64_t capacity_rows, float* dweights, const int32_t* expert_offset,
                                 const int32_t* expert_count, int zero_pad, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Norm settings.  Plain values, copied by every call. */
typedef struct moe_norm_desc {
  int64_t rows;          /* rows >= 0                                                      */
  int64_t cols;          /* a positive multiple of 16, at most MOE_MAX_NORM_COLS           */
  float eps;             /* 2^-126 .. 2^88: beside others what fp32 loses of squares counts */
  int32_t stream_fp32;   /* residual stream (residual, residual_out, z, dz): 0 bf16, 1 fp32 */
  int32_t weight_fp32;   /* weight: 0 bf16, 1 fp32                                         */
} moe_norm_desc;
#define MOE_MAX_NORM_COLS 32768

/*
 * Residual addition and root-mean-square norm, with the normed rows in bf16, in 8 bits
 * or both.  For every row:
 *   z = x + residual, rounded to the stream's type and written to residual_out
 *       (residual and residual_out both NULL: z = x, and the stream must be bf16);
 *   r = 1 / sqrt(mean_j z_j^2 + eps);  v_j = z_j * r * weight_j, in fp32;
 *   y = bf16(v);
 *   q, sf = v quantised as by moe_quantize_rows (sf_ld as there: 0 row-major for
 *       moe_dispatch_permute, > 0 column-major for moe_expert_gemm_fp8);
 *   rstd[row] = r, for moe_rms_norm_backward.
 *   x bf16 [rows, cols]; y, q (with sf) and rstd may each be NULL, but not both y and q.
 *   16-byte aligned bases (rstd, sf: 4).  residual_out may be residual itself, and any
 *   bf16 output any bf16 input; other overlaps are refused.
 * total_rows (device int32, may be NULL): rows in use; later rows are neither read nor
 * written.
 */
MOE_API int moe_rms_norm(const moe_norm_desc* norm, const void* x, const void* residual, const void* weight,
                         const int32_t* total_rows, void* residual_out, void* y, void* q, float* sf,
                         int64_t sf_ld, float* rstd, void* stream);

/* Bytes of the gradient's workspace (16-byte aligned; it need not be zero-filled; one
 * stream at a time). */
MOE_API int moe_rms_norm_workspace_bytes(const moe_norm_desc* norm, size_t* bytes);

/*
 * Gradient of moe_rms_norm.  z is the call's residual_out (its x, without a residual),
 * rstd its rstd, dy bf16 the gradient of v, dresidual that of residual_out from elsewhere
 * (the stream's type; may be NULL).  With g = dy * weight and h = z * rstd:
 *   dz = rstd * (g - h * mean_j(g_j h_j)) + dresidual: the gradient of x and of residual,
 *       in the stream's type;  dx: the same in bf16 (may be NULL);
 *   dweight[j] = sum over the rows of dy_j h_j in fp32 (may be NULL); accumulate != 0 adds
 *       to what it holds.  The order of the sum does not change from run to run.
 * dz may be dresidual, z or (bf16) dy, and dx dy; other overlaps are refused.  eps is not
 * used.  workspace may be NULL without dweight.
 */
MOE_API int moe_rms_norm_backward(const moe_norm_desc* norm, const void* dy, const void* z, const float* rstd,
                                  const void* weight, const void* dresidual, const int32_t* total_rows,
                                  void* dz, void* dx, float* dweight, int accumulate, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * bf16 rows to e4m3 with one fp32 scale for each 1x128 block (the last block of
 * a row may be shorter):
 *   sf = max(max|x|, 1e-30) / 448, q = e4m3(x * (1 / sf)), nearest even.
 *   x bf16 [rows, cols], q [rows, cols]: cols a positive multiple of 16, bases
 *   16-byte aligned; B = ceil(cols / 128) scales a row:
 *   sf_ld == 0: row-major [rows, B], as moe_dispatch_permute takes them;
 *   sf_ld > 0:  column-major [B, sf_ld], sf_ld >= rows and a multiple of 4, as
 *               moe_dispatch_sf_col_major writes them and moe_expert_gemm_fp8
 *               reads them.
 * total_rows (device int32, may be NULL): rows in use; later rows are neither
 * read nor written.
 */
MOE_API int moe_quantize_rows(const void* x, int64_t rows, int64_t cols, const int32_t* total_rows, void* q,
                              float* sf, int64_t sf_ld, void* stream);

/*
 * silu(gate) * up of rows [gate | up] (bf16 [rows, 2 * width]), quantised as by
 * moe_quantize_rows with column-major scales [ceil(width / 128), sf_ld].
 */
MOE_API int moe_swiglu_quantize(const void* gate_up, int64_t rows, int64_t width, const int32_t* total_rows,
                                void* q, float* sf, int64_t sf_ld, void* stream);

/*
 * Gradient of silu(gate) * up: gate_up bf16 [rows, 2 * width], dh bf16
 * [rows, width], dgate_up bf16 [rows, 2 * width]; width a multiple of 8.
 */
MOE_API int moe_swiglu_backward(const void* gate_up, const void* dh, int64_t rows, int64_t width,
                                const int32_t* total_rows, void* dgate_up, void* stream);

/*
 * Receive rows to transposed e4m3 with one scale for each block of 128 rows of a
 * column: the operands of moe_expert_wgrad_fp8.
 *   x bf16 [capacity_rows, cols], cols a multiple of 8; q [cols, ld] with
 *   ld >= capacity_rows rounded up to 128, a multiple of 128; sf
 *   [ceil(capacity_rows / 128), cols].  Rows in the alignment gaps count as
 *   zeros whatever they hold.  Row blocks past the last segment are not written.
 * desc->alignment must be a multiple of 128 (MOE_ERR_UNSUPPORTED otherwise).  With a
 * segment that does not start at a multiple of 128 nothing is written and
 * MOE_ERR_INVALID_ARG is recorded in the workspace.
 */
MOE_API int moe_quantize_cols(const moe_layout_desc* desc, const void* x, int64_t capacity_rows, int64_t cols,
                              const int32_t* expert_offset, const int32_t* expert_count, void* q, int64_t ld,
                              float* sf, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Expert product on the receive buffer.  For every row r of expert e
 * (expert_offset[e] <= r < expert_offset[e] + expert_count[e]) and output o:
 *   out[r, o] = bf16( sum_b x_sf[b, r] * w_sf[e, o / 128, b] *
 *                           sum_{i in block b} x[r, i] * w[e, o, i] )
 * over the 128-wide blocks b of width_in; products and sums in fp32, rounded
 * once.  Rows in the alignment gaps of out are set to zero; later rows are not
 * written.  Rows of x outside the segments' real rows are never used, whatever
 * they hold.
 *   x e4m3 [capacity_rows, width_in], x_sf fp32 [ceil(width_in / 128), sf_ld]
 *   (column-major), w e4m3 [E, width_out, width_in], w_sf fp32
 *   [E, ceil(width_out / 128), ceil(width_in / 128)], out bf16
 *   [capacity_rows, width_out]; width_in a multiple of 16, width_out of 8;
 *   x, w and out 16-byte aligned.
 * The input gradient is the same call with the weights (and their scales)
 * transposed.  A single dense product is E = 1.  desc->num_tokens * topk is the
 * number of pairs the layout was built for: it chooses the tiling, not the result's
 * meaning.
 */
MOE_API int moe_expert_gemm_fp8(const moe_layout_desc* desc, const void* x, const float* x_sf, int64_t sf_ld,
                                int64_t capacity_rows, int64_t width_in, const void* w, const float* w_sf,
                                int64_t width_out, const int32_t* expert_offset, const int32_t* expert_count,
                                void* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Weight gradient of the expert product.  For every expert e, with b over the
 * 128-row blocks of its segment:
 *   dw[e, o, i] = sum_b dy_sf[b, o] * x_sf[b, i] * sum_{r in block b} dy[o, r] * x[i, r]
 * (0 for an expert without rows), from operands as moe_quantize_cols writes
 * them: dy [width_out, ld], dy_sf [ceil(capacity_rows/128), width_out],
 * x [width_in, ld], x_sf [ceil(capacity_rows/128), width_in].
 * dw is [E, width_out, width_in], bf16 (dw_fp32 == 0) or fp32; accumulate != 0
 * adds to what an fp32 dw holds, in fp32 (values below 2^-126 in magnitude may
 * count as zeros there); an expert without rows then keeps its dw as it is.
 * width_in a multiple of 8.  desc->alignment must be a multiple of 128.
 */
MOE_API int moe_expert_wgrad_fp8(const moe_layout_desc* desc, const void* dy, const float* dy_sf, const void* x,
                                 const float* x_sf, int64_t ld, int64_t capacity_rows, int64_t width_out,
                                 int64_t width_in, const int32_t* expert_offset, const int32_t* expert_count,
                                 void* dw, int dw_fp32, int accumulate, void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * Synchronise `stream`, copy the workspace's sticky error word (the first
 * device-side error since the last read; MOE_OK if none) into
 * *device_error, and reset it to MOE_OK.
 */
MOE_API int moe_layout_get_error(void* workspace, int32_t* device_error, void* stream);

/* Static, human-readable name of a status code. */
MOE_API const char* moe_strerror(int status);

/* Number of kernels this library has launched in this process so far. */
MOE_API uint64_t moe_kernel_launches(void);

/*
 * Test hook for the bounded waits (not for normal use; process-wide; affects
 * launches made after the call).  Every wait inside the library's kernels
 * gives up after limit_ns nanoseconds (0: the default, 1 s; at most 1 s),
 * records MOE_ERR_TIMEOUT and lets the kernel finish.  barrier_extra > 0
 * raises the cooperative layout kernel's grid-barrier targets past the number
 * of CTAs, so its first barrier can only run out; extra_tx (a multiple of 16)
 * adds transaction bytes that no copy delivers to each CTA's first stage of
 * the dynamic permute and of the expert products, so that stage can only run
 * out.  A layout that timed
 * out leaves its workspace's barrier counter set: zero the workspace before
 * reusing it.  Call with (0, 0, 0) to restore normal operation.
 */
MOE_API int moe_debug_set_waits(uint64_t limit_ns, uint32_t barrier_extra, uint32_t extra_tx);

/*
 * The CUDA error code (cudaError_t) behind this thread's most recent
 * MOE_ERR_CUDA from any entry point, or 0 if there was none; *message (if
 * non-NULL) receives its description.  Diagnostics only: a status the pages
 * do not define.
 */
MOE_API int moe_last_cuda_error(const char** message);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYOUT_H_ */
