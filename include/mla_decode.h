/*
 * mla_decode.h -- C ABI of libmla_decode.so: absorbed multi-head latent
 * attention (MLA) decode on GB300 (sm_103a).
 *
 * The operation (one query token per request, per head):
 *
 *   for request b with context rows K_b = kv_cache[kv_indices[kv_indptr[b] .. kv_indptr[b+1])]
 *   and head h with q = [q_nope[b,h,0:512], q_rope[b,h,0:64]]:
 *       s_t        = sm_scale * (q_nope . c_t + q_rope . k_rope_t)     c_t = row[0:512], k_rope_t = row[512:576]
 *       lse[b,h]   = ln sum_t exp(s_t)
 *       out[b,h,:] = sum_t softmax(s)_t * c_t                            (the latent is also the value)
 *
 * Sources: "实现差距：MLA 与 DeepSeek V3", section 2.4 (MLA Pallas kernel V2,
 * core computation: dual-path score, FA2-style online softmax, kv_c reused as
 * the value) and section 2.1 (the 576-wide row: kv_latent 512 then k_rope 64);
 * "Attention backends", paragraphs "MLA" (one 576-wide vector per token shared
 * by all heads) and "Paged, ragged batches" (page size 1, kv_indptr /
 * kv_indices CSR, a host-side plan() that picks split-KV chunking and balances
 * long and short contexts across SMs); "Attention backends", paragraph
 * "FlashAttention" (Flash-Decoding: keys split across blocks, partial results
 * merged with the same rescaling).
 *
 * Conventions for every entry point:
 *   - All memory is owned by the caller; the library never allocates.
 *   - Device pointers must be 16-byte aligned; tensors are dense row-major.
 *   - bf16 means IEEE bfloat16 (the bits of the upper half of an fp32).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *   - No function throws or aborts; each returns an mla_status.  Arguments are
 *     checked on the host before any launch; on a bad argument nothing is
 *     launched and nothing is written.
 *   - Supported head counts: 16 and 32 (one CTA per SM) and 48..128 in steps
 *     of 16 (a two-CTA cluster per worker); both work in 64-token tiles.
 *     kv_lora_rank is 512 and qk_rope_head_dim is 64; nothing else is built.
 *     (The prompt side, further down, takes any head count.)
 *   - The natural log is used for every LSE.
 */
#ifndef MLA_DECODE_H_
#define MLA_DECODE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size, malformed kv_indptr, bad plan */
  MLA_ERR_UNSUPPORTED = 2,   /* head count or dtype the library does not build */
  MLA_ERR_WORKSPACE = 3,     /* plan or workspace buffer too small; as a device status: its counters were not zero */
  MLA_ERR_CUDA = 4,          /* a CUDA runtime call failed (launch, attribute, device query) */
  MLA_ERR_TIMEOUT = 5,       /* a device-side wait exceeded its limit (~1 s); the kernel returned early */
  MLA_ERR_INDEX_OOB = 6,     /* a kv_indices value was outside [0, num_slots); row 0 was read instead */
  MLA_ERR_PLAN_MISMATCH = 7, /* a plan work item does not lie inside its request's kv_indptr range */
  MLA_ERR_TREE = 8           /* a draft tree names a parent that is not an earlier draft or -1; that draft
                                was verified as a child of the context */
} mla_status;

/* Human-readable name of a status code (static string, never NULL). */
const char* mla_status_string(int status);

/* Library ABI version (currently 1). */
int mla_abi_version(void);

/* mla_decode_plan -- host only, no device work, deterministic.
 *
 * Builds the split-KV work plan for one decode batch ("Attention backends",
 * paragraph "Paged, ragged batches": plan() rebuilt on the CPU per batch,
 * choosing per-request chunking and balancing long and short contexts).
 *
 *   kv_indptr          host int32[batch+1]; kv_indptr[0] == 0, non-decreasing.
 *   batch              number of requests B >= 0.
 *   num_heads          H (see supported head counts above).
 *   num_sms            SMs to plan for; 0 = query the current CUDA device.
 *   plan               host int32 buffer of plan_words words that receives the
 *                      plan, or NULL to only report the sizes.
 *   plan_words_needed  out: words the plan takes (always written when non-NULL).
 *   workspace_bytes    out: device workspace bytes mla_decode_run needs for this
 *                      plan (fp32 partial states plus a 256-byte status header).
 *
 * Rule: tiles of T = 64 tokens; W workers = SMs (H <= 32) or SMs/2; a piece
 * of n tokens costs its whole tiles plus 32 tokens (its epilogue); requests,
 * in order, are poured into workers 0, 1, ... each up to a load budget, so a
 * request is cut only where a worker is full and only at a tile boundary of
 * the request (no cut piece shorter than 64 tokens); the budget starts at the
 * balanced share and grows in steps of 8 tokens until W workers suffice.
 * Requests left whole are written straight to out/lse; cut or empty requests
 * go through the LSE merge.
 *
 * Returns MLA_OK, MLA_ERR_INVALID_ARG (malformed kv_indptr, negative batch),
 * MLA_ERR_UNSUPPORTED (head count), MLA_ERR_WORKSPACE (plan too small; sizes
 * are still reported) or MLA_ERR_CUDA (num_sms == 0 and no device).
 */
int mla_decode_plan(const int32_t* kv_indptr, int32_t batch, int32_t num_heads, int32_t num_sms,
                    int32_t* plan, size_t plan_words, size_t* plan_words_needed,
                    size_t* workspace_bytes);

/* mla_decode_run -- asynchronous on `stream`.
 *
 *   plan_host     host copy of the plan words from mla_decode_plan (read now).
 *   plan_dev      device copy of the same words (read by the kernels).
 *   q_nope        device bf16 [batch, H, 512]: q_nope already multiplied by W_UK.
 *   q_rope        device bf16 [batch, H, 64]: the rotary part of the query.
 *   kv_cache      device bf16 [num_slots, 576]: latent [0,512) then rope key [512,576).
 *   num_slots     rows in kv_cache (1 .. 2^31-1).
 *   kv_indptr     device int32 [batch+1], equal to the host array the plan was built from.
 *   kv_indices    device int32 [kv_indptr[batch]]: slot of every context token.
 *   sm_scale      softmax scale applied to the summed score.
 *   out           device [batch, H, 512], fp32 (out_dtype 0) or bf16 (out_dtype 1).
 *   lse           device fp32 [batch, H] (natural log), or NULL to skip it.
 *   workspace     device buffer of at least the planned workspace_bytes; must be
 *                 zero-filled before its first use (its first 256 bytes hold the
 *                 sticky device status read by mla_check_errors).
 *
 * Launches the decode kernel and, when the plan cut or left empty any request,
 * the merge kernel.  An empty request (kv_indptr[b+1] == kv_indptr[b]) gets
 * out = 0 and lse = -inf.  When no request has a token the decode kernel is
 * not launched (q_nope, q_rope, kv_cache, kv_indptr and kv_indices may then be
 * NULL) and the merge alone writes out and lse; with batch == 0 nothing is
 * launched and only plan_dev and workspace are checked (the other device
 * pointers may be NULL).  Device-side faults are not possible from bad indices: an
 * index outside [0, num_slots) reads row 0 and sets MLA_ERR_INDEX_OOB in the
 * workspace status.  The call does not synchronise; read device-side status
 * with mla_check_errors.  Safe to capture in a CUDA graph (no host sync, no
 * allocation) as long as the plan words stay unchanged.
 */
int mla_decode_run(const int32_t* plan_host, const int32_t* plan_dev,
                   const void* q_nope, const void* q_rope,
                   const void* kv_cache, int64_t num_slots,
                   const int32_t* kv_indptr, const int32_t* kv_indices,
                   float sm_scale, void* out, int32_t out_dtype, float* lse,
                   void* workspace, size_t workspace_bytes, void* stream);

/* mla_decode_attend / mla_decode_merge -- the two launches of mla_decode_run,
 * callable separately (same arguments and checks).  mla_decode_attend runs
 * the decode kernel: requests the plan left whole get their out/lse, cut
 * requests leave fp32 partial states in the workspace.  mla_decode_merge then
 * combines the partials of every cut request (and writes out = 0, lse = -inf
 * for empty requests); it launches nothing when the plan has no such request.
 * mla_decode_run == mla_decode_attend followed by mla_decode_merge. */
int mla_decode_attend(const int32_t* plan_host, const int32_t* plan_dev,
                      const void* q_nope, const void* q_rope,
                      const void* kv_cache, int64_t num_slots,
                      const int32_t* kv_indptr, const int32_t* kv_indices,
                      float sm_scale, void* out, int32_t out_dtype, float* lse,
                      void* workspace, size_t workspace_bytes, void* stream);

int mla_decode_merge(const int32_t* plan_host, const int32_t* plan_dev, void* out,
                     int32_t out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                     void* stream);

/* mla_merge_states -- asynchronous on `stream`.
 *
 * Flash-Decoding merge ("Attention backends", paragraph "FlashAttention"):
 * for request b, partial states i in [merge_indptr[b], merge_indptr[b+1]):
 *   M = max_i s_i;  w_i = exp(s_i - M);  out = sum_i w_i v_i / sum_i w_i;
 *   lse = M + ln sum_i w_i.
 * Partials with s_i = -inf carry no weight; a request with no live partial
 * gets out = 0 and lse = -inf.
 *
 *   v_partial     device fp32 [P, H, 512], each partial already normalised.
 *   s_partial     device fp32 [P, H], the partial LSEs (natural log).
 *   merge_indptr  device int32 [batch+1], non-decreasing, merge_indptr[0] == 0.
 *   out, lse      as for mla_decode_run (lse may be NULL).
 */
int mla_merge_states(const float* v_partial, const float* s_partial, const int32_t* merge_indptr,
                     int32_t batch, int32_t num_heads, void* out, int32_t out_dtype, float* lse,
                     void* stream);

/* mla_decode_run_noalloc -- mla_decode_run without a caller-provided workspace.
 *
 * No counterpart on the pages: this entry point exists for callers that are
 * not allowed to allocate device memory at the point of the call -- code
 * running inside a memory arena owned by another runtime, plugins that only
 * receive tensors they did not allocate, or a decode step that must not call
 * cudaMalloc while it runs.  It takes the same arguments as mla_decode_run
 * except the workspace: the split-KV partial states and the device status go
 * to one static device buffer of MLA_NOALLOC_SCRATCH_BYTES (32 MiB) that is
 * part of the library image, so every GPU that loads the library holds it
 * until the process exits.
 *
 *   - The first call on a device looks the buffer's device address up for
 *     that device (a runtime query, no allocation); make that first call
 *     before any stream capture.  The address is cached per device and per
 *     CUDA context: after cudaDeviceReset (or anything else that replaces
 *     the device's context) the next call looks it up again, so that call,
 *     too, must not be inside a stream capture.
 *   - Plans whose partial states do not fit (256 B + P*H*513*4 bytes larger
 *     than MLA_NOALLOC_SCRATCH_BYTES) are rejected with MLA_ERR_WORKSPACE
 *     and nothing is launched.
 *   - Every call shares the one buffer: calls that overlap on the GPU (on
 *     different streams, or from different threads) race and corrupt each
 *     other's partial states.  Serialise them on one stream.
 *   - The buffer's status word starts at zero (static initialisation) and,
 *     like a caller workspace's, keeps the first device-side error (bad slot
 *     index, timeout, plan mismatch) of any call until
 *     mla_noalloc_check_errors reads and clears it.
 *   - Nothing here calls cudaMalloc, cudaFree or an allocating routine. */
#define MLA_NOALLOC_SCRATCH_BYTES (32u << 20)
int mla_decode_run_noalloc(const int32_t* plan_host, const int32_t* plan_dev,
                           const void* q_nope, const void* q_rope,
                           const void* kv_cache, int64_t num_slots,
                           const int32_t* kv_indptr, const int32_t* kv_indices,
                           float sm_scale, void* out, int32_t out_dtype, float* lse,
                           void* stream);

/* mla_noalloc_check_errors -- the device status of mla_decode_run_noalloc.
 *
 * Synchronises `stream`, then reads the status word of the static buffer on
 * the current device and clears it when it is non-zero (the same contract as
 * mla_check_errors on a caller workspace).  Returns MLA_OK, the first
 * MLA_ERR_* a kernel recorded since the last read, or MLA_ERR_CUDA when the
 * stream or the copy failed.  It allocates nothing: the word is copied into a
 * host int.  Like the entry point it reports on, it has no counterpart on the
 * pages. */
int mla_noalloc_check_errors(void* stream);

/* mla_merge_two_states -- asynchronous on `stream`.
 *
 * Row-wise merge of two attention states over disjoint key sets, for every
 * row r of `rows` (a row is a request-head pair, 512 wide):
 *   m = max(lse_a, lse_b);  w = exp(lse - m);
 *   out = (w_a o_a + w_b o_b) / (w_a + w_b);  lse = m + ln(w_a + w_b)
 * with -inf states weighing nothing (both -inf: out = 0, lse = -inf).  This
 * is the last step of a shared-prefix cascade ("[sglang] EAGLE 트리 검증
 * 어텐션 최적화", section "들어가며": prefix attention shared by every query,
 * suffix attention per query, the two merged by LSE): the prefix pass runs
 * mla_decode_run once over the prefix rows with the G x H query rows of G
 * requests as the heads of one request (each prefix row gathered once), the
 * suffix pass is an ordinary mla_decode_run, both with fp32 out.
 *   o_a, o_b    device fp32 [rows, 512];  lse_a, lse_b  device fp32 [rows].
 *   out         device [rows, 512], fp32 (0) or bf16 (1); may be o_a.
 *   lse         device fp32 [rows] or NULL; may be lse_a. */
int mla_merge_two_states(const float* o_a, const float* lse_a, const float* o_b, const float* lse_b, int64_t rows,
                         void* out, int32_t out_dtype, float* lse, void* stream);

/* mla_decode_run_multi_query -- asynchronous on `stream`.
 *
 * Verification of q_len draft tokens per request in one pass ("[sglang]
 * EAGLE 트리 검증 어텐션 최적화", section "들어가며": every query attends to
 * the shared context and to its ancestor drafts; this is the chain case).
 * Request b's context of L_b rows (kv_indptr / kv_indices) ends with its
 * q_len drafts; query i (0-based) attends to its first L_b - q_len + 1 + i
 * rows.  The q_len x H query rows are read as the heads of one request, so
 * each cache row is gathered once for all of them:
 *   plan        mla_decode_plan(kv_indptr, B, q_len * H, ...).
 *   q_nope      bf16 [B, q_len, H, 512];  q_rope  bf16 [B, q_len, H, 64].
 *   out, lse    [B, q_len, H, 512] (out_dtype as for mla_decode_run), [B, q_len, H].
 * A query row with no row to attend to (L_b < q_len) gets out = 0, lse = -inf.
 * Both decode kernels apply the per-row limit (q_len * H of 16 or 32: one CTA
 * per worker; 48..128: a two-CTA cluster).
 * Errors: MLA_ERR_INVALID_ARG when q_len < 1 or the plan's head count is not a
 * multiple of q_len; otherwise as for mla_decode_run (q_len = 1 is
 * mla_decode_run). */
int mla_decode_run_multi_query(const int32_t* plan_host, const int32_t* plan_dev, int32_t q_len,
                               const void* q_nope, const void* q_rope, const void* kv_cache, int64_t num_slots,
                               const int32_t* kv_indptr, const int32_t* kv_indices, float sm_scale, void* out,
                               int32_t out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                               void* stream);

/* mla_decode_run_tree -- asynchronous on `stream`.
 *
 * Verification of a TREE of W = q_len draft tokens per request in one pass
 * ("[sglang] EAGLE 트리 검증 어텐션 최적화", section "들어가며": with topk > 1
 * the drafts form a tree, and each query token attends to the verified
 * context and to its own ancestor chain among the drafts).  Request b's
 * context of L_b rows ends with its W drafts in generation order; query i
 * sees the first L_b - W rows and, among the last W, the drafts on its path
 * to the root and itself.  Layouts and plan as for mla_decode_run_multi_query
 * (the W x H query rows are the heads of one request, each cache row is
 * gathered once for all of them), plus:
 *   tree_parents  device int32 [B, W]: parents[b][i] = the draft that draft i
 *                 extends (0 <= parent < i), or -1 for a child of the context.
 *                 Read only.  An entry outside [-1, i) records MLA_ERR_TREE
 *                 (mla_check_errors) and draft i is verified as a child of
 *                 the context.
 *   tree_masks    device uint64 [B, W], 8-byte aligned, caller-owned scratch:
 *                 the call writes each draft's ancestor-or-self bits there
 *                 (a small kernel on `stream`) and the decode kernels read
 *                 them; it must stay allocated until the call's work is done.
 * W = 1 is mla_decode_run.  Both decode kernels apply the masks (W * H of 16
 * or 32: one CTA per worker; 48..128: a two-CTA cluster).
 * Errors: MLA_ERR_INVALID_ARG when W < 1, the plan's head count is not a
 * multiple of W, or tree_parents / tree_masks is null or misaligned;
 * MLA_ERR_UNSUPPORTED when W > 64; otherwise as for mla_decode_run. */
int mla_decode_run_tree(const int32_t* plan_host, const int32_t* plan_dev, int32_t q_len,
                        const int32_t* tree_parents, uint64_t* tree_masks, const void* q_nope, const void* q_rope,
                        const void* kv_cache, int64_t num_slots, const int32_t* kv_indptr, const int32_t* kv_indices,
                        float sm_scale, void* out, int32_t out_dtype, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream);

/* mla_decode_step_host -- one decode step from HOST buffers, asynchronous on `stream`.
 *
 * Plans the batch on the host (mla_decode_plan with the current device's SM
 * count) into `plan`, copies the plan words, q_nope, q_rope, kv_indptr and
 * kv_indices into the caller's device `staging` buffer, runs mla_decode_run
 * there, and copies out and lse back into host memory -- seven
 * cudaMemcpyAsync and the decode's launches.  The kernels go on `stream`,
 * the copies in on `copy_in_stream` and the copies out on `copy_out_stream`
 * when those are not NULL (ordered with the kernels through events), else on
 * `stream`.  With page-locked host buffers every copy is asynchronous: keep
 * the host buffers (and `plan`) unchanged until the copies have passed this
 * step.  A serving loop alternates two staging buffers over consecutive
 * steps with one copy-in and one copy-out stream, so one step's copies
 * overlap its neighbours' kernels.
 *
 *   q_nope, q_rope, kv_indptr, kv_indices, out, lse
 *               HOST buffers, same shapes and dtypes as for mla_decode_run.
 *   kv_cache    device, as for mla_decode_run.
 *   plan        host int32 buffer of plan_words (query the size with
 *               mla_decode_plan(..., plan = NULL, ...)).
 *   staging     device buffer of at least mla_step_staging_bytes(batch,
 *               num_heads, nnz, plan words, out_dtype) bytes.
 *   workspace   device, at least the plan's workspace bytes.
 * Errors: those of mla_decode_plan and mla_decode_run; MLA_ERR_WORKSPACE when
 * staging or workspace is too small; MLA_ERR_INVALID_ARG for null pointers or
 * batch < 1.  Nothing is copied or launched on an error found before the
 * first copy. */
size_t mla_step_staging_bytes(int32_t batch, int32_t num_heads, int64_t nnz, size_t plan_words, int32_t out_dtype);
int mla_decode_step_host(const void* q_nope, const void* q_rope, const int32_t* kv_indptr,
                         const int32_t* kv_indices, int32_t batch, int32_t num_heads, const void* kv_cache,
                         int64_t num_slots, float sm_scale, void* out, int32_t out_dtype, float* lse,
                         int32_t* plan, size_t plan_words, void* staging, size_t staging_bytes, void* workspace,
                         size_t workspace_bytes, void* stream, void* copy_in_stream, void* copy_out_stream);

/* mla_absorb_query -- asynchronous on `stream`.
 *
 * The query side of the absorbing path ("MLA and torch.compile: v0.3's two
 * sources", section "MLA: starting from a 439-line commit": q_nope is
 * multiplied by w_kc before attention): for every request b and head h,
 *   q_nope[b, h, :] = q_pre[b, h, 0:128] . w_kc[h]        (fp32 sums, bf16 result)
 * which is the q_nope that mla_decode_run takes.
 *
 *   q_pre     device bf16 [batch, num_heads, nope_dim], nope_dim = 128.
 *   w_kc      device bf16 [num_heads, nope_dim, 512], row-major per head.
 *   q_nope    device bf16 [batch, num_heads, 512] (written).
 *   workspace NULL, or a decode workspace whose status word records a timeout
 *             (read with mla_check_errors).
 * Errors: MLA_ERR_UNSUPPORTED for nope_dim != 128; MLA_ERR_INVALID_ARG for
 * null or non-16-byte-aligned pointers, batch < 0 or num_heads < 1; nothing
 * is launched then.  batch == 0 launches nothing. */
int mla_absorb_query(const void* q_pre, const void* w_kc, void* q_nope, int32_t batch, int32_t num_heads,
                     int32_t nope_dim, void* workspace, void* stream);

/* mla_project_output -- asynchronous on `stream`.
 *
 * The output side of the absorbing path (same section: the attention's
 * latent output is multiplied by w_vc): for every request b and head h,
 *   out[b, h, :] = o_lat[b, h, 0:512] . w_vc[h]            (fp32 sums)
 *
 *   o_lat     device bf16 [batch, num_heads, 512] (mla_decode_run with
 *             out_dtype 1).
 *   w_vc      device bf16 [num_heads, 512, v_dim], row-major per head, v_dim = 128.
 *   out       device [batch, num_heads, v_dim], fp32 (out_dtype 0) or bf16 (1).
 *   workspace as for mla_absorb_query.
 * Errors as for mla_absorb_query (v_dim != 128 or a bad out_dtype give
 * MLA_ERR_UNSUPPORTED). */
int mla_project_output(const void* o_lat, const void* w_vc, void* out, int32_t out_dtype, int32_t batch,
                       int32_t num_heads, int32_t v_dim, void* workspace, void* stream);

/* mla_append_kv -- asynchronous on `stream`.
 *
 * Writes a decode step's new cache rows: rows[b] (576 bf16: the 512-wide
 * latent, then the 64-wide rope key) goes to kv_cache[slots[b]]
 * ("实现差距：MLA 与 DeepSeek V3", section 2.4: the new token's kv_c and k_pe
 * are written to the cache before attention).  Run it before mla_decode_run
 * on the same stream when the new tokens' slots are in kv_indices.
 *
 *   kv_cache   device bf16 [num_slots, 576], written in place.
 *   slots      device int32 [batch], distinct (two rows to one slot: either may win).
 *   rows       device bf16 [batch, 576].
 *   workspace  NULL, or a decode workspace: a slot outside [0, num_slots) is
 *              skipped and recorded there as MLA_ERR_INDEX_OOB (mla_check_errors).
 * Errors: MLA_ERR_INVALID_ARG for null or non-16-byte-aligned pointers,
 * batch < 0 or num_slots < 1; nothing is launched then. */
int mla_append_kv(void* kv_cache, int64_t num_slots, const int32_t* slots, const void* rows, int32_t batch,
                  void* workspace, void* stream);

/* ---- decode with a device-only plan (CUDA-graph replays) -------------------
 * "Attention backends", paragraphs "Paged, ragged batches" and "The
 * interface": for decode the CSR arrays live in buffers sized for the largest
 * captured batch, so a captured graph replays kernels whose inputs change
 * every step; before each replay the runner writes the new plan into those
 * buffers.  mla_decode_run bakes the host plan's merge count and partial
 * layout into its launches; this variant reads everything that changes from
 * the device plan, so one capture serves every plan built for the same
 * (max_batch, num_heads, num_sms). */

/* mla_decode_graph_sizes -- host.  Capacities for plans of up to max_batch
 * requests: *plan_words (int32 words of the device plan buffer) and
 * *workspace_bytes (status header, then room for max_batch + W - 1 partial
 * states, W = the plan's workers).  Any plan mla_decode_plan builds for
 * batch <= max_batch with the same num_heads and num_sms fits.
 * Errors: MLA_ERR_INVALID_ARG for max_batch < 1 or num_sms < 1;
 * MLA_ERR_UNSUPPORTED for an unsupported num_heads. */
int mla_decode_graph_sizes(int32_t max_batch, int32_t num_heads, int32_t num_sms, size_t* plan_words,
                           size_t* workspace_bytes);

/* mla_decode_run_graph -- asynchronous on `stream`; capturable in a CUDA
 * graph and replayable after the buffers' contents change.
 *
 *   plan_dev   device int32 [plan_words]: a plan from mla_decode_plan (same
 *              num_heads and num_sms, batch <= max_batch), copied in before
 *              each launch or replay.  Read only on the device: the kernels
 *              check its header (magic, version, heads, workers, batch, item
 *              count against plan_words) and clamp its ranges; a bad plan
 *              computes nothing and records MLA_ERR_PLAN_MISMATCH.
 *   kv_indptr  device int32 [max_batch + 1]; entries past the plan's batch
 *              repeat its last value.
 *   q_nope, q_rope, out, lse: [max_batch, ...] as for mla_decode_run;
 *              rows of requests past the plan's batch are not written.
 *   workspace  >= the workspace_bytes of mla_decode_graph_sizes, 16-byte
 *              aligned, zero-filled before first use.
 *   other arguments as for mla_decode_run.
 * Launches the decode kernel on the plan's workers and the merge kernel over
 * max_batch possible entries (each block reads the plan's merge count).
 * Errors: MLA_ERR_WORKSPACE when plan_words or workspace_bytes are below the
 * capacities; otherwise as for mla_decode_run, with nothing launched. */
int mla_decode_run_graph(const int32_t* plan_dev, size_t plan_words, int32_t max_batch, int32_t num_heads,
                         int32_t num_sms, const void* q_nope, const void* q_rope, const void* kv_cache,
                         int64_t num_slots, const int32_t* kv_indptr, const int32_t* kv_indices, float sm_scale,
                         void* out, int32_t out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                         void* stream);

/* ---- FP8 latent cache ----------------------------------------------------
 * "MLA and torch.compile: v0.3's two sources", section "MLA: starting from a
 * 439-line commit": an FP8 KV cache is one of the four parts of the 3-7x
 * (the page's FP8 tensors are float8_e4m3fn); "实现差距：MLA 与 DeepSeek V3",
 * section 2.4: new rows are packed into the FP8 cache.  Format taken here:
 * one E4M3 code (OCP "fn" variant: no infinities, largest finite 448) per
 * value, 576 bytes per row (latent 0-511, rope key 512-575), and one float32
 * kv_scale for the whole cache: value = code value x kv_scale. */

/* mla_decode_fp8_workspace_bytes -- host.  Workspace mla_decode_run_fp8 needs
 * for `plan`: the plan's own workspace plus the per-request query images
 * (4 x H x 288 bytes) and per-head factors (H floats).
 * Errors: MLA_ERR_INVALID_ARG for a bad plan or null result pointer. */
int mla_decode_fp8_workspace_bytes(const int32_t* plan_host, size_t* workspace_bytes);

/* mla_decode_run_fp8 -- asynchronous on `stream`.
 *
 * mla_decode_run over an FP8 cache: the same out / lse as the bf16 decode of
 * the cache values (code value x kv_scale), with the bf16 query used as is.
 * Every head count of mla_decode_plan is supported (16 or 32: one CTA per
 * worker; 48..128: a two-CTA cluster; each CTA keeps its own partial score
 * exact and receives its peer's with an error of at most 2^-22 of the largest
 * partial in its 32-token half row).
 *
 *   kv_cache   device uint8 [num_slots, 576] E4M3 codes.
 *   kv_scale   finite, > 0.
 *   workspace  at least mla_decode_fp8_workspace_bytes(plan) bytes, 16-byte
 *              aligned, zero-filled before first use (status word as for
 *              mla_decode_run; the query images are rewritten every call, so
 *              calls sharing a workspace must not overlap on the GPU).
 *   all other arguments as for mla_decode_run.
 * Accuracy: a weight is held to 2^-8 of itself (H >= 48: 2^-9), and what the
 * smallest lose beyond that is at most 2^-5 of all weights together in the worst
 * order of them (measured: below 2^-7), however many rows there are and by
 * whatever factor one of them outweighs the others; the tensor core's sums as for
 * mla_decode_run_fp8_rows with a bf16 out.
 * Launches (H 16 / 32) a query-prep kernel (each request's query split into
 * two E4M3 parts after a per-head power-of-two scaling) and the decode kernel
 * as its programmatic dependent, or (H 48..128) the two-CTA kernel, which
 * splits the query itself; then the plan's merge.
 * Errors as for mla_decode_run; nothing is launched on an argument error. */
int mla_decode_run_fp8(const int32_t* plan_host, const int32_t* plan_dev, const void* q_nope, const void* q_rope,
                       const void* kv_cache, int64_t num_slots, float kv_scale, const int32_t* kv_indptr,
                       const int32_t* kv_indices, float sm_scale, void* out, int32_t out_dtype, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream);

/* mla_append_kv_fp8 -- asynchronous on `stream`.
 *
 * mla_append_kv into an FP8 cache: the codes of rows[b] go to slot slots[b],
 * each value divided by kv_scale in float32 (IEEE division) and rounded to
 * the nearest E4M3 value (ties to the even code, magnitudes past 448 to 448).
 *
 *   kv_cache   device uint8 [num_slots, 576], written in place.
 *   rows       device bf16 [batch, 576].
 *   kv_scale   finite, > 0.
 *   slots, workspace as for mla_append_kv.
 * Errors: MLA_ERR_INVALID_ARG for null or non-16-byte-aligned pointers,
 * batch < 0, num_slots < 1 or a bad kv_scale; nothing is launched then. */
int mla_append_kv_fp8(void* kv_cache, int64_t num_slots, const int32_t* slots, const void* rows, int32_t batch,
                      float kv_scale, void* workspace, void* stream);

/* ---- FP8 latent cache with a scale for every row -------------------------
 * The same 576 codes a row, and a float32 scale for every page of the cache
 * (a page is one row, shared by all heads): value = code value x
 * kv_scales[slot].  A loud token then neither clips nor coarsens the others, and
 * nothing has to be calibrated.  Rows are written by mla_rope_append_kv_fp8_rows
 * (further down, with mla_expand_kv_fp8_rows).  Readers take a scale outside
 * [2^-64, 2^64] as the nearer end, a NaN as 2^-64. */

/* mla_decode_run_fp8_rows -- asynchronous on `stream`.
 *
 * mla_decode_run_fp8 over such a cache.
 *   kv_scales  device float32 [num_slots], 4-byte aligned; read at the slots
 *              that kv_indices names (at slot 0 for one outside the cache).
 *   all other arguments, plan and workspace as for mla_decode_run_fp8.
 * Launches for every head count a kernel that prepares the queries, the decode
 * kernel as its programmatic dependent, and the merge of mla_decode_run; with a
 * bf16 out split requests are merged from float32 states.
 * Accuracy: a weight is held to 2^-8 of itself for a bf16 out, to 2^-16 for a
 * float32 out, and what the smallest lose beyond that is at most 2^-8 (2^-15) of
 * all weights together, however many rows there are (one row may outweigh each of
 * very many others by any factor); their sum is that of the unrounded ones.  The
 * tensor core cuts its sums to 24 bits, towards zero, two (four) times for every
 * 32 rows of an uncut request, so over n rows that add up to one side a result
 * is short of itself by up to n 2^-28 (n 2^-27) in the mean, twice that at most: 1e-3 for
 * a float32 out over 131072 rows, as with the other caches.  The scales of a
 * request's rows may be 2^100 apart (a row of zeros has 2^-64).
 * Errors as for mla_decode_run_fp8, and MLA_ERR_INVALID_ARG for a null or
 * misaligned kv_scales (not looked at when no request has a row). */
int mla_decode_run_fp8_rows(const int32_t* plan_host, const int32_t* plan_dev, const void* q_nope, const void* q_rope,
                            const void* kv_cache, int64_t num_slots, const float* kv_scales, const int32_t* kv_indptr,
                            const int32_t* kv_indices, float sm_scale, void* out, int32_t out_dtype, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream);

/* ---- the prompt side ------------------------------------------------------
 * What stands before the decode: rotary positions, a row's way into the cache,
 * and a prompt's attention in the EXPANDED form (per-head keys and values made
 * from the latents), which takes 192 + 128 multiply-adds a head and pair
 * instead of the absorbed form's 576 + 512 ("MLA and torch.compile: v0.3's two
 * sources", section "MLA: starting from a 439-line commit": prefill takes the
 * ordinary path, decode the absorbing one).  All activations and weights are
 * bf16; strides are in elements, non-negative multiples of 8 below 2^38 (that of
 * a dimension of one is not looked at). */

/* mla_rope_frequencies -- host only.  The rotary frequencies of the 64-wide
 * part, as the 64-bit fractions of a turn per position that the calls below
 * take: freqs[i] = 2^64 f_i / (2 pi), i = 0..31, with inv_i = theta^(-i/32) and
 *   scaling 0 (none)    f_i = inv_i
 *   scaling 1 (linear)  f_i = inv_i / factor
 *   scaling 2 (YaRN)    f_i = inv_i ((1 - r_i) + r_i / factor),
 *                       r_i = clamp((i - lo) / max(hi - lo, 0.001), 0, 1),
 *                       lo = max(floor(p(beta_fast)), 0),
 *                       hi = min(ceil(p(beta_slow)), 63),
 *                       p(beta) = 32 ln(original_positions / (2 pi beta)) / ln theta
 *   theta               finite, > 1;  factor finite, >= 1 (scaling 1 and 2);
 *                       original_positions >= 1, beta_fast >= beta_slow > 0,
 *                       beta_fast finite (scaling 2).  Unused values are not
 *                       looked at.
 *   freqs               host uint64[32], written.
 * The position times freqs[i] modulo 2^64 is the angle as a fraction of a
 * turn.  That product loses nothing at any position; freqs[i] itself comes from
 * double arithmetic and is within 2^-55 of a turn (2^-24 at the farthest position).
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED (another scaling). */
int mla_rope_frequencies(double theta, int32_t scaling, double factor, int32_t original_positions, double beta_fast,
                         double beta_slow, uint64_t* freqs);

/* mla_rope_query -- asynchronous on `stream`.
 *
 * Rotates the rotary part of every head's query by its token's position:
 * with x = the last 64 of the head's nope_dim + 64 values,
 *   (x0, x1) -> amplitude (x0 cos - x1 sin, x1 cos + x0 sin)
 * over pairs (2i, 2i + 1) (interleaved 1) or (i, i + 32) (interleaved 0), in
 * fp32 with one rounding.
 *   q          device bf16: head h of token t at q + t*q_token_stride +
 *              h*q_head_stride, nope_dim values and then the 64 rotary ones.
 *   positions  device int32 [tokens]; any value (a negative one turns back).
 *   nope_dim   a multiple of 8 (0 .. 65536).
 *   freqs      host uint64[32] from mla_rope_frequencies (read now; a captured
 *              graph keeps them).   amplitude  finite factor on cos and sin
 *              (1, or YaRN's ratio of attention scalings).
 *   q_rope     device bf16, written: (t, h) at q_rope + t*rope_token_stride +
 *              h*rope_head_stride.  [tokens, heads, 64] dense is what
 *              mla_decode_run takes; q + nope_dim with q's strides rotates in
 *              place.  Any other overlap with q is not allowed.
 *   q_nope     NULL, or device bf16 [tokens, heads, nope_dim] dense: the rest
 *              of each head is copied there (what mla_absorb_query takes).
 * Errors: MLA_ERR_INVALID_ARG for null or non-16-byte-aligned pointers
 * (positions: 4), tokens < 0, num_heads outside 1 .. 65535, bad strides
 * (q_rope's rows overlapping included); MLA_ERR_UNSUPPORTED for another nope_dim
 * or more than 2^30 - 1 blocks of work (a token and 32 heads; 128 heads where
 * there are many).  Nothing is launched then, nor for tokens == 0. */
int mla_rope_query(const void* q, int64_t q_token_stride, int64_t q_head_stride, const int32_t* positions,
                   int32_t tokens, int32_t num_heads, int32_t nope_dim, const uint64_t* freqs, float amplitude,
                   int32_t interleaved, void* q_rope, int64_t rope_token_stride, int64_t rope_head_stride,
                   void* q_nope, void* stream);

/* mla_rope_append_kv -- asynchronous on `stream`.
 *
 * mla_append_kv for rows as the projection leaves them: the latent is
 * normalised (y = x / sqrt(mean x^2 + eps) * norm_weight over its 512 values;
 * norm_weight NULL: unchanged), the rope key rotated as in mla_rope_query, and
 * the row written to its slot; fp32 arithmetic, one rounding (the sum of squares
 * included: a row whose values pass 2^59 may overflow it and becomes zeros).
 *   kv_cache     device bf16 [num_slots, 576], written in place.
 *   slots        device int32 [tokens], distinct (two rows to one slot: any
 *                part of either may win).
 *   rows         device bf16, token t at rows + t*row_stride: 512 latent
 *                values, then 64 of the rope key; row_stride >= 576 (not
 *                looked at for one token).
 *   norm_weight  device bf16 [512] or NULL;  eps finite, >= 0.
 *   workspace    NULL, or a decode workspace: a slot outside [0, num_slots) is
 *                skipped and recorded there as MLA_ERR_INDEX_OOB.
 *   positions, freqs, amplitude, interleaved: as for mla_rope_query.
 * Errors: MLA_ERR_INVALID_ARG for bad pointers (rows, cache, weight and
 * workspace 16-byte aligned; slots and positions 4), sizes, strides or scalars;
 * nothing is launched then, nor for tokens == 0. */
int mla_rope_append_kv(void* kv_cache, int64_t num_slots, const int32_t* slots, const void* rows, int64_t row_stride,
                       const int32_t* positions, int32_t tokens, const void* norm_weight, float eps,
                       const uint64_t* freqs, float amplitude, int32_t interleaved, void* workspace, void* stream);

/* mla_rope_append_kv_fp8 -- the same into an FP8 cache (uint8 [num_slots, 576]
 * E4M3 codes): the fp32 values are divided by kv_scale (finite, > 0) and
 * rounded once, as in mla_append_kv_fp8. */
int mla_rope_append_kv_fp8(void* kv_cache, int64_t num_slots, const int32_t* slots, const void* rows,
                           int64_t row_stride, const int32_t* positions, int32_t tokens, const void* norm_weight,
                           float eps, const uint64_t* freqs, float amplitude, int32_t interleaved, float kv_scale,
                           void* workspace, void* stream);

/* mla_rope_append_kv_fp8_rows -- the same into a cache with a scale for every
 * row: with m = the largest magnitude of the row's 576 fp32 values (a NaN is not
 * counted), kv_scales[slot] = m / 448 kept inside [2^-64, 2^64], and the codes
 * are those of value x (1 / kv_scales[slot]), rounded once, magnitudes past 448
 * to 448.  A row of zeros gets the scale 2^-64.
 *   kv_scales  device float32 [num_slots], 4-byte aligned, written at the slots. */
int mla_rope_append_kv_fp8_rows(void* kv_cache, float* kv_scales, int64_t num_slots, const int32_t* slots,
                                const void* rows, int64_t row_stride, const int32_t* positions, int32_t tokens,
                                const void* norm_weight, float eps, const uint64_t* freqs, float amplitude,
                                int32_t interleaved, void* workspace, void* stream);

/* mla_expand_kv -- asynchronous on `stream`.
 *
 * Per-head keys and values of cached rows: with c_t = the latent of row
 * kv_indices[t],
 *   k_nope[t, h, n] = sum_r c_t[r] w_kc[h, n, r]      (fp32 sums, bf16 result)
 *   v[t, h, n]      = sum_r c_t[r] w_vc[h, r, n]
 *   k_rope[t, :]    = the row's rope key (shared by all heads, copied)
 * -- what mla_prefill_run takes.  The weights are those of mla_absorb_query
 * and mla_project_output.
 *   kv_cache    device bf16 [num_slots, 576].
 *   kv_indices  device int32 [tokens]; repeats are allowed.  An index outside
 *               [0, num_slots) reads row 0 and records MLA_ERR_INDEX_OOB in the
 *               workspace status, when there is one.
 *   w_kc        device bf16 [num_heads, 128, 512];  w_vc  [num_heads, 512, 128].
 *   k_nope, v   device bf16 [tokens, num_heads, 128];  k_rope  [tokens, 64].
 *   workspace   NULL, or a decode workspace (its status word).
 * Errors: MLA_ERR_INVALID_ARG for null or misaligned pointers (16 bytes;
 * kv_indices 4), tokens < 0, num_heads outside 1 .. 65535, num_slots < 1;
 * MLA_ERR_UNSUPPORTED for more than 2^30 - 1 tiles of work (128 tokens and one
 * head's keys or values); nothing is launched then, nor for tokens == 0. */
int mla_expand_kv(const void* kv_cache, int64_t num_slots, const int32_t* kv_indices, int32_t tokens,
                  const void* w_kc, const void* w_vc, int32_t num_heads, void* k_nope, void* k_rope, void* v,
                  void* workspace, void* stream);

/* mla_expand_kv_fp8 -- the same from an FP8 cache: a value is its E4M3 code
 * times kv_scale (finite, > 0), applied to the fp32 sums. */
int mla_expand_kv_fp8(const void* kv_cache, int64_t num_slots, float kv_scale, const int32_t* kv_indices,
                      int32_t tokens, const void* w_kc, const void* w_vc, int32_t num_heads, void* k_nope,
                      void* k_rope, void* v, void* workspace, void* stream);

/* mla_expand_kv_fp8_rows -- the same from a cache with a scale for every row:
 * kv_scales device float32 [num_slots], 4-byte aligned; each token's fp32 sums
 * are multiplied by its row's scale. */
int mla_expand_kv_fp8_rows(const void* kv_cache, const float* kv_scales, int64_t num_slots, const int32_t* kv_indices,
                           int32_t tokens, const void* w_kc, const void* w_vc, int32_t num_heads, void* k_nope,
                           void* k_rope, void* v, void* workspace, void* stream);

/* mla_prefill_plan -- host only, no device work, deterministic.
 *
 * The work plan of one batch of the expanded attention: tiles of query rows,
 * heaviest first, and, where few rows meet long keys, the cut of their keys
 * into pieces that mla_prefill_run joins.
 *   q_indptr, kv_indptr  host int32 [batch + 1], each from 0, non-decreasing:
 *              request b's queries are rows q_indptr[b] .. q_indptr[b+1] and
 *              its keys kv_indptr[b] .. kv_indptr[b+1] of the packed arrays.
 *   causal     1: with L_q queries and L_k keys, query i sees keys
 *              j <= i + L_k - L_q (the ends aligned: a chunk that continues a
 *              cached context; with L_k < L_q the first rows see nothing);
 *              0: every key of its request.
 *   num_sms, plan, plan_words, plan_words_needed, workspace_bytes: as for
 *   mla_decode_plan.
 * Errors: those of mla_decode_plan; any num_heads of 1 .. 65535 is supported;
 * MLA_ERR_UNSUPPORTED for 2^30 - 1 or more queries or keys, more than 2^31 -
 * 2^16 - 1 tiles over all heads, or 2^16 or more of them with their keys cut. */
int mla_prefill_plan(const int32_t* q_indptr, const int32_t* kv_indptr, int32_t batch, int32_t num_heads,
                     int32_t causal, int32_t num_sms, int32_t* plan, size_t plan_words, size_t* plan_words_needed,
                     size_t* workspace_bytes);

/* mla_prefill_run -- asynchronous on `stream`.
 *
 *   s_ij = sm_scale (q_i . [k_nope_j, k_rope_j]);   lse_i = ln sum_j exp(s_ij);
 *   out_i = sum_j softmax(s_i)_j v_j                 over the keys row i sees.
 * A row that sees no key, or none with a score above -inf, gets out = 0 and
 * lse = -inf, whatever the values are.  Values of keys that a row does not see
 * never reach it.  An infinite or NaN value of a key that it sees with a score
 * above -inf leaves that column of its output infinite or NaN, however small
 * the key's weight (which of the two is not promised once the weight is below
 * 2^-126); with a score of -inf, beside others above it, it may or may not.
 *   plan_host, plan_dev  the words of mla_prefill_plan, on both sides
 *              (plan_dev 16-byte aligned).
 *   q          device bf16: head h of row i at q + i*q_token_stride +
 *              h*q_head_stride, 128 values and then the 64 rotary ones.
 *   k_nope, v  device bf16, 128 values of (row, head) each, with strides (the
 *              halves of one [rows, heads, 256] projection will do).
 *   k_rope     device bf16, 64 values of a row, shared by the heads.
 *              k_nope, k_rope and v are not looked at when there are no keys.
 *   Strides are at least the width of what lies there (192, 128, 64), where
 *   there is more than one row or head, and below 2^38.
 *   out        device bf16 [q rows, heads, 128] dense, apart from the inputs; the weights of the
 *              values are rounded to bf16, sums are fp32.
 *   lse        device fp32 [q rows, heads] or NULL.
 *   workspace  device, at least the plan's workspace_bytes, 16-byte aligned,
 *              zero-filled before first use (status word as for mla_decode_run,
 *              and counters that are zero between calls; calls sharing one must
 *              not overlap on the GPU).  Counters found otherwise are reported as
 *              MLA_ERR_WORKSPACE: rows may be missing, fill it with zeros again.
 * Safe to capture in a CUDA graph.  Errors as for mla_decode_run; with no
 * query row nothing is launched.  A plan_dev that does not lie inside the
 * arrays of plan_host is skipped item by item with MLA_ERR_PLAN_MISMATCH. */
int mla_prefill_run(const int32_t* plan_host, const int32_t* plan_dev, const void* q, int64_t q_token_stride,
                    int64_t q_head_stride, const void* k_nope, int64_t k_token_stride, int64_t k_head_stride,
                    const void* k_rope, int64_t k_rope_stride, const void* v, int64_t v_token_stride,
                    int64_t v_head_stride, float sm_scale, void* out, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream);

/* ---- between two steps ----------------------------------------------------
 * What a speculative serving step does once the target has scored its drafts
 * (mla_decode_run_multi_query, mla_decode_run_tree): decide which drafts hold,
 * cut the requests' lists of rows to them, fork and free requests, and keep the
 * pool of rows in order.  All of it stays on the device, without a host copy or
 * an allocation, and can be captured. */

/* mla_verify_drafts -- asynchronous on `stream`.
 *
 * The walk down each request's drafts ("[sglang] EAGLE 트리 검증 어텐션
 * 최적화", section "들어가며"), from given random numbers.  Draft 0 is the token
 * that the last step ended with: it stands, and target row i is the target's
 * distribution of the token after draft i (what the W = q_len queries of a
 * multi-query or tree decode give).  With node = 0 at first, the node's children
 * c are tried in their order:
 *   sampled drafts (draft_probs; a chain): accepted when u_c q_c(x_c) < t(x_c),
 *       q_c = the draft row c, which draft c was drawn from;
 *   chosen drafts (no draft_probs; a chain or a tree): accepted when
 *       u_c (1 - the t of the node's rejected children so far) < t(x_c); a child
 *       whose token a rejected sibling had counts t = 0;
 * with t = the node's target row, x = tokens, u = uniforms.  An accepted child
 * is the next node; without one the walk ends.  Of what is left of the node's
 * row,
 *   r_v = max(t_v - q_v, 0) after a rejected sampled draft, t_v off the rejected
 *         children's tokens for chosen ones, t_v where nothing was rejected,
 * the next token is the lowest v with sum_(w <= v) r_w > u_0 sum_w r_w, or -1
 * when nothing is left.  The drafts' tests are those of 64-bit arithmetic, and the sums are
 * good to about 2^-45 of the whole; entries are probabilities: values outside
 * [0, 1] count as the nearer end, NaN as 0.  With u_0 >= 1 or NaN the token is
 * the last one with r > 0; u_c is taken as 0 when it is negative or NaN.
 *   target_probs   device fp32: row i of request b at + b*target_batch_stride +
 *                  i*target_row_stride, vocab values together.  Strides in
 *                  elements, 0 .. 2^40 - 1.
 *   draft_probs    NULL, or device fp32 likewise (row 0 is not looked at).
 *   tokens         device int32 [batch, q_len].  A token of a draft other than
 *                  the first outside [0, vocab) is not accepted, and recorded as
 *                  MLA_ERR_INDEX_OOB.
 *   tree_parents   NULL (a chain: draft i extends draft i - 1), or device int32
 *                  [batch, q_len] as for mla_decode_run_tree: parents[0] = -1, an
 *                  earlier draft for the others.  -1 for another than the first
 *                  is a draft that nothing reaches; any other entry outside
 *                  [-1, i) is one too, and recorded as MLA_ERR_TREE.
 *   uniforms       device fp32 [batch, q_len], in [0, 1): entry 0 draws the next
 *                  token, entry c decides on draft c.
 *   path           device int32 [batch, q_len], written: the accepted drafts in
 *                  their order (the first is 0), then -1.
 *   accepted       device int32 [batch], written: how many (at least 1).
 *   next_token     device int32 [batch], written.
 *   workspace      NULL, or a workspace (its status word).
 * Pointers are 4-byte aligned (workspace 16); outputs apart from the inputs.
 * Errors: MLA_ERR_INVALID_ARG for bad pointers, sizes or strides;
 * MLA_ERR_UNSUPPORTED for q_len > 64, a vocab past 2^30, and draft_probs with
 * tree_parents.
 * Nothing is launched then, nor for batch == 0. */
int mla_verify_drafts(const float* target_probs, int64_t target_batch_stride, int64_t target_row_stride,
                      const float* draft_probs, int64_t draft_batch_stride, int64_t draft_row_stride,
                      const int32_t* tokens, const int32_t* tree_parents, const float* uniforms, int32_t batch,
                      int32_t q_len, int32_t vocab, int32_t* path, int32_t* accepted, int32_t* next_token,
                      void* workspace, void* stream);

/* mla_slots_workspace_bytes -- host.  Workspace of the calls below for a pool of
 * num_slots rows (0 for a num_slots outside 1 .. 2^31 - 1).  Zero-filled before
 * its first use; a status word as for mla_decode_run, and a set of slots that is
 * empty between calls, so that calls that share one must not overlap on the GPU.
 * One made for more slots serves a smaller pool as well, called with all of its
 * bytes. */
size_t mla_slots_workspace_bytes(int64_t num_slots);

/* mla_repack_requests -- asynchronous on `stream`.
 *
 * The lists of rows of the next step's requests: request r continues request
 * sources[r] of the old lists (any number may continue the same: forks; what
 * none continues is freed; -1 starts with no rows).  With path and accepted
 * (mla_verify_drafts), the last q_len rows of an old request are its drafts, and
 * its successors keep the rows before them and the accepted drafts' rows, in
 * the path's order; without, all rows.
 *   kv_indptr, kv_indices  device int32 [batch + 1], [entries].
 *   sources     device int32 [new_batch].
 *   path, accepted  both NULL, or device int32 [batch, q_len] and [batch].
 *   new_indptr, new_indices  device int32 [new_batch + 1], [capacity], written;
 *               entries of new_indices past the last list are left as they were.
 *   freed, freed_count  both NULL, or device int32 [freed_capacity] and [1],
 *               written: the slots of the old lists that no new list holds,
 *               ascending, and their number; entries past them are left as they
 *               were.
 *   num_slots   rows of the pool.   workspace  of mla_slots_workspace_bytes.
 * Bad contents are recorded (mla_check_errors), never followed:
 * MLA_ERR_PLAN_MISMATCH for a source outside [-1, batch) (taken as -1), a
 * kv_indptr that leaves [0, entries] or falls (clipped), a request with fewer
 * rows than drafts (kept whole); MLA_ERR_TREE for an accepted or path entry out
 * of range (clipped); MLA_ERR_INDEX_OOB for a slot outside the pool (copied, and
 * freed by no one; looked for only with freed); MLA_ERR_WORKSPACE when a list
 * passes capacity, or the freed slots freed_capacity (the rest is not written).
 * Pointers are 4-byte aligned (workspace 16); outputs apart from the inputs.
 * Errors: MLA_ERR_INVALID_ARG for bad pointers or sizes, one of a pair without
 * the other, a capacity past 2^31 - 2; MLA_ERR_UNSUPPORTED for q_len > 64 (with
 * path), more than 65536 requests with freed, or more than 2^20 new ones;
 * MLA_ERR_WORKSPACE for too small a workspace.  Nothing is launched then. */
int mla_repack_requests(const int32_t* kv_indptr, const int32_t* kv_indices, int64_t entries, int32_t batch,
                        const int32_t* sources, int32_t new_batch, const int32_t* path, const int32_t* accepted,
                        int32_t q_len, int32_t* new_indptr, int32_t* new_indices, int64_t capacity, int64_t num_slots,
                        int32_t* freed, int64_t freed_capacity, int32_t* freed_count, void* workspace,
                        size_t workspace_bytes, void* stream);

/* mla_copy_rows -- asynchronous on `stream`.
 *
 * dst[l, dst_slots[i]] = src[l, src_slots[i]] for i < rows and l < layers: rows
 * of any of the caches here, in all layers at once, with their scales.
 *   src_cache, dst_cache  device, row s of layer l at byte (l * layer_rows + s) *
 *               row_bytes; row_bytes 1152 (bf16) or 576 (FP8).  They may be the
 *               same, when no destination is also a source.
 *   src_scales, dst_scales  both NULL, or device fp32 [layers, layer_rows] (FP8
 *               rows with a scale each).
 *   src_num_slots, dst_num_slots  slots of a layer; layer_rows at least as many
 *               (not looked at for one layer).
 *   src_slots, dst_slots  device int32 [rows]; destinations distinct (of two
 *               rows to one slot any part of either may win).  A pair with a slot
 *               out of range is skipped, and recorded as MLA_ERR_INDEX_OOB.
 *   workspace   NULL, or a workspace (its status word).
 * Caches and workspace are 16-byte aligned, the rest 4.
 * Errors: MLA_ERR_INVALID_ARG; MLA_ERR_UNSUPPORTED for another row_bytes.
 * Nothing is launched then, nor for rows == 0 or layers == 0. */
int mla_copy_rows(const void* src_cache, const float* src_scales, int64_t src_num_slots, int64_t src_layer_rows,
                  const int32_t* src_slots, void* dst_cache, float* dst_scales, int64_t dst_num_slots,
                  int64_t dst_layer_rows, const int32_t* dst_slots, int32_t rows, int32_t layers, int32_t row_bytes,
                  void* workspace, void* stream);

/* mla_compact_cache -- asynchronous on `stream`.
 *
 * Moves the rows that lists name into the lowest slots of the pool, in all
 * layers, and rewrites the lists: with n distinct live slots, the k-th live slot
 * from n on (ascending) goes to the k-th free slot below n; what lies below n
 * stays.  Slots n .. num_slots - 1 are free afterwards (their rows as they were).
 *   kv_cache, kv_scales, layer_rows, layers, row_bytes  as for mla_copy_rows.
 *   kv_indptr   device int32 [batch + 1]: its last entry, at most `entries`, is
 *               how much of kv_indices is live (the lists of mla_repack_requests
 *               as they are).
 *   kv_indices, new_indices  device int32 [entries]; new_indices is written up
 *               to the last list, and may be kv_indices itself.  A slot outside
 *               the pool is recorded as MLA_ERR_INDEX_OOB and kept.
 *   live_count  device int32 [1], written: n.
 *   workspace   of mla_slots_workspace_bytes(num_slots).
 * Errors: MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED (row_bytes),
 * MLA_ERR_WORKSPACE; nothing is launched then. */
int mla_compact_cache(void* kv_cache, float* kv_scales, int64_t num_slots, int64_t layer_rows, int32_t layers,
                      int32_t row_bytes, const int32_t* kv_indptr, int32_t batch, const int32_t* kv_indices,
                      int64_t entries, int32_t* new_indices, int32_t* live_count, void* workspace,
                      size_t workspace_bytes, void* stream);

/* mla_check_errors -- synchronises `stream`, reads the workspace status word,
 * clears it, and returns it (MLA_OK when the kernels found nothing wrong), or
 * MLA_ERR_CUDA if the stream reports a CUDA error. */
int mla_check_errors(void* workspace, void* stream);

/* mla_probe_wait_limit -- asynchronous on `stream`.  A diagnostic of the
 * failure handling, not part of a decode.
 *
 * Every mbarrier wait of the decode and head-product kernels above is bounded:
 * after about 1 s of wall time it gives up, the kernel records MLA_ERR_TIMEOUT in the workspace
 * status word and returns, so a stalled pipeline becomes a status code, not a
 * hung GPU.  This launches one warp whose first thread waits, with that same
 * bounded wait, on a shared-memory barrier that nothing completes: after the
 * limit the status word holds MLA_ERR_TIMEOUT (read and clear it with
 * mla_check_errors) and the context stays usable.  Nothing but the status
 * word is written.
 *
 *   workspace  device, at least 4 bytes, 16-byte aligned (a decode workspace).
 * Errors: MLA_ERR_INVALID_ARG for a null or misaligned workspace; nothing is
 * launched then. */
int mla_probe_wait_limit(void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_DECODE_H_ */
