/*
 * libjfa -- Jagged Flash Attention and GDPA for GB300 (sm_103a).
 *
 * The operation (GEM training-efficiency article, aihot.vn, section "Jagged
 * Sequence Flash Attention"; vibekk.com GEM article, FAQ "Jagged tensor 是什么"):
 * attention computed directly on jagged tensors -- packed values plus offsets --
 * with no padding, where every sequence b attends only within itself.  Query and
 * key/value lengths may differ per sequence ("asymmetric query/key-value
 * lengths"), an additive per-head bias may apply ("custom attention bias"), and the
 * backward pass is provided.  The GDPA mode (same article, section "Generalized
 * Dot-Product Attention (GDPA)") replaces softmax by an elementwise GELU or SiLU
 * with no row normalisation.
 *
 * For sequence b, head h, query row i (0-based within the sequence), key row j:
 *   s_ij   = scale * <q_i, k_j> + bias[h, bucket(|i + (kv_len - q_len) - j|)]
 *   allowed(i, j) = (!causal || j <= i') && (W < 0 || j >= i' - W),  i' = i + (kv_len - q_len)
 *                   (bottom-right causal; optional sliding window of W keys before i')
 *   SOFTMAX: o_i = sum_j softmax_j(s_ij) v_j over allowed j;  lse_i = log sum exp s_ij
 *   GDPA:    o_i = sum_j act(s_ij) v_j over allowed j, act = tanh-GELU or SiLU
 *   bucket(r) = min(31, floor(log2((1 + r)^2)))   (exact integer arithmetic)
 * A row with no allowed key gets o = 0 (and lse = -inf); its gradients are 0.
 *
 * Layout and conventions (all calls):
 *  - Q, O, dO, dQ are [T_q, H, D] row-major (token-major), T_q = q_offsets[B];
 *    K, V, dK, dV are [T_kv, H, D], T_kv = kv_offsets[B].  Contiguous, 16-byte
 *    aligned DEVICE pointers owned by the caller.  lse is fp32 [T_q, H].
 *  - Element type: JFA_BF16 (bfloat16, head_dim 64 or 128; tensor-core products)
 *    or JFA_F32 (float, head_dim 32 or 64; plain fp32 arithmetic on the CUDA cores,
 *    no TF32 rounding; jfa_cache_fwd says what it does).  Accumulation is fp32.
 *  - Values must be finite: a key/value row of a neighbouring sequence is read
 *    (and multiplied by an exact zero weight) at jagged tile edges.
 *  - Calls are asynchronous on `stream` (a cudaStream_t, NULL = legacy default
 *    stream).  jfa_plan_create (which uploads the work lists), jfa_plan_destroy,
 *    jfa_plan_device_status and jfa_plan_kernel_times synchronise; jfa_fwd and
 *    jfa_bwd never do.
 *  - Every call returns a jfa_status; argument errors are detected on the host
 *    before anything is launched.  No call aborts the process.
 *  - A plan is not thread-safe: do not use one plan from two host threads at once.
 */
#ifndef JFA_H
#define JFA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    JFA_OK = 0,
    JFA_ERR_INVALID_ARG = 1,    /* null pointer, bad offsets, misaligned pointer, bad size */
    JFA_ERR_UNSUPPORTED = 2,    /* head_dim / dtype / mode combination not built */
    JFA_ERR_CUDA = 3,           /* a CUDA runtime or driver call failed */
    JFA_ERR_TIMEOUT = 4,        /* a kernel pipeline wait exceeded its limit (device status) */
    JFA_ERR_DEVICE_BOUNDS = 5,  /* a kernel's own bounds check fired (device status) */
    JFA_ERR_PLAN_MISMATCH = 6,  /* the call does not match the plan (mode, head_dim) */
    JFA_ERR_NO_DEVICE = 7,      /* no usable sm_100-family GPU */
    JFA_ERR_SCRATCH_LIMIT = 8   /* the problem needs more scratch than JFA_STATIC_SCRATCH_BYTES */
} jfa_status;

typedef enum { JFA_SOFTMAX = 0, JFA_GDPA_GELU_TANH = 1, JFA_GDPA_SILU = 2 } jfa_mode;
typedef enum { JFA_BF16 = 0, JFA_F32 = 1 } jfa_dtype;
/* JFA_BIAS_RELPOS32: a per-head table [H, 32] indexed by bucket(relative position).
 * JFA_BIAS_DENSE: one fp32 value per (head, sequence, query row, key row), the most
 *   general form of the article's "custom attention bias": [H, P] head-major, with
 *   P = sum_b q_len_b * kv_len_b (jfa_plan_info fact 15).  Sequence b's block starts at
 *   pair_off[b] = sum_{b' < b} q_len_b' * kv_len_b' within each head's row and is
 *   row-major [q_len_b, kv_len_b]: the pair (i, j) is at h * P + pair_off[b] + i * kv_len_b
 *   + j.  Values of masked pairs are never read.  Meant for short sequences: it moves
 *   4 bytes per pair (and 4 more for its gradient), where the table moves none. */
typedef enum { JFA_BIAS_NONE = 0, JFA_BIAS_RELPOS32 = 1, JFA_BIAS_DENSE = 2 } jfa_bias_kind;

typedef struct jfa_plan_t* jfa_plan;

/*
 * Builds the work lists for one batch shape (the planner): validates offsets,
 * splits every (sequence, head) into query tiles (forward, backward dQ) and
 * key/value tiles (backward dK/dV), costs each tile by the tensor-core products it
 * issues (causal tiles stop at the diagonal), and assigns them longest-first to the least loaded
 * CTA of a persistent grid, so that short sequences never leave SMs idle while a
 * long one finishes (the article's point that padding-free kernels otherwise idle
 * SMs when short sequences end early).
 *   q_offsets, kv_offsets: int32[B+1], non-decreasing, offsets[0] == 0; host
 *     pointers, or device pointers when offsets_on_device != 0 (then copied to the
 *     host on `stream`).  Copied; the caller keeps ownership.
 *   The plan's device memory (offsets, work lists, status word) is allocated here
 *   and uploaded on `stream`, which this call synchronises.
 *   B >= 0 sequences, H >= 1 heads, D head_dim, mode a jfa_mode, causal 0/1.
 *   out: receives a library-owned plan; free with jfa_plan_destroy.
 * Errors: INVALID_ARG (bad offsets or sizes), UNSUPPORTED (D not 32/64/128),
 * NO_DEVICE, CUDA.
 */
jfa_status jfa_plan_create(const int32_t* q_offsets, const int32_t* kv_offsets, int32_t B,
                           int32_t H, int32_t D, int32_t mode, int32_t causal,
                           int32_t offsets_on_device, void* stream, jfa_plan* out);

/*
 * jfa_plan_create with a sliding window (aihot.vn GEM article, section
 * "BlockAttention": each token limited to its neighbouring events, O(L * window)
 * work): with window W >= 0, query i attends only to keys i' - W <= j <= i', where
 * i' = i + (kv_len - q_len) is its aligned causal position; the kernels skip every
 * tile outside the band.  window = -1 is jfa_plan_create.  A window requires causal
 * = 1.  Errors: those of jfa_plan_create; INVALID_ARG for window < -1 or a window
 * without causal.
 */
jfa_status jfa_plan_create_ex(const int32_t* q_offsets, const int32_t* kv_offsets, int32_t B,
                              int32_t H, int32_t D, int32_t mode, int32_t causal, int32_t window,
                              int32_t offsets_on_device, void* stream, jfa_plan* out);

/*
 * Shared key/value attention: the in-kernel broadcast (IKBO) of the PyTorch blog
 * "In-Kernel Broadcast Optimization: Co-Designing Kernels for RecSys Inference",
 * section 3 "IKBO Flash Attention" and figure 1.  Many candidate query sets of a
 * request attend to the same user history, and the kernels read each user's keys and
 * values once per use instead of from a copy made per query set.
 *   Query set b (rows q_offsets[b] .. q_offsets[b+1] of Q, O, dO, dQ) attends to the
 *   rows of user u = kv_index[b], kv_offsets[u] .. kv_offsets[u+1] of K and V.  The
 *   results are those of jfa_fwd / jfa_bwd on the broadcast batch, with each query set
 *   holding its own copy of its user's rows.  dK and dV of a user's rows sum over all
 *   of its query sets, and are zero for a user that no query set uses.
 *   kv_offsets: int32[U+1] over the users (T_kv = kv_offsets[U]); kv_index: int32[B],
 *   each in [0, U).  Host arrays, or device arrays with offsets_on_device (copied to the
 *   host on `stream`, which this call synchronises).
 *   Causal alignment, the sliding window and the bias use each query set's q_len and
 *   its user's kv_len, as in jfa_plan_create_ex.  A dense bias (JFA_BIAS_DENSE) has one
 *   block per query set, q_len_b x kv_len_{kv_index[b]}.
 *   Planning: the forward and dQ passes work per query set, reading its user's rows.
 *   The dK/dV pass works per user key tile over the query tiles of all of that user's
 *   query sets, so dK and dV accumulate on chip and each user row is written once.
 *   Without causal masking or a window, a row's result does not depend on which query
 *   set it belongs to, except through the relative-position table.  The plan then
 *   also holds a merged view: each run of consecutive query sets of one user is one
 *   query sequence, so short query sets fill whole 128-row tiles.  Calls use it unless
 *   they pass JFA_BIAS_RELPOS32.  Query sets of a user placed next to each other in Q
 *   thus share tiles.
 *   jfa_plan_info fact 16 is U.
 *   The other calls take the plan as usual.  jfa_worklist_* and
 *   jfa_partition_sequences describe plain batches only; jfa_partition_users splits a
 *   shared key/value batch.
 * Errors: INVALID_ARG for bad offsets or an index outside [0, U); otherwise those of
 * jfa_plan_create_ex.
 */
jfa_status jfa_plan_create_shared_kv(const int32_t* q_offsets, int32_t B, const int32_t* kv_offsets,
                                     int32_t U, const int32_t* kv_index, int32_t H, int32_t D,
                                     int32_t mode, int32_t causal, int32_t window,
                                     int32_t offsets_on_device, void* stream, jfa_plan* out);

/* Frees a plan and its device memory (cudaFree synchronises the device, so launches
 * still using the plan finish first).  NULL is accepted. */
jfa_status jfa_plan_destroy(jfa_plan plan);

/*
 * Plan facts for callers and tests, written to info[0..n): T_q, T_kv, B, H, D,
 * mode, causal, forward work items, forward grid, backward dK/dV work items, its
 * grid, SM count, backward dQ work items, its grid, window (-1: none), P, the number
 * of (query, key) pairs sum_b q_len_b * kv_len_b, the number of users U of a
 * shared key/value plan (-1 for other plans), and the number of merged query sequences
 * of a shared key/value plan's merged view (-1 when it has none; see
 * jfa_plan_create_shared_kv), and 1 when the forward runs the kernel with split items
 * (sequences of one query tile whose key range is split in two halves that are merged
 * at the end; chosen when such items carry at least half the forward's tensor-core
 * products and the plan has no window), else 0, and 1 when jfa_bwd on JFA_BF16 inputs
 * (without a dense bias or a bias gradient) may run the fused backward, in which every
 * key tile also adds its part of dQ into an fp32 accumulator held in the workspace, else
 * 0.  The planner chooses the fused form when the backward's key tiles visit few query
 * tiles on average (short sequences), unless jfa_plan_set_deterministic chose the
 * two-pass form; see jfa_plan_set_deterministic.  Fact 20 is the query-tile rows (64 or
 * 128) of the short-query backward when jfa_bwd on JFA_BF16 inputs without a bias runs
 * it for this plan, else 0: one kernel per (sequence, head) for batches whose query sets
 * all fit one tile, with no causal mask, window or shared key/value (it then takes the
 * place of the fused form for calls without a bias).  Fact 21 is the same query-tile rows
 * when jfa_fwd on JFA_BF16 inputs without a bias runs a short-query forward for this plan,
 * else 0: in GDPA modes the scores formed transposed, with the keys on the tensor-core
 * accumulator's lanes; in SOFTMAX mode (head_dim 64, query sets of at most 64 rows) two key
 * tiles per score tile, one per half of the lanes.  Either way short query sets leave no
 * lane on padding rows.  n may be smaller than 22.
 */
jfa_status jfa_plan_info(jfa_plan plan, int64_t* info, int32_t n);

/*
 * Forward pass.
 *   Q [T_q,H,D], K, V [T_kv,H,D] (dtype); bias_table fp32 [H,32] when bias_kind is
 *   JFA_BIAS_RELPOS32, the dense bias fp32 [H,P] when it is JFA_BIAS_DENSE (see
 *   jfa_bias_kind), else ignored; scale multiplies <q,k> (typically 1/sqrt(D)); in
 *   SOFTMAX mode it must be finite and positive (the kernels bound each row's maximum by
 *   scale times the row's largest raw score), else INVALID_ARG.
 *   O [T_q,H,D] is written for every row covered by the offsets, in o_dtype:
 *   JFA_F32 (the fp32 accumulator, no output rounding) or JFA_BF16 (rounded to
 *   nearest even); with dtype JFA_F32, o_dtype must be JFA_F32.
 *   lse fp32 [T_q,H]: written in SOFTMAX mode (natural log, -inf for a row with
 *   no allowed key) and required there; ignored and may be NULL in GDPA modes.
 * Errors: INVALID_ARG, UNSUPPORTED, PLAN_MISMATCH, CUDA (launch failure).
 */
jfa_status jfa_fwd(jfa_plan plan, int32_t dtype, const void* Q, const void* K, const void* V,
                   int32_t bias_kind, const float* bias_table, float scale, void* O, int32_t o_dtype,
                   float* lse, void* stream);

/* Bytes of device workspace jfa_bwd needs for this plan and dtype: fp32 row terms
 * [T_q,H], and an fp32 dQ accumulator [T_q,H,D] for JFA_F32 and for plans whose bf16
 * backward may be fused (jfa_plan_info fact 19); 0 on a bad plan. */
size_t jfa_bwd_workspace_size(jfa_plan plan, int32_t dtype);

/*
 * Backward pass of L = sum(O * dO) for the forward with the same arguments.
 *   O (in o_dtype) and lse are the forward's outputs (both ignored in GDPA modes);
 *   dO is the upstream gradient [T_q,H,D] (dtype).  Writes dQ [T_q,H,D], dK, dV
 *   [T_kv,H,D] (dtype).
 *   workspace: caller-owned device memory of at least jfa_bwd_workspace_size bytes,
 *   256-byte aligned; its contents need not be initialised and are clobbered.
 * Errors: INVALID_ARG (incl. too small a workspace), UNSUPPORTED, PLAN_MISMATCH,
 * CUDA.
 */
jfa_status jfa_bwd(jfa_plan plan, int32_t dtype, const void* Q, const void* K, const void* V,
                   const void* O, int32_t o_dtype, const void* dO, const float* lse,
                   int32_t bias_kind, const float* bias_table, float scale, void* dQ, void* dK,
                   void* dV, void* workspace, size_t workspace_bytes, void* stream);

/*
 * jfa_bwd that also returns the gradient of the bias (the article's "custom attention
 * bias", aihot.vn GEM article, section "Jagged Sequence Flash Attention", made
 * trainable): a bias adds to the score, so its gradient is dS,
 *   ds_ij = p_ij (dp_ij - sum_l p_il dp_il) (softmax) or act'(s_ij) dp_ij (GDPA).
 * For the table of JFA_BIAS_RELPOS32, entry (h, k) receives the sum of ds_ij over the
 * allowed pairs (i, j) of head h, in every sequence, whose relative position falls in
 * bucket k:
 *   dbias[h, k] = sum_{b, i, j allowed, bucket(|i + kv_len - q_len - j|) = k} ds_ij.
 * For JFA_BIAS_DENSE, dbias has the dense bias's layout [H, P] and receives ds_ij at
 * every allowed pair and 0 at every masked one.
 *   dbias: fp32 device pointer, [H, 32] or [H, P] by bias_kind, 4-byte aligned,
 *     caller-owned; overwritten (not accumulated into).  NULL makes the call exactly
 *     jfa_bwd.  Requires bias_kind JFA_BIAS_RELPOS32 or JFA_BIAS_DENSE (the gradient
 *     is taken at the given bias).
 *   workspace: at least jfa_bwd_ex_workspace_size(plan, dtype, bias_kind) bytes when
 *     dbias is set (jfa_bwd_workspace_size otherwise), 256-byte aligned.
 *   The result is the same on every run: each CTA and warp sums its part in a fixed
 *   order, and a last kernel adds the parts in a fixed order.
 * Errors: those of jfa_bwd; INVALID_ARG for a dbias with bias_kind JFA_BIAS_NONE, a
 * misaligned dbias or too small a workspace.
 */
size_t jfa_bwd_ex_workspace_size(jfa_plan plan, int32_t dtype, int32_t bias_kind);
jfa_status jfa_bwd_ex(jfa_plan plan, int32_t dtype, const void* Q, const void* K, const void* V,
                      const void* O, int32_t o_dtype, const void* dO, const float* lse,
                      int32_t bias_kind, const float* bias_table, float scale, void* dQ, void* dK,
                      void* dV, float* dbias, void* workspace, size_t workspace_bytes, void* stream);

/* Size of the library-held scratch array that jfa_bwd_static_scratch uses on each
 * GPU (64 MiB).  A plan fits when jfa_bwd_workspace_size(plan, dtype) is at most
 * this.  With an fp32 dQ accumulator in the scratch (JFA_F32, and JFA_BF16 on a fused
 * backward) that is T_q * H up to about 130,000 (token, head) rows at head_dim 128 and
 * 258,000 at head_dim 64; with row terms alone (shared key/value plans on JFA_BF16),
 * about 16.7 million. */
#define JFA_STATIC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * jfa_bwd without a caller-supplied workspace, for callers that cannot allocate
 * device memory at all.  Examples are a host program whose device buffers are all
 * handed to it by another runtime, or one whose device memory is entirely reserved
 * by a pool at start-up, where one more cudaMalloc fails or defeats the pool.  The
 * paper has no counterpart to this call; it exists only for such callers.
 *   Arguments, layout, results and asynchrony are those of jfa_bwd.  The scratch is
 *   the library's own JFA_STATIC_SCRATCH_BYTES device array, which every GPU that
 *   loads the library holds until the process exits.  This call allocates nothing:
 *   no cudaMalloc, no cudaFree, no allocating library routine.  The plan's timing
 *   hook, when a caller has switched it on, creates CUDA events as it does for
 *   jfa_bwd; it is off by default.
 *   Set-up: the first call in a CUDA context (normally the device's primary
 *   context, made current by cudaSetDevice) looks up the array's device address
 *   and keeps it, keyed by the context's unique id, for later calls in that
 *   context.  A new context -- the primary context re-created after
 *   cudaDeviceReset, or a caller's own driver-API context -- gets a fresh look-up,
 *   and the array's contents do not survive a reset.  The look-up can load the
 *   library's module on the device, so make the first call in each context before
 *   any stream capture.
 *   Every call on a device uses the same array.  A call rewrites the row terms
 *   held there before reading them.  Where the scratch holds a dQ accumulator
 *   (JFA_F32, and JFA_BF16 on a fused backward) it also clears that on its stream
 *   before adding anything in.  So no call depends on
 *   what an earlier call left there.  Calls that may overlap on the GPU race on the
 *   array and corrupt each other's gradients: order them on one stream, or by
 *   events.
 *   The current device must be the plan's device.
 * Errors: SCRATCH_LIMIT when jfa_bwd_workspace_size(plan, dtype) exceeds
 * JFA_STATIC_SCRATCH_BYTES (checked before anything is launched); PLAN_MISMATCH
 * when another device is current; CUDA if the address look-up fails; otherwise
 * those of jfa_bwd.
 */
jfa_status jfa_bwd_static_scratch(jfa_plan plan, int32_t dtype, const void* Q, const void* K,
                                  const void* V, const void* O, int32_t o_dtype, const void* dO,
                                  const float* lse, int32_t bias_kind, const float* bias_table,
                                  float scale, void* dQ, void* dK, void* dV, void* stream);

/*
 * The bf16 backward has three forms (the articles leave the backward's accumulation open;
 * see jfa_bwd):
 *   fused: one kernel over key tiles forms dK, dV and each key tile's part of dQ, adding
 *     the parts into an fp32 accumulator in the workspace with reduce-adds at L2, and a
 *     conversion pass writes dQ.  The order of the additions varies from run to run, so
 *     dQ can differ in its last bit between runs; dK and dV do not.
 *   two-pass: a second kernel over query tiles recomputes S and dP and accumulates dQ
 *     on chip, with no atomics: every result is the same bit for bit on every run, at
 *     1.4x the tensor-core work of the backward.
 *   short-query: when every query set fits one tile of 64 or 128 rows (64 at head_dim
 *     64) and the plan has no causal mask, window or shared key/value, and the call has no
 *     bias: one kernel per (sequence, head) keeps the query set on chip while the key
 *     tiles stream past, and sums dQ in TMEM.  No atomics: the same bits on every run.
 * By default (enable = 0) the planner picks the faster form for the batch: short-query
 * where it applies; else fused when the key tiles visit few query tiles on average (short
 * sequences, where it saves the second pass); two-pass otherwise (long sequences, where
 * the reduce-adds cost more than the recomputation).  enable = 1 always runs the two-pass
 * form.  Shared key/value plans
 * (unless their merged view is used), a dense bias and bias gradients always run the
 * two-pass form.  The choice changes jfa_bwd_workspace_size (the fused backward needs the
 * fp32 accumulator); query it after this call.  jfa_plan_info facts 19 and 20 report the
 * form.
 * fp32 inputs are unaffected.
 * Errors: INVALID_ARG for a null plan or enable not 0 or 1.
 */
jfa_status jfa_plan_set_deterministic(jfa_plan plan, int32_t enable);

/*
 * Test hook for the kernels' own checks (not a counterpart of anything in the articles).
 * Every kernel checks each work item it reads against the plan -- sequence, head and
 * tile inside the batch, inner count equal to the one the tile ranges give -- before it
 * touches anything the item indexes.  It skips an item that fails and sets the status
 * that jfa_plan_device_status reports as JFA_ERR_DEVICE_BOUNDS.  The planner never writes
 * such an item; this call overwrites work item `index` of a pass (0 forward, 1 backward
 * dK/dV, 2 backward dQ, 3 the short-query backward, 4 the short-query forward; numbering as
 * jfa_plan_info facts 7, 9, 12, and for passes 3 and 4 as jfa_worklist_build's pass 3 on the
 * plan's offsets, grouped for each kernel's own grid) in the plan's device
 * memory so that a test can plant one.  The lists are the plan's own (a shared key/value
 * plan's merged view keeps its lists).  Synchronises.  A plan holding a changed item gives
 * wrong results for that item's rows until it is destroyed.
 *   item: int32[4] (sequence, head, tile, inner count), host memory.
 * Errors: INVALID_ARG for a bad pass, an index outside the list or a null pointer; CUDA.
 */
jfa_status jfa_plan_set_work_item(jfa_plan plan, int32_t pass, int64_t index, const int32_t* item);

/* Synchronises `stream`, then reads and clears the plan's device status word, which
 * the kernels set when a pipeline wait times out (TIMEOUT) or a bounds check fires
 * (DEVICE_BOUNDS).  Returns JFA_OK when no kernel reported anything. */
jfa_status jfa_plan_device_status(jfa_plan plan, void* stream);

/* Host-only planner, usable without a GPU (the same code jfa_plan_create runs).
 * pass 0 = forward (pairs of 128-row query tiles), 1 = backward dK/dV (key/value
 * tiles of 128 rows, visiting 128-row query tiles), 2 = backward dQ (128-row query
 * tiles), 3 = the short-query backward (one item (sequence, head, 0, key tiles) per
 * sequence with a query or a key; causal must be 0 and window -1).  jfa_worklist_size
 * gives the number of work items; jfa_worklist_build writes items as int32 quadruples
 * (sequence, head, tile index, inner tiles visited) grouped by CTA, cta_offsets[n_ctas+1]
 * delimiting each CTA's items, and optionally each CTA's total cost in units of
 * tensor-core products.  window as in jfa_plan_create_ex (-1: none).  With a window the
 * inner tiles are a band: a forward pair streams the union of its two query tiles' key
 * ranges.  Errors: INVALID_ARG for bad offsets, H < 1, n_ctas < 1, an unknown pass, or
 * pass 3 with a causal mask or a window. */
jfa_status jfa_worklist_size(const int32_t* q_offsets, const int32_t* kv_offsets, int32_t B,
                             int32_t H, int32_t causal, int32_t window, int32_t pass, int64_t* n_items);
jfa_status jfa_worklist_build(const int32_t* q_offsets, const int32_t* kv_offsets, int32_t B,
                              int32_t H, int32_t causal, int32_t window, int32_t pass, int32_t n_ctas,
                              int32_t* items, int32_t* cta_offsets, int64_t* cta_cost);

/* Data-parallel split, host only (no GPU needed).  Sequences are independent, so a
 * batch shards across GPUs with no exchange (GEM articles: jagged batches with long
 * and short sequences, where balance decides throughput).  Each sequence is costed by
 * the tensor-core products its forward and backward issue over all heads, and the
 * sequences are assigned longest-first to the least loaded of n_parts parts
 * (deterministic: ties go to the lower part and the lower sequence index).
 *   part_of_seq[B] receives each sequence's part; part_cost[n_parts] (may be NULL)
 *   each part's total cost.  The greedy bound holds: the most loaded part exceeds
 *   the least loaded by at most one sequence's cost.
 * window as in jfa_plan_create_ex (-1: none).
 * Errors: INVALID_ARG (bad offsets, H < 1, n_parts < 1, causal not 0/1, a window
 * without causal). */
jfa_status jfa_partition_sequences(const int32_t* q_offsets, const int32_t* kv_offsets, int32_t B,
                                   int32_t H, int32_t causal, int32_t window, int32_t n_parts,
                                   int32_t* part_of_seq, int64_t* part_cost);

/*
 * jfa_partition_sequences for a shared key/value batch (jfa_plan_create_shared_kv):
 * users, each with all of its query sets, split over n_parts GPUs by greedy LPT on
 * their cost, the cost of their query sets plus their key tiles.  A user's dK and dV sum
 * over its query sets, so keeping them together means no GPU exchanges anything.
 *   Host arrays: q_offsets int32[B+1], kv_offsets int32[U+1], kv_index int32[B].
 *   part_of_user: int32[U] out, each in [0, n_parts); part_cost: int64[n_parts] out
 *   (may be NULL).  Deterministic.
 * Errors: INVALID_ARG for bad offsets or sizes, or an index outside [0, U).
 */
jfa_status jfa_partition_users(const int32_t* q_offsets, int32_t B, const int32_t* kv_offsets,
                               int32_t U, const int32_t* kv_index, int32_t H, int32_t causal,
                               int32_t window, int32_t n_parts, int32_t* part_of_user,
                               int64_t* part_cost);

/* Kernel timing for measurement.  With timing enabled, every kernel launch made for
 * this plan is bracketed by a pair of CUDA events recorded on the launch stream.
 * jfa_plan_kernel_times synchronises those events and returns, per kernel kind
 * (0 forward, 1 backward preprocess, 2 backward dK/dV (fp32 inputs: backward main),
 * 3 fp32 dQ conversion, 4 bf16 backward dQ), the summed milliseconds and the number
 * of launches since the previous query, then forgets them.  Timing is off by
 * default; enabling it adds one event record before and after each launch.
 * total_ms and launches point to arrays of 5 (either may be NULL). */
jfa_status jfa_plan_set_timing(jfa_plan plan, int32_t enable);
jfa_status jfa_plan_kernel_times(jfa_plan plan, double* total_ms, int64_t* launches);

/* Static description of a status code. */
const char* jfa_status_string(int32_t status);

/*
 * Paged key/value cache: serving a jagged model token by token.
 *
 * A cache holds keys and values of many sequences in pages of `page_size` positions.
 * Sequence b's position p lies in page page_table[b * max_pages + p / page_size], slot
 * p % page_size.  Element (page, slot, head, d) of the keys is at
 *   K[page * k_strides[0] + slot * k_strides[1] + head * k_strides[2] + d]
 * (strides in elements), and likewise of the values, so token-major pages
 * [n_pages, page_size, Hkv, D], head-major pages [n_pages, Hkv, page_size, D] and keys
 * and values interleaved in one array are all served without a copy.
 *
 * A step of a served batch is two calls on the same arrays:
 *   jfa_cache_append  writes the new tokens' keys and values to their slots, with the
 *                     position rotation applied to keys and queries on the way;
 *   jfa_cache_fwd     attends from the new tokens to the cached positions.
 * Both take, as int32 DEVICE arrays read when the kernels run (so a captured graph can be
 * replayed on new contents), for B of at most 8192 sequences and T of at most 2^30 rows:
 *   q_offsets [B+1]  the new tokens of sequence b are rows q_offsets[b] .. q_offsets[b+1]
 *                    of Q, K and V (non-decreasing; rows from q_offsets[B] to T belong to
 *                    no sequence and are left alone);
 *   kv_lens [B]      positions of sequence b in the cache, its new tokens included: they are
 *                    its last q_len_b positions;
 *   page_table [B, max_pages]  only the first ceil(kv_len / page_size) entries of a row are
 *                    read, with a window only those that hold a position some new token sees.
 * The kernels check them: a sequence whose offsets leave [0, T], whose length leaves
 * [0, max_pages * page_size], or a page outside [0, n_pages) sets the status that
 * jfa_cache_device_status reports as JFA_ERR_DEVICE_BOUNDS.  Nothing outside the arrays is
 * read or written then; a bad sequence's rows stay as they were, and rows that needed a bad
 * page are wrong.  Offsets that decrease make a bad sequence and let others overlap: rows of
 * several sequences hold one's result, or, where the overlap asks for more work than can be
 * counted, nothing is computed.
 */
typedef struct jfa_cache_t* jfa_cache;

/* Rotation layouts: which elements of a head's first rot_dim form a pair (x_a, x_b).
 * HALF: (x_k, x_{k + rot_dim/2});  PAIRS: (x_{2k}, x_{2k+1}). */
typedef enum { JFA_ROT_HALF = 0, JFA_ROT_PAIRS = 1 } jfa_rot_kind;

/*
 * A handle on a cache whose K and V arrays the caller owns (they must outlive it).
 *   dtype JFA_BF16 (D 64 or 128) or JFA_F32 (D 32 or 64); Hkv >= 1 key/value heads;
 *   page_size a power of two from 8 to 1024; n_pages >= 1.
 *   K, V: DEVICE pointers of the current device (device memory of another one is refused with
 *   INVALID_ARG: the handle's kernels run where it was created), 16-byte aligned; k_strides, v_strides:
 *   host int64[3] (page, slot, head), each at least D and a multiple of 16 bytes.
 *   The handle allocates a status word on the current device (synchronises `stream`).
 *   It keeps no state between calls: calls on one handle may run at once on different
 *   streams, with a workspace each.
 * Errors: INVALID_ARG, UNSUPPORTED (dtype / D / page_size), NO_DEVICE, CUDA.
 */
jfa_status jfa_cache_create(int32_t dtype, int32_t Hkv, int32_t D, int32_t page_size, int64_t n_pages,
                            void* K, void* V, const int64_t* k_strides, const int64_t* v_strides,
                            void* stream, jfa_cache* out);

/*
 * A cache held in 4 bits: a history of 9 bytes for 16 elements, 3.6 times less than bf16 to keep
 * and to read.  The handle is used like any other: jfa_cache_append quantises the new rows,
 * jfa_cache_fwd attends over the values that the cache stands for, and workspaces, status and
 * destruction are the same calls.  Rows (K, V, Q, O of those calls) are as of a bf16 cache.
 *   A row of D elements of one (page, slot, head) is D / 2 bytes of e2m1 codes (a sign and 0, 0.5, 1,
 *   1.5, 2, 3, 4 or 6; element 2i in the low half of byte i) and D / 16 e4m3 scales, one for each 16
 *   elements; an element is  factor * scale * code,  with one factor for all keys (k_factor) and
 *   one for all values (v_factor), powers of two or not, in [2^-60, 2^60].  1 suits rows whose
 *   largest magnitudes lie in 0.02 .. 2688.
 *   K, V: the codes; k_strides, v_strides: host int64[3] (page, slot, head) in bytes, each at least
 *   D / 2 and a multiple of 16.  K_scales, V_scales: the scales, a head's page_size * D / 16 bytes of
 *   one page in one piece (slot by slot); ks_strides, vs_strides: host int64[2] (page, head) in
 *   bytes, each at least that size and a multiple of 16.  All DEVICE pointers of the current
 *   device, 16-byte aligned, owned by the caller.  Codes with a head's slots of a page in one piece
 *   ([n_pages, Hkv, page_size, D / 2]) are read fastest.
 *   D 64 or 128; Hkv, page_size, n_pages as in jfa_cache_create.
 * Appending: of each 16 elements y of a row (keys after their rotation, which is not rounded in
 *   between)  scale = e4m3(max|y| / (6 factor)), at most 448, and code = e2m1(y / (factor scale)), at
 *   most 6 in magnitude (0 where the scale is 0), both to nearest, ties to the even code, as if
 *   in exact arithmetic.
 * Attention: scale * code is exact in the products' types.  jfa_cache_fwd's text on bf16 caches
 *   holds, with each weight of the softmax rounded to fp16 for its product: off by 2^-11 of itself, or
 *   by 2^-31 of the row's largest where that is more, and queries taken to fp16 by a power of two for
 *   each row: exact but for elements below 2^-28 of its largest, which lose 2^-39 of that at
 *   most.  scale * k_factor must lie in [1e-37, 1e37].
 * Errors: those of jfa_cache_create.
 */
jfa_status jfa_cache_create_quantized(int32_t Hkv, int32_t D, int32_t page_size, int64_t n_pages, void* K, void* V,
                                      const int64_t* k_strides, const int64_t* v_strides, void* K_scales, void* V_scales,
                                      const int64_t* ks_strides, const int64_t* vs_strides, float k_factor, float v_factor,
                                      void* stream, jfa_cache* out);

/* Frees the handle (not K and V).  cudaFree synchronises the device.  NULL is accepted. */
jfa_status jfa_cache_destroy(jfa_cache cache);

/* As jfa_plan_device_status: synchronises `stream`, reads and clears the status word. */
jfa_status jfa_cache_device_status(jfa_cache cache, void* stream);

/*
 * Appends the new tokens' keys and values, rotating keys (and queries) by their position.
 *   K, V [T, Hkv, D] and, with a rotation, Q, Q_out [T, H, D] in the cache's dtype: heads
 *   dense, tokens *_stride elements apart (at least the row, a multiple of 16 bytes), so that
 *   slices of one fused projection are taken as they are.  Q_out may be Q itself, and
 *   overlaps nothing else.
 *   rot: NULL (keys stored as given, Q and Q_out must be NULL), or an fp32 table
 *   [rot_len, rot_dim], 16-byte aligned, whose row p holds the rot_dim / 2 cosines and then
 *   the sines of position p.  Of each pair of the first rot_dim elements of a head
 *     y_a = x_a cos - x_b sin,   y_b = x_b cos + x_a sin,
 *   in fp32, rounded once; the other elements are copied.  rot_dim is a multiple of 16, at
 *   most D.  A position at or past rot_len sets JFA_ERR_DEVICE_BOUNDS and its token is
 *   skipped.
 *   Q may be NULL with a rotation (keys alone); H and the two strides are then ignored.
 *   A sequence with fewer positions than new tokens (kv_len < q_len) is bad, as a whole.
 *   Two tokens must not share a slot (pages shared by sequences are for reading).
 * Errors: INVALID_ARG, PLAN_MISMATCH (another device is current), CUDA.
 */
jfa_status jfa_cache_append(jfa_cache cache, int32_t B, int64_t T, const int32_t* q_offsets,
                            const int32_t* kv_lens, const int32_t* page_table, int32_t max_pages,
                            const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                            const void* Q, int64_t q_stride, int32_t H, void* Q_out, int64_t qo_stride,
                            const float* rot, int32_t rot_dim, int64_t rot_len, int32_t rot_kind,
                            void* stream);

/*
 * The rows that jfa_cache_append wrote for the same arrays, as the cache holds them (a cache of any
 * type): row t of K and V [T, Hkv, D], in the type of the cache's rows, is the position of new token
 * t.  With kv_lens for lengths of new tokens (q_offsets their sums) these are whole histories.  Of a
 * 4-bit cache, factor * scale * code is rounded to bf16.  Strides, bad sequences and pages as in
 * jfa_cache_append (their rows are left alone); K and V overlap neither each other nor the cache.
 * Errors: INVALID_ARG, PLAN_MISMATCH (another device is current), CUDA.
 */
jfa_status jfa_cache_read(jfa_cache cache, int32_t B, int64_t T, const int32_t* q_offsets, const int32_t* kv_lens,
                          const int32_t* page_table, int32_t max_pages, void* K, int64_t k_stride, void* V, int64_t v_stride,
                          void* stream);

/* Bytes of device workspace jfa_cache_fwd needs, for any batch with H query heads (0: bad
 * arguments). */
size_t jfa_cache_workspace_size(jfa_cache cache, int32_t H);

/*
 * Attention of the new tokens over the cache: with i' = i + kv_len - q_len for row i of
 * sequence b and key head h / (H / Hkv) of query head h (H a multiple of Hkv, with bf16 at most 128 Hkv),
 *   s_ij = scale * <q_i, k_j> + bias[h, bucket(|i' - j|)],  o_i = sum_j softmax_j(s_ij) v_j
 * over the keys j < kv_len allowed as in jfa_plan_create_ex: causal (0/1) j <= i', window
 * W >= 0 (with causal) j >= i' - W, -1: none.  A row with no allowed key gets o = 0 and
 * lse = -inf.
 *   Q [T, H, D] in the cache's dtype (T H at most 2^31 - 257), tokens q_stride elements apart (a
 *   multiple of 16 bytes); O [T, H, D] dense, in o_dtype (JFA_F32, or JFA_BF16 with a bf16 cache);
 *   O must not overlap Q.
 *   With a bf16 cache each weight of the softmax is rounded to bf16 for its product with the
 *   values, after their sum has been taken in fp32, as in jfa_fwd: at most 2^-8 of sum_j p_j |v_j|.
 *   Scores, maxima, sums, partial outputs and lse are fp32.
 *   lse fp32 [T, H], or NULL.  bias_kind JFA_BIAS_NONE or JFA_BIAS_RELPOS32 (fp32 [H, 32]).
 *   scale must be finite and positive, and scores finite (so the bias too: it is no mask).
 *   fp32 is computed at fp32's accuracy, single tokens and short query sets (up to 16 rows of
 *   grouped heads) on the CUDA cores, longer ones on the tensor cores with each operand as the
 *   sum of three bf16 values, for magnitudes below 2^127.
 *   max_q_len: an upper bound of the batch's q_len, or 0 if unknown (T is taken).  It only
 *   chooses among kernels: results do not depend on it beyond rounding, and a longer
 *   sequence is still computed in full.
 *   Keys that no new token of a sequence may see -- slots at or past kv_len, positions
 *   before every row's window -- may hold anything, NaN included, and pages that hold only
 *   such positions may be unset in the table; the other values must be finite.
 *   workspace: at least jfa_cache_workspace_size bytes, 256-byte aligned.  Its first
 *   JFA_CACHE_ZERO_BYTES must be zero before its first use and are zero again after every
 *   call (zero them again after JFA_ERR_TIMEOUT; what was not zero can spoil results, and sets
 *   JFA_ERR_DEVICE_BOUNDS where it names rows that the call does not have, which are not
 *   written); the rest needs no initialisation.  Calls
 *   that may overlap on the GPU need a workspace each: order those that share one.
 *   The result is the same bit for bit on every run of the same call.  There is no backward
 *   pass: a cache is for serving (training keys and values go through jfa_fwd and jfa_bwd).
 *   Over a cache there is the softmax alone: the GDPA activations take packed keys (jfa_fwd).
 * Errors: INVALID_ARG, UNSUPPORTED (a dense bias, bf16 output of an fp32 cache, more than 128
 *   grouped heads with bf16, or row tiles x key tiles that max_pages and T allow past 2^31),
 *   PLAN_MISMATCH (another device is current), CUDA.  A call refused with one of the first
 *   three launches nothing and writes nothing.
 */
#define JFA_CACHE_ZERO_BYTES ((size_t)32768)
jfa_status jfa_cache_fwd(jfa_cache cache, int32_t B, int64_t T, int32_t max_q_len, const int32_t* q_offsets,
                         const int32_t* kv_lens, const int32_t* page_table, int32_t max_pages,
                         const void* Q, int64_t q_stride, int32_t H, int32_t causal, int32_t window,
                         int32_t bias_kind, const float* bias_table, float scale, void* O, int32_t o_dtype,
                         float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Attention over selected blocks: a long history is read in part, and every new token chooses
 * which part for each key head.  A block is a page (block k of a sequence is its positions
 * k * page_size on).  A step of a served batch is four calls on the same arrays:
 *   jfa_cache_append      as before;
 *   jfa_cache_summarize   brings the bounds of the pages that got new tokens up to date;
 *   jfa_cache_select      chooses blocks by a score from the bounds alone;
 *   jfa_cache_fwd_blocks  attends over the chosen blocks.
 * For bf16 and 4-bit caches with pages of at least 16 positions (UNSUPPORTED otherwise).  Bad sequences,
 * lengths and pages are reported as in the calls above.  Attention is causal, without a window.
 *
 * Bounds: bf16 [n_pages, Hkv, 2, D], 16-byte aligned, the caller's: the least and the largest of each
 * element over the keys of a page (of a 4-bit cache scale * code, without the factor).  Summarize
 * takes a page's positions below kv_len, all of them anew, so that a page that was given to another
 * sequence needs nothing else.  Bounds of other pages are left alone.
 */
jfa_status jfa_cache_summarize(jfa_cache cache, int32_t B, int64_t T, const int32_t* q_offsets, const int32_t* kv_lens,
                               const int32_t* page_table, int32_t max_pages, void* bounds, void* stream);

/* Bytes of device workspace jfa_cache_select needs (0: bad arguments, or more than it takes); it needs no
 * initialisation.  About 4 T Hkv max_pages. */
size_t jfa_cache_select_workspace_size(jfa_cache cache, int64_t T, int32_t max_pages);

/*
 * blocks [T, Hkv, n_blocks] int32, for new token i of sequence b at position i' = i + kv_len - q_len
 * and each key head: n_blocks of the blocks 0 .. c, c = i' / page_size its own, ascending.  If there
 * are no more than n_blocks, all of them and then -1.  Otherwise the first n_first, the last n_last (c
 * among them), and of the others those of the highest score
 *   sum_{h in the key head's group} sum_d max(q_hd lo_d, q_hd hi_d),
 * an upper bound of what the group's scores with a key of the block can sum to; of equal scores the lower index.
 * Scores are compared as in 64-bit arithmetic.  Bounds of blocks 0 .. c - 1 are read where they
 * decide, and must be finite.  Rows that belong to no sequence are left alone.
 *   Q [T, H, D] as in jfa_cache_fwd (with the rotation); max_q_len: an upper bound of the batch's
 *   q_len, or 0; it only chooses among kernels.
 *   n_last >= 1, n_first >= 0, n_first + n_last <= n_blocks, n_blocks * page_size <= 2^30.
 *   workspace: at least jfa_cache_select_workspace_size bytes, 256-byte aligned; calls that may
 *   overlap on the GPU need one each.
 *   The kernels are chosen, and the workspace sized, by max_pages, whatever the histories' lengths: a page
 *   table of no more columns than they need is fastest (64 tokens over up to 499 pages, 8 key heads of 128:
 *   25 us with 499 columns, 29 with 1024, 51 with 2048, 100 with 8192; four prompts of 1,312
 *   tokens over up to 313 pages: 64 us with 313, 105 with 1024, 448 with 2048 and more).
 *   (Lists for more than 16 grouped heads can be had here; jfa_cache_fwd_blocks does not take them.)
 * Errors: INVALID_ARG, UNSUPPORTED (the cache; more than 128 grouped heads; max_pages over 65535 * 64), PLAN_MISMATCH, CUDA.
 */
jfa_status jfa_cache_select(jfa_cache cache, int32_t B, int64_t T, int32_t max_q_len, const int32_t* q_offsets,
                            const int32_t* kv_lens, const int32_t* page_table, int32_t max_pages, const void* bounds,
                            const void* Q, int64_t q_stride, int32_t H, int32_t n_blocks, int32_t n_first, int32_t n_last,
                            int32_t* blocks, void* workspace, size_t workspace_bytes, void* stream);

/*
 * jfa_cache_fwd (causal) with the keys of row i of key head hk limited to the blocks listed for it in
 * blocks [T, Hkv, n_blocks]: indices that ascend strictly, then -1.  Listed positions after i' are
 * not seen, so a list may name the token's own block and later ones.  An entry that does not ascend, or
 * follows a -1, is left out where it is met, and sets JFA_ERR_DEVICE_BOUNDS (ascends: over all entries before
 * it, left out or not; as many entries are looked at as the token has blocks).  At most 16 grouped
 * heads.  Workspace (jfa_cache_workspace_size), outputs, bias, rounding and empty rows are as in
 * jfa_cache_fwd; the result is the same bit for bit on every run.
 *   Every token reads its blocks for itself, so this is a call for single tokens and drafts.  For prompts
 *   jfa_cache_fwd over everything is faster until histories are long.  With 2,048 listed keys, 32 query
 *   and 8 key heads of 128: one sequence over 20k keys, from about 64 tokens on (4 bits: 256); 16
 *   over 12k, from 8 each on (4 bits: past 16); four prompts of 1,312 tokens over 5k-20k 882 us against
 *   296 (4 bits: 601, 331).  One sequence over 100k: this call, up to 512 tokens at least.
 * Errors: those of jfa_cache_fwd; UNSUPPORTED also for the cache and for more than 16 grouped heads.
 */
jfa_status jfa_cache_fwd_blocks(jfa_cache cache, int32_t B, int64_t T, const int32_t* q_offsets, const int32_t* kv_lens,
                                const int32_t* page_table, int32_t max_pages, const void* Q, int64_t q_stride, int32_t H,
                                const int32_t* blocks, int32_t n_blocks, int32_t bias_kind, const float* bias_table, float scale,
                                void* O, int32_t o_dtype, float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* JFA_H */
