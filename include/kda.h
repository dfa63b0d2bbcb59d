/*
 * libkda — Kimi Delta Attention (KDA) recurrent decode for GB300 (sm_103a).
 *
 * One decode step of the KDA recurrence per (row, head) "unit".  The state
 * S of a unit is a 128 x 128 matrix stored as S[k][v]: row = key channel,
 * column = value channel, value channel contiguous.  With q, k L2-normalised
 * (eps 1e-6), g the per-key-channel log decay and beta the delta-rule rate:
 *
 *     S_d = diag(exp(g)) S
 *     u   = beta * (v - S_d^T k)
 *     S'  = S_d + k u^T                  (written back in place)
 *     o   = scale * S'^T q               (scale = 1/sqrt(128) by default)
 *
 * Sources, cited by page title and section:
 *   [P1] "flashinfer.kda_decode" (module overview): the Kimi-Linear T=1 gate
 *        -exp(A_log) * softplus(g + dt_bias), beta sigmoid and QK
 *        normalisation in-kernel; Q, K, V may be views into one padded
 *        projection row and raw G / beta may have independent row strides;
 *        packed cu_seqlens form with ragged lengths and null slots
 *        ("Frozen / speculative-verify mode").
 *   [P2] "flashinfer.kda_decode.fused_kda_decode" (Parameters): the fused
 *        conv + KDA + gated RMSNorm contract.
 *   [P3] "feat(cake_kda): add serving-native packed decode backend" ("Exact
 *        contract"): the packed Kimi K3 T=1 contract.
 *   [P4] "feat(kda): add fused speculative decode kernel - #4809": the
 *        packed fused operation (description) that updates conv and
 *        recurrent caches from accepted-token metadata; the review of the
 *        T=1 row mapping (token rows past the last sequence are padding
 *        that write zero and touch no slot); the bf16-state follow-up
 *        (float32 recurrence across tokens, one rounding per checkpoint).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensor data pointers are DEVICE memory owned by the caller.  The
 *   library allocates nothing, never synchronises the host, and never reads
 *   device memory on the host, so every call can be captured in a CUDA graph.
 * - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default
 *   stream) of the calling thread's current device, which must be a
 *   compute-capability 10.3 (GB300) device.  An unsupported device returns
 *   KDA_ERR_UNSUPPORTED; there is no fallback path.
 * - Every call launches exactly one kernel unless its comment says otherwise.
 *   Any contract breach (dtype,
 *   rank, shape, stride, alignment, aliasing) is detected on the host and
 *   returned as a status WITHOUT launching anything; kda_last_error_message()
 *   then describes it.  A launch failure returns KDA_ERR_CUDA.
 * - state_indices: contiguous int32, one entry per decode row (per sequence
 *   and checkpoint column for kda_packed_fused_decode).  A row whose
 *   index is <= 0 or >= num_slots is a null row: its output is zero and no
 *   cache slot is read or written (slot 0 is the reserved null slot).  Live
 *   indices must be unique; that is a caller contract the library does not
 *   check (it would need a device read).
 * - State pool [num_slots, H, 128, 128], float32 or bfloat16: each slot's
 *   [H, 128, 128] block is contiguous, the slot stride is any value >=
 *   H*128*128 that keeps 16-byte alignment.  The recurrence runs in float32;
 *   a bfloat16 state is rounded once (round-to-nearest-even) on write-back.
 * - Outputs are bfloat16 and contiguous, rounded to nearest even.
 * - Strides are in elements.  Activation vectors need unit stride on the
 *   channel axis and 16-byte (float32) or 8-byte (bfloat16) aligned rows.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kda_status {
  KDA_OK = 0,
  KDA_ERR_INVALID_ARG = 1, /* bad dtype / rank / shape / stride / alignment / null pointer */
  KDA_ERR_UNSUPPORTED = 2, /* valid request this build does not serve (device, head count) */
  KDA_ERR_ALIAS = 3,       /* a written tensor overlaps another argument */
  KDA_ERR_CUDA = 4         /* a CUDA runtime call or the launch failed */
} kda_status;

typedef enum kda_dtype { KDA_F32 = 0, KDA_BF16 = 1, KDA_I32 = 2 } kda_dtype;

/* A strided view of device memory.  shape/stride entries past ndim are ignored. */
typedef struct kda_tensor {
  void* data;        /* device address of element [0, ..., 0] */
  int32_t dtype;     /* kda_dtype */
  int32_t ndim;      /* 1..4 */
  int64_t shape[4];
  int64_t stride[4]; /* in elements */
} kda_tensor;

/*
 * kda_recurrent_decode — T=1 recurrent decode with split q, k, v.
 * [P1] Kimi-Linear T=1 equal-head schedules; [P2] "lower_bound" for the
 * bounded gate.
 *
 *   q, k, v     [B, H, 128] or [B, 1, H, 128], float32 or bfloat16 (one dtype
 *               for all three); any positive row and head strides.
 *   raw_gate    same shape as q, float32 or bfloat16 (pre-gate values).
 *   raw_beta    [B, H] or [B, 1, H], float32 or bfloat16 (logits).
 *   A_log       [H] float32, contiguous.
 *   dt_bias     [H*128] or [H, 128] float32, contiguous.
 *   state_indices [B] int32, contiguous.
 *   state       [num_slots, H, 128, 128] float32 or bfloat16, updated in place.
 *   out         [B, H, 128] or [B, 1, H, 128] bfloat16, contiguous (written).
 *   has_lower_bound = 0: g = -exp(A_log[h]) * softplus(raw_gate + dt_bias).
 *   has_lower_bound = 1: g = lower_bound * sigmoid(exp(A_log[h]) * (raw_gate + dt_bias)),
 *               lower_bound < 0.
 *   scale       output scale (> 0), normally 1/sqrt(128).
 */
kda_status kda_recurrent_decode(const kda_tensor* q, const kda_tensor* k, const kda_tensor* v,
                                const kda_tensor* raw_gate, const kda_tensor* raw_beta,
                                const kda_tensor* A_log, const kda_tensor* dt_bias,
                                const kda_tensor* state_indices, const kda_tensor* state,
                                const kda_tensor* out, int32_t has_lower_bound,
                                float lower_bound, float scale, void* stream);

/*
 * kda_packed_decode — serving-native packed Kimi K3 T=1 decode ([P3] "Exact
 * contract"): H = 12, K = V = 128, bfloat16 data and bfloat16 state, fixed
 * scale 1/sqrt(128), L2 eps 1e-6 and lower_bound -5.
 *
 *   mixed_qkv   [B, 4608] bfloat16: q | k | v, each 12 x 128 head-major;
 *               channel stride 1, any row stride.
 *   raw_gate    [B, 1536] bfloat16, channel stride 1, any row stride.
 *   raw_beta    [B, 12] bfloat16.
 *   A_log       [12] float32;  dt_bias [1536] float32.
 *   state_indices [B] int32 (-1 = inactive graph-padding row).
 *   state       [num_slots, 12, 128, 128] bfloat16, updated in place.
 *   out         [B, 1, 12, 128] or [B, 12, 128] bfloat16, contiguous.
 */
kda_status kda_packed_decode(const kda_tensor* mixed_qkv, const kda_tensor* raw_gate,
                             const kda_tensor* raw_beta, const kda_tensor* A_log,
                             const kda_tensor* dt_bias, const kda_tensor* state_indices,
                             const kda_tensor* state, const kda_tensor* out, void* stream);

/*
 * kda_fused_decode — width-4 depthwise causal conv + SiLU, one KDA step and
 * gated RMSNorm ([P2] "fused_kda_decode", Parameters).  conv_state and state
 * are updated in place; null rows touch neither.
 *
 *   x           [rows, 3*H*128] bfloat16 packed q|k|v projection, channel stride 1.
 *   conv_weight [3, 4, H*128] float32 contiguous (section q/k/v, tap, channel).
 *   conv_state  [num_slots, 3*H*128, 3] bfloat16 with strides
 *               [slot_stride, 1, 3*H*128]: cached raw samples, oldest first.
 *   raw_gate    [1, rows, H, 128] or [rows, H, 128] bfloat16.
 *   raw_beta    [1, rows, H] or [rows, H] bfloat16.
 *   A_log [H], dt_bias [H*128] float32;  state_indices [rows] int32.
 *   state       [num_slots, H, 128, 128] float32 or bfloat16 (same num_slots
 *               as conv_state).
 *   output_gate [rows, H, 128] or [1, rows, H, 128] bfloat16 (gate logits).
 *   norm_weight [128] float32.
 *   has_lower_bound / lower_bound: gate form as in kda_recurrent_decode
 *               (the pages' default is the bounded gate with -5).
 *   norm_eps    RMSNorm epsilon (>= 0, default 1e-5).
 *   out         [1, rows, H, 128] or [rows, H, 128] bfloat16 contiguous:
 *               RMSNorm(o) * norm_weight * sigmoid(output_gate).
 */
kda_status kda_fused_decode(const kda_tensor* x, const kda_tensor* conv_weight,
                            const kda_tensor* conv_state, const kda_tensor* raw_gate,
                            const kda_tensor* raw_beta, const kda_tensor* A_log,
                            const kda_tensor* dt_bias, const kda_tensor* state_indices,
                            const kda_tensor* state, const kda_tensor* output_gate,
                            const kda_tensor* norm_weight, int32_t has_lower_bound,
                            float lower_bound, float norm_eps, const kda_tensor* out,
                            void* stream);

/*
 * kda_spec_decode — packed speculative decode, T >= 1 tokens per row with
 * ragged cu_seqlens ([P1] Cake T=1..6 family with precomputed gates and
 * "Frozen / speculative-verify mode"'s packed cu_seqlens form; [P4] padding).
 *
 *   q, k, v     [R, H, 128] float32 or bfloat16 token rows (one dtype).
 *   g           [R, H, 128] float32 precomputed log decay (<= 0).
 *   beta        [R, H] float32 or bfloat16: logits if beta_is_logit, else rates.
 *   cu_seqlens  [N+1] int32 contiguous, read on the device: row n owns token
 *               rows cu[n] .. cu[n+1]-1, processed in order with the state
 *               kept in float32 on chip; its final state goes to its slot.
 *               Token rows outside [cu[0], cu[N]) are padding: zero output.
 *               Rows are clamped to [0, R); empty rows do nothing.
 *   t_max       host hint: longest row expected (>= 1); used for scheduling
 *               only, longer rows are still processed correctly.
 *   state_indices [N] int32;  state [num_slots, H, 128, 128] float32/bfloat16.
 *   out         [R, H, 128] bfloat16 contiguous.
 *   scale       output scale (> 0).
 */
kda_status kda_spec_decode(const kda_tensor* q, const kda_tensor* k, const kda_tensor* v,
                           const kda_tensor* g, const kda_tensor* beta, int32_t beta_is_logit,
                           const kda_tensor* cu_seqlens, int32_t t_max,
                           const kda_tensor* state_indices, const kda_tensor* state,
                           const kda_tensor* out, float scale, void* stream);

/*
 * kda_spec_verify_decode — speculative-verify mode ([P1] "Frozen /
 * speculative-verify mode"): the kda_spec_decode outputs for up to 16 tokens
 * per row computed from a read-only committed state pool; the state is never
 * written.  Arguments as kda_spec_decode (state is read only, t_max <= 16),
 * plus two optional slot-indexed out-params for a later commit of the
 * accepted tokens (either may be NULL):
 *   correction_cache [num_slots, H, T_cap, 128] float32 contiguous: for the
 *                token at position t < T_cap of a live row, its delta-rule
 *                correction u_t = beta (v - S_d^T k_hat);
 *   kg_cache     [num_slots, H, T_cap, 256] float32 contiguous: that token's
 *                raw key (128) followed by its log decay g (128).
 * T_cap (1..16) is the caches' third extent (equal when both are given).  The
 * state after accepting the first a tokens of a row is, token by token,
 * S <- diag(exp(g)) S + normalise(k) u^T.  Null and empty rows write no cache
 * entry; tokens at positions >= T_cap are decoded but not cached.
 */
kda_status kda_spec_verify_decode(const kda_tensor* q, const kda_tensor* k, const kda_tensor* v,
                                  const kda_tensor* g, const kda_tensor* beta, int32_t beta_is_logit,
                                  const kda_tensor* cu_seqlens, int32_t t_max,
                                  const kda_tensor* state_indices, const kda_tensor* state,
                                  const kda_tensor* out, const kda_tensor* correction_cache,
                                  const kda_tensor* kg_cache, float scale, void* stream);

/*
 * kda_packed_fused_decode — packed fused speculative decode with per-token
 * checkpoints ([P4] description, the review thread on the T=1 row mapping,
 * and its bf16-state follow-up): the kda_fused_decode step (conv + SiLU, KDA,
 * gated RMSNorm) run over the T >= 1 token rows of each of N packed
 * sequences, one sequence after another's rows in x.
 *
 *   x, conv_weight, conv_state, raw_gate, raw_beta, A_log, dt_bias,
 *   output_gate, norm_weight, has_lower_bound, lower_bound, norm_eps, out:
 *               as kda_fused_decode, with R token rows in place of rows.
 *   state_indices [N, C] int32, column stride 1: checkpoint slots of each
 *               sequence (C >= 1).
 *   query_start_loc [N+1] int32 contiguous, read on the device: sequence n
 *               owns token rows qsl[n] .. qsl[n+1]-1 (clamped to [0, R)).
 *   num_accepted_tokens [N] int32, read on the device: a_n.
 *   state       [num_slots, H, 128, 128] float32 or bfloat16.
 * Sequence n starts from the conv and recurrent caches of slot
 * state_indices[n, a_n - 1] and, after its j-th token (j < C), writes both
 * caches to slot state_indices[n, j]; a slot outside [1, num_slots) there is
 * skipped.  The recurrence stays in float32 across the tokens; a bfloat16
 * checkpoint is rounded once when stored.  A sequence whose start slot is
 * null, or whose a_n is outside 1..C, writes zero output rows and no cache;
 * empty sequences do nothing; token rows outside [qsl[0], qsl[N]) are
 * padding with zero output.  Checkpoint slots must be distinct across the
 * call (the start slot may be one of the sequence's own).  The rows of x,
 * raw_gate and output_gate are copied to shared memory in 16-byte pieces:
 * their base addresses and outer strides must be multiples of 16 bytes
 * (KDA_ERR_UNSUPPORTED otherwise).
 */
kda_status kda_packed_fused_decode(const kda_tensor* x, const kda_tensor* conv_weight,
                                   const kda_tensor* conv_state, const kda_tensor* raw_gate,
                                   const kda_tensor* raw_beta, const kda_tensor* A_log,
                                   const kda_tensor* dt_bias, const kda_tensor* state_indices,
                                   const kda_tensor* query_start_loc,
                                   const kda_tensor* num_accepted_tokens, const kda_tensor* state,
                                   const kda_tensor* output_gate, const kda_tensor* norm_weight,
                                   int32_t has_lower_bound, float lower_bound, float norm_eps,
                                   const kda_tensor* out, void* stream);

/* ---- attention layers and beams around the recurrent ones ----------------
 *
 * A decoder that mixes KDA layers with softmax-attention layers needs, per
 * new token: rotary positions and a paged key-value cache
 * (kda_rope_append), attention over it (kda_paged_attention_decode), and for
 * beam search the selection (kda_beam_select) and the copy of each surviving
 * beam's recurrent state, conv cache and pages (kda_pool_move).
 *
 * Pages follow the slot convention above: page_table [N, P] int32 (column
 * stride 1) lists the pages of each sequence in order; an entry <= 0 or >=
 * num_pages is a null page (page 0 is reserved): nothing is written to it and
 * its positions are not attended to.  k_pages and v_pages are [num_pages,
 * page_size, Hkv, D], float32 or bfloat16, unit channel stride, any other
 * positive strides that keep 4-element alignment, so a head-major page is a
 * transposed view, and keys and values may interleave in one allocation.
 */

/*
 * kda_rope_append: rotary positions of new tokens' q and k, and the write of
 * their k and v into the pages.
 *
 *   q           [R, Hq, D], k, v [R, Hkv, D], float32 or bfloat16 (one dtype),
 *               views into one packed row allowed; D a multiple of 4, <= 512.
 *   phase_steps [rot/2, 2] int32 contiguous: the rotation of pair i as turns
 *               per position in 64 fractional bits, low word first
 *               (kda_rope_phase_steps).  rot = twice its length, a multiple of
 *               8, <= D; channels past rot are copied; rot = 0 rotates nothing.
 *   cu_seqlens  [N+1] int32: sequence n owns rows cu[n] .. cu[n+1]-1 (clamped
 *               to [0, R)); NULL: row n is the one new token of sequence n.
 *   seq_lens    [N] int32: each sequence's length INCLUDING its new rows; its
 *               last row is at position seq_lens[n] - 1.
 *   k_pages, v_pages (written), page_table: as above; positions past the
 *               table's P * page_size are not written.  Two rows must not
 *               share a position of a live page.
 *   q_out       [R, Hq, D] of the pages' dtype (written); may be q itself.
 *   interleaved = 0: pair i is channels (i, i + rot/2); 1: (2i, 2i + 1).
 *   amplitude   factor on cosine and sine (1 unless a long-context scaling
 *               asks for more).
 * A pair (a, b) at position p turns by t = 2 pi frac(p * step):
 * (a cos t - b sin t, a sin t + b cos t) * amplitude.  Rows outside every
 * sequence and rows at a negative position give zero q_out and write nothing.
 */
kda_status kda_rope_append(const kda_tensor* q, const kda_tensor* k, const kda_tensor* v, const kda_tensor* phase_steps,
                           const kda_tensor* cu_seqlens, const kda_tensor* seq_lens, const kda_tensor* page_table,
                           const kda_tensor* k_pages, const kda_tensor* v_pages, const kda_tensor* q_out,
                           int32_t interleaved, float amplitude, void* stream);

/*
 * Rotation steps for kda_rope_append, computed on the host into steps[rot/2]:
 * f_i = base^(-2i/rot) radians per position; with turns r_i = original_len *
 * f_i / 2 pi over the original context and keep_i = clamp((r_i - low) / (high
 * - low), 0, 1), the step is f_i (keep_i + (1 - keep_i) / factor): fast pairs
 * keep their frequency, slow ones are stretched by `factor`.  original_len =
 * 0 stretches all pairs alike (low and high unused); factor = 1 changes none.
 */
kda_status kda_rope_phase_steps(int32_t rot_dim, double base, double factor, double original_len, double low,
                                double high, uint64_t* steps);

/*
 * kda_paged_attention_decode: softmax attention of one new token per
 * sequence over its pages.  Launches two kernels: one over the positions,
 * split over every SM whatever the lengths, and one that joins the parts.
 *
 *   q           [N, Hq, D] float32 or bfloat16, D = 64, 128 or 256, any row and
 *               head strides that keep 4-element alignment.
 *   k_pages, v_pages, page_table: as above, of q's dtype; Hq a multiple of Hkv,
 *               query head h reads key head h / (Hq / Hkv).
 *   seq_lens    [N] int32, the new token included.  Positions past the table's
 *               P * page_size, at most 2^30, are not there to be attended to; a
 *               window counts from seq_lens[n] all the same.
 *   workspace   float32, contiguous, at least the floats that
 *               kda_paged_attention_workspace names for the device's SM count;
 *               its contents matter only during the call, so calls on one
 *               stream may share one, concurrent calls may not.
 *   window      0: every position; w > 0: only the last w positions, t >=
 *               seq_lens[n] - w.
 *   scale       > 0 and at most 2.3e38, normally 1/sqrt(D).
 *   out         [N, Hq, D] bfloat16 contiguous (written).
 *   lse         [N, Hq] float32 contiguous (written), or NULL: the natural
 *               logarithm of the sum of exp(scale q.k) over the row's positions.
 * Positions past the length, outside the window or on null pages are never
 * read into the result, whatever their bytes hold.  A row without positions
 * gives zero and an lse of minus infinity.  At an attended position a NaN, a
 * score of +infinity and an infinite value make the row's result non-finite; a
 * score of -infinity weighs nothing.  Values are summed before they are divided
 * by the weights' sum, so finite ones whose weighted sum passes float32 overflow.
 */
kda_status kda_paged_attention_decode(const kda_tensor* q, const kda_tensor* k_pages, const kda_tensor* v_pages,
                                      const kda_tensor* page_table, const kda_tensor* seq_lens,
                                      const kda_tensor* workspace, int32_t window, float scale, const kda_tensor* out,
                                      const kda_tensor* lse, void* stream);

/* Floats of workspace of kda_paged_attention_decode on a device of sm_count SMs (dtype: KDA_F32 / KDA_BF16). */
kda_status kda_paged_attention_workspace(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t dtype,
                                         int32_t sm_count, int64_t* floats);

/*
 * kda_beam_select: the best continuations of each request's beams.  Launches
 * two kernels, over the logits and over the pieces' candidates.
 *
 *   logits      [N, B, V] float32 or bfloat16, unit stride on the vocabulary, any
 *               other positive strides; B <= 32, V <= 2^24.
 *   scores      [N, B] float32 contiguous: log probability of each beam so far.
 *   finished    [N, B] int32 contiguous, or NULL: non-zero marks a beam that has
 *               ended; its one continuation is eos_token, at its score unchanged.
 *   workspace   float32, contiguous, the floats of kda_beam_select_workspace;
 *               its contents matter only during the call.
 *   out_scores float32, out_parents int32, out_tokens int32 [N, M] contiguous
 *               (written), 1 <= M <= 64.
 * Continuation (b, t) is worth scores[b] + logits[b, t] - log sum exp(logits[b]);
 * the M largest of a request's B * V are returned in falling order, equal ones
 * by rising b, then t.  Candidates are compared as unrounded sums of two
 * float32, the returned score is rounded to float32.  A beam's log-sum is off
 * by 1.1e-6 at most, 3.5e-7 where all logits are equal, far less over a
 * vocabulary of unequal ones, so beams whose candidates are closer than that
 * may be taken in either order; beams of equal logits and scores are equal, wherever
 * their rows start.  A logit of minus infinity is no continuation, and a beam
 * whose score or log-sum is not finite (a dead beam; a NaN or +infinity among
 * its logits) has none.  Places without one get -infinity, -1 and -1.
 */
kda_status kda_beam_select(const kda_tensor* logits, const kda_tensor* scores, const kda_tensor* finished,
                           int32_t eos_token, const kda_tensor* workspace, const kda_tensor* out_scores,
                           const kda_tensor* out_parents, const kda_tensor* out_tokens, void* stream);

/* Floats of workspace of kda_beam_select on a device of sm_count SMs (dtype of the logits: KDA_F32 / KDA_BF16). */
kda_status kda_beam_select_workspace(int64_t requests, int32_t beams, int64_t vocab, int32_t num_out, int32_t dtype,
                                     int32_t sm_count, int64_t* floats);

/*
 * kda_pool_move: copies whole slots inside pools, in place; forks, compacts,
 * clears and, by parent beam, reorders recurrent states, conv caches and
 * pages alike.
 *
 *   pools       n_pools (1..256) descriptors, rank 1..4, of any kda_dtype (bytes
 *               are copied, so other types move as views of one): axis 0 is
 *               the slot (the same number of slots in every pool), the other
 *               axes dense in any order (a conv cache's [slot_stride, 1, 3*H*128]
 *               and a head-major page are), slot stride as large or larger.
 *   src_slots, dst_slots  [N, K] int32, column stride 1, K <= 32.
 *   parents     [N, K] int32, column stride 1, or NULL (parent j = j).
 * In every pool, for every row n and all its j at once: slot dst[n, j] takes
 * what slot src[n, parents[n, j]] held before the call.  A parent outside
 * [0, K), or a destination outside [1, num_slots), moves nothing; a source
 * outside [1, num_slots) clears the destination to zero bytes; a slot that is
 * its own source is not touched.
 * Rows are independent and unordered: a live destination may appear once in
 * the call, and may be a source only in its own row (as the null slots, a
 * caller contract the library does not check).  Sources may repeat.
 * Launches one kernel per 64 pools.
 */
kda_status kda_pool_move(const kda_tensor* const* pools, int32_t n_pools, const kda_tensor* src_slots,
                         const kda_tensor* dst_slots, const kda_tensor* parents, void* stream);

/* ---- host-only queries (no CUDA calls) ---------------------------------- */

/* Operation ids for kda_plan_split. */
typedef enum kda_op {
  KDA_OP_RECURRENT = 0,
  KDA_OP_PACKED = 1,
  KDA_OP_FUSED = 2,
  KDA_OP_SPEC = 3,
  KDA_OP_PACKED_FUSED = 4
} kda_op;

/*
 * Value-column split the dispatcher picks for `units` = rows * heads on a
 * device with `sm_count` SMs (state_dtype: KDA_F32 / KDA_BF16; t_max: tokens
 * per row, 1 for T=1).  Each CTA then owns 128/split value columns of one
 * unit.  Returns the split (1, 2, 4, 8 or 16), or 0 on invalid arguments.
 * Honors kda_set_split_override.  For KDA_OP_PACKED_FUSED (units =
 * sequences * heads) the split is the size of the thread-block cluster that
 * shares a unit (1, 2, 4 or 8; a forced 16 runs as 8); for KDA_OP_FUSED it
 * is the cluster size of the split schedule: 1 unless forced (2 or 4; a
 * forced 8 or 16 runs as 4).
 */
int32_t kda_plan_split(int32_t op, int64_t units, int32_t state_dtype, int32_t t_max,
                       int32_t sm_count);

/*
 * Force the split of every later call in this process (0 restores the
 * measured policy).  For sweeps and tests.  Returns KDA_ERR_INVALID_ARG for
 * a split this build has no kernel for.  A forced split selects the split
 * schedule for the T=1 entry points unless a schedule is forced too.
 */
kda_status kda_set_split_override(int32_t split);

/*
 * Kernel schedules of the T=1 entry points (kda_recurrent_decode,
 * kda_packed_decode, kda_fused_decode).  SPLIT: one CTA per (row, head,
 * value split; the fused entry point's splits form a thread-block cluster
 * that shares the RMSNorm), the state block streamed through registers;
 * best for latency-bound batches.
 * STREAM: one persistent CTA per SM, a loader warp moving whole state
 * blocks (TMA, swizzled) and the unit's activation vectors into
 * shared-memory stages with bulk asynchronous copies while consumer warps
 * update earlier ones; needs every activation head vector (and, fused, the
 * conv-cache slots and conv_weight) 16-byte aligned, otherwise the call uses SPLIT, or
 * returns KDA_ERR_UNSUPPORTED if STREAM is forced.
 * MMA (kda_spec_decode and kda_spec_verify_decode with a bfloat16 state
 * pool): the chunked form of the token loop on the tensor cores ([P1]
 * "Frozen / speculative-verify mode" names the WY-parallel tensor-core form
 * of these rows): per chunk of up to 8 tokens, S^T [P k | P q] and the
 * rank-T update run as tcgen05 MMAs with float32 accumulators in tensor
 * memory, every operand as three bf16 pieces (within 2^-24 of its float32
 * value); one persistent CTA per SM.  The dispatcher picks it for a bfloat16
 * state pool with t_max >= 14 (unless a split or the SPLIT/STREAM schedule is
 * forced); forcing MMA with a float32 state returns KDA_ERR_UNSUPPORTED.
 * The speculative entry points otherwise use SPLIT (one CTA per row, head
 * and value slab, the state in registers).
 */
typedef enum kda_schedule {
  KDA_SCHED_AUTO = 0,
  KDA_SCHED_SPLIT = 1,
  KDA_SCHED_STREAM = 2,
  KDA_SCHED_MMA = 3
} kda_schedule;

/* Schedule the dispatcher picks (same arguments as kda_plan_split); 0 on invalid arguments. */
int32_t kda_plan_schedule(int32_t op, int64_t units, int32_t state_dtype, int32_t t_max,
                          int32_t sm_count);

/* Force the schedule of later calls (KDA_SCHED_AUTO restores the policy):
 * SPLIT / STREAM apply to the T=1 entry points, SPLIT / MMA to the
 * speculative ones; a schedule an entry point does not have is ignored
 * there. */
kda_status kda_set_schedule_override(int32_t schedule);

/*
 * Device error word of the streaming kernels on the current device: bit 0 =
 * a wait for a filled stage timed out (2 s), bit 1 = a wait for a free stage
 * timed out, bit 2 = the kda_selftest_wait_timeout wait gave up (expected),
 * bit 3 = a wait of the tensor-core (MMA) speculative kernel timed out.  A
 * kernel that times out records the bit and returns early, its results for
 * the affected units are undefined.  Synchronises the device;
 * clears the word when `clear` is non-zero.
 */
kda_status kda_device_error(uint32_t* flags, int32_t clear);

/*
 * Diagnostic of the bounded waits: launches one warp on `stream` that waits
 * on a barrier nothing completes.  The wait gives up after 2 s and sets bit
 * 2 (value 4) of the device error word, so the timeout path can be checked
 * without faulting or hanging the GPU; the context stays usable.
 */
kda_status kda_selftest_wait_timeout(void* stream);

const char* kda_status_string(kda_status s);
/* Detail of the last non-OK status returned on the calling thread. */
const char* kda_last_error_message(void);
/* Library version string. */
const char* kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
