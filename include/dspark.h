/*
 * dspark.h -- C ABI of the GB300 (sm_103a) DSpark verify planner, ragged
 * verify pack, greedy / cap / sampling accept, compact-to-strided scatter and
 * calibration library (libdspark.so).
 *
 * Pages cited below (by title and section):
 *   [AVS]   "DSpark 自适应 Verify 怎样分配候选预算" -- DSpark adaptive
 *           verify: how the candidate budget is allocated
 *   [ROUND] "DeepSeek-V4 DSpark一轮 Draft、Verify、Accept 与 Commit" -- one
 *           DSpark round: draft, verify, accept and commit
 *   [SGL]   "DSpark接入SGLang：用置信度驱动可变长度验证" -- DSpark in SGLang
 *   [TUT]   charlestar.github.io tutorial "DSpark confidence-scheduled
 *           speculative decoding"
 *
 * Conventions shared by every entry point
 *   - Every pointer is DEVICE memory unless its comment says "host".
 *   - The caller owns every buffer; the library allocates nothing.  Scratch
 *     comes from a caller-provided device workspace whose size the matching
 *     *_workspace_bytes() function returns (256-byte aligned pointer).
 *   - All work is enqueued asynchronously on `stream` (a cudaStream_t passed
 *     as void*; NULL = the legacy default stream).  No call synchronises the
 *     host; every result, including the budget, stays in device memory.
 *   - Return value: DSPARK_OK or a negative DSPARK_ERR_* code.  Argument
 *     checks happen on the host before anything is enqueued, so a rejected
 *     call has no effect on the device.
 *   - `status` (device int32[1], zeroed by the caller) collects
 *     DSPARK_STATUS_* bits that the kernels OR in for conditions only the
 *     device can see.  Kernels never trap or assert; their only waits on
 *     memory (the scatter's copy barriers, and those between the warps of
 *     the attention) give up, after 200 ms and about a second, and set
 *     DSPARK_STATUS_TIMEOUT.
 *   - Calls are stateless and thread-safe; concurrent calls must not share
 *     workspaces.
 */
#ifndef DSPARK_H
#define DSPARK_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define DSPARK_API __attribute__((visibility("default")))
#else
#define DSPARK_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- errors */
#define DSPARK_OK               0
#define DSPARK_ERR_INVALID_ARG (-1) /* null pointer, size or range violation */
#define DSPARK_ERR_WORKSPACE   (-2) /* workspace missing, too small or misaligned */
#define DSPARK_ERR_CUDA        (-3) /* a CUDA launch or attribute call failed */
#define DSPARK_ERR_UNSUPPORTED (-4) /* outside the supported envelope (see each call) */

/* device status bits (OR-ed into *status) */
#define DSPARK_STATUS_CAPACITY    1  /* a row count exceeded the buffer's capacity */
#define DSPARK_STATUS_TOKEN_RANGE 2  /* a draft token outside [0, V) */
#define DSPARK_STATUS_NAN_LOGIT   4  /* a NaN in a target-logits row (NaN never wins the argmax) */
#define DSPARK_STATUS_BAD_INPUT   8  /* a NaN confidence logit or a temperature that is not > 0 */
#define DSPARK_STATUS_BAD_LEN     16 /* a verify length / cu_seqlens range outside [1, gamma+1] */
#define DSPARK_STATUS_BAD_COST    32 /* cost table not ascending, or a non-positive / non-finite cost used */
#define DSPARK_STATUS_INFEASIBLE  64 /* no budget in range: budget set to 0 */
#define DSPARK_STATUS_BAD_INDEX   128 /* a packed row's strided destination outside the buffer */
#define DSPARK_STATUS_TIMEOUT     256 /* a kernel's bounded wait gave up (its outputs are incomplete) */
#define DSPARK_STATUS_BAD_TIER    512 /* a shared verify tier below this rank's packed rows */
/* Set only by the bounds-checked build (libdspark_checked.so, compiled with
 * -DDSPARK_CHECKED): an index a kernel computed from data fell outside the
 * buffer (global or shared memory) it addresses; the access was skipped.  It
 * always marks a defect of the library, never of the inputs.  The normal
 * build carries no such checks and never sets it. */
#define DSPARK_STATUS_OUT_OF_BOUNDS 1024

/* Message for a DSPARK_ERR_* code (static string). */
DSPARK_API const char *dspark_strerror(int code);

/* Library version: major*10000 + minor*100 + patch. */
DSPARK_API int dspark_version(void);

/* 1 in the bounds-checked build (see DSPARK_STATUS_OUT_OF_BOUNDS), 0 in the
 * normal one.  The two builds export the same calls with the same results. */
DSPARK_API int dspark_checked_build(void);

/* ---------------------------------------------------------------- planner */

#define DSPARK_COST_SPS_1D   0
#define DSPARK_COST_ADDITIVE 1
#define DSPARK_COST_ADDITIVE_INTERP 2

/* Planner parameters (host struct).  [AVS] §一: ScheduleVerifyLensTopk is
 * bounded by min_verify_len, max_verify_len and survival_eps. */
typedef struct {
    int32_t B;              /* requests in this planner decision, >= 1 */
    int32_t gamma;          /* draft tokens per request, 1..31 */
    float survival_eps;     /* candidates with survival < eps are dropped; in [2^-14, 1] */
    int32_t min_verify_len; /* 1 <= min <= max */
    int32_t max_verify_len; /* <= gamma + 1; depths >= max-1 are never candidates */
    int32_t forced_budget;  /* < 0: budget = argmax theta; >= 0: this budget, clipped to range */
} dspark_plan_params;

/* Step-cost table (host struct pointing at DEVICE arrays M[n], val[n]).
 *   DSPARK_COST_SPS_1D ([AVS] §一 and §四 "1D SpsCostTable"):
 *     theta(b) = tau(b) * SPS(B + b); SPS is a floor lookup -- the sample
 *     with the largest M_j <= B + b, sample 0 below the first -- with no
 *     interpolation.  val = steps per second, must be > 0.
 *   DSPARK_COST_ADDITIVE ([AVS] §一/§四 "Additive SPS"; [TUT] T(bs,K)):
 *     theta(b) = tau(b) / T, T = (bias_ms + alpha_ms) + val[j] with j the
 *     smallest graph tier M_j >= B + b; budgets above the largest tier are
 *     infeasible.  alpha_ms is alpha(B) already evaluated for this B.
 *   DSPARK_COST_ADDITIVE_INTERP ([AVS] §四 "三个关键假设", the third: the
 *     exported additive table interpolates theta(M) linearly at runtime):
 *     T = (bias_ms + alpha_ms) + theta(B + b), with M_j <= M < M_{j+1}
 *     theta(M) = val[j] + (M - M_j) * slope_j, slope_j = (val[j+1] - val[j])
 *     / (M_{j+1} - M_j), in that fp64 order; val[j] at M = M_j; val[0] below
 *     M_0; budgets with B + b above the last sample are infeasible.  Every
 *     budget has its own cost, so theta is evaluated at every in-range
 *     budget (one fp64 division each, on one CTA).
 *   M must be strictly ascending (else DSPARK_STATUS_BAD_COST, all budgets
 *   infeasible).  A used entry whose SPS or T is not a positive finite
 *   number is infeasible and flagged DSPARK_STATUS_BAD_COST. */
typedef struct {
    int32_t kind;          /* DSPARK_COST_SPS_1D, _ADDITIVE or _ADDITIVE_INTERP */
    int32_t n;             /* entries, >= 1 */
    const int32_t *M;      /* device [n]: total verify rows (1-D) or graph tiers (additive) */
    const double *val;     /* device [n]: SPS (steps/s) or token-side cost theta(M) in ms */
    double bias_ms;        /* additive only */
    double alpha_ms;       /* additive only */
} dspark_cost_table;

/* Device scratch of one planner call: about 24 * B * gamma + 4 * B + 25 KB
 * (a completion counter, a 2048-bin histogram of the survivals, candidate
 * ranks, the sorted survivals and their prefix sums, and what passes of one
 * call hand over).  The workspace must be zero-filled
 * once before its first dspark_plan call (cudaMemset); every call that
 * returns DSPARK_OK leaves the histogram zero again, and a call that
 * returns DSPARK_ERR_CUDA after launching clears it on the stream, so the
 * buffer can be passed unchanged to the next call.  Do not reuse it for
 * other data between planner calls. */
DSPARK_API size_t dspark_plan_workspace_bytes(int32_t B, int32_t gamma);

/* The verify planner.  [AVS] §一 (budget by survival, tau, theta, argmax,
 * ScheduleVerifyLensTopk), §二 (STS c = sigmoid(z / T), S_k = prod c);
 * [ROUND] §三 (resolve_verify_token_budget, schedule_layout).
 *   conf_logits  [B, gamma] fp32 row-major: confidence-head logits z
 *   sts_temps    [gamma] fp32: per-depth STS temperature T_k > 0
 *   p, cost      host structs (above); cost->M / cost->val are device arrays
 *   survivals    out [B, gamma] fp32: S_k = prod_{i<=k} sigmoid(z_i / T_i),
 *                fp32 sequential product, 0 where S_k < eps
 *   verify_lens  out [B] int32: 1 (root) + candidates selected for the
 *                request, clamped to [min_verify_len, max_verify_len]
 *   budget       out [1] int32: extra verify rows b (argmax or forced)
 *   tau_theta    out [2] fp64: tau(budget) = B + sum of the budget largest
 *                survivals (exact), theta(budget) (0 if the budget is infeasible)
 * Candidates are ordered by survival descending, then depth ascending,
 * then request id ascending; theta ties go to the smaller budget.
 * Errors: INVALID_ARG (null pointer, B < 1, min/max out of order, cost n < 1
 * or unknown kind); UNSUPPORTED (gamma > 31, B*(gamma+1) > 65536,
 * B*gamma > 16384, eps outside [2^-14, 1]); WORKSPACE (missing, smaller than
 * dspark_plan_workspace_bytes(B, gamma) or not 256-byte aligned); CUDA.
 * Device flags: BAD_INPUT, BAD_COST, INFEASIBLE. */
DSPARK_API int dspark_plan(const float *conf_logits, const float *sts_temps,
                const dspark_plan_params *p /* host */, const dspark_cost_table *cost /* host */,
                float *survivals, int32_t *verify_lens, int32_t *budget, double *tau_theta,
                void *workspace, size_t workspace_bytes, int32_t *status, void *stream);

/* Options of the planner ([AVS] §三, the conditions under which the
 * executed budget departs from the plain plan).  Every field may be left
 * zero / NULL.
 *   conf_generation, req_generation  device [B] int32, both or neither: a
 *       request whose confidences were recorded for another generation of
 *       its pool slot plans with survivals of 1 at every depth (optimistic;
 *       [AVS] §三 "req_generation")
 *   lagged_conf_logits  device [B, gamma] fp32: the budget is chosen from
 *       these (lagged) confidences, then allocated over the current ones by
 *       the same ordering, as with a forced budget ([AVS] §三, overlap
 *       scheduler: lagged confidence sets the budget, the current one the
 *       allocation); tau/theta are reported for the allocation
 *   align_to_tiers  1: graph-tier alignment ([AVS] §三, §五 "paid-padding
 *       reclamation"): with T verify rows at the chosen budget and the
 *       smallest tier >= T, the executed budget takes one more candidate per
 *       spare row of that tier, as long as candidates remain in range; no
 *       tier holds T: unchanged.  Also applies to a forced budget.
 *   host_tiers, n_tiers  host: the tiers for alignment (dspark_plan_ex; the
 *       pack's tiers are used by dspark_plan_pack_ex) */
typedef struct {
    const int32_t *conf_generation;
    const int32_t *req_generation;
    const float *lagged_conf_logits;
    int32_t align_to_tiers;
    const int32_t *host_tiers;
    int32_t n_tiers;
} dspark_plan_options;

/* dspark_plan with options (opt may be NULL: dspark_plan).  Each option adds
 * planner passes over the same workspace: lagged confidences a survival
 * kernel and a pass, alignment a pass.  Errors: those of dspark_plan, and
 * INVALID_ARG for one generation array without the other or alignment
 * without a valid tier list. */
DSPARK_API int dspark_plan_ex(const float *conf_logits, const float *sts_temps,
                   const dspark_plan_params *p /* host */, const dspark_cost_table *cost /* host */,
                   const dspark_plan_options *opt /* host, nullable */, float *survivals,
                   int32_t *verify_lens, int32_t *budget, double *tau_theta, void *workspace,
                   size_t workspace_bytes, int32_t *status, void *stream);

/* ------------------------------------------------------------------ pack */

#define DSPARK_MAX_TIERS 64

/* Front-pack the verify rows and round the total up to a graph tier.
 * [ROUND] §三 (verify ids = [anchor, drafts]; BuildRaggedVerifyWindow /
 * compact_verify_ids), §四 (verify positions); [AVS] §六 (cu_seqlens_q with
 * a leading 0); [SGL] "Ragged verify"; [TUT] "变长批次如何与 CUDA Graph 共存".
 *   anchor [B], draft [B, gamma], prefix_lens [B], verify_lens [B]: int32
 *   host_tiers   host [n_tiers] ascending graph tiers (n_tiers <= 64; 0 = no
 *                rounding)
 *   capacity     rows available in each packed_* buffer
 *   packed_ids/pos/req/src  out [capacity] int32.  Row cu[r]+j (j < len_r):
 *                id = anchor[r] (j = 0) or draft[r][j-1]; pos = prefix_lens[r]
 *                + j; req = r; src = r*(gamma+1) + j (row in the strided
 *                [B, gamma+1] layout).  Rows [total, padded) are pad rows
 *                (0, 0, -1, -1); rows >= padded are not written.
 *   cu_seqlens   out [B+1] int32, cu[0] = 0
 *   totals       out [2] int32: {total, padded}
 * A length outside [1, gamma+1] is clamped and flagged BAD_LEN; rows past
 * capacity are dropped and flagged CAPACITY, as is a total above the
 * largest tier (then padded = total).
 * Errors: INVALID_ARG (null pointer, B < 1, gamma outside 1..31, capacity
 * < 0, n_tiers outside 0..64, tiers not ascending); CUDA. */
DSPARK_API int dspark_pack_verify(const int32_t *anchor, const int32_t *draft, const int32_t *prefix_lens,
                       const int32_t *verify_lens, int32_t B, int32_t gamma,
                       const int32_t *host_tiers /* host */, int32_t n_tiers, int32_t capacity,
                       int32_t *packed_ids, int32_t *packed_pos, int32_t *packed_req,
                       int32_t *packed_src, int32_t *cu_seqlens, int32_t *totals,
                       int32_t *status, void *stream);

/* dspark_plan followed by dspark_pack_verify on the planner's verify_lens,
 * in fewer launches: for cost tables of at most 6143 entries (interpolated:
 * 2048 samples) the planner's last kernel, which runs on one CTA, also packs
 * the window (one launch and one dependency wait fewer per step); larger
 * tables run the two calls' kernels back to back.
 * Arguments and outputs are those of the two calls (the planner's
 * workspace, which must be zero-filled once, serves both); the pages'
 * planner and pack are the same two steps ([AVS] §一, §五-§六; [ROUND]
 * §三).  Errors: those of dspark_plan, then of dspark_pack_verify's
 * arguments (checked before anything is launched). */
DSPARK_API int dspark_plan_pack(const float *conf_logits, const float *sts_temps,
                     const dspark_plan_params *p /* host */, const dspark_cost_table *cost /* host */,
                     float *survivals, int32_t *verify_lens, int32_t *budget, double *tau_theta,
                     const int32_t *anchor, const int32_t *draft, const int32_t *prefix_lens,
                     const int32_t *host_tiers /* host */, int32_t n_tiers, int32_t capacity,
                     int32_t *packed_ids, int32_t *packed_pos, int32_t *packed_req,
                     int32_t *packed_src, int32_t *cu_seqlens, int32_t *totals,
                     void *workspace, size_t workspace_bytes, int32_t *status, void *stream);

/* Scratch of one sampling accept: per-(CTA, row) softmax partials for up
 * to max_rows target rows and B*gamma draft rows, and B+1 offsets. */
DSPARK_API size_t dspark_sampling_workspace_bytes(int32_t max_rows, int32_t B, int32_t gamma);

/* Speculative sampling accept, compact mode ([ROUND] §五 AcceptSampling
 * with chain speculative sampling; [AVS] §一: a draft drawn from q is
 * accepted with probability min(1, p/q)).  The pages leave the rule to the
 * speculative algorithm; this is the textbook one:
 *   p_j = softmax(target row cu[r] + j), q_j = softmax(draft row r*gamma+j)
 *   draft j (token x) is accepted iff u_accept[r][j] * q_j(x) < p_j(x); the
 *   chain stops at the first rejection (correct_len = j)
 *   bonus: inverse-CDF draw with u_bonus[r] -- the smallest token whose
 *   cumulative weight exceeds u * W -- from max(0, p_j - q_j) after a
 *   rejection (from p_j when that residual's mass is below 2^-20), else from the last
 *   row's p; then num_accepted / commit_lens / new_seq_lens / out_tokens as
 *   dspark_greedy_accept.
 *   target_logits  [max_rows, ld_t] bf16 or fp32, draft_logits [B*gamma,
 *                  ld_d] of the same dtype: the proposal logits that produced
 *                  each draft (after any correction)
 *   u_accept [B, gamma], u_bonus [B]: fp32 uniforms in [0, 1) (the caller's
 *                  random numbers)
 * Softmax sums are fp32 per thread and fp64 beyond, the bonus weights are
 * summed exactly in units of 2^-40: a decision can differ from an exact
 * evaluation only within ~1e-6 relative of its threshold.  NaN logits weigh
 * 0 (DSPARK_STATUS_NAN_LOGIT); a draft token outside [0, V) is rejected
 * (TOKEN_RANGE); a bad cu range gives the greedy defaults (BAD_LEN).
 * Errors: INVALID_ARG (null pointer, dtype, B < 1, gamma outside 1..31,
 * V < 1, a stride below V, max_rows < 0); UNSUPPORTED (B > 4096 or
 * V > 2^20); WORKSPACE; CUDA. */
DSPARK_API int dspark_sampling_accept(const void *target_logits, int32_t dtype, int64_t ld_t,
                           int32_t V, int32_t max_rows, const int32_t *cu_seqlens,
                           const void *draft_logits, int64_t ld_d, const int32_t *draft,
                           const int32_t *prefix_lens /* nullable with new_seq_lens */,
                           int32_t B, int32_t gamma, const float *u_accept,
                           const float *u_bonus, int32_t *num_accepted, int32_t *bonus,
                           int32_t *commit_lens, int32_t *new_seq_lens /* nullable */,
                           int32_t *out_tokens, void *workspace, size_t workspace_bytes,
                           int32_t *status, void *stream);

/* dspark_sampling_accept with the draft rows' softmax normalizers supplied
 * by the caller -- the drafting step's sampler has them -- so that the
 * draft rows are not streamed to normalise them (only the target rows are;
 * a rejected request's draft row is still read for the residual bonus):
 *   draft_lse  [B*gamma] fp32 (nullable: dspark_sampling_accept):
 *              log(sum_y exp(z_y)) of draft row r*gamma + j (natural log);
 *              q_j(x) = exp(z_x - draft_lse[r*gamma + j]).  Read for the
 *              tested drafts only.  A non-finite value makes that row's q
 *              zero everywhere.
 * Everything else, including the workspace size, as dspark_sampling_accept. */
DSPARK_API int dspark_sampling_accept_ex(const void *target_logits, int32_t dtype, int64_t ld_t,
                           int32_t V, int32_t max_rows, const int32_t *cu_seqlens,
                           const void *draft_logits, int64_t ld_d, const float *draft_lse,
                           const int32_t *draft, const int32_t *prefix_lens, int32_t B,
                           int32_t gamma, const float *u_accept, const float *u_bonus,
                           int32_t *num_accepted, int32_t *bonus, int32_t *commit_lens,
                           int32_t *new_seq_lens, int32_t *out_tokens, void *workspace,
                           size_t workspace_bytes, int32_t *status, void *stream);

/* ScatterCompactToStrided ([ROUND] §三): after the target forward over the
 * compact verify rows, copy packed row i (i < totals[0]) to row
 * packed_src[i] = r*(gamma+1) + j of the [B x (gamma+1)] strided buffer, so
 * that the accept can address rows by fixed position (cap-accept); pad rows
 * and the strided rows no request selected are left untouched.
 *   src          device [max_rows, ld_src] rows of `width` elements of
 *                elem_bytes (2: bf16 logits or hidden states, 4: fp32)
 *   packed_src   device [max_rows] int32, the pack's output
 *   totals       device [>= 1] int32, totals[0] = real packed rows (clamped
 *                to [0, max_rows])
 *   dst          device [dst_rows, ld_dst], strides in elements
 * TMA bulk copies (16 KB segments staged in shared memory) when both
 * buffers, both strides and the row size are 16-byte multiples, else 2-byte
 * copies.  A destination outside [0, dst_rows) is skipped and flagged
 * DSPARK_STATUS_BAD_INDEX; DSPARK_STATUS_TIMEOUT if a copy did not complete
 * within 200 ms (that CTA then copies nothing more: the rows it had left are
 * not written).
 * Errors: INVALID_ARG (null pointer, elem_bytes not 2 or 4, width < 1, a
 * stride below width, negative row counts); CUDA. */
DSPARK_API int dspark_scatter_compact_to_strided(const void *src, int64_t ld_src, int32_t width,
                                      int32_t elem_bytes, const int32_t *packed_src,
                                      const int32_t *totals, int32_t max_rows, void *dst,
                                      int64_t ld_dst, int32_t dst_rows, int32_t *status,
                                      void *stream);

/* dspark_scatter_compact_to_strided with the limit of one pipeline wait of
 * the TMA path in the caller's hands (no counterpart on the pages: failure
 * detection).
 *   wait_limit_ns  < 0: 200 ms (the default); 0: each wait tests its copy
 *                  once, so a copy not yet landed at the first test gives
 *                  up -- how the tests exercise the give-up path.
 * A CTA that gives up flags DSPARK_STATUS_TIMEOUT, issues nothing more,
 * waits (up to 200 ms each, whatever wait_limit_ns) for the loads it still
 * has in flight and for its stores, and exits; the call returns normally and
 * the rows that CTA had left are not written.  The 2-byte path has no waits. */
DSPARK_API int dspark_scatter_compact_to_strided_ex(const void *src, int64_t ld_src,
                                      int32_t width, int32_t elem_bytes,
                                      const int32_t *packed_src, const int32_t *totals,
                                      int32_t max_rows, void *dst, int64_t ld_dst,
                                      int32_t dst_rows, int64_t wait_limit_ns, int32_t *status,
                                      void *stream);

/* The verify tier shared by data-parallel ranks.  [AVS] §六 "DP / DeepEP
 * 是第二层复杂度" (each rank's local verify tier is gathered and the
 * DP-global max token tier is what every rank replays); [SGL] "Ragged
 * verify" (under DP attention the ranks share one tier, the largest any rank
 * needs).  Each rank packs its own requests (dspark_pack_verify or
 * dspark_plan_pack: totals[1] = its local tier), the ranks take the max of
 * totals[1] (one int32 MAX all-reduce, e.g. NCCL, on the step's stream), and
 * this call pads the rank's window to the result:
 *   pad_to       device [1] int32: the shared tier.  May point at totals + 1
 *                (the all-reduce done in place).
 *   capacity     rows of the packed_* buffers
 *   packed_*     device [capacity], the pack's outputs; rows
 *                [totals[0], min(*pad_to, capacity)) become pad rows (id 0,
 *                position 0, request -1, source -1), other rows untouched
 *   totals       device [2] in/out: totals[0] (real rows) is read,
 *                totals[1] = *pad_to is written
 * A shared tier below totals[0] changes nothing and flags
 * DSPARK_STATUS_BAD_TIER; one above capacity writes up to capacity and flags
 * DSPARK_STATUS_CAPACITY.  No host synchronisation.
 * Errors: INVALID_ARG (null pointer, capacity < 0); CUDA. */
DSPARK_API int dspark_pad_to_tier(const int32_t *pad_to, int32_t capacity, int32_t *packed_ids,
                                  int32_t *packed_pos, int32_t *packed_req, int32_t *packed_src,
                                  int32_t *totals, int32_t *status, void *stream);

/* dspark_plan_pack with options (see dspark_plan_options; alignment uses
 * the pack's tiers). */
DSPARK_API int dspark_plan_pack_ex(const float *conf_logits, const float *sts_temps,
                        const dspark_plan_params *p /* host */,
                        const dspark_cost_table *cost /* host */,
                        const dspark_plan_options *opt /* host, nullable */, float *survivals,
                        int32_t *verify_lens, int32_t *budget, double *tau_theta,
                        const int32_t *anchor, const int32_t *draft, const int32_t *prefix_lens,
                        const int32_t *host_tiers /* host */, int32_t n_tiers, int32_t capacity,
                        int32_t *packed_ids, int32_t *packed_pos, int32_t *packed_req,
                        int32_t *packed_src, int32_t *cu_seqlens, int32_t *totals,
                        void *workspace, size_t workspace_bytes, int32_t *status, void *stream);

/* ---------------------------------------------------------------- accept */

#define DSPARK_DTYPE_BF16 0
#define DSPARK_DTYPE_F32  1

/* Scratch of one accept call over at most max_rows rows. */
DSPARK_API size_t dspark_accept_workspace_bytes(int32_t max_rows, int32_t V);

/* Compact-mode greedy accept.  [ROUND] §五 "Greedy" (target_predict =
 * argmax(target_logits); correct_len = leading drafts equal to the target
 * chain; bonus from the last valid input row; no acceptance past the first
 * mismatch), FinalizeAcceptLens and BuildOutTokens.
 *   logits       [max_rows, ld] bf16 or fp32 (dtype), row stride ld >= V
 *                elements; 16-byte aligned base and ld*elem % 16 == 0 take
 *                the vector path, anything else a scalar path.  Device
 *                memory, or pinned host memory (device-accessible at the
 *                same address under unified addressing): the kernels then
 *                read the packed rows over the host link, with no copy step
 *   cu_seqlens   [B+1]: request r owns packed rows [cu[r], cu[r+1]); rows
 *                = min(cu[B], max_rows) rows are read (CAPACITY if cu[B] >
 *                max_rows)
 *   draft        [B, gamma]; prefix_lens [B] (may be NULL iff new_seq_lens is)
 *   argmax       out [max_rows] (nullable): argmax of every row < rows --
 *                lowest index of the largest non-NaN value, -0 == +0, 0 for
 *                a row with nothing above -inf
 *   num_accepted out [B]: correct_len = first j < L-1 with argmax(row
 *                cu[r]+j) != draft[r][j], else L-1 (L = cu[r+1]-cu[r])
 *   bonus        out [B]: argmax of row cu[r] + correct_len
 *   commit_lens  out [B]: correct_len + 1
 *   new_seq_lens out [B] (nullable): prefix_lens + commit_lens
 *   out_tokens   out [B, gamma+1]: drafts, -1 in column gamma, then the
 *                bonus written at column correct_len
 * A request whose range is empty, longer than gamma+1 or beyond rows gets
 * correct 0, bonus -1, commit 0 (flag BAD_LEN).  Device flags also:
 * TOKEN_RANGE, NAN_LOGIT, CAPACITY.
 * Errors: INVALID_ARG (null pointer, B < 1, gamma outside 1..31, V < 1,
 * ld < V, max_rows < 0, unknown dtype, new_seq_lens without prefix_lens);
 * WORKSPACE; CUDA. */
DSPARK_API int dspark_greedy_accept(const void *logits, int32_t dtype, int64_t ld, int32_t V,
                         int32_t max_rows, const int32_t *cu_seqlens, const int32_t *draft,
                         const int32_t *prefix_lens, int32_t B, int32_t gamma, int32_t *argmax,
                         int32_t *num_accepted, int32_t *bonus, int32_t *commit_lens,
                         int32_t *new_seq_lens, int32_t *out_tokens, void *workspace,
                         size_t workspace_bytes, int32_t *status, void *stream);

/* cap-accept: verify the full block, commit only the window.  [AVS] §三
 * (capped_correct_len = min(raw_correct_len, verify_len - 1)), §五
 * "cap-accept"; [SGL] "三种 verify mode" (commits equal compact's and the
 * full-verify acceptance ceiling is exposed).
 *   logits       [B*(gamma+1), ld] strided verify rows, row r*(gamma+1)+j
 *   verify_lens  [B] (clamped to [1, gamma+1], flag BAD_LEN)
 *   outputs as dspark_greedy_accept, with L = gamma+1 for the raw count:
 *   num_accepted = capped; bonus = argmax of row r*(gamma+1) + capped
 *   ceiling      out [B]: raw correct_len over the full block
 *   totals       out [2] int32: {sum commit_lens, sum (ceiling + 1)}
 * Errors as dspark_greedy_accept. */
DSPARK_API int dspark_cap_accept(const void *logits, int32_t dtype, int64_t ld, int32_t V,
                      const int32_t *verify_lens, const int32_t *draft,
                      const int32_t *prefix_lens, int32_t B, int32_t gamma, int32_t *argmax,
                      int32_t *num_accepted, int32_t *bonus, int32_t *commit_lens,
                      int32_t *new_seq_lens, int32_t *out_tokens, int32_t *ceiling,
                      int32_t *totals, void *workspace, size_t workspace_bytes,
                      int32_t *status, void *stream);

/* ------------------------------------------------ allocation-free accept */

#define DSPARK_STATIC_MAX_ROWS 32768

/* dspark_greedy_accept without a workspace.  The pages have no counterpart:
 * this exists for callers that cannot allocate device memory (embeddings
 * that only pass in buffers they own, runtimes whose device memory is fixed
 * at start-up and that forbid cudaMalloc afterwards).
 *   Arguments, outputs and device flags are those of dspark_greedy_accept,
 *   minus workspace / workspace_bytes.
 *   Scratch: a file-scope device array of (4096 + 32768 + 1) * 8 bytes
 *   rounded up to 256 (~300 KB) that every GPU loading this library holds
 *   until the process exits.  max_rows may be at most DSPARK_STATIC_MAX_ROWS
 *   (else DSPARK_ERR_UNSUPPORTED, nothing enqueued); a device row count
 *   cu_seqlens[B] above max_rows is clamped to max_rows and flags
 *   DSPARK_STATUS_CAPACITY, as in dspark_greedy_accept.
 *   The first call on a device looks up the array's device address with
 *   cudaGetSymbolAddress (and so loads the module on that device) and keeps
 *   it for the life of the process; make that first call on each device
 *   before any stream capture.  cudaDeviceReset unloads the module and makes
 *   the kept address stale: a process that resets a device must not call
 *   this function on that device afterwards.
 *   Every call shares the one array: calls whose kernels may overlap on the
 *   GPU (different streams without ordering) race on it.  The array keeps the
 *   last call's contents; nothing in it needs clearing, because every slot a
 *   call reads is written earlier in the same call.
 *   Allocates nothing: no cudaMalloc, cudaFree or allocating library call. */
DSPARK_API int dspark_greedy_accept_static(const void *logits, int32_t dtype, int64_t ld, int32_t V,
                         int32_t max_rows, const int32_t *cu_seqlens, const int32_t *draft,
                         const int32_t *prefix_lens, int32_t B, int32_t gamma, int32_t *argmax,
                         int32_t *num_accepted, int32_t *bonus, int32_t *commit_lens,
                         int32_t *new_seq_lens, int32_t *out_tokens, int32_t *status,
                         void *stream);

/* ------------------------------------------------------------ calibration
 *
 * STS recorder, calibration statistics and the sequential temperature fit.
 *   [AVS] §二 "但 SGLang STS 校准的不是同一个 soft target" (the recorder's
 *   label: prefix_mask = positions < num_correct_drafts) and "STS
 *   更像运行时语义桥" (c_i = sigmoid(z_i / T_i); the fitter picks a
 *   temperature position by position, keeping the cumulative survival of the
 *   positions already fitted, by lowest ECE); §七 A (per-position and
 *   cumulative calibration, ECE, Brier).  [TUT] "为什么置信度必须校准"
 *   (ECE = sum_b |I_b|/n |acc(I_b) - conf(I_b)|), "截短会制造观测盲区"
 *   (positions past a compact window are censored), "置信度质量" (by depth;
 *   reliability diagram; ECE, Brier score or log loss).
 *
 * A recorded sample is one request of one step: its confidence logits
 * z[gamma] (fp32), `correct` = drafts accepted and `tested` = drafts the
 * target checked.  Definitions used by the statistics and the fit:
 *   - tested is clamped to [0, gamma] and correct to [0, tested] (BAD_LEN);
 *   - depth k is observed iff k < tested; its label is y_k = (k < correct);
 *   - flavour 0 (cumulative): prediction S_k = c_0 * ... * c_k (fp32, left
 *     to right, c as in dspark_plan), over observed samples; flavour 1
 *     (per-position): prediction c_k over observed samples with correct >= k
 *     (the prefix survived through k-1); a NaN prediction is left out;
 *   - n_bins equal-width bins over [0, 1]: bin = min(floor(p*n_bins),
 *     n_bins-1); each confidence enters the bin sums as floor(p * 2^32), so
 *     the bin sums are exact integers and ECE = sum_b |L_b 2^32 - C_b| /
 *     (n 2^32) is exact up to its final rounding (within 2^-32 of the
 *     real-number ECE);
 *   - Brier = mean (p - y)^2 and log loss = mean -[y ln p + (1-y) ln(1-p)]
 *     with p clamped to [2^-24, 1 - 2^-24]; each term is evaluated as a pair
 *     of floats (Brier to ~2^-47 relative, the log term to ~2^-43 absolute)
 *     and the sums end in fp64 (deterministic for a given GPU; within ~1e-13
 *     of a sequential fp64 sum);
 *   - a flavour/depth with no sample reports n = 0 and zeros. */

/* STS-calibrated confidences c[r][k] = sigmoid(conf_logits[r][k] /
 * sts_temps[k]) ([AVS] §二, c_i = sigmoid(z_i / T_i)), elementwise over
 * [n_rows, gamma] fp32 -- the same values the planner multiplies into its
 * survivals: IEEE fp32 division, then the fp64 formula 1 / (1 + exp(-t))
 * rounded once to fp32 (evaluated in fp32 arithmetic wherever that
 * certifies the same rounding).  Flags BAD_INPUT for a NaN logit or a
 * temperature that is not > 0.  Errors: INVALID_ARG (null pointer, n_rows <
 * 0, gamma < 1); CUDA. */
DSPARK_API int dspark_sts_confidence(const float *conf_logits, const float *sts_temps,
                                     int64_t n_rows, int32_t gamma, float *conf_out,
                                     int32_t *status, void *stream);

/* Append the selected requests of one step to ring buffers of recorded
 * samples, and optionally write the step's greedy prefix mask.
 *   conf_logits  [B, gamma] fp32 confidence logits of the step
 *   num_correct  [B] accepted drafts (num_accepted of the compact accept, or
 *                the cap-accept ceiling with verify_lens NULL)
 *   verify_lens  [B] (nullable): tested = verify_len - 1, verify_len clamped
 *                to [1, gamma+1] (BAD_LEN); NULL = the full block was tested
 *   select       [B] uint8 (nullable): record request r iff select[r] != 0;
 *                NULL records every request
 *   rec_logits   [capacity, gamma] fp32, rec_correct / rec_tested
 *                [capacity] int32: the ring; the i-th selected request of the
 *                call (request order) goes to slot (*cursor + i) % capacity;
 *                num_correct is stored clamped to [0, tested] (BAD_LEN)
 *   cursor       device uint64[1], advanced by the number selected (so a
 *                captured graph can record every step); when one call
 *                selects more than capacity requests only the last capacity
 *                are written (CAPACITY)
 *   prefix_mask  [B, gamma] uint8 (nullable): (k < clamped num_correct)
 * One CTA; any B.  Errors: INVALID_ARG (null required pointer, B < 1, gamma
 * outside 1..31, capacity < 1); CUDA. */
DSPARK_API int dspark_sts_record(const float *conf_logits, const int32_t *num_correct,
                                 const int32_t *verify_lens, const uint8_t *select, int32_t B,
                                 int32_t gamma, float *rec_logits, int32_t *rec_correct,
                                 int32_t *rec_tested, int64_t capacity, uint64_t *cursor,
                                 uint8_t *prefix_mask, int32_t *status, void *stream);

/* Workspace of dspark_calibration_stats (independent of N); 0 for gamma
 * outside 1..31 or n_bins outside 1..32.  Zero-fill it once before its first
 * use: every call leaves it zeroed again. */
DSPARK_API size_t dspark_calibration_workspace_bytes(int32_t gamma, int32_t n_bins);

/* Calibration of N recorded samples under temperatures sts_temps, by depth.
 *   rec_logits [N, gamma] fp32, rec_correct / rec_tested [N] int32 (may be
 *              NULL when N == 0)
 *   sts_temps  [gamma] fp32 (a value that is not > 0 flags BAD_INPUT and is
 *              used as given)
 *   hist       out [2][gamma][n_bins][3] uint64 (nullable): per flavour,
 *              depth and bin -- count, label sum, confidence sum in 2^-32
 *              units (a reliability diagram)
 *   metrics    out [2][gamma][4] fp64: n, ECE, Brier, log loss
 * Device flags: BAD_INPUT (NaN logit anywhere, temperature not > 0),
 * BAD_LEN.  Errors: INVALID_ARG (null required pointer, N outside
 * 0..2^31-1, gamma outside 1..31, n_bins outside 1..32); WORKSPACE; CUDA. */
DSPARK_API int dspark_calibration_stats(const float *rec_logits, const int32_t *rec_correct,
                                        const int32_t *rec_tested, int64_t N, int32_t gamma,
                                        const float *sts_temps, int32_t n_bins, uint64_t *hist,
                                        double *metrics, void *workspace,
                                        size_t workspace_bytes, int32_t *status, void *stream);

/* Workspace of dspark_sts_fit; 0 outside the envelope.  Zero-fill it once
 * before its first use: every call leaves the part that must be zero zeroed
 * again. */
DSPARK_API size_t dspark_sts_fit_workspace_bytes(int64_t N, int32_t n_temps, int32_t n_bins);

/* Sequential temperature scaling fit.  For depth k = 0, 1, ..., gamma-1 and
 * every grid temperature T_j: the cumulative survival S_k = S_{k-1} *
 * sigmoid(z_k / T_j), with S_{k-1} under the temperatures already chosen,
 * is scored by its ECE (flavour 0 above) over the samples observed at depth
 * k; the lowest ECE * n * 2^32 (an exact integer) wins, ties to the lower
 * grid index.  A depth with no observed sample gets T = 1 and choice -1.
 *   rec_*         as in dspark_calibration_stats (NULL allowed when N == 0)
 *   temp_grid     HOST [n_temps] fp32, each positive and finite
 *   sts_temps_out out [gamma] fp32: the fitted temperatures (grid values)
 *   choice        out [gamma] int32: grid index per depth, -1 = none
 *   ece_curve     out [gamma][n_temps] fp64 (nullable): ECE of every candidate
 *   n_obs         out [gamma] int64 (nullable): samples observed per depth
 * gamma launches (one per depth), N * n_temps fp32-rounded fp64 sigmoids
 * each.  Device flags: BAD_INPUT (NaN logit), BAD_LEN.  Errors: INVALID_ARG
 * (null required pointer, N outside 0..2^31-1, gamma outside 1..31, n_temps outside
 * 1..256, a grid value not positive and finite, n_bins outside 1..32);
 * WORKSPACE; CUDA. */
DSPARK_API int dspark_sts_fit(const float *rec_logits, const int32_t *rec_correct,
                              const int32_t *rec_tested, int64_t N, int32_t gamma,
                              const float *temp_grid /* host */, int32_t n_temps, int32_t n_bins,
                              float *sts_temps_out, int32_t *choice, double *ece_curve,
                              int64_t *n_obs, void *workspace, size_t workspace_bytes,
                              int32_t *status, void *stream);

/* --------------------------------------------- verify window over a cache
 *
 * What a target layer does with the packed window between the pack and the
 * accept ([ROUND] §三, §四: the target forward over the compact verify rows
 * at their own positions): norms and rotation of queries and keys, the write
 * of the drafted tokens' keys and values into a paged cache, and attention
 * of the drafted tokens over that cache.  The pages describe no kernel for
 * these; the formulas are below.  Every index (requests, positions, window
 * lengths) is read on the device, from the pack's outputs. */

#define DSPARK_DTYPE_E4M3 2 /* 8-bit cache entries: 4 exponent, 3 mantissa bits, +-448, no infinity */
#define DSPARK_MAX_HEAD_DIM 256
#define DSPARK_MAX_WINDOW 32 /* drafted tokens of one request in dspark_tree_attention */

/* One layer's paged cache (host struct pointing at DEVICE memory).  Position
 * p of request r lies in page g = block_table[r * table_width + p / page_size]
 * at token p % page_size; element d of head h is at
 *   g * page_stride + (p % page_size) * token_stride + h * head_stride + d
 * elements from k (and from v: both have the same layout), so either order of
 * tokens and heads inside a page is a choice of strides.  An E4M3 entry has
 * one fp32 scale for each token and head, at
 *   (g * n_kv_heads + h) * page_size + p % page_size
 * of k_scale / v_scale, and stands for code * scale. */
typedef struct {
    int32_t dtype;       /* DSPARK_DTYPE_BF16, _F32 or _E4M3 */
    int32_t n_pages;     /* pages in the pool, >= 1 */
    int32_t page_size;   /* tokens a page, >= 1 */
    int32_t n_kv_heads;  /* >= 1 */
    int32_t head_dim;    /* 2..DSPARK_MAX_HEAD_DIM, even */
    int32_t n_requests;  /* rows of block_table, >= 1 */
    int32_t table_width; /* pages a row of block_table lists, >= 1 */
    int64_t page_stride, token_stride, head_stride; /* elements, >= 0 */
    void *k, *v;
    float *k_scale, *v_scale;   /* E4M3 only, else NULL */
    const int32_t *block_table; /* [n_requests, table_width] */
} dspark_kv_cache;

/* Norm and rotation of one call (host struct).  In 32 bits, rounded once at
 * the end, for each row and head:
 *   y_d = x_d / sqrt(mean(x^2) + eps) * weight_d    (weight given, else y = x)
 *   the first rope_dim elements in pairs (a, b), pair i with the cosine
 *   c = cos_sin[pos * rope_dim + i] and the sine s = cos_sin[pos * rope_dim +
 *   rope_dim / 2 + i]:  (a, b) -> (a c - b s, b c + a s). */
typedef struct {
    const void *q_weight, *k_weight; /* [head_dim], type of the rows; NULL = no norm */
    float eps;                       /* >= 0 */
    const float *cos_sin;            /* device [n_pos, rope_dim]; NULL = no rotation */
    int32_t n_pos;
    int32_t rope_dim;                /* even, 2..head_dim (ignored without cos_sin) */
    int32_t interleaved;             /* pair i: 0 = elements (i, i + rope_dim/2), 1 = (2i, 2i+1) */
} dspark_norm_rope;

/* Norms and rotation of queries and keys, in one pass.
 *   q, k         [max_rows, heads * head_dim] rows of `dtype` (BF16 or F32), ld_*
 *                elements apart (slices of one projection's rows will do).
 *                Either may be NULL with its output (and 0 heads)
 *   q_out, k_out outputs of the same type; may be q and k themselves (in
 *                place) and must not overlap them in any other way
 *   pos          device [max_rows] int32: the rows' positions (the pack's
 *                packed_pos); may be NULL without cos_sin
 *   totals       device int32 (nullable): rows from totals[0] on are pads and
 *                left alone; NULL = all max_rows rows
 * A row whose position is outside [0, n_pos) is not written and flags
 * DSPARK_STATUS_BAD_INDEX.
 * Errors: INVALID_ARG (null pointer, dtype, a stride below a row's elements,
 * negative counts, rope_dim odd or outside 2..head_dim, eps negative or NaN);
 * UNSUPPORTED (head_dim odd or outside 2..DSPARK_MAX_HEAD_DIM); CUDA. */
DSPARK_API int dspark_qk_norm_rope(const void *q, int64_t ld_q, const void *k, int64_t ld_k,
                                   int32_t dtype, int32_t n_q_heads, int32_t n_kv_heads,
                                   int32_t head_dim, const dspark_norm_rope *nr /* host */,
                                   const int32_t *pos, const int32_t *totals, int32_t max_rows,
                                   void *q_out, int64_t ld_q_out, void *k_out, int64_t ld_k_out,
                                   int32_t *status, void *stream);

/* The same pass with the keys, and the values as they are, going into the
 * cache.
 *   k, v         [max_rows, n_kv_heads * head_dim] rows of `dtype`
 *   q, q_out     as above; NULL with n_q_heads = 0 when only the cache is written
 *   nr           host, nullable: keys (and queries) are written unchanged
 *   req          device [max_rows]: a row's request (the pack's packed_req); a
 *                negative one marks a pad row, which is left alone
 *   pos          device [max_rows]: positions for the rotation
 *   cache_pos    device [max_rows] (nullable: pos): positions in the cache.  A
 *                tree's nodes rotate by depth and are stored in window order
 * An E4M3 entry: scale = max(max_d |x_d| / 448, 2^-100), codes x / scale
 * rounded to nearest even, all from the 32-bit values.  A head with a NaN or
 * an infinity reads back as NaN and flags DSPARK_STATUS_BAD_INPUT.
 * A request >= n_requests, a cache position outside the block table or a page
 * outside the pool flags DSPARK_STATUS_BAD_INDEX, and that row's keys and
 * values are not written; with cos_sin, a position outside [0, n_pos) flags the
 * same, and nothing of that row is written.  Two rows of a call must not share a slot.
 * Errors as above, and for the cache: INVALID_ARG (null pointers, dtype,
 * counts < 1, negative strides, E4M3 without scales). */
DSPARK_API int dspark_kv_append(const void *q, int64_t ld_q, const void *k, int64_t ld_k,
                                const void *v, int64_t ld_v, int32_t dtype, int32_t n_q_heads,
                                const dspark_kv_cache *cache /* host */,
                                const dspark_norm_rope *nr /* host */, const int32_t *req,
                                const int32_t *pos, const int32_t *cache_pos,
                                const int32_t *totals, int32_t max_rows, void *q_out,
                                int64_t ld_q_out, int32_t *status, void *stream);

/* Cache entries back as rows: positions start[r], start[r]+1, ... of request
 * r < B go to rows cu_rows[r]..cu_rows[r+1]-1.
 *   start        device [B]; cu_rows device [B+1], ascending from 0
 *   k_out, v_out [max_rows, n_kv_heads * head_dim] rows of out_dtype (BF16 or
 *                F32), ld_out elements apart: code * scale in 32 bits,
 *                rounded once
 * Rows from min(cu_rows[B], max_rows) on are left alone (CAPACITY if cu_rows[B]
 * is larger); a position outside the block table or a page outside the pool
 * flags BAD_INDEX and its row is not written.
 * Errors: INVALID_ARG (null pointer, B outside 1..n_requests, out_dtype,
 * ld_out below a row, max_rows < 0, the cache's); UNSUPPORTED (head_dim); CUDA. */
DSPARK_API int dspark_kv_read(const dspark_kv_cache *cache /* host */, const int32_t *start,
                              const int32_t *cu_rows, int32_t B, int32_t max_rows,
                              int32_t out_dtype, void *k_out, void *v_out, int64_t ld_out,
                              int32_t *status, void *stream);

/* Workspace of dspark_tree_attention, for any number of requests, rows and
 * positions; need not be cleared. */
DSPARK_API size_t dspark_tree_attention_workspace_bytes(int32_t n_q_heads, int32_t head_dim);

/* Attention of the drafted tokens over the cache that holds their requests'
 * prefixes and the tokens themselves (dspark_kv_append first).  Packed row
 * cu_seqlens[r] + i is token i of request r's window of L <= 32 tokens, at
 * cache position prefix_lens[r] + i.  It sees every position below
 * prefix_lens[r], and token j of the window iff bit j of its ancestors word is
 * set (j < L); ancestors NULL = a chain, bits 0..i.  For query head h, with
 * kv head h / (n_q_heads / n_kv_heads), over the visible positions p:
 *   s_p = scale * q . k_p    m = max s_p    l = sum exp(s_p - m)
 *   out = sum exp(s_p - m) v_p / l          lse = m + ln l
 * A row that sees nothing gets out = 0 and lse = -inf.  What a row does not
 * see has no effect on it, NaN and infinities included.
 *   q, out       [max_rows, n_q_heads * head_dim] rows of `dtype` (BF16 or
 *                F32), ld_* elements apart; out must not share an element with
 *                q (slices of one buffer's rows will do)
 *   lse          [max_rows, n_q_heads] fp32, nullable
 *   prefix_lens  device [B], >= 0; cu_seqlens device [B+1], ascending; window
 *                length 0 is a request without rows
 * Sums and softmax statistics are held in 32 bits.  BF16 rows over a BF16 or
 * E4M3 cache with head_dim 64 or 128, at most 128 query heads a kv head,
 * page_size a multiple of 16 and 16-byte aligned bases and strides run on the
 * tensor cores, the weights exp(s - m) rounded to the 16-bit type of the
 * products (BF16; over E4M3 a half, whose smallest step is 2^-30 of the
 * largest weight times scale); anything else in 32 bits throughout.  Over
 * E4M3 a query's elements below 2^-9 of its largest are taken to 2^-17 of it
 * (where few rows a kv head leave the products to a second kernel, with at most
 * 8 query heads a kv head and 16-byte aligned scales: below 2^-31, to 2^-39).
 * The order of all sums is fixed by the lengths: a call repeated gives the
 * same bits.
 * A window of more than 32 tokens or outside max_rows (BAD_LEN), and positions
 * past the block table, positions from 2^31 - 8192 on or a page outside the pool
 * (BAD_INDEX): that request's rows are unspecified, the others not affected.
 * Rows of no request are left alone.
 * Errors: INVALID_ARG (null pointer, B outside 1..n_requests, n_q_heads not a
 * positive multiple of n_kv_heads, dtype, a stride below a row, max_rows < 0,
 * scale not finite, out over q, the cache's); UNSUPPORTED (head_dim, more than
 * 65535 query heads); WORKSPACE; CUDA. */
DSPARK_API int dspark_tree_attention(const void *q, int64_t ld_q, int32_t dtype, int32_t n_q_heads,
                                     int32_t max_rows, const int32_t *cu_seqlens,
                                     const int32_t *prefix_lens, int32_t B,
                                     const uint32_t *ancestors, float scale,
                                     const dspark_kv_cache *cache /* host */, void *out,
                                     int64_t ld_out, float *lse, void *workspace,
                                     size_t workspace_bytes, int32_t *status, void *stream);

/* ------------------------------------------------ attention, latent cache
 *
 * Models whose keys and values are projections of one latent vector a token,
 * shared by all heads, keep only that vector c (latent_dim elements) and a key
 * part r (rope_dim elements) that is rotated and shared too.  A window of
 * drafted tokens attends in the absorbed form: the key projection is taken into
 * the queries and the value projection is applied to the outputs, both by the
 * caller's own products.  A prompt attends in the expanded form, over keys and
 * values of every head.  The formulas are below. */

#define DSPARK_MAX_LATENT_DIM 512
#define DSPARK_MAX_LATENT_ROPE 128

/* One layer's paged latent cache (host struct pointing at DEVICE memory).
 * Position p of request r lies in page g = block_table[r * table_width + p /
 * page_size]: its latent vector, and its rotated key part directly behind it, from
 * element g * page_stride + (p % page_size) * token_stride of data. */
typedef struct {
    int32_t dtype;       /* DSPARK_DTYPE_BF16 or _F32 */
    int32_t n_pages;     /* pages in the pool, >= 1 */
    int32_t page_size;   /* tokens a page, >= 1 */
    int32_t latent_dim;  /* 2..DSPARK_MAX_LATENT_DIM, even */
    int32_t rope_dim;    /* 2..DSPARK_MAX_LATENT_ROPE, even */
    int32_t n_requests;  /* rows of block_table, >= 1 */
    int32_t table_width; /* pages a row of block_table lists, >= 1 */
    int64_t page_stride, token_stride; /* elements, >= 0 */
    void *data;
    const int32_t *block_table; /* [n_requests, table_width] */
} dspark_latent_cache;

/* Rows [latent | key part] into the cache, and the queries' rotated parts, in one
 * pass.  In 32 bits, rounded once at the end:
 *   c_d = x_d / sqrt(mean(x^2) + eps) * weight_d over the latent part (k_weight
 *   given, else c = x); the key part, and each head's query part, rotated.
 *   x            [max_rows, latent_dim + rope_dim] rows of `dtype` (BF16 or F32),
 *                ld_x elements apart
 *   q, q_out     the rope_dim elements of n_q_heads heads a row, rows ld_* and
 *                heads hs_* elements apart, so that q may be a slice of the
 *                queries' projection and q_out of the absorbed queries.  They may
 *                be the same (in place) and must not overlap in any other way; within
 *                the spans of each other's rows they have the same strides.
 *                Both NULL with n_q_heads = 0 when only the cache is written
 *   nr           host: k_weight is [latent_dim] or NULL, q_weight NULL; cos_sin and
 *                its rope_dim, which is the cache's, are required
 *   req, pos, cache_pos, totals   as in dspark_kv_append
 * A request >= n_requests, a cache position outside the block table or a page
 * outside the pool flags DSPARK_STATUS_BAD_INDEX, and that row is not stored (its
 * query part is written); a position outside [0, n_pos) flags the same, and
 * nothing of that row is written.  Two rows of a call must not share a slot.
 * Errors: INVALID_ARG (null pointer, dtype, a stride below what it spans, negative
 * counts, rope_dim not the cache's, eps negative or NaN, a query weight, q_out over a
 * part of q, and for the cache null pointers, dtype, counts < 1, negative strides);
 * UNSUPPORTED (latent_dim, rope_dim); CUDA. */
DSPARK_API int dspark_latent_append(const void *x, int64_t ld_x, const void *q, int64_t ld_q,
                                    int64_t hs_q, int32_t dtype, int32_t n_q_heads,
                                    const dspark_latent_cache *cache /* host */,
                                    const dspark_norm_rope *nr /* host */, const int32_t *req,
                                    const int32_t *pos, const int32_t *cache_pos,
                                    const int32_t *totals, int32_t max_rows, void *q_out,
                                    int64_t ld_q_out, int64_t hs_q_out, int32_t *status,
                                    void *stream);

/* Workspace of dspark_latent_attention, for any number of requests, rows and
 * positions; need not be cleared. */
DSPARK_API size_t dspark_latent_attention_workspace_bytes(int32_t n_q_heads, int32_t latent_dim);

/* dspark_tree_attention in the absorbed form: for a query q of latent_dim + rope_dim
 * elements over the visible positions p, with [c_p | r_p] their cache entries,
 *   s_p = scale * q . [c_p | r_p]    m = max s_p    l = sum exp(s_p - m)
 *   out = sum exp(s_p - m) c_p / l (latent_dim elements)     lse = m + ln l
 * Windows, visibility, rows that see nothing, what is not seen, bad windows and bad
 * positions as there.
 *   q            [max_rows, n_q_heads * (latent_dim + rope_dim)] rows of `dtype` (BF16
 *                or F32), ld_q elements apart
 *   out          [max_rows, n_q_heads * latent_dim] rows, ld_out elements apart; must
 *                not share an element with q
 *   lse          [max_rows, n_q_heads] fp32, nullable
 * BF16 rows over a BF16 cache with latent_dim 512, rope_dim 64, page_size a multiple
 * of 16, 16-byte aligned bases and strides and fewer than 2^31 tiles of 128 positions
 * and 128 (row, head) pairs in full block tables run on the tensor cores, the weights
 * exp(s - m) rounded to BF16; anything else in 32 bits throughout.  The order of all
 * sums is fixed by the lengths: a call repeated gives the same bits.
 * Errors: INVALID_ARG (null pointer, B outside 1..n_requests, n_q_heads < 1, dtype, a
 * stride below a row, max_rows < 0, scale not finite, out over q, the cache's);
 * UNSUPPORTED (latent_dim, rope_dim, more than 65535 heads); WORKSPACE; CUDA. */
DSPARK_API int dspark_latent_attention(const void *q, int64_t ld_q, int32_t dtype,
                                       int32_t n_q_heads, int32_t max_rows,
                                       const int32_t *cu_seqlens, const int32_t *prefix_lens,
                                       int32_t B, const uint32_t *ancestors, float scale,
                                       const dspark_latent_cache *cache /* host */, void *out,
                                       int64_t ld_out, float *lse, void *workspace,
                                       size_t workspace_bytes, int32_t *status, void *stream);

/* Causal attention of prompts, ragged: request r's queries are rows
 * cu_seqlens[r]..cu_seqlens[r+1]-1 of q, its keys and values rows
 * cu_keys[r]..cu_keys[r+1]-1 of k and v, and its last query stands at its last key:
 * of n queries and m keys, query i sees keys 0..m - n + i (none if that is
 * negative).  Of any length.  For query head h, with kv head g = h / (n_q_heads /
 * n_kv_heads), and a query of key_dim + shared_dim elements:
 *   s_j = scale * (q[0:key_dim] . k_jg + q[key_dim:] . k_shared_j)
 *   out = softmax(s) . v_g (value_dim elements)     lse = ln sum exp(s_j)
 * shared_dim = 0 (k_shared NULL) is attention over keys and values as they are; with
 * it, the expanded form over a latent cache's rows, k_shared their rotated part.
 *   q            [max_rows, n_q_heads * (key_dim + shared_dim)], ld_q elements apart
 *   k, v         heads hs_k and hs_v elements apart (they may be the two parts of one
 *                projection's heads), rows ld_k and ld_v; max_keys rows
 *   k_shared     [max_keys, shared_dim] rows ld_shared elements apart
 *   out          [max_rows, n_q_heads * value_dim], ld_out elements apart; must not
 *                share an element with an input
 *   lse          [max_rows, n_q_heads] fp32, nullable
 * A row that sees nothing gets out = 0 and lse = -inf.  What a row does not see has
 * no effect on it, NaN and infinities included; an infinite value that it sees with a
 * weight of 0 (a score of -inf) gives NaN, as the formula does, and a weight below 2^-126
 * may count as 0.  BF16 with key_dim 128, shared_dim 64 or 0, value_dim 128 and 16-byte
 * aligned bases and strides runs on the tensor cores, the weights rounded to BF16;
 * anything else in 32 bits throughout, and so, where max_rows + max_keys is below 46 B,
 * requests of up to 512 (query, key) pairs.
 * A range outside the rows or the keys (BAD_LEN): that request's rows are unspecified,
 * the others not affected.  Ranges that descend (BAD_LEN) or overlap: all rows are
 * unspecified.  Rows of no request are left alone.
 * Errors: INVALID_ARG (null pointer, dtype, B < 1, n_q_heads not a positive multiple
 * of n_kv_heads, a stride below what it spans, negative counts, scale not finite, out
 * over an input); UNSUPPORTED (key_dim, shared_dim or value_dim above
 * DSPARK_MAX_HEAD_DIM, key_dim or value_dim < 1, more than 65535 heads); CUDA. */
DSPARK_API int dspark_prompt_attention(const void *q, int64_t ld_q, const void *k, int64_t ld_k,
                                       int64_t hs_k, const void *k_shared, int64_t ld_shared,
                                       const void *v, int64_t ld_v, int64_t hs_v, int32_t dtype,
                                       int32_t n_q_heads, int32_t n_kv_heads, int32_t key_dim,
                                       int32_t shared_dim, int32_t value_dim, int32_t max_rows,
                                       int32_t max_keys, const int32_t *cu_seqlens,
                                       const int32_t *cu_keys, int32_t B, float scale, void *out,
                                       int64_t ld_out, float *lse, int32_t *status, void *stream);

/* --------------------------------------------- a cache that is kept short
 *
 * Which positions of a cache a request attends to is gathered step by step, for each
 * kv head; those that gathered least can then be evicted.  A head's entries need no
 * order (keys carry their rotation), so an eviction moves entries from behind the new
 * end into the places that became free before it and touches nothing else.  Later
 * tokens are appended with cache_pos from the new length on and pos as before. */

/* Adds the attention of a window's rows (dspark_tree_attention first, for lse) to what
 * each position of the cache has gathered.  For request r with prefix P and the
 * first n = counts[r] rows of its window, kv head h and position p:
 *   weights_out[r][h][p] = (p < P ? decay * weights[r][h][p] : 0)
 *       + sum over those rows and the head's query heads that see p of
 *         exp(scale * q . k_p - lse)                     for p < P + n
 *   weights_out[r][h][p] = 0                             from P + n on
 *   positions[r][h][P + i] = pos[cu_seqlens[r] + i]      for i < n (with positions)
 *   q, cu_seqlens, prefix_lens, ancestors, scale, cache   as in dspark_tree_attention
 *   lse          [max_rows, n_q_heads] fp32, as it left them
 *   counts       device [B] (nullable: whole windows): how many of a window's rows
 *                count (the accepted ones: commit_lens)
 *   decay        finite
 *   weights, weights_out   [B, n_kv_heads, length] fp32, the same or apart
 *   pos, positions         device [max_rows] and [B, n_kv_heads, length] int32,
 *                both or neither
 * Sums are held in 32 bits and their order is fixed.  BF16 rows over BF16 or E4M3 keys of
 * 64 or 128 elements with 16-byte aligned bases and strides run on the tensor cores, their
 * products exact; beside E4M3 keys an element of a query may lose what is below 2^-39 of its
 * row's largest.  Anything else runs in 32 bits throughout.  What a row does not see has no
 * effect.  A window as dspark_tree_attention flags it, counts outside the window (BAD_LEN)
 * and P + n > length (CAPACITY): that request's weights and positions are left alone.
 * A page outside the pool flags BAD_INDEX; its positions gather nothing.
 * Errors: those of dspark_tree_attention (there is no workspace and no out), and
 * INVALID_ARG (length < 1, decay not finite, pos without positions, weights_out over a
 * part of weights); UNSUPPORTED (more than 65535 requests, length above 2^30). */
DSPARK_API int dspark_attention_weights(const void *q, int64_t ld_q, int32_t dtype,
                                        int32_t n_q_heads, int32_t max_rows,
                                        const int32_t *cu_seqlens, const int32_t *prefix_lens,
                                        int32_t B, const uint32_t *ancestors, float scale,
                                        const dspark_kv_cache *cache /* host */, const float *lse,
                                        const int32_t *counts, float decay, const float *weights,
                                        float *weights_out, int32_t length, const int32_t *pos,
                                        int32_t *positions, int32_t *status, void *stream);

/* Workspace of dspark_kv_evict; need not be cleared. */
DSPARK_API size_t dspark_kv_evict_workspace_bytes(int32_t B, int32_t n_kv_heads, int32_t length);

/* Cuts each request's cache down to `keep` entries a kv head.  Of the n = lens[r]
 * entries of a head, those stay that rank first by: position >= now[r] - recent; then
 * the larger weight (a NaN below all others; BAD_INPUT); then the lower place.  With
 * n' = min(n, keep), the i-th entry in order that stays from place n' on moves to the i-th
 * free place below n'; the others lie as they did.
 *   cache        keys, values and scales move; places from n' on keep what they held.  Two
 *                requests must not share a page
 *   lens, now    device [B]: entries in the cache, and tokens so far
 *   weights, positions          [B, n_kv_heads, length], as dspark_attention_weights left
 *                them (positions of a cache that has never been cut: 0, 1, 2, ...)
 *   weights_out, positions_out  the same after the eviction, 0 from n' on; weights and
 *                positions themselves, or apart
 *   new_lens     device [B]: n'; may be lens
 * lens below 0 or above length or the block table (BAD_LEN): that request, its
 * entries, ledger and length are left as they are (new_lens = lens).  A page outside
 * the pool flags BAD_INDEX, and the entry is not moved.
 * Errors: INVALID_ARG (null pointer, B outside 1..n_requests, length < 1, keep < 1,
 * recent outside 0..keep, an output over a part of its input, the cache's);
 * UNSUPPORTED (head_dim, length above 2^30, more than 65535 requests); WORKSPACE; CUDA. */
DSPARK_API int dspark_kv_evict(const dspark_kv_cache *cache /* host */, const int32_t *lens,
                               const int32_t *now, int32_t B, int32_t keep, int32_t recent,
                               const float *weights, float *weights_out, const int32_t *positions,
                               int32_t *positions_out, int32_t length, int32_t *new_lens,
                               void *workspace, size_t workspace_bytes, int32_t *status,
                               void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_H */
