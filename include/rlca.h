/*
 * rlca.h -- C ABI of the GB300 (sm_103a) credit-assignment scans.
 *
 * The operation behind every entry point is the first-order linear
 * recurrence of "rl-triton: High-Performance Triton GPU Kernels for
 * Reinforcement Learning Credit Assignment" (arXiv:2608.17641),
 * §1 Introduction and §3.1 Shared scan formulation:
 *
 *     backward:  A_t = alpha_t + beta_t * A_{t+1}      (A_T given)
 *     forward:   A_t = alpha_t + beta_t * A_{t-1}      (A_{-1} given)
 *
 * evaluated independently for each of E environment rows of T steps, with
 * each estimator's (alpha_t, beta_t) built on chip from raw rollout inputs
 * (§3.3 Algorithm-specific recurrences) and the episode-boundary rules of
 * §3.2 Episode-boundary semantics:
 *
 *   terminated[e,t] != 0  the episode ended at t: successor value 0, beta_t = 0.
 *   truncated[e,t]  != 0  the episode was cut at t: the successor value is the
 *                         caller's trunc_value[e,t], beta_t = 0.  Where both
 *                         flags are set, termination wins.
 *   t = T-1, no flag      the rollout window ends: the successor value is
 *                         bootstrap[e] (0 when bootstrap is NULL).
 *   forward scans         restart after a flagged step; no bootstrap.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pointers are DEVICE pointers owned by the caller; the library keeps no
 *    reference after the call returns.  Inputs are read once, outputs are
 *    written once, every output element is written (steps after a boundary
 *    included).  Outputs must not overlap any input or each other.
 *  - Layout: env-major [E, T] (t fastest) by default; with RLCA_TIME_MAJOR
 *    every [E, T] array is [T, E] (e fastest) and every per-action array is
 *    [T, E, A] instead of [E, T, A].  Per-environment vectors (bootstrap,
 *    carry) are [E] in both layouts.  Arrays are dense and contiguous.
 *  - Element types: float32 values (bfloat16 with RLCA_BF16), uint8 flags
 *    (nonzero = set), int32 actions.  Any pointer alignment is accepted;
 *    16-byte aligned bases with T % 4 == 0 take the vectorised load paths
 *    (env-major rows; time-major rows staged through shared memory).
 *  - Sizes: 0 <= E <= 2^31-1, 0 <= T <= 2^30.
 *  - Work is enqueued on `stream` (NULL = the legacy default stream) and the
 *    call returns without synchronising.  No host or device memory is
 *    allocated by any entry point.  Kernels are launched with programmatic
 *    stream serialization: they may be scheduled while the previous kernel
 *    of the stream drains, but touch no memory before it has completed, so
 *    stream order is kept.
 *  - Workspace: an entry point may need device scratch for the two-pass
 *    segmented path (long rows on few environments, or RLCA_MULTIPASS).
 *    Query its size with rlca_workspace_size() using the same E, T,
 *    num_actions and flags, and pass a device buffer of at least that many
 *    bytes (16-byte aligned).  A NULL workspace is valid when the size is 0.
 *    The workspace is scratch: its contents on entry are ignored and on exit
 *    are unspecified; calls that share one workspace must not overlap on the
 *    GPU.  It shares no memory with the arrays of its call: one that overlaps
 *    an output is refused everywhere, one that overlaps an input by the calls
 *    of a recurrent policy's trunk.
 *  - E == 0 or T == 0 returns RLCA_OK and enqueues nothing.
 *  - Errors: RLCA_ERR_INVALID_ARG (NULL required pointer, negative or
 *    oversized E/T, overlapping outputs, workspace too small or misaligned,
 *    unknown flags) and RLCA_ERR_UNSUPPORTED (num_actions above
 *    RLCA_MAX_ACTIONS, RLCA_BF16 where noted) are detected on the host
 *    before anything is enqueued.  RLCA_ERR_CUDA reports a failed CUDA runtime call (device
 *    query or launch); the CUDA error itself is left readable through
 *    cudaGetLastError()/cudaPeekAtLastError().
 *  - Entry points are thread-safe and hold no global state except a
 *    per-device cache of device attributes filled on first use.
 */
#ifndef RLCA_H
#define RLCA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *rlca_stream_t;

/* ---- status codes ------------------------------------------------------ */
#define RLCA_OK               0
#define RLCA_ERR_INVALID_ARG  1
#define RLCA_ERR_UNSUPPORTED  2
#define RLCA_ERR_CUDA         3

/* ---- flags (bitwise OR) -------------------------------------------------- */
/* Arrays are time-major [T, E] ([T, E, A]) instead of env-major [E, T]. */
#define RLCA_TIME_MAJOR          0x1u
/* Use the two-pass segmented path even where one pass would do (the library
 * picks it by itself for long rows on few environments).  Needs workspace. */
#define RLCA_MULTIPASS           0x2u
/* The caller asserts that this call's inputs were not written by the kernel
 * that precedes it on the stream (they were complete before that kernel was
 * enqueued).  The kernel may then read its inputs while the preceding kernel
 * is still running, and only waits for it before writing anything, so
 * back-to-back calls on independent batches overlap.  Without the flag a
 * call reads nothing before the preceding kernel has completed.  Ignored by
 * the two-pass path.  A false assertion gives wrong results (never an
 * out-of-bounds access). */
#define RLCA_INPUTS_READY        0x10u
/* Every floating-point array of the call -- per-step inputs and outputs and
 * the per-environment [E] vectors (bootstrap, carry) -- holds IEEE bfloat16
 * values (2 bytes each, the upper half of a float32) instead of float32; the
 * pointers keep their declared float type and point at the bfloat16 data.
 * Arithmetic and the scan state stay float32; each output is rounded to
 * nearest-even bfloat16 once.  Flags and int32 arrays are unchanged.  With
 * rlca_episodic_prefix_sum it applies to RLCA_F32 data only (RLCA_I32:
 * RLCA_ERR_INVALID_ARG); rlca_gae_static_scratch returns
 * RLCA_ERR_UNSUPPORTED.  With rlca_retrace it covers q, pi and mu_a as well
 * (the expectation and the ratio are formed in float32).  The paper defers bfloat16 I/O to future work and
 * keeps scans in float32 (rl-triton (arXiv:2608.17641) §9 Discussion and
 * Future Work; §4 Implementation, numerical requirements): only storage is
 * narrowed here. */
#define RLCA_BF16                0x20u
/* rlca_episodic_prefix_sum: output the sum over the steps BEFORE t in t's
 * episode instead of the inclusive sum. */
#define RLCA_PSUM_EXCLUSIVE      0x4u
/* rlca_episodic_prefix_sum: a flagged step is the FIRST step of a new
 * episode (default: a flagged step is the LAST step of its episode). */
#define RLCA_PSUM_FLAG_IS_START  0x8u

/* ---- estimator ids (for rlca_workspace_size) ---------------------------- */
#define RLCA_EST_GAE               1
#define RLCA_EST_DISCOUNTED_RETURN 2
#define RLCA_EST_TD_LAMBDA         3
#define RLCA_EST_VTRACE            4
#define RLCA_EST_RETRACE           5
#define RLCA_EST_ELIG_TRACE        6
#define RLCA_EST_PREFIX_SUM        7
#define RLCA_EST_AFFINE_SCAN       8
#define RLCA_EST_VALUE_TARGETS     9
/* the policy-update operators: E = rows, T = row width, num_actions = vocabulary
 * (RLCA_EST_CLIP_GRADS: E = number of tensors, T ignored unless 0) */
#define RLCA_EST_TOKEN_LOGPROB          10
#define RLCA_EST_TOKEN_LOGPROB_BACKWARD 11
#define RLCA_EST_LAYER_NORM_BACKWARD    12
#define RLCA_EST_CLIP_GRADS             13
#define RLCA_EST_RMS_NORM_BACKWARD      14
/* the gated scans: E, T, num_actions = channels */
#define RLCA_EST_GATED_SCAN             15
#define RLCA_EST_GATED_SCAN_BACKWARD    16

/* ---- prefix-sum element types ------------------------------------------- */
#define RLCA_F32 0
#define RLCA_I32 1

/* Largest num_actions accepted by rlca_retrace. */
#define RLCA_MAX_ACTIONS 64

/* Human-readable text of a status code (static storage, never NULL). */
const char *rlca_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int rlca_version(void);

/* Device status bits (see rlca_device_status). */
#define RLCA_STATUS_WAIT_TIMEOUT 0x1u /* a bounded wait on a tile copy gave up */
#define RLCA_STATUS_INDEX        0x2u /* index-check build: an out-of-range index was skipped */

/*
 * Device-side status of the kernels launched so far on the CURRENT device:
 * writes to *status the OR of the status words the kernels keep in device
 * memory (0: nothing to report), and zeroes them when `clear` is nonzero.
 * No counterpart in the paper: it reports conditions that a kernel records
 * instead of trapping.  The only one in the product build is
 * RLCA_STATUS_WAIT_TIMEOUT: a kernel that waits for its own copies (the
 * time-major bulk driver, the norms' gradients, the gated scans) or matrix instructions
 * (the policy head) gives up after 0.2 s instead of hanging and leaves that
 * call's outputs incomplete.  The copies are synchronous: the
 * call waits for the device's earlier work.  Errors: RLCA_ERR_INVALID_ARG
 * for a NULL `status`, RLCA_ERR_CUDA when a copy fails.
 */
int rlca_device_status(unsigned int *status, int clear);

/* 1 in the index-check build of this library (compiled with
 * RLCA_INDEX_CHECK: kernels check every index of the staged and two-pass
 * paths, record a miss as RLCA_STATUS_INDEX instead of trapping, and each
 * call waits for its kernels, returning RLCA_ERR_CUDA if any recorded a
 * condition), 0 in the product build.  A debugging aid; no counterpart in
 * the paper. */
int rlca_index_checks(void);

/*
 * Bytes of device workspace that the call of `estimator` (RLCA_EST_*) with
 * these sizes and flags needs on the CURRENT device (0 for the one-pass
 * path).  num_actions is read for RLCA_EST_RETRACE (actions) and the
 * RLCA_EST_TOKEN_LOGPROB (vocabulary) and RLCA_EST_GATED_SCAN (channels) ids
 * only.  Writes the size to *bytes.  Errors: RLCA_ERR_INVALID_ARG for a NULL `bytes`, an unknown
 * estimator, bad sizes or flags; RLCA_ERR_CUDA if the device cannot be
 * queried.
 */
int rlca_workspace_size(int estimator, int64_t E, int64_t T,
                        int32_t num_actions, uint32_t flags, size_t *bytes);

/*
 * Generalized Advantage Estimation (rl-triton §2.1 Motivation, §3.2;
 * Schulman et al. 2016), backward scan with the bootstrap in alpha_{T-1}:
 *   delta_t = r_t + gamma * V_next(t) - V_t
 *   adv_t   = delta_t + gamma * lambda * (1 - d_t) * [t < T-1] * adv_{t+1}
 *   ret_t   = adv_t + V_t
 * V_next(t) = 0 / trunc_value[t] / bootstrap / values[t+1] per the boundary
 * rules above.
 *   rewards, values        [E,T] f32, required
 *   terminated             [E,T] u8, NULL = no terminations
 *   truncated              [E,T] u8, NULL = no truncations (fast path)
 *   trunc_value            [E,T] f32, required iff truncated != NULL; read
 *                          only where truncated is set
 *   bootstrap              [E] f32, NULL = 0
 *   advantages             [E,T] f32 output, required
 *   returns                [E,T] f32 output, NULL = not written
 */
int rlca_gae(const float *rewards, const float *values,
             const uint8_t *terminated, const uint8_t *truncated,
             const float *trunc_value, const float *bootstrap,
             float *advantages, float *returns,
             int64_t E, int64_t T, float gamma, float lambda,
             uint32_t flags, void *workspace, size_t workspace_bytes,
             rlca_stream_t stream);

/*
 * Fused value targets: GAE advantages and returns, discounted returns and
 * TD(lambda) returns of the same rollout in one pass that reads rewards,
 * values and flags once (rl-triton §4 Fusion: constructing coefficients on
 * chip removes intermediate HBM round trips).  The recurrences of rlca_gae
 * and rlca_discounted_return are scanned side by side; the TD(lambda) return
 * is written as advantages + values, which equals it exactly under every
 * boundary rule, so it needs no third scan.  Results equal those of the
 * separate calls within floating-point rounding.
 *   rewards, values, terminated, truncated, trunc_value, bootstrap  as rlca_gae
 *   advantages, returns        [E,T] f32 outputs of rlca_gae, each nullable
 *   disc_returns               [E,T] f32 output of rlca_discounted_return, nullable
 *   td_lambda_returns          [E,T] f32 output of rlca_td_lambda, nullable
 * At least one output must be given.  Workspace (two-pass path): 16 bytes
 * per row per segment (rlca_workspace_size with RLCA_EST_VALUE_TARGETS).
 */
int rlca_value_targets(const float *rewards, const float *values,
                       const uint8_t *terminated, const uint8_t *truncated,
                       const float *trunc_value, const float *bootstrap,
                       float *advantages, float *returns, float *disc_returns,
                       float *td_lambda_returns, int64_t E, int64_t T,
                       float gamma, float lambda, uint32_t flags,
                       void *workspace, size_t workspace_bytes,
                       rlca_stream_t stream);

/*
 * GAE with library-owned scratch, for callers that cannot allocate.
 *
 * The paper has no counterpart to this entry point.  It computes exactly
 * what rlca_gae computes, with the same arguments minus the workspace, for
 * callers that have no way to hand this library a device buffer: a plain C
 * or Fortran host linked only against this library, a simulator callback
 * that must not touch the device heap, a service that reserved all device
 * memory at start-up.  When the two-pass path needs scratch, it uses one
 * array that the library defines in device memory: RLCA_STATIC_SCRATCH_BYTES
 * (1 MiB) on every GPU that loads the library, held until the process exits.
 * Nothing is allocated, on the host or the device, by this call.
 *
 *  - The first call on a device looks up that array's device address (the
 *    set-up); make that first call before any stream capture on the device.
 *    The address is kept with the id of the device context it was found in
 *    and looked up again when that context has changed (after
 *    cudaDeviceReset, for instance): the first call after such a change is
 *    a set-up call too.
 *  - Problems whose two-pass path needs more than RLCA_STATIC_SCRATCH_BYTES
 *    (8 bytes per row per segment; rlca_workspace_size with RLCA_EST_GAE
 *    gives the figure) return RLCA_ERR_UNSUPPORTED and enqueue nothing;
 *    use rlca_gae with a workspace for those.
 *  - All calls on a device share the array and it keeps whatever the last
 *    call left there.  No slot needs to start at zero: the first pass writes
 *    every slot the second pass reads.  Calls whose work overlaps on the GPU
 *    (other streams, other host threads) race on the array and give wrong
 *    results: serialise them.
 * Flags: RLCA_TIME_MAJOR and RLCA_MULTIPASS (RLCA_INPUTS_READY and other
 * bits: RLCA_ERR_INVALID_ARG; RLCA_BF16: RLCA_ERR_UNSUPPORTED).  Arguments,
 * layouts and errors otherwise as rlca_gae.
 */
#define RLCA_STATIC_SCRATCH_BYTES (1u << 20)

int rlca_gae_static_scratch(const float *rewards, const float *values,
                            const uint8_t *terminated,
                            const uint8_t *truncated,
                            const float *trunc_value, const float *bootstrap,
                            float *advantages, float *returns, int64_t E,
                            int64_t T, float gamma, float lambda,
                            uint32_t flags, rlca_stream_t stream);

/*
 * Discounted return (rl-triton §3.2: continuation split between the local
 * update and the boundary carry):
 *   G_t = r_t + gamma * G_next(t),  G_next = 0 / trunc_value[t] /
 *   bootstrap (t = T-1) / G_{t+1}.
 * Scan form: alpha_t = r_t + gamma * trunc_t * trunc_value_t,
 * beta_t = gamma * (1 - d_t), carry A_T = bootstrap.
 * Arguments as rlca_gae; `returns` [E,T] f32 output, required.
 */
int rlca_discounted_return(const float *rewards, const uint8_t *terminated,
                           const uint8_t *truncated, const float *trunc_value,
                           const float *bootstrap, float *returns,
                           int64_t E, int64_t T, float gamma,
                           uint32_t flags, void *workspace,
                           size_t workspace_bytes, rlca_stream_t stream);

/*
 * TD(lambda) return (rl-triton §3.2: continuation split between alpha and
 * the boundary carry):
 *   G_t = r_t + gamma * [(1 - lambda) * V_{t+1} + lambda * G_{t+1}]
 * inside an episode, the bracket replaced by the boundary value at an edge
 * (at t = T-1: (1-lambda)*gamma*bootstrap in alpha, lambda*gamma*bootstrap
 * through the carry A_T = bootstrap).  Arguments as rlca_gae; `returns`
 * [E,T] f32 output, required.
 */
int rlca_td_lambda(const float *rewards, const float *values,
                   const uint8_t *terminated, const uint8_t *truncated,
                   const float *trunc_value, const float *bootstrap,
                   float *returns, int64_t E, int64_t T, float gamma,
                   float lambda, uint32_t flags, void *workspace,
                   size_t workspace_bytes, rlca_stream_t stream);

/*
 * V-Trace (rl-triton §8 Related Work; Espeholt et al. 2018), backward scan
 * with the bootstrap in alpha_{T-1}:
 *   ratio_t = exp(logp_target_t - logp_behaviour_t)
 *   rho_t = min(rho_bar, ratio_t),  c_t = lambda * min(c_bar, ratio_t)
 *   D_t   = rho_t (r_t + gamma V_next(t) - V_t) + gamma c_t (1-d_t)[t<T-1] D_{t+1}
 *   vs_t  = V_t + D_t
 *   pg_t  = rho_t (r_t + gamma vs_next(t) - V_t)   (vs_next: vs_{t+1} inside
 *                                                   an episode, boundary
 *                                                   value at an edge)
 *   logp_target, logp_behaviour  [E,T] f32 log-probabilities of the taken
 *                                action, required
 *   vs                           [E,T] f32 output, required
 *   pg_advantages                [E,T] f32 output, NULL = not written
 * Other arguments as rlca_gae (lambda = 1 gives plain V-Trace).
 */
int rlca_vtrace(const float *rewards, const float *values,
                const float *logp_target, const float *logp_behaviour,
                const uint8_t *terminated, const uint8_t *truncated,
                const float *trunc_value, const float *bootstrap,
                float *vs, float *pg_advantages,
                int64_t E, int64_t T, float gamma, float rho_bar,
                float c_bar, float lambda, uint32_t flags, void *workspace,
                size_t workspace_bytes, rlca_stream_t stream);

/*
 * Retrace(lambda) (rl-triton §3.3: the decay sits on the next step's
 * importance weight; Munos et al. 2016), backward scan with the bootstrap in
 * alpha_{T-1}:
 *   EV_t = sum_a pi[t,a] Q[t,a],  c_t = lambda * min(1, pi[t,a_t] / mu_a[t])
 *   G_t  = r_t + gamma [EV_{t+1} + c_{t+1} (G_{t+1} - Q[t+1, a_{t+1}])]
 * inside an episode, the bracket replaced by the boundary value at an edge
 * (trunc_value: E_pi Q of the truncated episode's last state; bootstrap:
 * E_pi Q of the state after the window).  The action dimension is reduced
 * per step on chip before the scan, so registers do not grow with T.
 *   q, pi        [E,T,A] f32, or bf16 with RLCA_BF16 (A = num_actions
 *                fastest), required
 *   mu_a         [E,T] f32 (bf16 with RLCA_BF16) behaviour probability of
 *                the taken action (> 0)
 *   actions      [E,T] int32 in [0, A); values outside are clamped into
 *                range (memory-safe, result unspecified)
 *   q_ret        [E,T] f32 output, required
 *   num_actions  1 .. RLCA_MAX_ACTIONS (larger: RLCA_ERR_UNSUPPORTED)
 */
int rlca_retrace(const float *q, const float *pi, const float *mu_a,
                 const int32_t *actions, const float *rewards,
                 const uint8_t *terminated, const uint8_t *truncated,
                 const float *trunc_value, const float *bootstrap,
                 float *q_ret, int64_t E, int64_t T, int32_t num_actions,
                 float gamma, float lambda, uint32_t flags, void *workspace,
                 size_t workspace_bytes, rlca_stream_t stream);

/*
 * Accumulating eligibility trace, forward scan (rl-triton §1 forward-time
 * mirror; §5 forward-scan boundaries: beta_t = 0 when d_{t-1} = 1):
 *   e_t = x_t + gamma * lambda * (1 - d_{t-1}) * e_{t-1},  e_{-1} = 0.
 *   x           [E,T] f32 per-step signal, required
 *   terminated  [E,T] u8, NULL = none;  truncated [E,T] u8, NULL = none
 *   out         [E,T] f32 output, required
 */
int rlca_elig_trace(const float *x, const uint8_t *terminated,
                    const uint8_t *truncated, float *out, int64_t E,
                    int64_t T, float gamma, float lambda, uint32_t flags,
                    void *workspace, size_t workspace_bytes,
                    rlca_stream_t stream);

/*
 * Episodic prefix sum, segmented forward scan (rl-triton §3.3: configurable
 * boundary conventions):
 *   S_t = x_t + (1 - d_{t-1}) S_{t-1}       (default, flag = last step)
 *   S_t = x_t + (1 - d_t) S_{t-1}           (RLCA_PSUM_FLAG_IS_START)
 * RLCA_PSUM_EXCLUSIVE writes S_t - x_t (the sum over the earlier steps of t's
 * episode).  d = terminated | truncated (either may be NULL).
 *   x, out  [E,T] of `dtype`: RLCA_I32 (int32, wraps modulo 2^32,
 *           bit-exact) or RLCA_F32 (float32)
 */
int rlca_episodic_prefix_sum(const void *x, int dtype,
                             const uint8_t *terminated,
                             const uint8_t *truncated, void *out,
                             int64_t E, int64_t T, uint32_t flags,
                             void *workspace, size_t workspace_bytes,
                             rlca_stream_t stream);

/*
 * Generic affine scan over precomputed coefficients (rl-triton §4 Scan
 * procedure: the generic kernel consuming precomputed alpha and beta).
 *   reverse != 0: A_t = alpha_t + beta_t A_{t+1}, A_T    = carry[e]
 *   reverse == 0: A_t = alpha_t + beta_t A_{t-1}, A_{-1} = carry[e]
 *   alpha, beta  [E,T] f32, required;  carry [E] f32, NULL = 0
 *   out          [E,T] f32 output, required
 */
int rlca_affine_scan(const float *alpha, const float *beta,
                     const float *carry, float *out, int64_t E, int64_t T,
                     int reverse, uint32_t flags, void *workspace,
                     size_t workspace_bytes, rlca_stream_t stream);

/* ---- the policy update around the scans ----------------------------------
 *
 * A policy over a vocabulary of tokens trains on the scans' advantages.  The
 * entry points below are the operators of such an update that stand next to
 * the scans: the final layer norm, the head's log-probabilities and entropy
 * (V-Trace's logp_target), the gradients of both, and the clipping of all
 * gradients by their global norm.  No counterpart in the paper.
 *
 * Conventions: as above (device pointers, caller's stream, no allocation, no
 * synchronisation, host-side argument errors), and
 *  - matrices are row-major; an input matrix has a row stride in elements (at
 *    least its width), outputs are dense;
 *  - with RLCA_BF16 the arrays documented as "x" hold bfloat16; statistics,
 *    log-probabilities and per-row factors are float32 always.  Arithmetic is
 *    float32 or better, and an output is rounded once (one exception, stated
 *    at rlca_token_logprob_backward);
 *  - RLCA_BF16 is the only flag;
 *  - results do not depend on scheduling: no floating-point atomics.
 */

/*
 * Layer norm of N rows of width D:
 *   y = (x - mean) * rstd * weight + bias,  rstd = 1 / sqrt(var + eps)
 * with the biased variance over the row (computed from the centred row).
 *   x                      [N,D] x, row stride x_stride, required
 *   weight                 [D] x, required
 *   bias                   [D] x, NULL = 0
 *   y                      [N,D] x output, required
 *   mean, rstd             [N] f32 outputs, NULL = not written
 * N == 0 or D == 0 returns RLCA_OK and enqueues nothing.  Errors:
 * RLCA_ERR_INVALID_ARG also for x_stride < D and eps not in [0, inf).
 */
int rlca_layer_norm(const float *x, const float *weight, const float *bias,
                    float *y, float *mean, float *rstd, int64_t N, int64_t D,
                    int64_t x_stride, float eps, uint32_t flags,
                    rlca_stream_t stream);

/*
 * Gradient of rlca_layer_norm from its saved statistics.  With
 * g = dy * weight and xh = (x - mean) * rstd:
 *   dx = rstd * (g - mean_D(g) - xh * mean_D(g * xh))
 *   dweight = sum_N dy * xh,  dbias = sum_N dy
 *   dy                     [N,D] x, row stride dy_stride, required
 *   x                      [N,D] x, row stride x_stride, required
 *   weight                 [D] x, required
 *   mean, rstd             [N] f32, required
 *   dx                     [N,D] x output, NULL = not written
 *   dweight, dbias         [D] x outputs, NULL = not written
 * Workspace: RLCA_EST_LAYER_NORM_BACKWARD.  N == 0 writes zeros to dweight
 * and dbias; D == 0 enqueues nothing.
 */
int rlca_layer_norm_backward(const float *dy, const float *x,
                             const float *weight, const float *mean,
                             const float *rstd, float *dx, float *dweight,
                             float *dbias, int64_t N, int64_t D,
                             int64_t dy_stride, int64_t x_stride,
                             uint32_t flags, void *workspace,
                             size_t workspace_bytes, rlca_stream_t stream);

/*
 * Log-probabilities of taken tokens and entropies of a policy head, straight
 * from its input rows; the N x V logits are never stored:
 *   z_ij   = inv_temperature * <hidden_i, weight_j>
 *   lse_i  = log sum_j exp(z_ij)
 *   logp_i = z_i,tokens[i] - lse_i     (the cross entropy is -logp)
 *   ent_i  = lse_i - sum_j softmax(z_i)_j z_ij
 * A row whose token is outside [0, V) takes no part: its three results are
 * 0 and its hidden row is not used.
 *   hidden                 [N,D] x, row stride hidden_stride, required
 *   weight                 [V,D] x, row stride weight_stride, required
 *   tokens                 [N] i32, required
 *   logp, lse              [N] f32 outputs, required
 *   entropy                [N] f32 output, NULL = not written
 * Workspace: RLCA_EST_TOKEN_LOGPROB.  N == 0 enqueues nothing.  Errors:
 * RLCA_ERR_INVALID_ARG also for D < 1, V < 1, a row stride below D,
 * inv_temperature not positive and finite; RLCA_ERR_UNSUPPORTED for D above
 * RLCA_MAX_HEAD_DIM, N or V above RLCA_MAX_HEAD_ROWS.
 */
#define RLCA_MAX_HEAD_DIM  65536
#define RLCA_MAX_HEAD_ROWS 16777216
int rlca_token_logprob(const float *hidden, const float *weight,
                       const int32_t *tokens, float *logp, float *lse,
                       float *entropy, int64_t N, int64_t D, int64_t V,
                       int64_t hidden_stride, int64_t weight_stride,
                       float inv_temperature, uint32_t flags, void *workspace,
                       size_t workspace_bytes, rlca_stream_t stream);

/*
 * Gradient of rlca_token_logprob, for factors g = d_logp and e = d_entropy
 * and the saved lse and entropy; the logits are recomputed in pieces of the
 * vocabulary:
 *   dz_ij    = inv_temperature * (g_i ([j = tokens[i]] - p_ij)
 *                                 - e_i p_ij (z_ij - lse_i + ent_i))
 *   d_hidden = dz weight,   d_weight = dz^T hidden
 * A row that takes no part has gradient 0 and adds nothing to d_weight,
 * whatever its inputs hold.  With RLCA_BF16 and N above 128, dz is rounded to
 * bfloat16 before its two products (sums stay float32): results are then
 * about 2.4e-3 off in the 2-norm, where their own rounding alone is 1.7e-3.
 *   hidden, weight, tokens as above, required
 *   lse                    [N] f32, required
 *   entropy, d_entropy     [N] f32, both or neither NULL (NULL = e is 0)
 *   d_logp                 [N] f32, required
 *   d_hidden               [N,D] x output, NULL = not written
 *   d_weight               [V,D] x output, NULL = not written
 * Workspace: RLCA_EST_TOKEN_LOGPROB_BACKWARD.  N == 0 writes zeros to
 * d_weight.  Errors as for rlca_token_logprob.
 */
int rlca_token_logprob_backward(const float *hidden, const float *weight,
                                const int32_t *tokens, const float *lse,
                                const float *entropy, const float *d_logp,
                                const float *d_entropy, float *d_hidden,
                                float *d_weight, int64_t N, int64_t D,
                                int64_t V, int64_t hidden_stride,
                                int64_t weight_stride, float inv_temperature,
                                uint32_t flags, void *workspace,
                                size_t workspace_bytes, rlca_stream_t stream);

/*
 * Global norm of `count` gradient tensors, and the tensors scaled by it:
 *   norm  = sqrt(sum over all elements of g^2)
 *   scale = min(1, max_norm / (norm + eps)), or 1 when norm is not finite
 *   out_k = scale * grad_k
 * so a step whose norm overflowed or met a NaN is left for the caller to
 * judge by the norm.  Squares are summed in float32 over short runs and in
 * float64 beyond, in a fixed order.
 *   grads                  host array of count device pointers
 *   outs                   host array of count device pointers; NULL = only
 *                          the norm.  outs[k] == grads[k] scales in place; any
 *                          other overlap is an error where it is within one
 *                          pair, and the caller's to avoid across pairs
 *   sizes                  host array of element counts (0 allowed; the
 *                          pointers are then not read)
 *   dtypes                 host array: 0 (float32) or RLCA_BF16, of both
 *                          grads[k] and outs[k]
 *   max_norm               >= 0 (infinity: scale 1)
 *   norm                   [1] f32 output, required
 * The host arrays are read before the call returns.  Workspace:
 * RLCA_EST_CLIP_GRADS.  count == 0 writes 0 to norm.
 */
int rlca_clip_grads(const void *const *grads, void *const *outs,
                    const int64_t *sizes, const uint32_t *dtypes,
                    int64_t count, float max_norm, float eps, float *norm,
                    void *workspace, size_t workspace_bytes,
                    rlca_stream_t stream);

/* ---- a recurrent policy's trunk -------------------------------------------
 *
 * The layers in front of a token policy's head, where they are recurrent: the
 * norm of the residual stream, with the stream's addition and 8-bit results,
 * and a gated linear recurrence over each rollout's steps, which starts anew
 * behind an episode's end as the forward scans above do.  No counterpart in
 * the paper.  Conventions as for the policy update; matrices below have a row
 * stride where one is named.
 *
 * Rows in 8 bits: a row of D values is D e4m3 values q (1 byte each: sign, 4
 * exponent and 3 mantissa bits, largest 448) and one float32 scale for each
 * group of RLCA_GROUP consecutive columns (the last group may be narrower):
 *   scale = max(max |v| * (1 / 448), 2^-126)
 *   q     = v * (1 / scale), to the nearest e4m3, ties to the even one
 * with 1 / 448, 1 / scale and the products rounded to float32: a value whose
 * ratio to the scale lies within 2^-22 of a border between two e4m3 may go to
 * either side of it.  A value is read back as q * scale.  NaN stays NaN (and does not count in the
 * group's maximum); a group that holds an infinity reads back as NaN.  Both
 * arrays are dense: q [N,D], scale [N, ceil(D / RLCA_GROUP)].
 */
#define RLCA_GROUP 128

/*
 * Root-mean-square norm of N rows of width D, with the residual's addition:
 *   total = x + residual, rounded to its type   (x itself without a residual)
 *   rstd  = 1 / sqrt(mean_D(total^2) + eps)
 *   y     = total * rstd * weight
 *   x                      [N,D] x, row stride x_stride, required
 *   residual               [N,D] x, row stride residual_stride, NULL = none
 *   weight                 [D] x, required
 *   total                  [N,D] x output, required iff residual is given;
 *                          may be the residual's own buffer (then dense)
 *   y                      [N,D] x output, NULL = not written
 *   y8, y8_scale           y as rows in 8 bits, from its float32 values; both
 *                          or neither NULL
 *   total8, total8_scale   total (as stored) as rows in 8 bits, to be kept for
 *                          rlca_rms_norm_backward; both or neither NULL
 *   rstd                   [N] f32 output, NULL = not written
 * At least one output must be given.  N == 0 or D == 0 enqueues nothing.
 * Errors: RLCA_ERR_INVALID_ARG also for a row stride below D and eps not in
 * [0, inf).
 */
int rlca_rms_norm(const float *x, const float *residual, const float *weight,
                  float *total, float *y, uint8_t *y8, float *y8_scale,
                  uint8_t *total8, float *total8_scale, float *rstd,
                  int64_t N, int64_t D, int64_t x_stride,
                  int64_t residual_stride, float eps, uint32_t flags,
                  rlca_stream_t stream);

/*
 * Gradient of rlca_rms_norm from its saved statistic and its total, as stored
 * or kept in 8 bits.  With g = dy * weight and s = total * rstd:
 *   dx = d_total + rstd * (g - s * mean_D(g * s))   (of x and the residual)
 *   dweight = sum_N dy * s
 *   dy                     [N,D] x, row stride dy_stride, required
 *   d_total                [N,D] x, row stride d_total_stride: the gradient
 *                          that reaches total from elsewhere, NULL = 0
 *   total                  [N,D] x, row stride total_stride, or NULL and
 *   total8, total8_scale   total as rows in 8 bits
 *   weight                 [D] x, required
 *   rstd                   [N] f32, required
 *   dx                     [N,D] x output, NULL = not written
 *   dweight                [D] x output, NULL = not written
 * Workspace: RLCA_EST_RMS_NORM_BACKWARD.  N == 0 writes zeros to dweight;
 * D == 0 enqueues nothing.
 */
int rlca_rms_norm_backward(const float *dy, const float *d_total,
                           const float *total, const uint8_t *total8,
                           const float *total8_scale, const float *weight,
                           const float *rstd, float *dx, float *dweight,
                           int64_t N, int64_t D, int64_t dy_stride,
                           int64_t d_total_stride, int64_t total_stride,
                           uint32_t flags, void *workspace,
                           size_t workspace_bytes, rlca_stream_t stream);

/*
 * Gated linear recurrence over E rows of T steps of D channels, a forward
 * scan (rl-triton §1 forward-time mirror, with beta_t = 0 behind an episode's
 * end as in §5):
 *   a_t = 1 / (1 + exp(-gate_t))
 *   h_t = a_t h_{t-1} + (1 - a_t) x_t,   h_{-1} = state
 * where h_{t-1} counts as 0 if step t-1 of the call is flagged (terminated or
 * truncated).  A row may be shorter than T: steps at and behind lengths[e]
 * take no part, whatever their inputs and flags hold, and their h is 0.
 *   last = h at the row's last step (state for a row of length 0), or 0 if
 *          that step is flagged
 * so that a rollout cut into several calls gives the results of one, each
 * call's last being the next one's state.  T = 1 is the form for acting, one
 * token of E sequences at a time; last may then (and always) be the state's
 * own buffer.  a_t and 1 - a_t are formed in float32, each relatively exact to
 * 2^-20 (bfloat16 gates g: to (4 + 1.2 |g|) 2^-23) however small it is, down to
 * 2^-125; bfloat16 gates below -86 count as -86.  A state or an x that is not
 * finite reaches every later h of its channel up to an episode's end: an
 * infinity stays one wherever a_t is not 0 in float32.
 *   x, gate                [E,T,D] x ([T,E,D] with RLCA_TIME_MAJOR), rows of D
 *                          at row strides x_stride and gate_stride, required
 *   terminated, truncated  [E,T] ([T,E]) u8, NULL = none
 *   state                  [E,D] f32, NULL = 0
 *   lengths                [E] i32, NULL = T; values outside [0, T] count as
 *                          the nearer end
 *   h                      [E,T,D] x output, dense, required
 *   last                   [E,D] f32 output, NULL = not written
 * Flags: RLCA_TIME_MAJOR, RLCA_BF16 (x, gate and h).  E * T is at most
 * 2^31 - 1.  E == 0 or D == 0 enqueues nothing; T == 0 writes last only.
 * Workspace: RLCA_EST_GATED_SCAN (nothing unless a few rows are long).
 */
int rlca_gated_scan(const float *x, const float *gate,
                    const uint8_t *terminated, const uint8_t *truncated,
                    const float *state, const int32_t *lengths, float *h,
                    float *last, int64_t E, int64_t T, int64_t D,
                    int64_t x_stride, int64_t gate_stride, uint32_t flags,
                    void *workspace, size_t workspace_bytes,
                    rlca_stream_t stream);

/*
 * Gradient of rlca_gated_scan from its inputs and its h, for the gradients dh
 * and d_last of its outputs, a backward scan.  With k_t = 0 where h_{t-1}
 * counts as 0 and 1 elsewhere:
 *   G_t     = dh_t + k_{t+1} a_{t+1} G_{t+1},  behind a row's last step
 *             d_last (0 if that step is flagged) in place of k a G
 *   dx_t    = (1 - a_t) G_t
 *   dgate_t = a_t (1 - a_t) G_t (k_t h_{t-1} - x_t)
 *   d_state = k_0 a_0 G_0                     (d_last for a row of length 0)
 * Steps that take no part have gradient 0.
 *   dh, x, gate, h         [E,T,D] x ([T,E,D]) at their row strides, required
 *   terminated, truncated, state, lengths  as in the forward call
 *   d_last                 [E,D] f32, NULL = 0
 *   dx, dgate              [E,T,D] x outputs at their row strides, required;
 *                          with one stride they may be parts of one wider
 *                          matrix's rows
 *   d_state                [E,D] f32 output, NULL = not written; may be
 *                          d_last's own buffer
 * Otherwise as rlca_gated_scan; T == 0 writes d_state only.  Workspace:
 * RLCA_EST_GATED_SCAN_BACKWARD.
 */
int rlca_gated_scan_backward(const float *dh, const float *x,
                             const float *gate, const float *h,
                             const uint8_t *terminated,
                             const uint8_t *truncated, const float *state,
                             const int32_t *lengths, const float *d_last,
                             float *dx, float *dgate, float *d_state,
                             int64_t E, int64_t T, int64_t D,
                             int64_t dh_stride, int64_t x_stride,
                             int64_t gate_stride, int64_t h_stride,
                             int64_t dx_stride, int64_t dgate_stride,
                             uint32_t flags, void *workspace,
                             size_t workspace_bytes, rlca_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RLCA_H */
