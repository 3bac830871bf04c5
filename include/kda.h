/*
 * kda.h — C ABI of the MI355X (gfx950) KDA library, libkda.so.
 *
 * KDA (Kimi Delta Attention) is a gated delta-rule linear attention: each
 * head keeps a fixed-size state S (K x V, fp32) instead of a KV cache, and
 * every token applies, per batch row b and head h,
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t
 *
 * with a per-key-channel forget gate alpha_t = exp(g_t), g clamped to
 * [-5, 0] (alpha in [e^-5, 1]) inside the library.
 *
 * Page: "Kimi K3 — открытая модель, которая обошла закрытых лидеров рынка"
 * (aiblin.ru).  Section "Как хранить миллион токенов в памяти": the state
 * matrix S of fixed size, the delta rule (partly erase, then write), beta as
 * write strength in [0, 1], alpha as forgetting coefficient and its clamp to
 * [e^-5, 1].  Section "Как распараллелили последовательное обновление":
 * chunk-parallel evaluation (all tokens of a chunk at once, then the state
 * passed on, in parallel over heads) and the one-card segment planner for
 * long prefill (per segment a local state and a transition matrix,
 * recombined exactly).  The update formula itself is lost on the page; the
 * equation above is the reading used throughout.
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE pointers (HIP), row-major, contiguous.
 *     Alignment: states and the workspace 16 bytes; for prefill q, k, v, g
 *     and o 16 bytes and beta its element size; for decode every token
 *     tensor its element size.  The caller owns every buffer, the workspace
 *     included; the library allocates no device memory.
 *   - Work is enqueued asynchronously on `stream` (NULL is the default
 *     stream) of the current HIP device.  Nothing is synchronised.
 *   - Arguments are validated on the host before anything is launched; on an
 *     error nothing is launched.  KDA_ERR_INVALID_ARG: a null pointer, a
 *     negative size, a misaligned pointer, a partially overlapping state
 *     pair.  KDA_ERR_UNSUPPORTED: sizes or a dtype the kernels do not
 *     implement.  KDA_ERR_WORKSPACE: workspace missing or too small.
 *     KDA_ERR_HIP: a HIP launch or query failed.
 *   - Token tensors (q, k, v, g, beta, o) share one dtype `dt`; states are
 *     always fp32.  o is rounded to `dt` (round to nearest even).
 *   - Results are deterministic: no floating-point atomics.
 *   - The library keeps no state between calls and every call is reentrant,
 *     with one opt-in exception: the launch timing of kda_profile_start /
 *     kda_profile_stop below keeps one process-wide record (guarded by a
 *     mutex) while it is on.
 *   - Non-finite inputs propagate; they are not detected.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <hip/hip_runtime_api.h>   /* hipStream_t */

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,
    KDA_ERR_UNSUPPORTED = 2,
    KDA_ERR_WORKSPACE = 3,
    KDA_ERR_HIP = 4,
    /* never returned: they stretch the enum's value range over all of int,
     * so that any code a caller passes to kda_status_string is a valid
     * kda_status (in C++ a value outside the range is undefined) */
    KDA_STATUS_RANGE_MIN_ = -2147483647 - 1,
    KDA_STATUS_RANGE_MAX_ = 2147483647
} kda_status;

typedef enum kda_dtype {
    KDA_F32 = 0,
    KDA_BF16 = 1,
    /* never valid: the same value range as kda_status, so that an unknown
     * code reaches the argument checks (which reject it) with defined
     * behaviour */
    KDA_DTYPE_RANGE_MIN_ = -2147483647 - 1,
    KDA_DTYPE_RANGE_MAX_ = 2147483647
} kda_dtype;

/*
 * Execution plan of a prefill call.
 *   split:   1 = single pass: one kernel per (b, h, segment, column block)
 *            walks the chunks and does all chunk work in order;
 *            2 = two passes: an intra-chunk pass over every (b, h, chunk) at
 *            once writes per-chunk operands to the workspace, then a state
 *            pass walks the chunks (the workspace holds those records);
 *            3 = token-serial: one workgroup per (b, h, 64-column block)
 *            applies the recurrence token by token (the defining equation of
 *            the page's section "Как хранить миллион токенов в памяти"), the
 *            state in registers; no workspace, n_seg 1, v_block 64.  The
 *            library's choice only where no chunk kernel exists (fp32 with
 *            K = 128); a chain's time grows with its length;
 *            4 = fused: one workgroup per (b, h, segment) in which four waves
 *            prepare chunk c + 1 (gate cumsum, in-chunk products, the
 *            triangular solve) while four waves carry the state through
 *            chunk c, the operands passed through LDS: the inputs are read
 *            once and nothing per chunk touches HBM.  bf16 with K = V = 128
 *            only, v_block 128 (0 or V); the library's choice for those
 *            sizes.
 *   n_seg:   number of sequence segments evaluated side by side on one card
 *            (1 = none; > 1 adds the segment summary and segment scan passes).
 *   v_block: value columns per workgroup of the state-carrying pass (64 or
 *            128; at most V, and with n_seg > 1 it must divide K).
 * Any field 0 means "let the library choose".  Any valid plan gives the same
 * result up to fp32/bf16 rounding.
 */
typedef struct kda_plan {
    int n_seg;
    int v_block;
    int split;
} kda_plan;

/* Sizes supported by the kernels: K, V in {64, 128}; bf16 or fp32 inputs
 * (fp32 with K = 128 runs the token-serial form, split 3).  T >= 0 is
 * arbitrary (the tail chunk is masked); B, H >= 0. */

/*
 * The plan kda_chunk_fwd uses for these sizes on the current device.
 * Fills *plan.  Returns KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED or
 * KDA_ERR_HIP (device query failed).
 */
kda_status kda_chunk_fwd_plan(int B, int T, int H, int K, int V, kda_dtype dt,
                              kda_plan* plan);

/*
 * Bytes of device workspace kda_chunk_fwd needs for these sizes in the plan
 * the library picks on the current device (kda_chunk_fwd_plan).  0 when none
 * is needed; (size_t)-1 for invalid or unsupported arguments or a failed
 * device query.
 */
size_t kda_chunk_fwd_workspace_size(int B, int T, int H, int K, int V, kda_dtype dt);

/*
 * Chunked prefill (the page's chunk-parallel form, section "Как
 * распараллелили последовательное обновление"), optionally resuming from an
 * initial state and returning the final state (the prefix-cache mechanism),
 * in the plan the library picks for the current device.
 *
 *   q, k, g : [B, T, H, K]  dtype dt   (g = log alpha before the clamp)
 *   v       : [B, T, H, V]  dtype dt
 *   beta    : [B, T, H]     dtype dt   (write strength; not clamped)
 *   initial_state : [B, H, K, V] fp32, or NULL for zeros
 *   o       : [B, T, H, V]  dtype dt   (written; may be NULL only if T == 0)
 *   final_state   : [B, H, K, V] fp32, or NULL (not written).  It may alias
 *                   initial_state exactly (in-place resume); a partial
 *                   overlap is KDA_ERR_INVALID_ARG.
 *   workspace / workspace_bytes : device scratch of at least
 *             kda_chunk_fwd_workspace_size(...) bytes (may be NULL when that
 *             size is 0); its contents on entry do not matter.
 * T == 0 writes final_state = initial_state (or zeros) and nothing else.
 */
kda_status kda_chunk_fwd(int B, int T, int H, int K, int V, kda_dtype dt,
                         const void* q, const void* k, const void* v,
                         const void* g,
                         const void* beta,
                         const float* initial_state,
                         void* o,
                         float* final_state,
                         void* workspace, size_t workspace_bytes,
                         hipStream_t stream);

/*
 * kda_chunk_fwd in a caller-chosen execution plan, and its workspace size.
 *   plan : NULL or a kda_plan; fields 0 are the library's choice.  A plan the
 *          kernels cannot run is KDA_ERR_INVALID_ARG (a field out of range) or
 *          KDA_ERR_UNSUPPORTED (a valid field these sizes have no kernel for).
 * The workspace size in a plan: with split = 2 one record per (b, h, chunk)
 * (for K = V = 128 bf16, 72.5 KiB; splits 1, 3 and 4 keep none); with
 * n_seg > 1 the segment transitions
 * and local states ((n_seg - 1) * B * H * K * (K + V) fp32) plus
 * B * H * K * V fp32 (a redirected final state).  Every other argument, and
 * the result up to fp32/bf16 rounding, as kda_chunk_fwd.
 */
size_t kda_chunk_fwd_planned_workspace_size(int B, int T, int H, int K, int V, kda_dtype dt,
                                            const kda_plan* plan);
kda_status kda_chunk_fwd_planned(int B, int T, int H, int K, int V, kda_dtype dt,
                                 const void* q, const void* k, const void* v,
                                 const void* g, const void* beta,
                                 const float* initial_state,
                                 void* o, float* final_state,
                                 const kda_plan* plan,
                                 void* workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/*
 * kda_chunk_fwd_planned for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  No workspace argument: the workspace comes from a device array
 * of KDA_NOALLOC_SCRATCH_BYTES (64 MiB) that the library defines and that
 * each GPU it runs on holds until the process ends; the call allocates
 * nothing.
 *   plan : NULL = the plan kda_chunk_fwd picks when its workspace
 *          (kda_chunk_fwd_planned_workspace_size) fits the array, else the
 *          single-pass plan (split 1) with as many of the library's segments
 *          as fit (one segment needs none, so every size runs); an explicit
 *          plan whose workspace exceeds the array is KDA_ERR_WORKSPACE.
 * All calls on one GPU share that GPU's array: calls that overlap in time on
 * one GPU (from several streams or host threads) race and give wrong
 * results; calls ordered on one stream are safe (nothing in the array needs
 * to start at zero).  Every other argument, and the result, as
 * kda_chunk_fwd_planned in the same plan.
 */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
kda_status kda_chunk_fwd_noalloc(int B, int T, int H, int K, int V, kda_dtype dt,
                                 const void* q, const void* k, const void* v,
                                 const void* g, const void* beta,
                                 const float* initial_state,
                                 void* o, float* final_state,
                                 const kda_plan* plan,
                                 hipStream_t stream);

/*
 * kda_chunk_fwd_planned with the output gate of the KDA block fused into the
 * store of o (aiblin.ru page, section "KV‑кэш все‑таки не исчез полностью":
 * after the attention a gate decides what share of its result passes on into
 * the model's main stream, and the KDA blocks use the same gate; its form is
 * not given there, the plainest reading is taken):
 *
 *   o[b,t,h,:] = RNE_dt( RNE_dt(S_t^T q_t) * sigmoid(gate[b,t,h,:]) )
 *
 *   gate : [B, T, H, V] dtype dt, the gate pre-activation, 16-byte aligned;
 *          NULL is KDA_ERR_INVALID_ARG when there is work.
 * The same result as kda_chunk_fwd followed by an elementwise o * sigmoid(gate)
 * in fp32 rounded to dt, up to the 1-ulp exp2 and reciprocal of the sigmoid;
 * it saves that pass over o.  Every other argument as kda_chunk_fwd_planned
 * (workspace size: kda_chunk_fwd_planned_workspace_size).
 */
kda_status kda_chunk_fwd_gated(int B, int T, int H, int K, int V, kda_dtype dt,
                               const void* q, const void* k, const void* v,
                               const void* g, const void* beta, const void* gate,
                               const float* initial_state,
                               void* o, float* final_state,
                               const kda_plan* plan,
                               void* workspace, size_t workspace_bytes,
                               hipStream_t stream);

/*
 * Prefill of a packed batch of N variable-length sequences (the
 * prefix-caching and multi-token-verification use: every sequence resumes
 * from its own state and returns its own final state).  The habr.com
 * article on the Kimi K3 technical report notes that KDA needs its own
 * prefix-caching support in serving engines; this is that call.
 *
 *   cu_seqlens : DEVICE int32 [N + 1]: sequence i is tokens
 *                [cu_seqlens[i], cu_seqlens[i+1]) of the packed axis;
 *                cu_seqlens[0] = 0, non-decreasing, cu_seqlens[N] = T_total.
 *                Read on the device (nothing is synchronised).  Offsets
 *                outside that contract are clamped to [0, T_total] (results
 *                for such sequences are then unspecified, but every access
 *                stays inside the buffers).
 *   q, k, g    : [T_total, H, K] dtype dt;  v, o : [T_total, H, V];
 *   beta       : [T_total, H]
 *   initial_state : [N, H, K, V] fp32 or NULL (zeros)
 *   final_state   : [N, H, K, V] fp32 or NULL; may alias initial_state exactly
 *   workspace  : device scratch of at least
 *                kda_chunk_fwd_varlen_workspace_size(...) bytes
 * Runs the two-pass plan (intra-chunk pass over every chunk of every
 * sequence, then one state-carrying workgroup column block per (sequence,
 * head)); sequences of length 0 copy their state.  Same conventions, dtypes
 * and error codes as kda_chunk_fwd; sizes: K, V in {64, 128}, bf16 or fp32.
 * fp32 other than K = V = 64 runs the token-serial form per (sequence, head)
 * and needs no workspace (the size function returns 0).
 */
size_t kda_chunk_fwd_varlen_workspace_size(int N, int T_total, int H, int K, int V, kda_dtype dt);
kda_status kda_chunk_fwd_varlen(int N, const int* cu_seqlens, int T_total, int H, int K, int V, kda_dtype dt,
                                const void* q, const void* k, const void* v,
                                const void* g, const void* beta,
                                const float* initial_state,
                                void* o, float* final_state,
                                void* workspace, size_t workspace_bytes,
                                hipStream_t stream);

/*
 * kda_chunk_fwd_varlen with the output gate fused as in kda_chunk_fwd_gated;
 * gate : [T_total, H, V] dtype dt.
 */
kda_status kda_chunk_fwd_varlen_gated(int N, const int* cu_seqlens, int T_total, int H, int K, int V,
                                      kda_dtype dt, const void* q, const void* k, const void* v,
                                      const void* g, const void* beta, const void* gate,
                                      const float* initial_state, void* o, float* final_state,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * kda_chunk_fwd_varlen that also returns state snapshots at fixed block
 * boundaries (prefix caching: a later request sharing the first m tokens of
 * a sequence resumes from the snapshot at the largest boundary <= m).
 *
 *   snapshot_interval : tokens between snapshots; a positive multiple of 64
 *                       (the chunk length), else KDA_ERR_INVALID_ARG.
 *   snapshots         : DEVICE fp32 [max_snapshots, H, K, V], 16-byte aligned
 *                       (may be NULL when max_snapshots == 0).
 *   max_snapshots     : capacity in snapshots (>= 0); slots past it are not
 *                       written.  With valid cu_seqlens the count needed is
 *                       sum_i floor(len_i / snapshot_interval) <=
 *                       floor(T_total / snapshot_interval).
 * Snapshot m (m = 0, 1, ...) of sequence i, the state after its first
 * (m + 1) * snapshot_interval tokens, is written to slot snap_off_i + m with
 * snap_off_i = sum_{j < i} floor(len_j / snapshot_interval); nothing else in
 * `snapshots` is touched.  o and final_state are exactly those of
 * kda_chunk_fwd_varlen with the same arguments; the workspace is the same.
 * Snapshots come from the chunk state pass: sizes that run the token-serial
 * form (fp32 other than K = V = 64) return KDA_ERR_UNSUPPORTED.
 */
kda_status kda_chunk_fwd_varlen_snapshots(int N, const int* cu_seqlens, int T_total, int H, int K, int V,
                                          kda_dtype dt, const void* q, const void* k, const void* v,
                                          const void* g, const void* beta, const float* initial_state,
                                          void* o, float* final_state, int snapshot_interval,
                                          float* snapshots, int max_snapshots,
                                          void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One decode step for N independent sequences (page section "Как хранить
 * миллион токенов в памяти": the fixed-size state replaces the KV cache).
 * Reads and writes the state once.
 *
 *   q, k, g : [N, H, K] dtype dt;  v : [N, H, V] dtype dt;  beta : [N, H] dtype dt
 *   state   : [N, H, K, V] fp32, updated IN PLACE to S_t
 *   o       : [N, H, V] dtype dt (written), o = S_t^T q
 */
kda_status kda_recurrent_step(int N, int H, int K, int V, kda_dtype dt,
                              const void* q, const void* k, const void* v,
                              const void* g, const void* beta,
                              float* state, void* o, hipStream_t stream);

/*
 * T consecutive tokens of each of N sequences in one call (multi-token
 * verification of a draft, as in speculative decoding): the same update as T
 * calls of kda_recurrent_step, with the state read once and written once.
 *
 *   q, k, g : [N, T, H, K] dtype dt;  v : [N, T, H, V];  beta : [N, T, H]
 *   state   : [N, H, K, V] fp32, updated IN PLACE to the state after token T
 *   o       : [N, T, H, V] dtype dt (written), o_t = S_t^T q_t
 *   step_states : [N, T, H, K, V] fp32, the state after each token (so that a
 *                 caller can resume after any accepted prefix), or NULL.  It
 *                 must not overlap state.
 * T == 0 or N * H == 0 does nothing.  Sizes and dtypes as kda_recurrent_step.
 */
kda_status kda_recurrent_steps(int N, int T, int H, int K, int V, kda_dtype dt,
                               const void* q, const void* k, const void* v,
                               const void* g, const void* beta,
                               float* state, void* o, float* step_states, hipStream_t stream);

/*
 * Backward of kda_chunk_fwd: the gradients of a loss L with respect to q, k,
 * v, g (log alpha before the clamp), beta and the initial state, given dL/do
 * and dL/dS_T.  The pages give no backward; this is the chain rule applied
 * to the recurrence (section "Как хранить миллион токенов в памяти") in its
 * chunk form (section "Как распараллелили последовательное обновление"): the
 * forward's state after every chunk, a reverse state pass for dL/dS at every
 * chunk boundary, then every chunk's gradients at once.  fp32 with K or V =
 * 128 (no two-pass forward) runs a token-level form instead.  The clamp
 * passes the gradient inside its closed range [-5, 0] and blocks it outside.
 *
 *   q, k, g, v, beta, initial_state : the forward's inputs (same layouts)
 *   d_o           : [B, T, H, V] dtype dt, dL/do, or NULL (zeros)
 *   d_final_state : [B, H, K, V] fp32, dL/dS_T, or NULL (zeros)
 *   dq, dk, dg    : [B, T, H, K] dtype dt (written)
 *   dv            : [B, T, H, V] dtype dt (written)
 *   dbeta         : [B, T, H] dtype dt (written)
 *   d_initial_state : [B, H, K, V] fp32 (written) or NULL.  It must not
 *                     overlap d_final_state (not even exactly: the reverse
 *                     pass reads dL/dS_T while it writes dL/dS_0), else
 *                     KDA_ERR_INVALID_ARG.
 *   workspace     : at least kda_chunk_bwd_workspace_size(...) bytes (the
 *                   size does not depend on the device).  Chunk form: the
 *                   forward plan's segment arrays (with n_seg > 1, the
 *                   transitions of all n_seg segments: one K x K fp32 slot
 *                   per (b, h) more than the forward's), its chunk records, the
 *                   state and dL/dS after every chunk (2 B*H*ceil(T/64)*K*V
 *                   values) and per-chunk fp32 intermediates.  bf16 at
 *                   K = V = 128: one workgroup computes every gradient of a
 *                   chunk from bf16 states and adjoints, and the workspace
 *                   holds those bf16, dL/dU (fp32, 64 x V per chunk) and bf16
 *                   copies of S0 and dL/dS_T.  Otherwise the states and
 *                   adjoints are fp32 and the products the three chunk stages
 *                   hand on are kept too.
 *                   Token-level
 *                   form: the state every 8 tokens (B*H*ceil(T/8)*K*V fp32)
 *                   and the per-16-column partial sums
 *                   (V/16 * B*T*H*(3K+1) fp32).
 * Sizes: K, V in {64, 128}; bf16 or fp32.  The forward states are recomputed
 * (no saved activations are needed).  Results are deterministic.
 */
size_t kda_chunk_bwd_workspace_size(int B, int T, int H, int K, int V, kda_dtype dt);
kda_status kda_chunk_bwd(int B, int T, int H, int K, int V, kda_dtype dt,
                         const void* q, const void* k, const void* v, const void* g, const void* beta,
                         const float* initial_state, const void* d_o, const float* d_final_state,
                         void* dq, void* dk, void* dv, void* dg, void* dbeta, float* d_initial_state,
                         void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- mixer operators ----------------------------------------------------------
 *
 * What stands around the recurrence in a layer, and its sibling with a scalar
 * decay a head: the short causal convolution on its inputs, the selective scan,
 * and the group norm with its gate on its output.
 *
 * Conventions, beyond those at the top of this file:
 *   - Token tensors share the dtype `dt`; parameters (weights, biases, A, D,
 *     dt_bias) and their gradients are fp32; convolution states are `dt` (they
 *     hold inputs), scan states fp32.
 *   - Sequences: with cu_seqlens NULL a call has N sequences of T tokens each,
 *     in order; else cu_seqlens is a DEVICE int32 [N + 1] array as in
 *     kda_chunk_fwd_varlen, T is the number of token rows, and rows at or
 *     behind cu_seqlens[N] are neither read nor written (they pad a batch).
 *     Offsets outside the contract are clamped: every access stays in bounds.
 *   - x_stride, delta_stride, b_stride, c_stride, gate_stride: elements between consecutive
 *     token rows of an input (at least the row's width), so that a slice of a
 *     wider projection is passed as it is.  Outputs are contiguous unless they
 *     have a stride of their own.
 *   - Outputs must not overlap inputs or each other unless a call says so: a
 *     shared byte is KDA_ERR_INVALID_ARG (rows of one spacing that keep to
 *     columns of their own share none).
 *   - All work goes to `stream`; a call may be captured into a graph.  Calls
 *     that run at the same time need workspaces of their own.
 *   - Results are deterministic: parameter gradients are summed in a fixed
 *     order.
 */
typedef enum kda_activation {
    KDA_ACT_NONE = 0,
    KDA_ACT_SILU = 1,               /* v sigmoid(v) */
    KDA_ACT_SIGMOID = 2,
    KDA_ACT_RANGE_MIN_ = -2147483647 - 1,   /* never valid, as in kda_dtype */
    KDA_ACT_RANGE_MAX_ = 2147483647
} kda_activation;

/*
 * Short causal depthwise convolution over the tokens of each sequence:
 *
 *   y_t[d] = act( bias[d] + sum_{w < W} weight[d, w] x_{t - (W-1) + w}[d] )
 *
 *   W in {2, 3, 4}; D up to 2^21; tokens and sequences up to 2^31 - 2^26
 *   (more are KDA_ERR_UNSUPPORTED).  Sums in fp32, rounded once.
 *   x      : [tokens, D] dt, row stride x_stride
 *   weight : [D, W] fp32;  bias : [D] fp32 or NULL
 *   initial_state : [N, W-1, D] dt, the W - 1 rows before each sequence, or
 *                   NULL (zeros)
 *   y      : [tokens, D] dt
 *   final_state   : [N, W-1, D] dt, the last W - 1 rows of (initial_state, x),
 *                   or NULL.  It must not overlap initial_state.
 * Pointers aligned to their element size; with every pointer 16-byte aligned
 * and D and x_stride multiples of 16 bytes, accesses are 16 bytes wide.
 */
kda_status kda_short_conv_fwd(int N, const int* cu_seqlens, int T, int D, int W, kda_dtype dt, kda_activation act,
                              const void* x, long long x_stride, const float* weight, const float* bias,
                              const void* initial_state, void* y, void* final_state, hipStream_t stream);

/*
 * Its gradients, from dL/dy (d_y, [tokens, D]) and dL/dfinal_state
 * (d_final_state or NULL):
 *   dx : [tokens, D] dt;  dweight : [D, W] fp32;  dbias : [D] fp32 or NULL
 *   d_initial_state : [N, W-1, D] dt or NULL
 *   workspace : kda_short_conv_bwd_workspace_size(...) bytes (packed: 1 for a
 *               call with cu_seqlens)
 * The convolution is recomputed from x.  Accesses are eight bytes wide where
 * pointers, D and x_stride are multiples of eight bytes.  No tokens: dweight
 * and dbias are zero, and dL/dfinal_state passes to d_initial_state.
 */
size_t kda_short_conv_bwd_workspace_size(int N, int packed, int T, int D, int W, kda_dtype dt);
kda_status kda_short_conv_bwd(int N, const int* cu_seqlens, int T, int D, int W, kda_dtype dt, kda_activation act,
                              const void* x, long long x_stride, const float* weight, const float* bias,
                              const void* initial_state, const void* d_y, const void* d_final_state, void* dx,
                              float* dweight, float* dbias, void* d_initial_state, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/*
 * One token of N sequences: y [N, D] from x [N, D] (row stride x_stride) and
 * state [N, W-1, D], whose rows move up IN PLACE.
 */
kda_status kda_short_conv_step(int N, int D, int W, kda_dtype dt, kda_activation act, const void* x,
                               long long x_stride, const float* weight, const float* bias, void* state, void* y,
                               hipStream_t stream);

/*
 * Selective scan: a state space recurrence with a scalar decay a head and
 * input-dependent step size and projections.  Per sequence and head h, with
 * delta_t = softplus(dt_t + dt_bias) (dt_softplus != 0) or dt_t + dt_bias:
 *
 *   S_t = exp(delta_t A) S_{t-1} + delta_t B_t x_t^T       (K x P, fp32)
 *   y_t = S_t^T C_t + D x_t
 *
 *   x     : [tokens, H, P] dt, row stride x_stride;  P in {64, 128}
 *   delta : [tokens, H] dt (row stride delta_stride), the step sizes dt_t before bias and softplus
 *   A     : [H] fp32;  D, dt_bias : [H] fp32 or NULL (none)
 *   B, C  : [tokens, G, K] dt, row strides b_stride, c_stride; K in {64, 128};
 *           G divides H, and heads h G / H .. share a group
 *   initial_state : [N, H, K, P] fp32 or NULL (zeros)
 *   y     : [tokens, H, P] dt
 *   final_state   : [N, H, K, P] fp32 or NULL; it may be initial_state exactly
 *   workspace : kda_selective_scan_fwd_workspace_size(...) bytes
 * x, B, C, y, states and workspace 16-byte aligned, strides of x, B and C
 * multiples of 16 bytes; every row stride, and H P, at most 2^23 elements in the
 * prompt and gradient calls (more are KDA_ERR_UNSUPPORTED).  Meant for
 * A delta <= 0 (decay); a growing state is computed as far as e^{sum A delta}
 * over 64 tokens stays finite.  Non-finite inputs propagate to their sequence
 * from the start of their 64-token chunk on, never to another sequence.  A
 * sequence without tokens passes its state on.
 * bf16 tokens: states, decays, step sizes and sums are fp32; y, dx, dB and dC
 * are off by their rounding to bf16 and 2^-16 of the sum of the absolute values
 * of their terms.
 */
size_t kda_selective_scan_fwd_workspace_size(int N, int packed, int T, int H, int G, int K, int P, kda_dtype dt);
kda_status kda_selective_scan_fwd(int N, const int* cu_seqlens, int T, int H, int G, int K, int P, kda_dtype dt,
                                  int dt_softplus, const void* x, long long x_stride, const void* delta,
                                  long long delta_stride, const float* A, const void* B, long long b_stride, const void* C,
                                  long long c_stride, const float* D, const float* dt_bias,
                                  const float* initial_state, void* y, float* final_state, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream);

/*
 * Its gradients, from dL/dy (d_y, [tokens, H, P] dt) and dL/dfinal_state
 * (d_final_state fp32 or NULL):
 *   dx : [tokens, H, P];  d_delta : [tokens, H] (of dt_t, before bias and
 *        softplus);  dB, dC : [tokens, G, K], summed over the group's heads;
 *        all dt, row strides dx_stride, db_stride, dc_stride (multiples of 16
 *        bytes, dx_stride at most 2^23 elements; columns of one wider buffer are fine)
 *   dA : [H] fp32;  dD, d_dt_bias : [H] fp32 or NULL
 *   d_initial_state : [N, H, K, P] fp32 or NULL
 *   workspace : kda_selective_scan_bwd_workspace_size(...) bytes: the state
 *        before and the adjoint behind every chunk of 64 tokens (fp32), and
 *        fp32 parts of dB and dC
 * The states are recomputed from the inputs.  No tokens: dA, dD and d_dt_bias
 * are zero, and dL/dfinal_state passes to d_initial_state.
 */
size_t kda_selective_scan_bwd_workspace_size(int N, int packed, int T, int H, int G, int K, int P, kda_dtype dt);
kda_status kda_selective_scan_bwd(int N, const int* cu_seqlens, int T, int H, int G, int K, int P, kda_dtype dt,
                                  int dt_softplus, const void* x, long long x_stride, const void* delta,
                                  long long delta_stride, const float* A, const void* B, long long b_stride,
                                  const void* C, long long c_stride, const float* D, const float* dt_bias,
                                  const float* initial_state, const void* d_y, const float* d_final_state, void* dx,
                                  long long dx_stride, void* d_delta, float* dA, void* dB, long long db_stride,
                                  void* dC, long long dc_stride, float* dD, float* d_dt_bias,
                                  float* d_initial_state, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream);

/*
 * One token of N sequences: state [N, H, K, P] is updated IN PLACE and read
 * and written once.  x [N, H, P], delta [N, H], B, C [N, G, K], y [N, H, P],
 * with row strides up to 2^37 elements.
 */
kda_status kda_selective_scan_step(int N, int H, int G, int K, int P, kda_dtype dt, int dt_softplus, const void* x,
                                   long long x_stride, const void* delta, long long delta_stride, const float* A,
                                   const void* B,
                                   long long b_stride, const void* C, long long c_stride, const float* D,
                                   const float* dt_bias, float* state, void* y, hipStream_t stream);

/*
 * Group norm of token rows (channels last), with an activation or a gate.
 * Each row's C channels form `groups` groups, normalised each by itself
 * (statistics a token: over tokens they would look ahead):
 *
 *   u = x, or x act(gate) with gate_first
 *   n = (u - m) / sqrt(mean((u - m)^2) + eps) weight + bias,
 *       m = mean(u) with center, else 0 (root mean square)
 *   y = act(n) without a gate; n act(gate); n with gate_first
 *
 *   x, gate : [rows, C] dt, row strides x_stride, gate_stride; gate or NULL
 *   weight, bias : [C] fp32 or NULL (1, 0);  y : [rows, C] dt
 *   groups at most 65535
 * fp32 inside, rounded once.  y may be x or the gate exactly.  C / groups at
 * most 4096 channels, or 16384 where 16-byte accesses work (C / groups and
 * strides multiples of 16 bytes, pointers 16-byte aligned); wider groups are
 * KDA_ERR_UNSUPPORTED.
 */
kda_status kda_group_norm_fwd(int rows, int C, int groups, kda_dtype dt, kda_activation act, int center,
                              int gate_first, float eps, const void* x, long long x_stride, const float* weight,
                              const float* bias, const void* gate, long long gate_stride, void* y,
                              hipStream_t stream);

/*
 * Its gradients from dL/dy (d_y, [rows, C]): dx [rows, C], dweight and dbias
 * [C] fp32 (each or NULL), d_gate [rows, C] (exactly where there is a gate).
 * workspace : kda_group_norm_bwd_workspace_size(...) bytes, needed where
 * dweight or dbias is asked for.
 */
size_t kda_group_norm_bwd_workspace_size(int rows, int C, int groups, kda_dtype dt);
kda_status kda_group_norm_bwd(int rows, int C, int groups, kda_dtype dt, kda_activation act, int center,
                              int gate_first, float eps, const void* x, long long x_stride, const float* weight,
                              const float* bias, const void* gate, long long gate_stride, const void* d_y, void* dx,
                              float* dweight, float* dbias, void* d_gate, void* workspace, size_t workspace_bytes,
                              hipStream_t stream);

/* ---- paged cache ----------------------------------------------------------------
 *
 * The layers between the recurrent ones that attend to every position keep
 * their keys and values: writing a paged cache (as it is or in 8 bits), reading
 * it back, and the attention of new tokens over it, from one token a sequence
 * to whole prompts.  The sequences, token rows, row strides, overlaps and
 * streams follow the mixer operators' conventions; results are deterministic.
 *
 * A sequence has seq_lens[i] positions, its new tokens among them: token t of n
 * is at position seq_lens[i] - n + t.  Position j is row j % page_size of page
 * block_table[i][j / page_size].  A position below zero, and one whose page is
 * outside [0, pages), is not there: it is not written, reads as zeros, and no
 * token attends to it.  seq_lens outside [0, blocks * page_size] are clamped to
 * it.  Pages may be shared by sequences that read them; two tokens of one
 * write must not name the same row (which of them it then holds, and whether
 * its scale is that one's, is not defined).
 *
 * 8-bit caches hold a row (one position's head_dim values of one head) as codes
 * and the exponent of one power of two: code * 2^(byte - 127), with the least
 * power from 2^-117 that takes the row's largest magnitude to 448 (e4m3) or 127
 * (int8), codes rounded to nearest even.  Byte 255 stands for NaN: a row with a
 * NaN or an infinity gets it, with codes 0.  Every value that is held is exact
 * in bf16.  Magnitudes of 2^127 and more may round up to infinity.
 */
typedef enum kda_kv_dtype {
    KDA_KV_F32 = 0,
    KDA_KV_BF16 = 1,
    KDA_KV_E4M3 = 2,                /* OCP e4m3: no infinities, largest 448 */
    KDA_KV_I8 = 3,
    KDA_KV_RANGE_MIN_ = -2147483647 - 1,    /* never valid, as in kda_dtype */
    KDA_KV_RANGE_MAX_ = 2147483647
} kda_kv_dtype;

/*
 *   k, v : [pages, heads, page_size, head_dim] dt, pages k_page_stride and
 *          v_page_stride elements apart (views of one buffer of both are fine);
 *          16-byte aligned, strides multiples of 16 bytes and at most 2^40
 *   k_scale, v_scale : [pages, heads, page_size] bytes, 16-byte aligned, exactly
 *          where dt has 8 bits; else NULL
 *   block_table : DEVICE int32 [N, blocks], rows block_table_stride apart
 *   seq_lens : DEVICE int32 [N]
 *   head_dim in {64, 128}; page_size in {16, 32, 64, 128, 256}; blocks *
 *   page_size at most 2^30: others are KDA_ERR_UNSUPPORTED, as is a dt that is
 *   neither the tokens' own nor one of 8 bits
 */
typedef struct kda_paged_cache {
    kda_kv_dtype dt;
    int pages, heads, page_size, head_dim, blocks;
    void* k;
    void* v;
    long long k_page_stride, v_page_stride;
    unsigned char* k_scale;
    unsigned char* v_scale;
    const int* block_table;
    long long block_table_stride;
    const int* seq_lens;
} kda_paged_cache;

/*
 * Writes the new tokens' keys and values to their positions.
 *   k, v : [tokens, heads, head_dim] dt, row strides k_stride, v_stride;
 *          16-byte aligned, strides multiples of 16 bytes
 */
kda_status kda_kv_cache_write(int N, const int* cu_seqlens, int T, kda_dtype dt, const void* k, long long k_stride,
                              const void* v, long long v_stride, const kda_paged_cache* cache, hipStream_t stream);

/*
 * Reads the last positions of every sequence (a sequence of n token rows: its
 * last n positions) back into k, v [tokens, heads, head_dim] dt, contiguous and
 * 16-byte aligned.
 */
kda_status kda_kv_cache_read(int N, const int* cu_seqlens, int T, kda_dtype dt, void* k, void* v,
                             const kda_paged_cache* cache, hipStream_t stream);

/*
 * Attention of the new tokens over the cache, which holds them already:
 *
 *   o_t[h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q_t[h] . k_j),
 *   over the positions j up to the token's own, k and v of cache head
 *   h / (H / heads);  times sigmoid(gate_t[h]) with a gate
 *
 *   q    : [tokens, H, head_dim] dt, row stride q_stride; heads divides H
 *   gate : [tokens, H, head_dim] dt or NULL, row stride gate_stride
 *   o    : [tokens, H, head_dim] dt, contiguous; a token with no position to
 *          attend to gets zeros
 *   scale: above zero, scale log2(e) finite; where it takes a finite q.k out of
 *          fp32's range, that token's output is not defined
 *   workspace : kda_paged_attn_workspace_size(...) bytes
 * q, gate, o and workspace 16-byte aligned, strides multiples of 16 bytes.
 * What is at positions that a token does not attend to (behind it, or not
 * there) does not reach it, NaN and infinities included; an infinite value at a
 * position that it does attend to makes its sum that infinity (NaN beside a NaN
 * or the other infinity, and maybe under a weight below 2^-126).  A token whose
 * scores are all -infinity is as one without a position.  bf16: scores, maxima
 * and sums are fp32; weights are rounded to bf16 for their product with v, so o
 * is off by its own rounding and 2^-8 of the weighted mean of |v|; where a batch
 * has up to 16 rows (tokens times H / heads) a sequence on average, they go into
 * it as two bf16, and o is off by its own rounding and 2^-16 of that mean.
 */
size_t kda_paged_attn_workspace_size(int N, int packed, int T, int H, kda_dtype dt, const kda_paged_cache* cache);
kda_status kda_paged_attn(int N, const int* cu_seqlens, int T, int H, kda_dtype dt, float scale, const void* q,
                          long long q_stride, const void* gate, long long gate_stride, void* o,
                          const kda_paged_cache* cache, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Optional per-launch timing, for benchmarks and tracing.  After
 * kda_profile_start(max_launches), each kernel launched by the library
 * (up to max_launches of them) is bracketed by two HIP
 * events recorded on its own stream; launches beyond that are not timed.
 * kda_profile_stop waits for the recorded events, writes up to `cap` launch
 * names (static strings: "intra_chunk", "state_output", "state_summary",
 * "chunk_output", "chunk_summary", "segment_scan", "copy_state",
 * "varlen_prep", "decode_step", "decode_steps", "backward"; the chunk-form
 * backward's "bwd_intra_chunk", "bwd_state_summary", "bwd_segment_scan",
 * "bwd_states", "bwd_reverse_summary", "bwd_reverse_scan", "bwd_state_reverse",
 * "bwd_value_side", "bwd_solve", "bwd_gated"; the mixer operators'
 * "short_conv", "short_conv_bwd", "short_conv_bwd_sums", "short_conv_step",
 * "scan_prep", "scan_gates", "scan_summary", "scan_combine", "scan_output", "scan_final", "scan_step",
 * "scan_bwd_summary", "scan_bwd_combine", "scan_bwd_states", "scan_bwd_grads",
 * "scan_bwd_join", "scan_bwd_sums",
 * "group_norm", "group_norm_bwd", "group_norm_bwd_sums"; the paged cache's
 * "cache_write", "cache_read", "attn_step", "attn_chunk", "attn_f32",
 * "attn_join") and durations in milliseconds, releases the
 * events, and returns the number of timed launches (-1: profiling was not
 * started or a HIP event query failed).  The record is process-wide (the one
 * piece of state the library keeps, opt-in): launches from several threads
 * while it is on are each recorded whole (a mutex guards it), in the order
 * they took their slots.  Profiling is off unless started.
 * kda_profile_start returns KDA_ERR_INVALID_ARG for max_launches outside
 * [1, 2^20] and KDA_ERR_HIP if an event cannot be created.
 */
kda_status kda_profile_start(int max_launches);
int kda_profile_stop(const char** names, float* ms, int cap);

/* Static description of a status code. */
const char* kda_status_string(kda_status s);

/* Library version string. */
const char* kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
