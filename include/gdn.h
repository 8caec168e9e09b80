/*
 * gdn.h -- C ABI of the GB300 GatedDeltaNet record / replay library (libgdn.so).
 *
 * The library runs the gated delta-rule recurrence step with innovation-tape
 * capture ("record"), the speculative-decode rollback that re-folds an
 * accepted tape prefix onto a state snapshot ("replay"), and the tiled GQA
 * head broadcast ("repeat"), as hand-written sm_103a CUDA kernels.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every tensor argument is a pointer to caller-owned, densely packed,
 *   row-major DEVICE memory (any pointer the CUDA runtime can dereference
 *   from a kernel).  The library never allocates, frees, copies to the host
 *   or synchronises: it validates its arguments on the host, enqueues one
 *   kernel on `stream` (gdn_chunk_prefill: two) and returns.  Results are
 *   ready when the stream has reached that point.
 * - `stream` is a cudaStream_t (the typedef below is the same type);
 *   NULL means the legacy default stream.
 * - Kernels are enqueued as programmatic dependent launches: a kernel may
 *   be scheduled while the kernel before it on the stream is still running,
 *   but it reads and writes no global memory until that kernel has
 *   completed and its writes are visible, so the stream order of every
 *   memory access is that of ordinary launches (a kernel of the caller's
 *   between two calls is waited for as usual).
 * - Dimensions are int64_t and must be > 0 (a zero or negative dimension is
 *   GDN_ERR_INVALID_ARGUMENT, the rule the tiled-repeat page applies to its
 *   own shapes).
 * - Validation happens before any launch.  A non-GDN_OK status means nothing
 *   was enqueued, except GDN_ERR_CUDA, which reports a failed launch.
 *   gdn_last_error() returns a message for the last failure on the calling
 *   host thread.
 * - Floating-point tensors share one element type `dtype` (f32, bf16 or
 *   f16); the recurrent state is float32 (or `dtype` in the _tstate calls).
 *   The state and every step's scalars are float32 (see gdn_step_record for
 *   the bf16 tensor-core paths' split operands); values written in bf16/f16
 *   are rounded to nearest-even.
 *
 * Notation: B batch, T timesteps, Hk key heads, Hv value heads (Hv % Hk == 0,
 * G = Hv / Hk, key head of value head hv is hk = hv / G), Dk key dim, Dv
 * value dim.  The source page for record and replay is "metaltile-std 0.1.0
 * -- src/ffai/gated_delta_replay.rs" (module doc, kernels
 * gated_delta_step_record and state_replay); the source page for the repeat
 * is "mlx-native 0.6.5 -- ops/repeat_tiled.rs" (module doc "Mapping",
 * dispatch_repeat_tiled_f32).
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 7

/* Same type as cudaStream_t. */
typedef struct CUstream_st *gdn_stream_t;

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARGUMENT = 1, /* bad shape, null pointer, overflow, overlap  */
    GDN_ERR_UNSUPPORTED = 2,      /* dtype or Dk outside the compiled set        */
    GDN_ERR_MISALIGNED = 3,       /* a pointer breaks its alignment requirement  */
    GDN_ERR_CUDA = 4              /* the CUDA runtime rejected the launch        */
} gdn_status;

typedef enum gdn_dtype {
    GDN_DTYPE_F32 = 0,
    GDN_DTYPE_BF16 = 1,
    GDN_DTYPE_F16 = 2
} gdn_dtype;

/* Which key head a value head reads (G = Hv / Hk). */
typedef enum gdn_gqa_mapping {
    GDN_GQA_BLOCK = 0, /* hk = hv / G: the record kernel's own rule             */
    GDN_GQA_TILED = 1  /* hk = hv % Hk: the head order of the tiled repeat
                          ("mlx-native repeat_tiled.rs", module doc "Mapping"),
                          read in place instead of materialised             */
} gdn_gqa_mapping;

/*
 * gdn_step_record -- T recurrence steps with delta-tape capture
 * (page: gated_delta_step_record; tape layout: module doc).
 *
 * For every state row s = state[b,hv,dv,:] (float32, Dk entries) and every
 * step t in 0..T-1 whose mask is on:
 *     s        <- g[b,t,hv] * s
 *     kv        = s . k[b,t,hk,:]
 *     delta     = (v[b,t,hv,dv] - kv) * beta[b,t,hv]
 *     delta_log[b,t,hv,dv] = delta
 *     s        <- s + k[b,t,hk,:] * delta
 *     y[b,t,hv,dv] = s . q[b,t,hk,:]
 * and state_out[b,hv,dv,:] = s after the last step.
 *
 * Arguments (shape, element type, alignment):
 *   q, k       [B,T,Hk,Dk]  dtype, 16-byte aligned
 *   v          [B,T,Hv,Dv]  dtype
 *   g, beta    [B,T,Hv]     dtype (g is a multiplicative decay, not a log)
 *   state_in   [B,Hv,Dv,Dk] float32, 16-byte aligned (the snapshot)
 *   mask       [B,T] uint32 or NULL.  NULL: every step is on.  A step with
 *              mask 0 is skipped: the state is unchanged and y, delta_log,
 *              k_log, g_log at (b,t) are NOT written (they keep whatever the
 *              caller put there).  Any nonzero value means on.
 *   y          [B,T,Hv,Dv]  dtype (output)
 *   state_out  [B,Hv,Dv,Dk] float32, 16-byte aligned (output).  May be the
 *              same pointer as state_in (in place); any other overlap with
 *              state_in is GDN_ERR_INVALID_ARGUMENT.
 *   delta_log  [B,T,Hv,Dv]  dtype (output, the innovation tape)
 *   k_log      [B,T,Hv,Dk]  dtype or NULL, 16-byte aligned (output): k
 *              expanded to value heads, k_log[b,t,hv,:] = k[b,t,hv/G,:],
 *              written where delta_log is
 *   g_log      [B,T,Hv]     dtype or NULL (output): copy of g, written where
 *              delta_log is
 *   Dk         32, 64, 128, 192 or 256 (else GDN_ERR_UNSUPPORTED); Dv any > 0
 * Outputs must not overlap inputs (other than the in-place state).
 *
 * Kernels and precision.  The call picks one of three kernels; all keep the
 * state in float32 and take every step's scalars (the decay products, the
 * reciprocals, the innovation) in float32:
 *   - FP32 steps (f32 / f16 inputs; bf16 calls the two below do not take):
 *     every product in float32, one rounding per state entry per step.
 *   - bf16, 7 <= T <= 16, Dk = 128, Dv a multiple of 128, v 16-byte aligned,
 *     state in float32: the tcgen05 kernel (one 16-step chunk per call,
 *     TMA-fed, accumulators in tensor memory).
 *   - other bf16 calls with T >= 12 and Dk of 64 or 128: mma.sync 16-step
 *     chunks.
 * The two tensor-core forms regroup a chunk's steps into products in which
 * the f32 state and the f32 per-row solve values enter as two bf16 terms
 * (hi + lo, 16 significant bits) against the exact bf16 k and q rows, with
 * f32 accumulation: each such product carries a relative error of about
 * 2^-17, well inside the 1e-3 that bf16 inputs are held to, but the results
 * are not bit-identical to the FP32-step kernel (and a bf16 tape is rounded
 * in either case).  The tcgen05 kernel solves each row's chunk in FP32.
 * Every kernel is deterministic run to run.
 */
gdn_status gdn_step_record(const void *q, const void *k, const void *v,
                           const void *g, const void *beta,
                           const float *state_in, const uint32_t *mask,
                           void *y, float *state_out, void *delta_log,
                           void *k_log, void *g_log,
                           int64_t B, int64_t T, int64_t Hk, int64_t Hv,
                           int64_t Dk, int64_t Dv, gdn_dtype dtype,
                           gdn_stream_t stream);

/*
 * gdn_step_record_mapped -- gdn_step_record with a choice of GQA mapping.
 *
 * Identical to gdn_step_record (same arguments, layouts, errors) except that
 * the key head of value head hv is chosen by `mapping`:
 *   GDN_GQA_BLOCK  hk = hv / (Hv/Hk)  (gdn_step_record itself)
 *   GDN_GQA_TILED  hk = hv % Hk       (the result equals gqa_repeat_tiled of
 *                  q and k to Hv heads followed by gdn_step_record with
 *                  Hk = Hv, without the expanded copies)
 * k_log, when given, receives k[b,t,hk,:] under the same mapping.  An
 * unknown mapping value is GDN_ERR_INVALID_ARGUMENT.
 */
gdn_status gdn_step_record_mapped(const void *q, const void *k, const void *v,
                                  const void *g, const void *beta,
                                  const float *state_in, const uint32_t *mask,
                                  void *y, float *state_out, void *delta_log,
                                  void *k_log, void *g_log,
                                  int64_t B, int64_t T, int64_t Hk, int64_t Hv,
                                  int64_t Dk, int64_t Dv, gdn_gqa_mapping mapping,
                                  gdn_dtype dtype, gdn_stream_t stream);

/*
 * gdn_step_record_tstate / gdn_state_replay_tstate -- record and replay with
 * the state stored in the input element type ("state in T", as the page's
 * kernels keep it) instead of float32.
 *
 * state_in / state_out are [B,Hv,Dv,Dk] in `dtype` (16-byte aligned).  The
 * state is widened exactly on load, every step runs in float32 as in
 * gdn_step_record, and the final state is rounded to nearest-even once on
 * store.  With dtype = GDN_DTYPE_F32 these are gdn_step_record_mapped and
 * gdn_state_replay (or _per_seq) exactly.  Everything else -- arguments,
 * layouts, mask rule, tape, errors -- is as documented for those calls;
 * gdn_state_replay_tstate takes the per-sequence counts of
 * gdn_state_replay_per_seq when accepted_per_seq is non-NULL (then
 * `accepted` is only checked to be >= 0), else the single count `accepted`.
 */
gdn_status gdn_step_record_tstate(const void *q, const void *k, const void *v,
                                  const void *g, const void *beta,
                                  const void *state_in, const uint32_t *mask,
                                  void *y, void *state_out, void *delta_log,
                                  void *k_log, void *g_log,
                                  int64_t B, int64_t T, int64_t Hk, int64_t Hv,
                                  int64_t Dk, int64_t Dv, gdn_gqa_mapping mapping,
                                  gdn_dtype dtype, gdn_stream_t stream);

gdn_status gdn_state_replay_tstate(const void *delta_log, const void *k_log,
                                   const void *g_log, const void *state_in,
                                   const uint32_t *mask, void *state_out,
                                   int64_t B, int64_t T, int64_t Hv, int64_t Dk,
                                   int64_t Dv, int64_t accepted,
                                   const int32_t *accepted_per_seq,
                                   gdn_dtype dtype, gdn_stream_t stream);

/*
 * gdn_chunk_prefill -- the record recurrence for long calls, computed in
 * chunks of 16 steps on the tensor cores.
 *
 * Same mathematics, arguments, layouts, mask rule and errors as
 * gdn_step_record_mapped, with these differences:
 *   - delta_log, k_log and g_log are optional (NULL: not written); y and
 *     state_out are required.
 *   - The chunk form re-associates the sums of the step form (the pages give
 *     only the step form; the chunk form follows from it algebraically), so
 *     results agree with the step form to float32 rounding, not bit for bit:
 *     replaying its tape reproduces state_out to rounding, where a float32
 *     tape of gdn_step_record replays exactly.
 *   - It needs a caller-owned DEVICE workspace of at least
 *     gdn_chunk_prefill_workspace_size(B, T, Hv) bytes, 16-byte aligned
 *     (too small or NULL: GDN_ERR_INVALID_ARGUMENT).  Its contents on entry
 *     and exit are irrelevant to the caller; two calls in flight at once
 *     need two workspaces.
 * It enqueues two kernels on `stream` (the chunk-local matrices, then the
 * sequential scan over chunks).
 */
size_t gdn_chunk_prefill_workspace_size(int64_t B, int64_t T, int64_t Hv);

gdn_status gdn_chunk_prefill(const void *q, const void *k, const void *v,
                             const void *g, const void *beta,
                             const float *state_in, const uint32_t *mask,
                             void *y, float *state_out, void *delta_log,
                             void *k_log, void *g_log,
                             int64_t B, int64_t T, int64_t Hk, int64_t Hv,
                             int64_t Dk, int64_t Dv, gdn_gqa_mapping mapping,
                             void *workspace, size_t workspace_bytes,
                             gdn_dtype dtype, gdn_stream_t stream);

/*
 * gdn_chunk_prefill_noalloc -- gdn_chunk_prefill without a caller workspace.
 *
 * The source pages have no counterpart to this entry point.  It is for
 * callers that cannot allocate device memory when they call: an inference
 * runtime that hands its whole HBM budget to its own pool allocator at start
 * and forbids allocations afterwards, a plugin or script host that receives
 * tensors but has no handle on the allocator that made them, or a serving
 * loop with a latency budget in which cudaMalloc (which may synchronise the
 * device) is not allowed.
 *
 * The workspace is a file-scope device array of 32 MiB inside the library (a
 * static __device__ object): every GPU on which the library's device code is
 * loaded holds those 32 MiB until the process exits, and no call allocates,
 * frees or synchronises anything.  Each call looks up the array's device
 * address for the current device (cudaGetSymbolAddress); the first call on a
 * device may also load the library's device code there, so make that first
 * call before any stream capture begins.  Problems whose workspace
 * (gdn_chunk_prefill_workspace_size) exceeds 32 MiB return
 * GDN_ERR_UNSUPPORTED before anything is launched.
 *
 * All calls on one device share the array, and each call leaves its contents
 * behind; a call writes every workspace entry it reads before reading it, so
 * nothing needs clearing between calls.  Calls whose kernels overlap in time
 * on one device race on the array and give wrong results: issue them on one
 * stream (or use gdn_chunk_prefill with a workspace per stream).  Results are
 * identical, bit for bit, to gdn_chunk_prefill with the same arguments; every
 * other argument, rule and error is as documented there.
 */
gdn_status gdn_chunk_prefill_noalloc(const void *q, const void *k, const void *v,
                                     const void *g, const void *beta,
                                     const float *state_in, const uint32_t *mask,
                                     void *y, float *state_out, void *delta_log,
                                     void *k_log, void *g_log,
                                     int64_t B, int64_t T, int64_t Hk, int64_t Hv,
                                     int64_t Dk, int64_t Dv, gdn_gqa_mapping mapping,
                                     gdn_dtype dtype, gdn_stream_t stream);

/*
 * gdn_state_replay -- rebuild the state after an accepted prefix of the tape
 * (page: state_replay; module doc: "re-folds the accepted prefix").
 *
 * For every state row and t in 0..T-1:
 *     do_step = (t < accepted) && (mask == NULL || mask[b,t] != 0)
 *     s <- do_step ? s * g_log[b,t,hv] + k_log[b,t,hv,:] * delta_log[b,t,hv,dv] : s
 * The select is a true select: tape slots of skipped steps are never read,
 * so they may hold anything (NaN, stale data).
 *
 *   delta_log  [B,T,Hv,Dv]  dtype
 *   k_log      [B,T,Hv,Dk]  dtype, 16-byte aligned (key rows expanded to value heads)
 *   g_log      [B,T,Hv]     dtype
 *   state_in   [B,Hv,Dv,Dk] float32, 16-byte aligned (the pre-record snapshot)
 *   mask       [B,T] uint32 or NULL (the mask record was given)
 *   state_out  [B,Hv,Dv,Dk] float32, 16-byte aligned; may equal state_in
 *   accepted   >= 0; values above T act as T; 0 copies state_in to state_out
 *
 * With a float32 tape written by gdn_step_record from the same snapshot and
 * mask, replay with accepted >= T reproduces record's state_out bit for bit,
 * and replay with accepted = a reproduces a record over the first a steps.
 *
 * Kernels: calls folding 2 to 16 steps with Dk = 128, a float32 state and
 * 16-byte aligned delta_log rows (base aligned, Dv * element size a multiple
 * of 16) run on a persistent kernel that streams 64-row state blocks and the
 * tape rows by TMA (one CTA per SM); the others on the FP32 kernel (one CTA
 * per 64-row block).  Both apply the same f32 operations in the same order,
 * so their results are bit-identical.  The persistent kernel's waits are
 * bounded as described at gdn_wait_status.  Past a fixed first share per
 * CTA, the persistent kernel hands its blocks out from a counter in library
 * memory, one of 256 slots taken round robin per launch and reset by the
 * launch itself; two launches that run at the same time must not share a
 * slot, so at most 255 other launches of this kernel may be in flight
 * alongside one (on any streams), and one captured graph that contains it
 * must not be instantiated twice and run concurrently.
 */
gdn_status gdn_state_replay(const void *delta_log, const void *k_log,
                            const void *g_log, const float *state_in,
                            const uint32_t *mask, float *state_out,
                            int64_t B, int64_t T, int64_t Hv, int64_t Dk,
                            int64_t Dv, int64_t accepted, gdn_dtype dtype,
                            gdn_stream_t stream);

/*
 * gdn_state_replay_per_seq -- gdn_state_replay with one accepted count per
 * sequence (speculative decoding accepts a different draft prefix in every
 * sequence of the batch; the page's kernel takes one count per dispatch).
 *
 *   accepted   [B] int32, DEVICE memory, 4-byte aligned, non-NULL.  Sequence
 *              b folds the steps t < accepted[b] whose mask is on; an entry
 *              < 0 acts as 0 (the sequence's state_out is its snapshot) and
 *              an entry > T acts as T.  Read by the kernel, so it may be
 *              produced by earlier work on the same stream.
 * Every other argument, layout and error is as for gdn_state_replay.  With
 * the same tape, sequence b's result equals gdn_state_replay with
 * accepted = accepted[b] (bit for bit).
 */
gdn_status gdn_state_replay_per_seq(const void *delta_log, const void *k_log,
                                    const void *g_log, const float *state_in,
                                    const uint32_t *mask, float *state_out,
                                    int64_t B, int64_t T, int64_t Hv, int64_t Dk,
                                    int64_t Dv, const int32_t *accepted,
                                    gdn_dtype dtype, gdn_stream_t stream);

/*
 * gdn_chunk_replay -- gdn_state_replay for long accepted prefixes, as one
 * tensor-core contraction.
 *
 * The replay fold is linear in the state and its updates do not read the
 * state, so it closes to
 *     s_out = Gam s_in + sum_t w_t delta_t k_t
 * over the folded steps t (t < accepted, mask on), with w_t the product of
 * g_log over the folded steps after t and Gam the product over all of them.
 * The library forms w and Gam, then runs the sum for every (b, hv) tile as a
 * (Dv x T) by (T x Dk) product on the tensor cores (tcgen05, tf32 operands
 * split into high and low parts, float32 accumulation).  Results agree with
 * gdn_state_replay to float32 rounding, not bit for bit; results are
 * run-to-run deterministic.
 *
 * Arguments, layouts and errors are those of gdn_state_replay, plus:
 *   accepted_per_seq  [B] int32 (device) or NULL: when given, sequence b folds
 *                     the steps t < accepted_per_seq[b] (entries < 0 act as 0,
 *                     > T as T) and `accepted` is only checked to be >= 0
 *   workspace         caller-owned device memory of at least
 *                     gdn_chunk_replay_workspace_size(B, T, Hv, Dk, Dv) bytes,
 *                     16-byte aligned; one workspace per call in flight
 * Only state_in, state_out and workspace need 16-byte alignment here.  It
 * enqueues two or three kernels on `stream` (the decay weights, the
 * contraction, and a fixed-order sum of partial results when the steps are
 * split over several CTAs per tile).
 */
size_t gdn_chunk_replay_workspace_size(int64_t B, int64_t T, int64_t Hv, int64_t Dk,
                                       int64_t Dv);

gdn_status gdn_chunk_replay(const void *delta_log, const void *k_log,
                            const void *g_log, const float *state_in,
                            const uint32_t *mask, float *state_out,
                            int64_t B, int64_t T, int64_t Hv, int64_t Dk,
                            int64_t Dv, int64_t accepted,
                            const int32_t *accepted_per_seq, void *workspace,
                            size_t workspace_bytes, gdn_dtype dtype,
                            gdn_stream_t stream);

/*
 * gqa_repeat_tiled -- tiled GQA broadcast (page: repeat_tiled.rs, "Mapping"):
 *     dst[t, hh, x] = src[t, hh % hg, x],  src [seq,hg,k] -> dst [seq,h,k]
 * A bit-exact copy.  Errors follow dispatch_repeat_tiled_f32: any dimension
 * <= 0, h % hg != 0, an element count or byte size that overflows, or
 * src_bytes / dst_bytes smaller than the shapes need ->
 * GDN_ERR_INVALID_ARGUMENT.  Any dtype of the enum is accepted; pointers
 * need only the element alignment (16-byte alignment with k * elemsize a
 * multiple of 16 takes the vector path).  src and dst must not overlap.
 */
gdn_status gqa_repeat_tiled(const void *src, void *dst,
                            int64_t seq, int64_t hg, int64_t h, int64_t k,
                            gdn_dtype dtype, size_t src_bytes, size_t dst_bytes,
                            gdn_stream_t stream);

/*
 * The operators around the recurrence.  A recurrent layer takes its
 * projections through gdn_causal_conv, runs a recurrence (gdn_step_record, or
 * gdn_selective_scan for layers of the state space family), normalises the
 * result with gdn_gated_norm; gdn_sample draws the tokens whose matches with
 * a draft are the `accepted` counts of the replay calls.  The conventions
 * above hold, and:
 *   - Inputs that a layer has as slices of a wider projection may have
 *     strides (in elements) on their outer dimensions, in either order; the
 *     inner dimensions are dense.  Strides that let rows overlap are
 *     GDN_ERR_INVALID_ARGUMENT.
 *   - `lengths` ([B] int32, DEVICE memory, or NULL for T) is the number of
 *     steps that a sequence has; an entry < 0 acts as 0, an entry > T as T.
 *     Steps at or past it change nothing: y is not written there, and their
 *     inputs are not used.  To roll a sequence back to an accepted prefix,
 *     repeat the call from the state before it with lengths = accepted (y may
 *     be NULL).
 *   - Pointers need the alignment of their element type unless 16 bytes are
 *     asked for; 16-byte aligned rows take the vector paths.
 *   - An output must not overlap an input, except where a call says so.
 *   - silu, the decays of the scan's tensor-core form and sampling's
 *     exponentials use the hardware's approximate float32 functions: silu(v) is
 *     within 8 + 2 |v| units (2^-24) of its value, a logprob within 2e-5 and 4
 *     units of its own.  The cut by min_p and the race compare exact float32
 *     exponentials.
 */
typedef enum gdn_activation { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1 } gdn_activation;

/*
 * gdn_causal_conv -- depthwise causal convolution of W taps with its state.
 *     y[b,t,c] = act(bias[c] + sum_j weight[c,j] * in[b, t-W+1+j, c])
 * where in[b,t] is x[b,t] for t >= 0 and state_in[b, W-1+t] for t < 0.
 *
 *   x          [B,T,C] dtype, strides x_stride_b, x_stride_t, 1
 *   weight     [C,W] dtype, tap W-1 on the current step; W from 2 to 8 (else
 *              GDN_ERR_UNSUPPORTED)
 *   bias       [C] dtype or NULL
 *   state_in   [B,W-1,C] dtype, the last W-1 inputs, oldest first, or NULL
 *              (zeros: the start of a sequence)
 *   lengths    [B] int32 or NULL
 *   y          [B,T,C] dtype or NULL (only the state is wanted)
 *   state_out  [B,W-1,C] dtype or NULL: the last W-1 inputs after the call, a
 *              bit-exact copy; may be state_in's own buffer
 * Sums are float32, rounded once.  One kernel.
 */
gdn_status gdn_causal_conv(const void *x, const void *weight, const void *bias,
                           const void *state_in, const int32_t *lengths,
                           void *y, void *state_out,
                           int64_t B, int64_t T, int64_t C, int64_t W,
                           int64_t x_stride_b, int64_t x_stride_t,
                           gdn_activation activation, gdn_dtype dtype,
                           gdn_stream_t stream);

/*
 * gdn_selective_scan -- the selective state space scan with one decay per
 * head and step.  For every state row s = state[b,h,p,:] (N entries), with
 * g = h / (H/G) and every step t < lengths[b]:
 *     dl  = softplus(dt[b,t,h] + dt_bias[h])      (softplus = 0: without it)
 *     s   <- exp(dl * A[h]) * s + (dl * x[b,t,h,p]) * B[b,t,g,:]
 *     y[b,t,h,p] = s . C[b,t,g,:] + D[h] * x[b,t,h,p]
 * and state_out[b,h,p,:] = s after the last step.
 *
 *   x          [B,T,H,P] dtype      dt       [B,T,H] dtype
 *   B, C       [B,T,G,N] dtype      A        [H] float32 (negative: a decay)
 *   D, dt_bias [H] float32 or NULL  lengths  [B] int32 or NULL
 *   state_in   [B,H,P,N] float32, 16-byte aligned, or NULL (zeros)
 *   y          [B,T,H,P] dtype or NULL (only the state is wanted)
 *   state_out  [B,H,P,N] float32, 16-byte aligned, or NULL; may be
 *              state_in's own buffer
 *   N          16, 32, 64, 128 or 256 (else GDN_ERR_UNSUPPORTED); P any > 0
 *   strides    batch and step strides of x, dt, B and C, or NULL (dense)
 *   workspace  at least gdn_selective_scan_workspace_size bytes, 16-byte
 *              aligned; not looked at when that call gives 16
 * The state and all sums are float32 and results do not change from run to
 * run.  bf16 calls of 32 steps or more with N of 64 or 128, P a multiple of 8
 * and 16-byte aligned rows take 32 steps at a time on the tensor cores: the
 * state stays as accurate as float32, the part of y that comes through the
 * state from before those steps is off by 2^-17 of its terms at most before y
 * is rounded (2^-16 in a call that is split along its steps), and an infinity
 * or NaN among a sequence's inputs may show in y from the start of its
 * 32 steps on.  One kernel, or three where a long call is split along its
 * steps.
 */
typedef struct gdn_scan_strides {
    int64_t x_b, x_t, dt_b, dt_t, B_b, B_t, C_b, C_t;
} gdn_scan_strides;

size_t gdn_selective_scan_workspace_size(int64_t B, int64_t T, int64_t H, int64_t P,
                                         int64_t N);

gdn_status gdn_selective_scan(const void *x, const void *dt, const float *A,
                              const void *Bm, const void *Cm, const float *D,
                              const float *dt_bias, const float *state_in,
                              const int32_t *lengths, void *y, float *state_out,
                              int64_t B, int64_t T, int64_t H, int64_t P,
                              int64_t G, int64_t N,
                              const gdn_scan_strides *strides, int softplus,
                              void *workspace, size_t workspace_bytes,
                              gdn_dtype dtype, gdn_stream_t stream);

/*
 * gdn_gated_norm -- root-mean-square norm with a gate and a residual sum.
 * For every token m and head k, over D entries:
 *     u = x                       (gate_first: u = x * silu(gate))
 *     u = residual + residual_scale * u      (with a residual)
 *     residual_out = u
 *     y = u / sqrt(mean(u^2) + eps) * weight (gate, not first: * silu(gate))
 * The norm takes u in float32, before it is rounded to residual_out.
 *
 *   x             [M,K,D] dtype, token stride x_stride_m
 *   gate          [M,K,D] dtype, token stride gate_stride_m, or NULL
 *   weight        [weight_rows,D] dtype; weight_rows is 1 (shared by the
 *                 heads) or K
 *   residual      [M,K,D] dtype or NULL; residual_out with it, else NULL
 *   y             [M,K,D] dtype
 * y and residual_out may each be the dense buffer of x, gate or residual.
 * One kernel.
 */
gdn_status gdn_gated_norm(const void *x, const void *weight, const void *gate,
                          const void *residual, void *y, void *residual_out,
                          int64_t M, int64_t K, int64_t D, int64_t x_stride_m,
                          int64_t gate_stride_m, int64_t weight_rows,
                          int gate_first, float residual_scale, float eps,
                          gdn_dtype dtype, gdn_stream_t stream);

/*
 * gdn_sample -- one token per row of logits, from given noise.
 *
 * With max the row's largest logit and e_i = exp((l_i - max) / temperature),
 * the tokens in the order (l descending, index ascending) are cut three
 * times, each time to a prefix that holds the first token at least:
 *     top_k  the first top_k tokens (<= 0 or >= V: all)
 *     top_p  a token stays while the mass of those before it is below top_p
 *            times the mass of the top_k tokens (>= 1: all)
 *     min_p  tokens with e_i >= min_p (<= 0: all)
 * token[r] is then the largest e_i / noise[r,i], ties to the lowest index:
 * with independent standard exponential noise, token i comes out with
 * probability e_i over the mass of the tokens that are left.  A temperature
 * of 0 or less takes the largest logit (lowest index), whatever the noise,
 * and 1 stands in its place for logprob.
 * logprob[r] = (l - max)/temperature - log(sum of e_i over the whole row).
 *
 *   logits   [R,V] dtype, row stride logits_stride; V at most 2^22.  A NaN
 *            counts as -inf (a masked token), +inf as the largest
 *            finite value of its type.
 *   noise    [R,V] float32, row stride noise_stride; > 0 (anything else
 *            counts as the smallest normal float)
 *   temperature, top_k, top_p, min_p  [R] DEVICE memory, or NULL: then the
 *            *_all value holds for every row
 *   token    [R] int32; -1 in a row whose logits are all -inf
 *   logprob  [R] float32 or NULL; -inf in such a row
 * Masses are summed as integers and ties are broken by index, so results do
 * not change from run to run.  One kernel.
 */
gdn_status gdn_sample(const void *logits, const float *noise,
                      const float *temperature, const int32_t *top_k,
                      const float *top_p, const float *min_p,
                      float temperature_all, int32_t top_k_all,
                      float top_p_all, float min_p_all,
                      int32_t *token, float *logprob, int64_t R, int64_t V,
                      int64_t logits_stride, int64_t noise_stride,
                      gdn_dtype dtype, gdn_stream_t stream);

/*
 * The operators of an attention layer.  A hybrid model puts attention layers
 * between its recurrent ones; their keys and values stay in pages of 4-bit
 * values.  In a serving step gdn_page_slots finds the pages and places of the
 * new tokens from the requests' lengths, gdn_rotary turns queries and keys,
 * gdn_kv_append writes keys and values to their places and gdn_kv_attention
 * reads them; gdn_kv_read gives them back.  The conventions above hold, and
 * those of the operators around the recurrence on strides, alignment and
 * overlap.
 *
 * The cache is [pages, H, page, 9 D/8] bytes for H key heads of D channels (D
 * of 64, 128 or 256, H at most 65535; page, the tokens of a page, of 16, 32, 64
 * or 128), 16-byte aligned.  Page and head make one block: the keys' codes [page, D/2] (element
 * 2i in the low half of byte i), the keys' scales [page, D/16], the values'
 * codes and the values' scales.  16 neighbouring channels of a token share a
 * scale s, an e4m3 byte; a code is e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and, in bit
 * 3, the sign), and an element's value is head scale * s * code, where the
 * float32 head scales k_scale[H] and v_scale[H] (finite, > 0; NULL: 1) keep s in
 * its range.  The cache holds finite values: an infinity is written as the
 * largest value (2688 head scales), a NaN as zero.
 *
 * Token j of sequence b stands in place j % page of page block_table[b, j /
 * page]; its slot is that page * page + j % page, an int32 (so pages * page
 * < 2^31).  A slot below 0 or past the last page is no slot: its token is not
 * written and not read.
 */

/*
 * gdn_page_slots -- block tables and slots of a step's tokens, from lengths.
 * Sequence b holds lengths[b] tokens in held[b] pages (more than it needs after
 * a rollback: to roll back, shorten its length), the first held[b] entries of
 * its row of block_table, and gets add[b] more:
 *     need[b] = max(0, ceil((lengths[b] + add[b]) / page) - held[b])
 * It is served if its row has room for them and need[b] is 0, or need[0] + ... +
 * need[b] (over sequences whose rows have room) is at most the number of free
 * pages; then granted[b] = add[b], and 0 if not.  add[b] < 0 ends the sequence:
 * its pages are free from the next call on, and its length is 0.
 *
 * Free pages stand in a ring of `pages` places, ring_state[1] of them from place
 * ring_state[0] on; pages are taken there in the order of the batch, and those
 * of ended sequences put behind the last one.
 *
 *   lengths, held   [B] int32         add        [B] int32 or NULL (T for each);
 *                                                above T counts as T
 *   ring_state      [2] int32         ring       [pages] int32, changed in place
 *   block_table     [B,width] int32, changed in place: entries held[b] on are
 *                   filled, no other is written
 *   slots           [B,T] int32: slot of token lengths[b] + t, -1 for t >=
 *                   granted[b] (and of an entry that names no page)
 *   positions       [B,T] int32: lengths[b] + t, -1 for t >= granted[b]
 *   granted         [B] int32: the `lengths` of the recurrent layers' calls, the
 *                   `fresh` of gdn_kv_attention
 *   lengths_out, held_out [B], ring_state_out [2]: after the call; each may be
 *                   its input's own buffer.  With other buffers a repeated call
 *                   gives the same results.
 * Counts that are negative or too large act as the nearest that is possible.
 * One kernel, two for more than 2048 slots.
 */
gdn_status gdn_page_slots(const int32_t *lengths, const int32_t *add,
                          const int32_t *held, const int32_t *ring_state,
                          int32_t *block_table, int32_t *ring, int32_t *slots,
                          int32_t *positions, int32_t *granted,
                          int32_t *lengths_out, int32_t *held_out,
                          int32_t *ring_state_out, int64_t B, int64_t T,
                          int64_t width, int64_t pages, int64_t page,
                          gdn_stream_t stream);

/* Which channels make a pair, i from 0 to R/2 - 1. */
typedef enum gdn_rotary_layout {
    GDN_ROTARY_HALF = 0,       /* i and i + R/2  */
    GDN_ROTARY_INTERLEAVED = 1 /* 2i and 2i + 1  */
} gdn_rotary_layout;

/* Batch and step strides, in elements. */
typedef struct gdn_rotary_strides {
    int64_t q_b, q_t, k_b, k_t, q_out_b, q_out_t, k_out_b, k_out_t;
} gdn_rotary_strides;

/*
 * gdn_rotary -- rotary positions of queries and keys: each pair (x, y) of the
 * first R channels of every head becomes
 *     scale * (x cos - y sin,  x sin + y cos),  angle = positions[b,t] * inv_freq[i]
 * and the channels from R on are copied.  `inverse` turns by minus the angles
 * (what a gradient takes).
 *
 *   q          [B,T,Hq,D] dtype      k  [B,T,Hk,D] dtype or NULL
 *   positions  [B,T] int32; a token with a negative one is left out: nothing of
 *              it is written
 *   inv_freq   [R/2] float32, R even, at most D and 8192 (above:
 *              GDN_ERR_UNSUPPORTED); frequencies stretched for long contexts
 *              are simply others, with their factor as `scale`
 *   q_out, k_out  like q and k; each may be its input's own rows (same pointer
 *              and strides), and the two may be slices of the same wider rows.
 *              Where one is in place, the other input is apart from it or
 *              another slice of the same rows
 *   strides    of the four, or NULL (dense)
 * An angle's fraction of a turn is exact to 2^-32 and 2^-53 of inv_freq per
 * step for every position; sines and products are float32, rounded once.  One
 * kernel.
 */
gdn_status gdn_rotary(const void *q, const void *k, const int32_t *positions,
                      const float *inv_freq, void *q_out, void *k_out,
                      int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                      int64_t R, const gdn_rotary_strides *strides,
                      gdn_rotary_layout layout, float scale, int inverse,
                      gdn_dtype dtype, gdn_stream_t stream);

/*
 * gdn_kv_append -- writes keys and values to their slots of the cache.  With
 * u = x / head scale (rounded to float32), each 16 channels get the scale s, the
 * nearest e4m3 of max|u| / 6 (at most 448), and each of them the nearest e2m1 of
 * u / s (at most 6); both of the exact quotient, ties to even.
 *
 *   k, v     [B,T,H,D] dtype, batch and step strides given
 *   slots    [B,T] int32; a slot may stand there once (of two tokens with the
 *            same slot, parts of either may be written)
 *   cache    in out; only the slots' bytes are written
 * One kernel.
 */
gdn_status gdn_kv_append(const void *k, const void *v, const int32_t *slots,
                         void *cache, const float *k_scale,
                         const float *v_scale, int64_t B, int64_t T, int64_t H,
                         int64_t D, int64_t page, int64_t pages,
                         int64_t k_stride_b, int64_t k_stride_t,
                         int64_t v_stride_b, int64_t v_stride_t,
                         gdn_dtype dtype, gdn_stream_t stream);

/*
 * gdn_kv_read -- the keys and values of N slots ([N] int32), as dense [N,H,D]
 * dtype: the float32 product, rounded to nearest-even.  The rows of a slot that is
 * none are not written.  One kernel.
 */
gdn_status gdn_kv_read(const void *cache, const int32_t *slots,
                       const float *k_scale, const float *v_scale, void *k,
                       void *v, int64_t N, int64_t H, int64_t D, int64_t page,
                       int64_t pages, gdn_dtype dtype, gdn_stream_t stream);

/*
 * gdn_kv_attention -- attention of new tokens over the cache.  Query token t of
 * sequence b (t < n, n = fresh[b]) stands at position p = lengths[b] - n + t and
 * sees the tokens j <= p with j > p - window (window 0: all of them):
 *     y[b,t,hq] = sum_j softmax_j(scale q . k_j) v_j,  key head hq / (Hq/H)
 *     lse[b,t,hq] = log sum_j exp(scale q . k_j)
 * A token that sees nothing (its position is below 0) has y = 0 and lse = -inf.
 *
 *   q            [B,T,Hq,D] dtype, batch and step strides given
 *   block_table  [B,width] int32; an entry that names no page takes its tokens
 *                out of sight
 *   lengths      [B] int32: the tokens in the cache, the new ones among them; at
 *                most width * page count
 *   fresh        [B] int32 or NULL (T): an entry < 0 acts as 0, > T as T.  y and
 *                lse are not written at or past it
 *   y            [B,T,Hq,D] dtype    lse [B,T,Hq] float32 or NULL
 *   workspace    at least gdn_kv_attention_workspace_size bytes, 16-byte
 *                aligned, one per call in flight; not looked at when that call
 *                gives 16
 * Scores (of less than 2^127), maxima and sums are float32, outputs are rounded
 * once.  What tensor cores cut off sums is at most 2^-12 of sum p |v| in f16
 * calls, 2^-9 in bf16 and 2^-22 in float32 calls, however many tokens there are.
 * The products take the cache's values exactly, the queries to 2^-23 of their
 * row's largest channel (if that is 2^-100 at least) and the probabilities
 * rounded to f16 (two f16 terms for float32 calls).  A query row that holds an
 * infinity or a NaN has NaN for y and lse if it sees a token.  What stands in
 * places that no token sees does not matter.  Results do not change from run to
 * run.  One kernel, or two where a call's tokens are shared out among blocks.
 */
size_t gdn_kv_attention_workspace_size(int64_t B, int64_t T, int64_t Hq,
                                       int64_t H, int64_t D);

gdn_status gdn_kv_attention(const void *q, const void *cache,
                            const int32_t *block_table, const int32_t *lengths,
                            const int32_t *fresh, const float *k_scale,
                            const float *v_scale, void *y, float *lse,
                            int64_t B, int64_t T, int64_t Hq, int64_t H,
                            int64_t D, int64_t width, int64_t page,
                            int64_t pages, int64_t q_stride_b,
                            int64_t q_stride_t, float scale, int64_t window,
                            void *workspace, size_t workspace_bytes,
                            gdn_dtype dtype, gdn_stream_t stream);

/* Static name of a status code ("GDN_OK", ...); never NULL. */
const char *gdn_status_string(gdn_status status);

/* Message for the last non-OK status returned on the calling host thread
 * ("" if none).  Valid until the next call from the same thread. */
const char *gdn_last_error(void);

/* GDN_ABI_VERSION of the loaded library. */
int gdn_abi_version(void);

/*
 * gdn_wait_status -- whether a bounded wait of a pipelined (TMA / tcgen05) kernel ran out.
 *
 * The pipelined paths (the tcgen05 record kernel behind gdn_step_record and
 * gdn_step_record_mapped, the persistent replay behind gdn_state_replay and
 * gdn_state_replay_per_seq, gdn_chunk_replay, and gdn_kv_attention's kernel for
 * many query rows) run stages that wait on
 * each other through mbarriers.  Every such wait gives up after a
 * bound (about a second of GPU clock by default) instead of hanging; the
 * kernel then writes NaN to the state or output rows it could not finish, lets its
 * copies and products in flight land, and raises a device-side flag.  The
 * call that launched it still returned GDN_OK (it only enqueues work), so a
 * caller that wants to know reads the flag here: *expired is set to 1 if any
 * kernel raised it since the last call, else 0, and the flag is cleared.
 * The read is a synchronous device-to-host copy: call it after synchronising
 * the streams that ran the calls.  The pages have no counterpart.
 */
gdn_status gdn_wait_status(int *expired);

/*
 * Testing hooks (the pages have no counterpart).
 *
 * gdn_set_wait_bound -- the bound, in GPU clock cycles, on the pipeline
 * waits of the pipelined kernels launched after this call (0 restores the
 * default of 2e9 cycles).  A bound far below a kernel's normal waiting time
 * makes its waits run out, which exercises the expiry path above without any
 * fault: the drain after a failed wait always uses the default bound.
 * Process-wide; not meant for production calls.
 *
 * gdn_inject_wait_expiry -- while on (nonzero), every pipelined kernel
 * launched takes, before its pipeline starts, one wait on a barrier that
 * nothing completes, so that its bound runs out deterministically (pair it
 * with a short gdn_set_wait_bound: with the default bound each such kernel
 * waits about a second).  0 turns it off.
 *
 * gdn_force_launch_failures -- the next n calls that pass their argument
 * checks return GDN_ERR_CUDA (with a gdn_last_error message) before touching
 * the device, so a caller's handling of launch failures can be tested.
 * Process-wide; 0 cancels.
 */
gdn_status gdn_set_wait_bound(int64_t cycles);
gdn_status gdn_inject_wait_expiry(int on);
gdn_status gdn_force_launch_failures(int n);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
