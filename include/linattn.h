/*
 * linattn.h -- C ABI of the GB300 (sm_103a) library for normalised causal
 * linear attention with a positive feature map and a recurrent S/z state.
 *
 * The method (sources cited by page title and section):
 *   [LA] "Linear attention：把历史写进状态" (hs-black.github.io/posts/linear-attention)
 *   [LC] "45. Linear Attention and Recurrent State | 线性注意力与递推状态" (datawhalechina, ch. 45)
 *
 *   phi(x)  = ELU(x) + 1  (x + 1 for x > 0, e^x otherwise)        [LA] "关键改写：让求和先发生"
 *   S_t     = alpha_t S_{t-1} + phi(k_t) v_t^T                     [LA] "公式里的每个维度",
 *   z_t     = alpha_t z_{t-1} + phi(k_t)                                "加一个门：让旧记忆逐渐淡出"
 *   y_t     = phi(q_t)^T S_t / (phi(q_t)^T z_t + eps)              [LA] "ε 是数值保护"
 * The state is updated before it is read, so y_t sees token t ([LA]
 * "每来一个 token，更新两个累加器"; [LC] TODO 3).  alpha_t == 1 is the ungated
 * form.  Prefill evaluates the recurrence chunk by chunk ([LA] "一个 chunk 的输出由
 * 两部分组成"); decode applies one step of it to a stored state ([LA]
 * "训练时，状态更新也能按块并行": the token recurrence suits decode).
 *
 * Conventions shared by every entry point:
 *  - Pointers marked "device" are CUDA device (or managed) memory owned by the
 *    caller; all arrays are dense, row-major and contiguous.  The library keeps
 *    no pointer after a call returns and allocates no device memory.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy default
 *    stream).  No call synchronises except la_last_device_status.
 *  - Errors are return codes.  Argument errors are detected on the host before
 *    anything is enqueued, and leave every output untouched.  LA_ERR_CUDA
 *    reports a failed launch or an earlier asynchronous CUDA error; kernels that
 *    give up waiting on an on-chip barrier record LA_ERR_TIMEOUT in a device
 *    status word that la_last_device_status reads.
 *  - Element types: q, k, v and y share `dtype` (BF16 or FP32).  States S, z and
 *    gates alpha are always FP32.  Arithmetic is FP32 with FP32 accumulation;
 *    on the BF16 path the features phi(q), phi(k) and the in-chunk score matrix
 *    enter the tensor cores as BF16.
 */
#ifndef LINATTN_H
#define LINATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *la_stream_t;

typedef enum {
    LA_OK = 0,
    LA_ERR_NULL = 1,        /* a required pointer is NULL                                      */
    LA_ERR_SHAPE = 2,       /* a size is < 1, out of range, or sizes disagree                    */
    LA_ERR_DTYPE = 3,       /* unknown element type                                            */
    LA_ERR_ALIGN = 4,       /* a pointer is not aligned as the chosen kernel requires           */
    LA_ERR_UNSUPPORTED = 5, /* a valid request that this build does not implement              */
    LA_ERR_CUDA = 6,        /* a CUDA runtime call or launch failed                            */
    LA_ERR_TIMEOUT = 7,     /* a kernel gave up waiting on an on-chip barrier                   */
    LA_ERR_WORKSPACE = 8    /* workspace NULL or smaller than the entry point needs             */
} la_status;

typedef enum { LA_DTYPE_BF16 = 0, LA_DTYPE_FP32 = 1 } la_dtype;

/*
 * la_state_init -- S = 0, z = 0 (the empty history; [LA] "每来一个 token，更新两个累加器":
 * the state starts from S0 = 0, z0 = 0; [LC] the zero-initialised state and normaliser).
 *   S  device, FP32 [B,H,r,dv]  (row i = feature index, column j = value index)
 *   z  device, FP32 [B,H,r]
 * Requires B, H, r, dv >= 1.  Errors: LA_ERR_NULL, LA_ERR_SHAPE, LA_ERR_CUDA.
 */
la_status la_state_init(float *S, float *z, int B, int H, int r, int dv, la_stream_t stream);

/*
 * la_prefill_workspace_bytes -- device scratch that la_prefill_chunked needs for
 * these sizes on the current device.  It is non-zero only for the BF16 path
 * when B*H*(dv/64) CTAs would leave at least half of the device's SMs idle and
 * T is long enough (>= 2048 tokens): the kernel then splits every sequence
 * into segments that run in parallel ([LA] "门控递推为什么能做并行 scan？": the
 * per-token updates are affine maps of the state, so a segment's map (the
 * product A of its gates and the state dS, dz it writes from a zero state)
 * can be computed first, scanned, and each segment started from its state).
 * The scratch holds A, dS, dz per segment part and every segment's start
 * state: FP32, about 66 KB per head per entry at r = dv = 128.  The answer
 * depends on the device's SM count: ask with the device current that will run
 * the call.  Returns 0 for sizes the BF16 path does not support.
 */
size_t la_prefill_workspace_bytes(int B, int H, int T, int r, int dv, int chunk);

/*
 * la_prefill_chunked -- run T tokens of every (b, h) sequence through the
 * recurrence, starting from (S0, z0), and return every output y_t and the final
 * state ([LA] "一个 chunk 的输出由两部分组成": per chunk, the read of the carried
 * state Q~c Sprev plus the masked in-chunk product [(Q~c K~c^T) . M] Vc, the same
 * two parts for the denominator, and the hand-off Snext, znext; with a gate, each
 * term is scaled by the product of the gates between its write and its read).
 *
 *   q, k   device [B,H,T,r]  dtype          v, y   device [B,H,T,dv]  dtype
 *   alpha  device FP32 [B,H,T], 0 <= alpha <= 1, or NULL for alpha == 1.
 *          alpha_t scales the state carried into token t (alpha of the first
 *          token scales S0, z0).
 *   S0     device FP32 [B,H,r,dv] or NULL (zero);  z0 device FP32 [B,H,r] or NULL.
 *          S0 may equal S_out and z0 may equal z_out (in-place continuation).
 *   S_out  device FP32 [B,H,r,dv] final state;  z_out device FP32 [B,H,r].
 *   eps    added once to the whole denominator: y = num / (den + eps).
 *   chunk  chunk length in tokens, >= 1.  The result does not depend on it
 *          beyond rounding ([LA] "动手实验": chunk boundaries do not change the
 *          semantics), so the BF16 kernel computes in chunks of 64 tokens
 *          whatever value is given; the FP32 path runs token by token.
 *   workspace, workspace_bytes: device scratch of at least
 *          la_prefill_workspace_bytes(...) bytes, 256-byte aligned, owned by the
 *          caller and not read after the call's kernels finish (may be NULL
 *          when that is 0).  Calls sharing one workspace must be ordered.
 *
 * Kernels:
 *   BF16: tensor-core kernel (tcgen05 MMAs with TMEM accumulators, TMA tile
 *         loads), chunks of 64 tokens.  Requires r == 128, dv in {64, 128}, q, k,
 *         v, y, S_out 16-byte aligned.  With a workspace (see above) three launches:
 *         the state pass, the scan of segment start states, and the chunk
 *         kernel over all segments at once.
 *   FP32: exact FP32 token recurrence on CUDA cores (chunk is not used).
 *         Requires 1 <= r <= 256, 1 <= dv <= 256, 4-byte alignment.
 * T may be any length >= 1 (a final partial chunk is masked).
 * Errors: LA_ERR_NULL, LA_ERR_SHAPE (B, H, T, r, dv or chunk < 1), LA_ERR_DTYPE,
 *         LA_ERR_ALIGN, LA_ERR_UNSUPPORTED, LA_ERR_WORKSPACE, LA_ERR_CUDA.
 */
la_status la_prefill_chunked(const void *q, const void *k, const void *v, la_dtype dtype,
                             const float *alpha, const float *S0, const float *z0,
                             int B, int H, int T, int r, int dv, int chunk, float eps,
                             void *y, float *S_out, float *z_out,
                             void *workspace, size_t workspace_bytes, la_stream_t stream);

/*
 * la_prefill_varlen_workspace_bytes -- device scratch that la_prefill_varlen needs
 * for a batch of B sequences, H heads and total_T tokens (total_T >= 0) on the
 * current device: the plan's tables and, when sequences can be split, their
 * segment states (0: the call needs none, dv = 64 with nothing to split).  It
 * depends on the sizes and the device's SM count only, not on the lengths, which
 * stay on the device.  Returns 0 for sizes la_prefill_varlen rejects.
 */
size_t la_prefill_varlen_workspace_bytes(int B, int H, int total_T, int r, int dv);

/*
 * la_prefill_varlen -- la_prefill_chunked for a batch of sequences of different
 * lengths packed one after another, e.g. the prompts of a serving batch, each
 * prefilled in large blocks and continuing from its own state ([LA]
 * "训练时，状态更新也能按块并行": token-by-token steps suit decode, prefill is
 * organised in chunks that hand the state on).  Sequence b is tokens cu_seqlens[b] ..
 * cu_seqlens[b+1]-1; it starts from S0[b], z0[b] and leaves its final state in
 * S_out[b], z_out[b] (an empty sequence copies S0, z0).
 *
 *   q, k       device BF16 [total_T, H, r]   (token-major: row t*H + h)
 *   v, y       device BF16 [total_T, H, dv]
 *   alpha      device FP32 [total_T, H] or NULL (alpha == 1)
 *   S0, z0     device FP32 [B, H, r, dv], [B, H, r] or NULL (zero); may alias S_out, z_out
 *   S_out, z_out  device FP32 [B, H, r, dv], [B, H, r]
 *   cu_seqlens device int32 [B + 1]: 0 = cu_seqlens[0] <= ... <= cu_seqlens[B] = total_T.
 *              The host cannot read it; a kernel finding a sequence outside
 *              [0, total_T] or of negative length skips it and records LA_ERR_SHAPE
 *              (read it with la_last_device_status).
 *   workspace  device scratch of la_prefill_varlen_workspace_bytes(B, H, total_T, r, dv)
 *              bytes, 256-byte aligned, owned by the caller and not read by the
 *              caller afterwards; may be NULL when that is 0.  Calls that may
 *              overlap in time need their own.
 * Long sequences are split into segments, as la_prefill_chunked splits a long T
 * ([LA] "门控递推为什么能做并行 scan？": a run of tokens composes into one affine map
 * of the state): a plan kernel reads the lengths and picks the segment length from
 * the batch's own chunk count, so that a long prompt among short ones no longer
 * holds up the batch; a state pass over the segments that end before a sequence's
 * last one and a scan give every segment its start state.  When no sequence is
 * long enough, or any sequence's bounds are invalid, nothing is split.  At dv = 128
 * with S0 16-byte aligned (or NULL), a sequence of at most 32 tokens (a short
 * continuation of one request, empty ones included) is walked token by token with
 * its state in registers (the walk of la_prefill_chunked), beside the others, on a
 * second stream of the library's (one per host thread and device, ordered against
 * `stream` by events): the first such call on a device from a host thread creates
 * it and must not be made inside a stream capture.
 * Requires BF16, r == 128, dv in {64, 128}, chunk >= 1 (computed in chunks of 64
 * tokens, as la_prefill_chunked); q, k, v, y, S_out 16-byte aligned.  total_T may be 0.
 * Rows of y outside every sequence are not written.
 * Errors: LA_ERR_NULL, LA_ERR_SHAPE, LA_ERR_DTYPE, LA_ERR_ALIGN, LA_ERR_UNSUPPORTED
 *         (FP32 or other sizes), LA_ERR_WORKSPACE (workspace missing or too small),
 *         LA_ERR_CUDA.
 */
la_status la_prefill_varlen(const void *q, const void *k, const void *v, la_dtype dtype,
                            const float *alpha, const float *S0, const float *z0, const int *cu_seqlens,
                            int B, int H, int total_T, int r, int dv, int chunk, float eps,
                            void *y, float *S_out, float *z_out,
                            void *workspace, size_t workspace_bytes, la_stream_t stream);

/*
 * la_prefill_chunked_noalloc -- la_prefill_chunked without caller scratch: the
 * workspace is a 32 MiB buffer compiled into the library (a static device array),
 * one per device for the whole process.  The pages have no counterpart; it is an
 * integration aid for callers that must not allocate device memory per call,
 * such as a serving loop that reserved its whole memory budget up front, or C
 * code without a caching allocator, where cudaMalloc/cudaFree would add
 * device-wide synchronisation and can fail under memory pressure.
 *   Arguments, results and errors are those of la_prefill_chunked, without
 *   workspace.  LA_ERR_WORKSPACE when la_prefill_workspace_bytes for these sizes
 *   exceeds the 32 MiB (the largest workspace la_prefill_workspace_bytes returns on
 *   devices with up to about 240 SMs).
 *   The first call on a device looks up the buffer's device address with that
 *   device current; make it before any stream capture.  The look-up is cached
 *   per device in an atomic, so first calls from several host threads are safe.
 *   Nothing in the buffer has to start at zero: a call writes every entry before
 *   reading it.  Calls that may overlap in time (other streams, other threads)
 *   race on the one buffer; the caller must serialise them.
 */
la_status la_prefill_chunked_noalloc(const void *q, const void *k, const void *v, la_dtype dtype,
                                     const float *alpha, const float *S0, const float *z0,
                                     int B, int H, int T, int r, int dv, int chunk, float eps,
                                     void *y, float *S_out, float *z_out, la_stream_t stream);

/*
 * la_decode_step -- one new token per (b, h), state updated in place:
 *   S <- alpha S + phi(k) v^T,  z <- alpha z + phi(k),  y = phi(q)^T S / (phi(q)^T z + eps)
 * ([LA] "公式里的每个维度" and "查询时，分子和分母一起读"; update before read).
 *   q, k   device [B,H,1,r] dtype;  v, y device [B,H,1,dv] dtype
 *   alpha  device FP32 [B,H] or NULL (alpha == 1)
 *   S      device FP32 [B,H,r,dv], read and overwritten;  z device FP32 [B,H,r], likewise.
 * Requires 1 <= r <= 256, 1 <= dv <= 256; 4-byte alignment (the r = dv = 128 fast
 * path is taken when S is 16-byte aligned).
 * Errors: LA_ERR_NULL, LA_ERR_SHAPE, LA_ERR_DTYPE, LA_ERR_ALIGN, LA_ERR_UNSUPPORTED, LA_ERR_CUDA.
 */
la_status la_decode_step(const void *q, const void *k, const void *v, la_dtype dtype,
                         const float *alpha, float *S, float *z, int B, int H, int r, int dv,
                         float eps, void *y, la_stream_t stream);

/*
 * la_backward_workspace_bytes -- device scratch that la_prefill_backward needs for
 * these sizes on the current device, for any r, dv <= 128 and either dtype: the
 * FP32 per-token terms and one value per head (4 * B*H*(3T + 1) bytes), the maps
 * of the z_t pass (4 * B*H*ceil(T/128)*257 bytes), and, when B*H whole-head CTAs
 * would leave enough SMs idle and T is long enough, the two state passes of the
 * sequence-segmented tensor-core sweeps (forward and reversed: per head and part
 * or segment 4 * (128*128 + 128) bytes).  The size depends on the device's SM
 * count; it is 0 only for invalid sizes.
 */
size_t la_backward_workspace_bytes(int B, int H, int T);

/*
 * la_prefill_backward -- gradients of la_prefill_chunked's outputs for training.
 * Given dy = dL/dy and optionally dS_T = dL/dS_T, dz_T = dL/dz_T, returns
 * dL/dq, dL/dk, dL/dv, dL/dalpha, dL/dS0 and dL/dz0.  The pages give no backward
 * formula; this is the chain rule through the recurrence of [LA] "公式里的每个维度"
 * and "加一个门：让旧记忆逐渐淡出", with y_t = n_t / d_t:
 *   dn_t = dy_t / d_t,  dd_t = -(dy_t . y_t) / d_t,
 *   G_t = phi(q_t) dn_t^T + alpha_{t+1} G_{t+1},  g_t = dd_t phi(q_t) + alpha_{t+1} g_{t+1},
 *   dq_t = phi'(q_t) * (S_t dn_t + dd_t z_t),  dk_t = phi'(k_t) * (G_t v_t + g_t),
 *   dv_t = G_t^T phi(k_t),  dS0 = alpha_1 G_1,  dz0 = alpha_1 g_1,
 *   dalpha_u = (sum_{t >= u} (phi(q_t) . dq~_t - phi(k_t) . dk~_t) + <dS_T, S_T> + <dz_T, z_T>) / alpha_u
 * (dq~, dk~: the gradients before the phi' factor).
 *   q, k, v, alpha, S0, z0, eps: as passed to the forward call.
 *   y      device [B,H,T,dv] dtype: the forward's output (used for dd_t).
 *   dy     device [B,H,T,dv] dtype.
 *   dS_T, dz_T  device FP32 [B,H,r,dv], [B,H,r], or NULL (zero).
 *   dq, dk device [B,H,T,r] dtype;  dv_out device [B,H,T,dv] dtype.
 *   dalpha device FP32 [B,H,T], or NULL (not computed; ignored without alpha).
 *          Defined where alpha > 0 (it is the log-gate derivative over alpha).
 *   dS0, dz0  device FP32 [B,H,r,dv], [B,H,r] (written also when S0, z0 are NULL).
 *   workspace: >= la_backward_workspace_bytes device bytes, 16-byte aligned, owned by
 *          the caller; calls sharing it must be ordered.
 * Kernels: the z_t recurrence over segments of 128 tokens (maps, scan, products)
 * for d_t, one pass for dd_t, then the three gradients as causal linear
 * attentions over chunks of 64 tokens (dq forward in time, dk and dv in
 * reverse), then a reverse running sum for dalpha.  BF16 with r = dv = 128 runs
 * the three on the tensor cores (BF16 operands, FP32 accumulators and state), and
 * for few long sequences over sequence segments whose entering states a forward
 * and a reversed state pass compute ([LA] "门控递推为什么能做并行 scan？"); the
 * other shapes and FP32 run them as gated rank-1 recurrences in FP32 on the CUDA
 * cores.  With segments, the state passes run on a second stream of the library's
 * (one per host thread and device, ordered against `stream` by events), beside
 * the z pass and the dq sweep; the call's work is still complete, in order, on
 * `stream`.  The first call on a device from a host thread creates that stream
 * and must not be made inside a stream capture.  Requires r, dv in {32, 64, 128}, T >= 1, 16-byte aligned
 * token arrays (q, k, v, y, dy, dq, dk, dv_out), 4-byte aligned FP32 arrays
 * (dS_T 8-byte aligned).
 * Errors: LA_ERR_NULL, LA_ERR_SHAPE, LA_ERR_DTYPE, LA_ERR_ALIGN, LA_ERR_UNSUPPORTED,
 *         LA_ERR_WORKSPACE, LA_ERR_CUDA.
 */
la_status la_prefill_backward(const void *q, const void *k, const void *v, la_dtype dtype, const float *alpha,
                              const float *S0, const float *z0, int B, int H, int T, int r, int dv, float eps,
                              const void *y, const void *dy, const float *dS_T, const float *dz_T, void *dq,
                              void *dk, void *dv_out, float *dalpha, float *dS0, float *dz0, void *workspace,
                              size_t workspace_bytes, la_stream_t stream);

/*
 * la_backward_states_bytes -- bytes of the states buffer that la_prefill_chunked_save
 * can fill for la_prefill_backward_saved: the backward splits a sequence into
 * segments when few long sequences would leave SMs idle, and this is the state
 * [S | z] (FP32, 128 x 128 then 128) entering each segment of every (b, h).
 * 0 when the backward would not split (then there is nothing to keep).
 */
size_t la_backward_states_bytes(int B, int H, int T);

/*
 * la_prefill_chunked_save -- la_prefill_chunked that also keeps, for training, the
 * denominator of every output row: d_t = phi(q_t) . z_t + eps, the normaliser of
 * [LA] "公式里的每个维度" (y_t = phi(q_t)^T S_t / d_t), in FP32, and optionally the
 * states at which the backward's sequence segments start.
 * la_prefill_backward_saved takes them instead of recomputing them.
 *   d_out      device FP32 [B,H,T], 4-byte aligned, owned by the caller.
 *   states_out device buffer of la_backward_states_bytes(B, H, T) bytes, 16-byte
 *              aligned, or NULL (not kept).  Written for BF16 with r = dv = 128
 *              when that size is not 0; otherwise left untouched.
 *   Everything else as for la_prefill_chunked.
 * BF16: the chunk kernel's own denominator (the BF16 operands of its products,
 * FP32 accumulation), the one y was divided by, and its FP32 state; FP32: the
 * exact recurrence's denominator.
 * Errors: those of la_prefill_chunked; LA_ERR_NULL when d_out is NULL.
 */
la_status la_prefill_chunked_save(const void *q, const void *k, const void *v, la_dtype dtype, const float *alpha,
                                  const float *S0, const float *z0, int B, int H, int T, int r, int dv, int chunk,
                                  float eps, void *y, float *S_out, float *z_out, float *d_out, float *states_out,
                                  void *workspace, size_t workspace_bytes, la_stream_t stream);

/*
 * la_prefill_backward_saved -- la_prefill_backward with d_t taken from
 * la_prefill_chunked_save instead of recomputed: the z_t recurrence over the
 * sequence (three of the backward's launches) is skipped, and with states, the
 * forward state pass and scan of a segmented backward too.
 *   d      device FP32 [B,H,T] from la_prefill_chunked_save on the same inputs
 *          (eps is included in it, so there is no eps argument).
 *   states the states_out of that call, or NULL (recomputed when needed).
 *   Everything else as for la_prefill_backward.
 * Errors: those of la_prefill_backward; LA_ERR_NULL when d is NULL; LA_ERR_ALIGN
 *         when states is not 16-byte aligned.
 */
la_status la_prefill_backward_saved(const void *q, const void *k, const void *v, la_dtype dtype, const float *alpha,
                                    const float *S0, const float *z0, int B, int H, int T, int r, int dv,
                                    const void *y, const void *dy, const float *d, const float *states,
                                    const float *dS_T, const float *dz_T, void *dq, void *dk, void *dv_out,
                                    float *dalpha, float *dS0, float *dz0, void *workspace, size_t workspace_bytes,
                                    la_stream_t stream);

/*
 * la_delta_rule -- the delta-rule memory ([LA] "Delta rule：先读旧答案，再写误差"): a
 * state without the normaliser that, per token, reads its current answer for the
 * key, writes back beta times the error, and is then read by the query:
 *     p_t = S_{t-1}^T k_t,   S_t = S_{t-1} + beta_t k_t (v_t - p_t)^T,   y_t = S_t^T q_t
 * q and k are used as given (no feature map); the read follows the write, as in
 * the other entry points.  With a unit key and beta = 1 the memory returns v
 * exactly for that key; the error left on k after a step is (1 - beta |k|^2)
 * times the error before it, so the update contracts for 0 < beta |k|^2 < 2.
 *   q, k   device [B,H,T,r] dtype          v, y  device [B,H,T,dv] dtype
 *   beta   device FP32 [B,H,T] write strength, or NULL for beta == 1
 *   S0     device FP32 [B,H,r,dv] or NULL (zero); may equal S_out (in place)
 *   S_out  device FP32 [B,H,r,dv] final state
 * Kernel: the token recurrence in FP32 on CUDA cores (the pages give no block
 * algorithm for this rule, [LA] "训练时，状态更新也能按块并行"), the state in
 * registers, the value columns split over CTAs.  Requires r in {32, 64, 128, 256},
 * dv a multiple of 32, q, k, v, y 16-byte aligned, S0, S_out 8-byte aligned,
 * beta 4-byte aligned.  T may be 0 (S_out = S0; q, k, v, y may then be NULL and are not touched).
 * Errors: LA_ERR_NULL, LA_ERR_SHAPE (B, H, r, dv < 1, T < 0), LA_ERR_DTYPE,
 *         LA_ERR_ALIGN, LA_ERR_UNSUPPORTED (other r or dv), LA_ERR_CUDA.
 */
la_status la_delta_rule(const void *q, const void *k, const void *v, la_dtype dtype, const float *beta,
                        const float *S0, int B, int H, int T, int r, int dv, void *y, float *S_out,
                        la_stream_t stream);

/*
 * la_delta_chunked_workspace_bytes -- bytes of device workspace la_delta_rule_chunked
 * needs for (B, H, T): 32 KB per chunk of 64 tokens per (b, h); 0 when T < 1.
 */
size_t la_delta_chunked_workspace_bytes(int B, int H, int T);

/*
 * la_delta_rule_chunked -- the memory of la_delta_rule, computed in chunks of 64
 * tokens on the tensor cores.  The pages give no block algorithm for this rule
 * ([LA] "训练时，状态更新也能按块并行"); this one follows from the update: for a
 * chunk with rows K, Q, V and the state S_prev before it, the written rows
 * V' = beta (V - K S) of the chunk's tokens solve (I + L) V' = diag(beta) X with
 * X = V - K S_prev and L = diag(beta) strictly-lower(K K^T), so
 *     V' = T X,  T = (I + L)^{-1} diag(beta),
 *     S_next = S_prev + K^T V',   Y = Q S_prev + (Q K^T masked causally, diagonal kept) V'.
 * The state chain evaluates V' as U - W S_prev with W = T K and U = T V, which
 * do not depend on the state.  The products take BF16 operands (q, k, v as
 * given, S_prev, W, T and V' rounded to BF16) with FP32 accumulation; U and the
 * state stay FP32 and T is solved in FP32.  Same arguments, layouts and ownership as
 * la_delta_rule, plus
 *   workspace  device buffer of >= la_delta_chunked_workspace_bytes(B, H, T) bytes,
 *              16-byte aligned, owned by the caller (may be NULL when T == 0);
 *              calls sharing it must be ordered.
 * Kernels: T, the masked scores (Q K^T) . M and -W of every chunk (one CTA per
 * chunk) into the workspace, then the state chain, one CTA per (b, h, 64-column
 * slice of v).  Requires dtype BF16,
 * r == 128, dv a multiple of 64, q, k, v, y, S0 and S_out 16-byte aligned, beta
 * 4-byte aligned.  T may be 0 (S_out = S0).
 * Errors: LA_ERR_NULL, LA_ERR_SHAPE, LA_ERR_DTYPE (not BF16), LA_ERR_ALIGN,
 *         LA_ERR_UNSUPPORTED (other r or dv), LA_ERR_WORKSPACE, LA_ERR_CUDA.
 */
la_status la_delta_rule_chunked(const void *q, const void *k, const void *v, la_dtype dtype, const float *beta,
                                const float *S0, int B, int H, int T, int r, int dv, void *y, float *S_out,
                                void *workspace, size_t workspace_bytes,
                                la_stream_t stream);

/*
 * Linear attention with a constant decay per head: the recurrence without a feature
 * map and without a normaliser,
 *     S_t = g S_{t-1} + k_t v_t^T,    y_t = scale q_t^T S_t        (g = decay[h])
 * so a write made n tokens ago counts g^n ([LA] "加一个门：让旧记忆逐渐淡出" with a gate that
 * is a constant of the head).  q and k are used as given; the read follows the
 * write, as in the other entry points.
 *   decay  device FP32 [H], 0 <= decay <= 1 (not checked: it stays on the device).
 *          It is a constant of the model: no gradient is formed for it.
 *   scale  any finite value, typically 1/sqrt(r).
 * Inputs are finite; a row with an infinity or NaN may spoil the outputs of the 128
 * tokens around it as well as all later ones.  Outputs do not overlap inputs, but for the
 * states where it says so.
 * Kernels:
 *   BF16, r in {64, 128}, dv a multiple of 64, token arrays 16-byte aligned, more than 16
 *         tokens: chunks of 128 tokens on the tensor cores.  The scores of a chunk and the state that enters
 *         it are rounded to BF16 once; the state itself is FP32, each write to it kept to 2^-16
 *         of its size (passed as FP32, the same values take the recurrence below and are kept to 2^-24).
 *         Few heads run their sequences in segments, which needs the workspace.
 *   else  the token recurrence in FP32 on CUDA cores, in segments side by side where few heads
 *         have 128 tokens or more and are not packed (for one token of la_decay_decode_step a
 *         kernel of its own, bound by the state's traffic, when dv is a multiple of 4 and
 *         S 16-byte aligned).
 * The first call of each kind on a device sets kernel attributes: make it before any stream
 * capture.
 */

/*
 * la_decay_prefill -- T tokens of every (b, h) sequence from S0 (a chunk's output is
 * the read of the carried state plus the masked in-chunk product, [LA] "一个 chunk
 * 的输出由两部分组成", each term times the decay between its write and its read).
 *   q, k   device [B,H,T,r] dtype          v, y   device [B,H,T,dv] dtype
 *   S0     device FP32 [B,H,r,dv] or NULL (zero); may equal S_out (in place)
 *   S_out  device FP32 [B,H,r,dv] final state
 *   workspace  device scratch of la_decay_prefill_workspace_bytes(...) bytes, 256-byte
 *              aligned, owned by the caller; may be NULL when that is 0.  Calls
 *              sharing one workspace must be ordered.  The size depends on the
 *              device's SM count (0 for sizes the call rejects).
 * Requires 1 <= r, dv <= 256, B, H <= 65535, T <= 2^30; BF16 arrays 2-byte, FP32 arrays 4-byte
 * aligned.  T may be 0 (S_out = S0; q, k, v, y may then be NULL).
 * Errors: LA_ERR_NULL, LA_ERR_SHAPE (B, H, r, dv < 1, T < 0, scale not finite),
 *         LA_ERR_DTYPE, LA_ERR_ALIGN, LA_ERR_UNSUPPORTED (other sizes),
 *         LA_ERR_WORKSPACE, LA_ERR_CUDA.
 */
size_t la_decay_prefill_workspace_bytes(int B, int H, int T, int r, int dv, la_dtype dtype);
la_status la_decay_prefill(const void *q, const void *k, const void *v, la_dtype dtype, const float *decay,
                           const float *S0, int B, int H, int T, int r, int dv, float scale, void *y, float *S_out,
                           void *workspace, size_t workspace_bytes, la_stream_t stream);

/*
 * la_decay_prefill_varlen -- the same for sequences of different lengths packed one after
 * another: sequence b is tokens cu_seqlens[b] .. cu_seqlens[b+1]-1, from S0[b] into
 * S_out[b] (an empty sequence copies its state).
 *   q, k       device [total_T, H, r] dtype (token-major)     v, y  device [total_T, H, dv]
 *   S0, S_out  device FP32 [B,H,r,dv]; S0 NULL (zero) or equal to S_out (in place) or apart
 *   cu_seqlens device int32 [B + 1], 0 <= cu_seqlens[0] <= .. <= cu_seqlens[B] <= total_T.  A
 *              sequence outside [0, total_T] or of negative length is skipped and
 *              recorded as LA_ERR_SHAPE in the device status word.
 * Rows of y outside every sequence are not written, and what q, k, v hold there (or in
 * another sequence) reaches no output.  Up to 256 sequences run the longest first; a sequence is
 * not split.  Needs no workspace.
 * Sizes, alignment and errors as for la_decay_prefill (total_T * H < 2^31).
 */
la_status la_decay_prefill_varlen(const void *q, const void *k, const void *v, la_dtype dtype, const float *decay,
                                  const float *S0, const int *cu_seqlens, int B, int H, int total_T, int r, int dv,
                                  float scale, void *y, float *S_out, la_stream_t stream);

/*
 * la_decay_decode_step -- one new token per (b, h), the state updated in place.
 *   q, k  device [B,H,1,r] dtype    v, y  device [B,H,1,dv] dtype    S  device FP32 [B,H,r,dv]
 * Requirements and errors as for la_decay_prefill.
 */
la_status la_decay_decode_step(const void *q, const void *k, const void *v, la_dtype dtype, const float *decay,
                               float *S, int B, int H, int r, int dv, float scale, void *y, la_stream_t stream);

/*
 * la_decay_backward -- gradients of la_decay_prefill's outputs.  Given dy = dL/dy and
 * optionally dS_T = dL/dS_T, with G_T = scale q_T dy_T^T + dS_T,
 *     G_t = scale q_t dy_t^T + g G_{t+1},
 *     dq_t = scale S_t dy_t,   dk_t = G_t v_t,   dv_t = G_t^T k_t,   dS0 = g G_1.
 *   q, k, v, decay, S0, scale: as passed to the forward call (its outputs are not needed).
 *   dy       device [B,H,T,dv] dtype         dS_T  device FP32 [B,H,r,dv] or NULL (zero)
 *   dq, dk   device [B,H,T,r] dtype          dv_out  device [B,H,T,dv] dtype
 *   dS0      device FP32 [B,H,r,dv] (written also when S0 is NULL); overlaps neither S0 nor dS_T.
 *   workspace  la_decay_backward_workspace_bytes(...) bytes, as for la_decay_prefill.
 * Three sweeps like the forward one, each with two of the arrays as keys and a third as values: dq
 * forwards in time, dk and dv backwards, in one launch where they take the same kernel.  On the tensor
 * cores a sweep's keys are 64 or 128 wide and its values a multiple of 64 (dq and dk: dv keys, r values).
 * Sizes, alignment and errors as for la_decay_prefill.  T may be 0 (dS0 = dS_T).
 */
size_t la_decay_backward_workspace_bytes(int B, int H, int T, int r, int dv, la_dtype dtype);
la_status la_decay_backward(const void *q, const void *k, const void *v, la_dtype dtype, const float *decay,
                            const float *S0, int B, int H, int T, int r, int dv, float scale, const void *dy,
                            const float *dS_T, void *dq, void *dk, void *dv_out, float *dS0, void *workspace,
                            size_t workspace_bytes, la_stream_t stream);

/*
 * The gated delta rule: the delta-rule memory of la_delta_rule with a gate per token and head, as
 * la_prefill_chunked's ([LA] "Delta rule：先读旧答案，再写误差" and "加一个门：让旧记忆逐渐淡出"):
 *     S' = alpha_t S_{t-1},  S_t = S' + beta_t k_t (v_t - S'^T k_t)^T,  y_t = scale S_t^T q_t
 * The memory fades, reads its answer for the key, writes beta times the error back and is then read by
 * the query.  q and k are used as given (models bring them to length one; the update contracts for
 * 0 <= beta |k|^2 <= 2).
 * Shared heads: q and k have Hk heads, v, the gates and the state H, a multiple of Hk; value head h reads key
 * head h / (H / Hk), and the gradients of a key head are summed over its value heads.
 *   alpha  device FP32, 0 <= alpha <= 1, or NULL (1)      beta  device FP32 write strength, or NULL (1)
 *   scale  any finite value, typically 1/sqrt(r)
 * Inputs are finite; a row with an infinity or NaN may spoil its whole chunk of 64 tokens as well as all later ones.
 * Outputs overlap neither inputs nor one another, but for the states where it says so.
 * Kernels:
 *   prompts in chunks of 64 tokens on the tensor cores, the state in FP32, for BF16 with r 64 or 128, dv a multiple of 64
 *   (la_gated_delta_backward: 64 or 128), every token array on a 16-byte boundary and T > 16 (packed sequences: any length);
 *   the token recurrence in FP32 on CUDA cores for everything else.  Dense prompts whose heads leave SMs idle go in segments there
 *   (the workspace is then not 0 bytes for FP32 either, and depends on the current device);
 *   for one token of la_gated_delta_decode_step a kernel of its own, bound by the state's traffic, when dv is a multiple of 4
 *   and S 16-byte aligned.
 * In the chunked kernels what is derived from the inputs enters the tensor cores as two BF16 parts (16 bits of it) where
 * it reaches an FP32 result, and as one where it reaches a BF16 one only: relative 2-norms of the errors about 4e-6 (dalpha and dbeta
 * 7e-6) and 2e-3 to 3e-3.
 * The first call of each kind on a device sets kernel attributes: make it before any stream capture.
 * Requires 1 <= r, dv <= 256, B, H <= 65535, T <= 2^30 and, but for packed sequences, B H (T + 1) <= 2^30; BF16 arrays
 * 2-byte, FP32 and int32 arrays 4-byte aligned, workspaces 256-byte.
 * Errors of every entry point: LA_ERR_NULL, LA_ERR_SHAPE (B, H, Hk, r, dv < 1, T < 0, H not a multiple of Hk,
 * scale not finite), LA_ERR_DTYPE, LA_ERR_ALIGN, LA_ERR_UNSUPPORTED (other sizes), LA_ERR_WORKSPACE, LA_ERR_CUDA.
 */

/*
 * la_gated_delta_prefill -- T tokens of every (b, h) sequence from S0.
 *   q, k   device [B,Hk,T,r] dtype         v, y   device [B,H,T,dv] dtype
 *   alpha, beta  device FP32 [B,H,T] or NULL
 *   S0     device FP32 [B,H,r,dv] or NULL (zero); may equal S_out (in place)
 *   S_out  device FP32 [B,H,r,dv] final state
 *   workspace  device scratch of la_gated_delta_prefill_workspace_bytes(...) bytes, owned by the caller; may be
 *              NULL when that is 0.  Calls sharing one workspace must be ordered.
 * T may be 0 (S_out = S0; q, k, v, y may then be NULL).
 */
size_t la_gated_delta_prefill_workspace_bytes(int B, int H, int Hk, int T, int r, int dv, la_dtype dtype);
la_status la_gated_delta_prefill(const void *q, const void *k, const void *v, la_dtype dtype, const float *alpha,
                                 const float *beta, const float *S0, int B, int H, int Hk, int T, int r, int dv,
                                 float scale, void *y, float *S_out, void *workspace, size_t workspace_bytes,
                                 la_stream_t stream);

/*
 * la_gated_delta_prefill_varlen -- the same for sequences of different lengths packed one after
 * another: sequence b is tokens cu_seqlens[b] .. cu_seqlens[b+1]-1, from S0[b] into
 * S_out[b] (an empty sequence copies its state).
 *   q, k         device [total_T, Hk, r] dtype (token-major)     v, y  device [total_T, H, dv]
 *   alpha, beta  device FP32 [total_T, H] or NULL
 *   S0, S_out    device FP32 [B,H,r,dv]; S0 NULL (zero) or equal to S_out (in place) or apart
 *   cu_seqlens   device int32 [B + 1], 0 <= cu_seqlens[0] <= .. <= cu_seqlens[B] <= total_T.  A
 *                sequence outside [0, total_T] or of negative length is skipped and
 *                recorded as LA_ERR_SHAPE in the device status word.
 *   workspace    la_gated_delta_prefill_varlen_workspace_bytes(...) bytes, as above
 * Rows of y outside every sequence are not written, and what q, k, v hold there (or in
 * another sequence) reaches no output.  total_T * H < 2^31.
 */
size_t la_gated_delta_prefill_varlen_workspace_bytes(int B, int H, int Hk, int total_T, int r, int dv, la_dtype dtype);
la_status la_gated_delta_prefill_varlen(const void *q, const void *k, const void *v, la_dtype dtype, const float *alpha,
                                        const float *beta, const float *S0, const int *cu_seqlens, int B, int H, int Hk,
                                        int total_T, int r, int dv, float scale, void *y, float *S_out, void *workspace,
                                        size_t workspace_bytes, la_stream_t stream);

/*
 * la_gated_delta_decode_step -- one new token per (b, h), the state updated in place.
 *   q, k  device [B,Hk,1,r] dtype    v, y  device [B,H,1,dv] dtype    alpha, beta  device FP32 [B,H] or NULL
 *   S     device FP32 [B,H,r,dv]
 */
la_status la_gated_delta_decode_step(const void *q, const void *k, const void *v, la_dtype dtype, const float *alpha,
                                     const float *beta, float *S, int B, int H, int Hk, int r, int dv, float scale,
                                     void *y, la_stream_t stream);

/*
 * la_gated_delta_backward -- gradients of la_gated_delta_prefill's outputs, by the chain rule through the
 * recurrence.  Given dy = dL/dy and optionally dS_T = dL/dS_T, with e_t = v_t - S'^T k_t,
 *     G_t = scale q_t dy_t^T + alpha_{t+1} (G_{t+1} - k_{t+1} dv_{t+1}^T),   G_T = scale q_T dy_T^T + dS_T,
 *     dv_t = beta_t G_t^T k_t,   dk_t = beta_t G_t e_t - S'_t dv_t,   dq_t = scale S_t dy_t,
 *     dbeta_t = (G_t^T k_t) . e_t,   dS0 = alpha_1 (G_1 - k_1 dv_1^T),
 *     dalpha_t = <S_{t-1}, G_t - k_t dv_t^T>.
 *   q, k, v, alpha, beta, S0, scale: as passed to the forward call (its outputs are not needed).
 *   dy       device [B,H,T,dv] dtype         dS_T  device FP32 [B,H,r,dv] or NULL (zero)
 *   dq, dk   device [B,Hk,T,r] dtype         dv_out  device [B,H,T,dv] dtype
 *   dalpha   device FP32 [B,H,T] or NULL (not formed; ignored without alpha).  It is as accurate at a gate near 0 (denormal numbers
 *            included) as at 1: off by 1e-7 of |S_{t-1}| |G_t - k_t dv_t^T| / sqrt(r dv) in the recurrence, 2e-6 in chunks (2-norms over all
 *            tokens), beside at most 2^-62 of what several nearly closed gates shut out together.  A gate of exactly 0 is taken for a
 *            constant: 0 is written there.  Who wants the derivative at a reset passes the smallest normal number for it,
 *            1.2e-38, which keeps nothing of the state either.
 *   dbeta    device FP32 [B,H,T] or NULL (not formed)
 *   dS0      device FP32 [B,H,r,dv] (written also when S0 is NULL)
 *   workspace  la_gated_delta_backward_workspace_bytes(...) bytes, as above
 * T may be 0 (dS0 = dS_T).  Repeated calls give the same bits.
 */
size_t la_gated_delta_backward_workspace_bytes(int B, int H, int Hk, int T, int r, int dv, la_dtype dtype);
la_status la_gated_delta_backward(const void *q, const void *k, const void *v, la_dtype dtype, const float *alpha,
                                  const float *beta, const float *S0, int B, int H, int Hk, int T, int r, int dv,
                                  float scale, const void *dy, const float *dS_T, void *dq, void *dk, void *dv_out,
                                  float *dalpha, float *dbeta, float *dS0, void *workspace, size_t workspace_bytes,
                                  la_stream_t stream);

/*
 * la_beam_select -- a beam search's choice: the best K of a request's K beams x V tokens.
 * Candidate (k, v) of request b scores
 *     scores[b,k] + logits[b,k,v] - log sum_u exp logits[b,k,u]
 * and the K best, best first, become the request's beams; equal scores go to the lower
 * k * V + v.  (Within one beam candidates rank by their logits.)  Scores are compared in 64
 * bits, the log-sum-exp carrying the error of its FP32 exponentials; a row's largest logit is taken off
 * first, so that rows of one huge value (masks of the type's lowest) keep their log-probabilities.
 *   logits      device [B,K,V] dtype, row (b, k) at element (b K + k) row_stride
 *   scores      device FP32 [B,K] cumulative log-probabilities
 *   done        device uint8 [B,K], non-zero: beam k has ended; its one candidate is token
 *               eos with its score unchanged.  NULL: none has.
 *   eos         the token that ends a beam, 0 .. V-1, or -1 (none; done must be NULL).
 *   next_scores, parents, tokens   device FP32, int32, int32 [B,K]: slot j's score, the beam it
 *               continues and the token it appends
 *   done_out    device uint8 [B,K] or NULL: 1 where the parent has ended or the token is eos
 * A logit of -infinity (a masked token) is no candidate; nor is any token of a beam whose
 * score or log-sum-exp is not finite (all its tokens masked, or a NaN or +infinity
 * among its logits).  A slot left without a candidate gets score -infinity, its own
 * beam as parent, token 0 and its own done.
 * next_scores may equal scores, done_out may equal done.
 * One launch, one cluster of 2 to 8 CTAs per request, the logits read once; rows that start on
 * 16-byte boundaries are read fastest.
 * Requires 1 <= K <= 32, 1 <= V <= 2^30, row_stride >= V, B <= 65535; logits aligned to their
 * element size, FP32 and int32 arrays 4-byte aligned.
 * Errors: LA_ERR_NULL, LA_ERR_SHAPE (sizes < 1, row_stride < V, eos out of range or missing),
 *         LA_ERR_DTYPE, LA_ERR_ALIGN, LA_ERR_UNSUPPORTED (K > 32, other sizes), LA_ERR_CUDA.
 */
la_status la_beam_select(const void *logits, la_dtype dtype, long long row_stride, const float *scores,
                         const unsigned char *done, int B, int K, int V, int eos, float *next_scores, int *parents,
                         int *tokens, unsigned char *done_out, la_stream_t stream);

/*
 * la_token_logprobs -- scores of given tokens under rows of logits (what a model answered with, or is trained
 * on):  lse = log sum_v exp x_v,  logprob = x_token - lse,  entropy = lse - sum_v p_v x_v  with p_v = exp(x_v - lse),
 * and the best alternatives of the row.
 *   logits    device [N,V] dtype, row n at element n row_stride
 *   tokens    device int32 [N].  A negative token skips its row (padding), which is not read: its logprob,
 *             entropy and lse are 0 and it has no alternatives.  A token >= V does the same and is
 *             recorded as LA_ERR_SHAPE in the device status word.
 *   top       alternatives per row, 0 .. 32
 *   logprobs  device FP32 [N];  entropy, lse  device FP32 [N] or NULL
 *   top_logprobs, top_tokens  device FP32, int32 [N,top] (may be NULL when top is 0): the top most probable
 *             tokens, best first, equal logits in the order of their indices
 * A logit of -infinity (a masked token) has probability 0 and is no alternative; slots left over get -infinity and token -1.
 * A row of nothing else has lse and logprob -infinity and entropy 0.  A row with a NaN or +infinity gives NaN
 * and no alternatives.
 * One launch, the logits read once (blocks that hold an alternative once more, out of the L2 cache); rows that start on
 * 16-byte boundaries are read fastest.  A row's results do not depend on the other rows' values.  How many rows there are decides
 * how many CTAs share one, and with that the order of its sums: among more or fewer rows its results differ in the last bits
 * (2^-20 of their size, the entropy 2^-19; its best tokens and their order do not differ).  The same N, V, layout and device give
 * the same bits.
 * Requires N >= 0, 1 <= V <= 2^30, row_stride >= V; logits aligned to their element size, other arrays 4-byte.
 * Errors: LA_ERR_NULL, LA_ERR_SHAPE (N < 0, V < 1, top < 0, row_stride < V), LA_ERR_DTYPE, LA_ERR_ALIGN,
 *         LA_ERR_UNSUPPORTED (top > 32, other sizes), LA_ERR_CUDA.
 */
la_status la_token_logprobs(const void *logits, la_dtype dtype, long long row_stride, const int *tokens, int N, int V,
                            int top, float *logprobs, float *entropy, float *lse, float *top_logprobs, int *top_tokens,
                            la_stream_t stream);

/*
 * la_token_logprobs_backward -- the gradient of la_token_logprobs' logprobs and entropies: from dlogprobs = dL/dlogprobs
 * and dentropy = dL/dentropy,
 *     dlogits_v = dlogprob (1[v = token] - p_v) - dentropy p_v (log p_v + entropy).
 *   logits, tokens, row_stride: as passed to the forward call       lse, entropy  device FP32 [N]: its results
 *             (entropy may be NULL without dentropy)
 *   dlogprobs device FP32 [N];  dentropy  device FP32 [N] or NULL (zero)
 *   dlogits   device [N,V] dtype, row n at element n grad_stride; may equal logits (with the same stride)
 * A skipped row (and one of -infinity only) gets zeros; masked logits get 0.
 * Requirements and errors as for la_token_logprobs (grad_stride as row_stride).
 */
la_status la_token_logprobs_backward(const void *logits, la_dtype dtype, long long row_stride, const int *tokens,
                                     const float *lse, const float *entropy, const float *dlogprobs,
                                     const float *dentropy, int N, int V, void *dlogits, long long grad_stride,
                                     la_stream_t stream);

/*
 * la_state_reorder -- moves recurrent states after a beam search's choice: slot j of
 * request b receives the state of its slot parents[b,j].
 *   S, S_out   device FP32 [B*K, H, r, dv]       z, z_out  device FP32 [B*K, H, r], or both NULL
 *   parents    device int32 [B,K], values 0 .. K-1.  A slot whose parent is out of range is
 *              left as it is and recorded as LA_ERR_SHAPE in the device status word.
 * S_out may equal S and z_out z (in place: slots that keep their state are not touched);
 * otherwise they must not overlap.  Any parents are allowed, repeated ones too.
 * The states of la_decode_step (S and z), la_delta_rule, la_decay_decode_step and
 * la_gated_delta_decode_step (S) all have this layout.
 * Requires 1 <= K <= 32, B <= 65535, 4-byte alignment (16-byte accesses when every slot is
 * 16-byte aligned).
 * Errors: LA_ERR_NULL, LA_ERR_SHAPE, LA_ERR_ALIGN, LA_ERR_UNSUPPORTED (K > 32), LA_ERR_CUDA.
 */
la_status la_state_reorder(const float *S, const float *z, const int *parents, int B, int K, int H, int r, int dv,
                           float *S_out, float *z_out, la_stream_t stream);

/*
 * la_last_device_status -- synchronise `stream`, then read and clear the device
 * status word of the current device: LA_OK, or LA_ERR_TIMEOUT when a kernel
 * gave up waiting on an on-chip barrier since the last read.  Returns
 * LA_ERR_CUDA when the synchronisation itself reports an error.
 */
la_status la_last_device_status(la_stream_t stream);

/* la_status_string -- a static, human-readable name for a status code. */
const char *la_status_string(la_status status);

/*
 * la_debug_wait_probe -- diagnostic: launches one block that waits on an
 * on-chip barrier that nothing ever completes, with a limit of `limit_ns`
 * nanoseconds (at most 1e9).  The wait runs out and records LA_ERR_TIMEOUT in the
 * device status word exactly as a stuck kernel would; the context stays usable.
 * Used to test the timeout path without faulting or hanging a GPU.
 */
la_status la_debug_wait_probe(unsigned long long limit_ns, la_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LINATTN_H */
