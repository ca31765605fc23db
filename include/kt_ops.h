/*
 * kt_ops.h -- C ABI of the operators around the fused MLP on one GB300 (sm_103a):
 *
 *   kt_layernorm_forward / kt_layernorm_backward   layer norm with its row statistics, and its
 *                                                  gradients;
 *   kt_quantize_rows / kt_linear_i8                each token's activations in 8-bit integers,
 *                                                  and the linear layer on 8-bit weights;
 *   kt_moe_plan / kt_moe_run / ...                 a whole mixture-of-experts feed-forward layer
 *                                                  for a few tokens (decoding), router included.
 *
 * They share the library, the status codes, kt_last_error(), the kt_dtype and kt_act values and
 * the [out][in] weight order (KT_W_OUT_IN) of kt_mlp.h.  All pointers are device pointers that
 * the caller owns.  A row pitch ("ld...") counts elements from one row to the next; a row of C
 * columns needs ld >= C.  Every call that computes is asynchronous on `stream` (a cudaStream_t; NULL = the
 * legacy default stream) of the current device, may be captured into a CUDA graph, reads its
 * inputs and writes its outputs in stream order only, and returns KT_ERR_INVALID or
 * KT_ERR_UNSUPPORTED before anything is launched where its arguments do not fit.  Results are
 * the same bits from run to run: every sum has a fixed order.  Outputs must not overlap inputs
 * except where a call says so.
 */
#ifndef KT_OPS_H
#define KT_OPS_H

#include "kt_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KT_LAYERNORM_MAX_D 16384  /* longest row of the layer norm calls and of kt_quantize_rows */

/*
 * kt_layernorm_forward -- for each row of X[M][D]:
 *   mean = avg(x),  rstd = 1 / sqrt(avg((x - mean)^2) + eps),
 *   y = (x - mean) * rstd * gamma + beta
 * in fp32 (biased variance, deviations taken before they are squared), rounded once to dtype.
 *   M >= 0 (0: nothing is done), 1 <= D <= KT_LAYERNORM_MAX_D; any D and any pitch.
 *   gamma, beta : [D] of dtype, both or neither (NULL, NULL: no affine step).
 *   Y           : [M][D], pitch ldy; may be X itself (same pointer and pitch).
 *   mean, rstd  : [M] fp32, each may be NULL.
 * Rows, gamma and beta that are 16-byte aligned (pointers, and pitches a multiple of 8) take
 * 16-byte loads; anything else takes the same kernel with 2-byte loads.
 * Errors: INVALID (NULL or misaligned pointer, negative size, pitch below D, unknown dtype, eps
 * negative or not finite, gamma without beta), UNSUPPORTED (D too long, device not sm_103),
 * CUDA (launch failed).
 */
kt_status kt_layernorm_forward(int64_t M, int64_t D, kt_dtype dtype, const void* X, int64_t ldx, const void* gamma,
                               const void* beta, float eps, void* Y, int64_t ldy, float* mean, float* rstd,
                               void* stream);

/*
 * kt_layernorm_backward -- the gradients of kt_layernorm_forward.  With xhat = (x - mean) * rstd
 * and g = dy * gamma (g = dy without gamma), per row
 *   dx = rstd * (g - avg(g) - xhat * avg(g * xhat)),
 * and over all rows  dgamma = sum dy * xhat,  dbeta = sum dy,  in fp32.
 *   mean, rstd     : [M] fp32, as the forward call wrote them.
 *   dX             : [M][D] of dtype; may be dY or X itself (same pointer and pitch).
 *   dgamma, dbeta  : [D] fp32 (sums of many rows: an optimiser rounds them, if it wants to);
 *                    both or neither.  M = 0 writes zeros.
 *   workspace      : kt_layernorm_backward_workspace(M, D) bytes, 16-byte aligned, its content
 *                    irrelevant before and after; NULL with dgamma = dbeta = NULL.
 * Errors as the forward call's, plus INVALID for a workspace that is too small.
 */
kt_status kt_layernorm_backward(int64_t M, int64_t D, kt_dtype dtype, const void* dY, int64_t lddy, const void* X,
                                int64_t ldx, const void* gamma, const float* mean, const float* rstd, void* dX,
                                int64_t lddx, float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Bytes of workspace that kt_layernorm_backward needs for M rows of D columns (0 for sizes that it refuses). */
size_t kt_layernorm_backward_workspace(int64_t M, int64_t D);

/*
 * kt_quantize_rows -- each row of the activations in signed 8-bit integers with one scale:
 *   v = act(X[m][:]) (fp32),  scale[m] = max|v| / 127,
 *   Q[m][k] = the integer nearest to v / scale[m] (ties to even), in [-127, 127].
 * The division's rounding never decides: the nearest integer is that of the exact quotient.  A
 * row of zeros has scale 0 and Q = 0.  A row with a NaN or an infinity has scale NaN and Q = 0,
 * so that whatever is computed from it shows it.
 *   act = KT_ACT_NONE quantises X[M][K]; an activation quantises the hidden layer of an MLP as
 *   it is computed: X is then the up projection's output, [M][K], or [M][2K] for KT_ACT_GEGLU
 *   (value columns, then gate columns).
 *   M >= 0, 1 <= K <= KT_LAYERNORM_MAX_D.  Q: int8, pitch ldq.  scale: [M] fp32.
 */
kt_status kt_quantize_rows(int64_t M, int64_t K, kt_dtype dtype, kt_act act, const void* X, int64_t ldx, int8_t* Q,
                           int64_t ldq, float* scale, void* stream);

/*
 * kt_linear_i8 -- the linear layer on 8-bit integers with a scale for each token and channel:
 *   Y[m][n] = round( scale_x[m] * scale_w[n] * sum_k Q[m][k] * W[n][k]  (+ bias[n]) )
 *   Q: int8 [M][K], pitch ldq.  W: int8 [N][K] ([out][in]), pitch ldw.  scale_x [M], scale_w [N]
 *   fp32.  bias: [N] of dtype or NULL.  Y: [M][N] of dtype, pitch ldy.
 *   M >= 0, N >= 1, K >= 16 and a multiple of 16; Q and W 16-byte aligned, ldq and ldw multiples
 *   of 16 (16-byte loads); Y, bias and the scales need their element's alignment only.
 * Any int8 value may appear, -128 included.  The sums are exact (32-bit integers) for M up to
 * KT_LINEAR_I8_DOT_ROWS; above, they run on the tensor cores as 16-bit floats, which hold every
 * int8 and every product, into fp32: exact as long as the partial sums stay below 2^24 (always
 * for K <= 1024; for longer rows unless |Q| and |W| are near 127 throughout with equal signs),
 * and beyond that rounded as fp32 sums are.  Where the sums are exact a row's result does not hang
 * on M; where they are not, it may differ between calls of few and of many rows, within these
 * roundings.  One rounding to dtype at the end.
 */
#define KT_LINEAR_I8_DOT_ROWS 16
kt_status kt_linear_i8(int64_t M, int64_t N, int64_t K, kt_dtype dtype, const int8_t* Q, int64_t ldq, const int8_t* W,
                       int64_t ldw, const float* scale_x, const float* scale_w, const void* bias, void* Y, int64_t ldy,
                       void* stream);

/*
 * kt_linear_i8_status -- wait for `stream` and read the current device's error word of kt_linear_i8,
 * as kt_mlp_status does a plan's: KT_ERR_TIMEOUT if a bounded device-side wait ran out in any of
 * the device's calls since it was last asked (the word is cleared).  Such a call stores NaN in every
 * element of Y that it could not compute, so that what is computed from it shows it as well.
 */
kt_status kt_linear_i8_status(void* stream);

/*
 * kt_linear_i8_debug_stall -- failure-injection hook for tests, as kt_mlp_debug_stall.  With enable = 1
 * the following calls of this process with more than KT_LINEAR_I8_DOT_ROWS rows wait, in the block
 * of their first tile, on a barrier nobody signals, bounded as every other wait then is by `limit_us`
 * microseconds; the wait runs out and the call ends with that block's tiles NaN.  enable = 0
 * restores normal calls.  No GPU fault is involved.
 */
kt_status kt_linear_i8_debug_stall(int enable, int64_t limit_us);

/*
 * The mixture-of-experts feed-forward layer for a few tokens.  For each token x of X[T][D]:
 *   logits[e] = x . W_router[e]                     (exact to about 48 bits, as an order hangs on them)
 *   its experts: the top_k largest logits, a tie going to the lower index
 *   weight_j = exp(logit_j) / sum of exp over all experts, or over the chosen ones (normalize)
 *   y = sum_j weight_j * ( act(x . W_up[e_j]^T + b_up[e_j]) . W_down[e_j]^T + b_down[e_j] )  (+ R)
 * in fp32 with one rounding to dtype at the end.  The hidden layer is kept as two 16-bit parts, its
 * rounding and the remainder's: to 2^-17 of its value with KT_BF16 (about 2e-6 of an output, which
 * is itself rounded to 2^-9), to 2^-22 with KT_F16, there never better than 2^-25 in absolute terms;
 * with KT_F16 a hidden value beyond 65504 is infinite, as in kt_mlp_run.  A NaN among a token's logits makes that
 * token's weights and outputs NaN; its experts are still valid indices.
 */
#define KT_MOE_MAX_TOKENS 64
#define KT_MOE_MAX_EXPERTS 256
#define KT_MOE_MAX_TOP_K 16

typedef struct kt_moe_plan_s* kt_moe_plan_t;

typedef struct {
    int64_t max_tokens;   /* most tokens of a run: 1 .. KT_MOE_MAX_TOKENS                          */
    int64_t D, F;         /* model dim, hidden dim: multiples of 8, at least 8                      */
    int64_t experts;      /* E: 1 .. KT_MOE_MAX_EXPERTS                                              */
    int64_t top_k;        /* 1 .. min(E, KT_MOE_MAX_TOP_K)                                           */
    int32_t act;          /* kt_act; KT_ACT_GEGLU: W_up holds F value rows, then F gate rows         */
    int32_t dtype;        /* kt_dtype                                                                */
    int32_t bias;         /* 1: b_up and b_down                                                      */
    int32_t normalize;    /* 1: a token's weights sum to one                                         */
} kt_moe_options;

typedef struct {
    int64_t tokens;         /* T: 0 .. max_tokens (0: nothing is done)                               */
    const void* X;          /* [T][D], pitch ldx                                                     */
    int64_t ldx;            /* elements, a multiple of 8                                             */
    const void* W_router;   /* [E][D]                                                                */
    const void* W_up;       /* [E][F_up][D], F_up = F, or 2F for KT_ACT_GEGLU                        */
    const void* W_down;     /* [E][D][F]                                                             */
    const void* b_up;       /* [E][F_up], iff bias                                                   */
    const void* b_down;     /* [E][D], iff bias                                                      */
    const void* R;          /* [T][D] contiguous, or NULL: a residual added to the fp32 result       */
    void* Y;                /* [T][D] contiguous; may be R, or X where ldx = D or T = 1              */
    int32_t* ids;           /* [T][top_k] the chosen experts, best first, or NULL                    */
    float* weights;         /* [T][top_k] their weights, or NULL                                     */
} kt_moe_tensors;

/*
 * kt_moe_plan -- check the problem and allocate the plan's workspace on the current device.
 * Errors: INVALID, UNSUPPORTED (sizes beyond the limits above, device not sm_103), CUDA, NOMEM;
 * *out is NULL then.
 */
kt_status kt_moe_plan(const kt_moe_options* options, kt_moe_plan_t* out);

/*
 * kt_moe_run -- enqueue the layer on `stream`.  16-byte aligned pointers (ids and weights: 4).
 * A plan has one workspace: it must not run on two streams at a time.
 */
kt_status kt_moe_run(kt_moe_plan_t plan, const kt_moe_tensors* tensors, void* stream);

/*
 * kt_moe_status -- wait for the plan's device (all its streams: a captured run may have been replayed
 * on any) and read the plan's error word: KT_ERR_TIMEOUT if a bounded device-side wait ran out (the
 * word is cleared, the plan usable again).  Y of that run, and of runs behind it, is not written.
 */
kt_status kt_moe_status(kt_moe_plan_t plan);

/*
 * kt_moe_debug_stall -- failure-injection hook for tests, as kt_mlp_debug_stall.  With enable = 1 the
 * first block of the plan's following runs waits on a barrier nobody signals, bounded as every
 * other wait then is by `limit_us` microseconds; the wait runs out, the other blocks give up,
 * and the run ends without its output.  enable = 0 restores normal runs.  No GPU fault is involved.
 */
kt_status kt_moe_debug_stall(kt_moe_plan_t plan, int enable, int64_t limit_us);

/* kt_moe_destroy -- free the plan's workspace (after synchronising its device). */
kt_status kt_moe_destroy(kt_moe_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* KT_OPS_H */
