/*
 * gemm_f32_ffn.h -- operators of a transformer's feed-forward half on AMD
 * MI355X (gfx950): the root-mean-square norm with the residual's addition (and
 * its gradient), rows in 8 bits with a scale each, the product of such
 * rows with 8-bit weights, and the gated pair of projections (with its
 * gradient), dense or per group of rows.
 *
 * Same library, conventions and return codes as gemm_f32_rows.h: row-major
 * matrices of the types GEMM_F32_TYPE_* with leading dimensions, device
 * pointers owned by the caller, every call only enqueues work on `stream` (a
 * stream of the current device) and returns, nothing is allocated.  Calls are
 * safe from several host threads; calls that share a workspace must not run
 * concurrently.  Every result is deterministic.  All entry points may be
 * captured into HIP graphs.  Weights of the norm, scales and biases are
 * binary32 vectors.
 *
 * Outputs must not overlap inputs, with one exception: where a matrix
 * of the norms, of their gradient or of gemm_f32_gate_grad() goes in and one of the same shape
 * comes out, both may be the same (address and leading dimension).
 *
 * Factors of a result are binary32 and round as such: where S r (of the norm), act(g)
 * or act'(g) is under 2^-126, it is off by up to 2^-149, 2^-119 or 2^-117, and the
 * result by that times its other factors.  (8-bit rows have no such error.)
 *
 * Validation order: the element type (GEMM_F32_ERR_TYPE), sizes
 * (GEMM_F32_ERR_DIM: negative, over 2^31 - 4096, or more tiles than a grid
 * has), leading dimensions and strides (GEMM_F32_ERR_LD), options
 * (GEMM_F32_ERR_OPTION), NULL pointers (GEMM_F32_ERR_NULL), alignment
 * (GEMM_F32_ERR_ALIGN: pointers must be aligned to their elements), the
 * workspace (GEMM_F32_ERR_WORKSPACE).  The first failure is returned and
 * nothing is enqueued.
 */
#ifndef GEMM_F32_FFN_H
#define GEMM_F32_FFN_H

#include "gemm_f32_rows.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Gates: what act(g) is. */
#define GEMM_F32_GATE_NONE      0
#define GEMM_F32_GATE_SILU      1   /* g / (1 + exp(-g))                                        */
#define GEMM_F32_GATE_GELU      2   /* g (1 + erf(g / sqrt 2)) / 2                              */
#define GEMM_F32_GATE_GELU_TANH 3   /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2        */

#define GEMM_F32_MAX_INT8_DEPTH 131071   /* K of the 8-bit product: its sums are exact in 32 bits */

/*
 * Root-mean-square norm of the T rows, N long, of S = X + residual:
 *
 *   S(t,n) = X(t,n) + residual(t,n), rounded to the type     (residual NULL: S = X)
 *   r(t)   = 1 / sqrt(sum over n of S(t,n)^2 / N + eps)
 *   Y(t,n) = S(t,n) * r(t) * weight[n], rounded to the type     (weight NULL: 1)
 *
 * The norm is that of the stored S, so that the two steps give what they would
 * one after the other, and that a gradient reads the same numbers.
 * sum receives S; it may be NULL, and is not written without a residual.  Squares
 * are summed in binary64: finite rows do not overflow.  eps must be positive and finite
 * (GEMM_F32_ERR_OPTION).
 */
GEMM_F32_API int gemm_f32_rms_norm(int type, int T, int N,
                                   const void *X, int ldx, const void *residual, int ldr,
                                   const float *weight, float eps,
                                   void *sum, int lds, void *Y, int ldy, hipStream_t stream);

/*
 * The same with each row y = S r weight in 8 bits, computed in binary64 and never
 * rounded in between:
 *
 *   scale[t] = max(largest |y(t,n)| / 127, 2^-126), rounded to binary32
 *   Q(t,n)   = y(t,n) / scale[t] to the nearest whole number, ties to even, in -127..127
 *
 * so that Q * scale is y to within half a scale.  A row whose y has a NaN or an
 * infinity, or whose scale would be one, gets scale NaN and Q = 0: it shows in every result.
 */
GEMM_F32_API int gemm_f32_rms_norm_int8(int type, int T, int N,
                                        const void *X, int ldx, const void *residual, int ldr,
                                        const float *weight, float eps,
                                        void *sum, int lds, int8_t *Q, int ldq, float *scale,
                                        hipStream_t stream);

/*
 * Gradients of gemm_f32_rms_norm() from dY, at the S of the forward call (X
 * without a residual) with its weight and eps; dsum is the gradient that reaches S
 * otherwise (NULL: none).  With m(t) = sum over n of weight[n] dY(t,n) S(t,n) / N:
 *
 *   dX(t,n)    = r(t) (weight[n] dY(t,n) - S(t,n) r(t)^2 m(t)) + dsum(t,n)
 *   dweight[n] = sum over t of dY(t,n) S(t,n) r(t)
 *
 * dX is the gradient of X and of the residual.  dX or dweight may be NULL (not
 * computed).  dweight's sums are binary32 within a workgroup's rows and binary64
 * over the workgroups, in a fixed order.  The workspace is
 * gemm_f32_rms_norm_grad_ws_size(T, N) bytes, 16-byte aligned, needed for dweight only; its
 * contents on return are unspecified.  dX may be dY, S or dsum itself.
 */
GEMM_F32_API size_t gemm_f32_rms_norm_grad_ws_size(int T, int N);
GEMM_F32_API int gemm_f32_rms_norm_grad(int type, int T, int N,
                                        const void *dY, int lddy, const void *S, int lds,
                                        const float *weight, float eps,
                                        const void *dsum, int ldds,
                                        void *dX, int lddx, float *dweight,
                                        void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Rows in 8 bits: y(t,n) = X(t,n), or with a gate act(X(t,n)) X(t,N+n) of rows 2N
 * long; scale and Q as above.
 */
GEMM_F32_API int gemm_f32_quantize(int type, int gate, int T, int N, const void *X, int ldx,
                                   int8_t *Q, int ldq, float *scale, hipStream_t stream);

/*
 * The product of 8-bit rows and 8-bit weights with a scale for each token
 * (row of Q) and channel (row of W):
 *
 *   Y(t,n) = (sum over k of Q(t,k) W(n,k)) * (scale[t] * w_scale[n]) + bias[n]
 *
 * rounded to the type; Q [T x K], W [N x K], both with k contiguous (W as
 * gemm_f32_quantize() makes it from a weight's rows, one per output channel);
 * bias NULL: 0.  The sums are exact (K over GEMM_F32_MAX_INT8_DEPTH is
 * GEMM_F32_ERR_DIM).  Binary32 results are computed in binary64 and rounded once.
 * For the 16-bit types the sums are rounded to binary32 and scaled there, so that
 * scales whose product is no binary32 number give infinities (NaN for a sum of 0) or lose digits.
 */
GEMM_F32_API int gemm_f32_int8(int type, int T, int N, int K,
                               const int8_t *Q, int ldq, const float *scale,
                               const int8_t *W, int ldw, const float *w_scale,
                               const float *bias, void *Y, int ldy, hipStream_t stream);

/*
 * Gated projections per group of rows.  Places, offsets, order, per_row and rows as in
 * gemm_f32_grouped(); offsets NULL with G = 1: all P places are in the one group
 * (a dense block).  W_g [K x 2N] holds the gate's columns and then the others:
 *
 *   [g u](p,:) = X(r(p),:) . W_g                              2N binary32 sums
 *   H(p,n)     = act(g(p,n)) * u(p,n), rounded once           [P x N]
 *   pre(p,:)   = [g u](p,:) rounded to the type               [P x 2N], NULL: not kept
 *
 * Rows of H and pre that belong to no group are left as they were.  Its gradients,
 * with pre as kept: dpre = gemm_f32_gate_grad(), then gemm_f32_grouped_grad_x() and
 * _grad_w() of dpre (2N columns):
 *
 *   dpre(p,n)   = dH(p,n) * u * act'(g),   dpre(p,N+n) = dH(p,n) * act(g)
 *
 * rounded once (the products' results then have the errors of two roundings); row by
 * row for all P rows (those of no group give what stands in them).
 * gemm_f32_grouped_grad_x() and _grad_w() take offsets NULL with G = 1 too.
 */
GEMM_F32_API int gemm_f32_gated(int type, int gate, int G, int P, int N, int K,
                                const int *offsets, const int *order, int per_row, int rows,
                                const void *X, int ldx, const void *W, int ldw, int64_t stride_w,
                                void *H, int ldh, void *pre, int ldp, hipStream_t stream);
GEMM_F32_API int gemm_f32_gate_grad(int type, int gate, int P, int N,
                                    const void *pre, int ldp, const void *dH, int lddh,
                                    void *dpre, int lddp, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F32_FFN_H */
