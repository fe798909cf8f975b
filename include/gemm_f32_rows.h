/*
 * gemm_f32_rows.h -- products whose second matrix is chosen row by row, on
 * AMD MI355X (gfx950): routing of rows ("tokens") to experts, the experts'
 * products with their gradients, the weighted sum of a token's results, and
 * low-rank adapters of many requests beside a shared product.
 *
 * Same library, conventions and return codes as gemm_f32.h: row-major
 * operands with leading dimensions, device pointers owned by the caller,
 * every call only enqueues work on `stream` (a stream of the current device)
 * and returns, nothing is allocated.  Outputs must not overlap inputs.  Calls
 * are safe from several host threads; calls that share a workspace must not
 * run concurrently.  Every result is deterministic: no atomics touch outputs.
 * All entry points may be captured into HIP graphs.
 *
 * Element types: matrices are binary32, bfloat16 or IEEE half (GEMM_F32_TYPE_*),
 * the type of every `void *` matrix of a call.  Sums are binary32 on the matrix
 * cores whatever the type (adapters: see there), rounded once to it at the end; routing computes in
 * binary64.  Pointers must be aligned to their elements; rows that are 16-byte
 * aligned (base, leading dimensions and strides) load faster.  16-bit rows that start on
 * odd elements take loads through registers, 2 to 4 times slower; so do an X of the products
 * that spans 2^31 bytes or more, and operands 256 rows of which do, 1.3 to 1.6 times slower.
 *
 * Arguments are validated in this order: the element type
 * (GEMM_F32_ERR_TYPE), sizes (GEMM_F32_ERR_DIM), leading dimensions and
 * strides (GEMM_F32_ERR_LD), options (GEMM_F32_ERR_OPTION), NULL pointers
 * (GEMM_F32_ERR_NULL), alignment (GEMM_F32_ERR_ALIGN), the workspace
 * (GEMM_F32_ERR_WORKSPACE).  The first failure is returned and nothing is
 * enqueued.  GEMM_F32_ERR_DIM also refuses what is too large:
 *   - of the products, sums and adapters N and K, P of the products, k of the sums:
 *     over 2^31 - 4096;
 *   - tiles of a product's output, 32 x 64 elements or larger: over 8388607 less the
 *     device's compute units; of the adapters', 256 x 256 (binary32 64 x 64): over 8387583
 *     (16776191);
 *   - T of routing: over 67108859, of the adapters: over 2^25.
 * Offsets, orders, positions and adapter numbers live in device
 * memory and are not validated: kernels clamp or skip what is out of range,
 * so wrong ones give wrong results but no access outside the operands.
 */
#ifndef GEMM_F32_ROWS_H
#define GEMM_F32_ROWS_H

#include <stdint.h>

#include "gemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define GEMM_F32_TYPE_F32  0   /* IEEE binary32 */
#define GEMM_F32_TYPE_BF16 1   /* bfloat16      */
#define GEMM_F32_TYPE_F16  2   /* IEEE binary16 */

/* Scores of gemm_f32_route(). */
#define GEMM_F32_SCORE_SOFTMAX 0
#define GEMM_F32_SCORE_SIGMOID 1

#define GEMM_F32_MAX_EXPERTS 1024   /* E of routing and of the slot map */
#define GEMM_F32_MAX_CHOSEN    64   /* k, and groups, of routing        */
#define GEMM_F32_MAX_RANK     256   /* R of the adapters                */

/*
 * Routing: k of E experts for each of T tokens.
 *
 *   s(t,e) = softmax over e of logits(t,e), or 1 / (1 + exp(-logits(t,e)));
 *   c(t,e) = s(t,e) + bias[e]   (bias NULL: 0), both in binary64.
 *
 * An expert is available to a token unless its logit or its bias is -inf.
 * With groups > 1 the experts form groups of E / groups consecutive ones; a
 * group's score is the sum of the group_top (1 or 2) largest c of its available
 * experts (what is not there adds nothing), and only the keep_groups groups
 * with the highest scores stay.  Of the available experts that stay, the k
 * with the largest key are chosen: the key is c with a bias and the logit
 * itself without one.  Ties go to the lowest index, of groups and of experts.
 * NaN ranks above every number, so that it shows in the weights.
 *
 *   index[t*k + j]  = the expert with the j-th largest key, -1 when fewer are
 *                     available;
 *   weight[t*k + j] = scale * s(t, index), or with `normalize` scale *
 *                     s(t, index) / sum over j of s(t, index); 0 where the index
 *                     is -1 and where that sum is 0.
 *
 * The bias chooses and does not weigh.  A normalised softmax is that of the chosen alone (the row's
 * sum cancels): NaN among the others does not reach it, and it does not underflow.
 * GEMM_F32_ERR_DIM: E outside
 * 1..GEMM_F32_MAX_EXPERTS, k outside 1..min(E, GEMM_F32_MAX_CHOSEN).
 * GEMM_F32_ERR_OPTION: unknown score; groups outside 1..GEMM_F32_MAX_CHOSEN or
 * no divisor of E; keep_groups outside 1..groups; group_top not 1 or 2.
 */
GEMM_F32_API int gemm_f32_route(int type, int T, int E, int k,
                                const void *logits, int ldl, const float *bias,
                                int score, int groups, int keep_groups, int group_top,
                                int normalize, float scale,
                                float *weight, int *index, hipStream_t stream);

/*
 * The gradient of the logits from that of the weights: dlogits(t,e) = sum over j of
 * dweight[t*k + j] * d weight[t*k + j] / d logits(t,e), for the choice `index`
 * that gemm_f32_route() made (the choice itself and the bias have none).
 * Computed in binary64 and rounded once.  Entries of index outside 0..E-1
 * count nothing.  Every element of the T x E window of dlogits is written.
 */
GEMM_F32_API int gemm_f32_route_grad(int type, int T, int E, int k,
                                     const void *logits, int ldl,
                                     int score, int normalize, float scale,
                                     const int *index, const float *dweight,
                                     void *dlogits, int lddl, hipStream_t stream);

/*
 * Slots in the order of their experts.  index[s] is slot s's expert, s < S
 * (slot t*k + j for the j-th choice of token t); slots whose expert is outside
 * 0..E-1 are left out.
 *
 *   offsets[e] = number of slots of experts below e, e = 0..E;
 *   order[p]   = the slot at place p: expert by expert, slots of an expert in
 *                rising order; -1 for p >= offsets[E];
 *   position[s] = the place of slot s, -1 if it is left out.
 *
 * The workspace is gemm_f32_expert_map_ws_size(S, E) bytes (0 for few
 * slots: then it may be NULL), 16-byte aligned; its contents on return are unspecified.
 */
GEMM_F32_API size_t gemm_f32_expert_map_ws_size(int S, int E);
GEMM_F32_API int gemm_f32_expert_map(int S, int E, const int *index,
                                     int *offsets, int *order, int *position,
                                     void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One product per group of rows.  Place p belongs to group g when
 * offsets[g] <= p < offsets[g+1] (offsets: G + 1 rising numbers within
 * 0..P).  Row r(p) of X is order[p] / per_row, or p when order is NULL; a
 * negative order[p] or a row outside 0..rows-1 reads as zeros.
 *
 *   gemm_f32_grouped:         Y(p,:)  = X(r(p),:) . W_g           [K] x [K x N]
 *   gemm_f32_grouped_grad_x:  dX(p,:) = dY(p,:) . W_g^T           [N] x [N x K]
 *   gemm_f32_grouped_grad_w:  dW_g    = sum over the p of group g of
 *                                       X(r(p),:)^T . dY(p,:)     [K x N]
 *
 * W_g(k,n) = W[g * stride_w + k * ldw + n], with stride_w >= K * ldw when G > 1
 * (of grad_w: of dW).
 * Rows of Y (dX) that belong to no group are left as they were; dW of an empty group
 * is set to +0.0.  The gradient of X itself is gemm_f32_combine() of dX.
 */
GEMM_F32_API int gemm_f32_grouped(int type, int G, int P, int N, int K,
                                  const int *offsets, const int *order, int per_row, int rows,
                                  const void *X, int ldx, const void *W, int ldw, int64_t stride_w,
                                  void *Y, int ldy, hipStream_t stream);
GEMM_F32_API int gemm_f32_grouped_grad_x(int type, int G, int P, int N, int K,
                                         const int *offsets,
                                         const void *dY, int lddy, const void *W, int ldw, int64_t stride_w,
                                         void *dX, int lddx, hipStream_t stream);
GEMM_F32_API int gemm_f32_grouped_grad_w(int type, int G, int P, int N, int K,
                                         const int *offsets, const int *order, int per_row, int rows,
                                         const void *X, int ldx, const void *dY, int lddy,
                                         void *dW, int lddw, int64_t stride_dw, hipStream_t stream);

/*
 * The weighted sum of a token's k results, which stand at places of Y (P rows):
 *
 *   out(t,:) = sum over j < k of weight[t*k + j] * Y(position[t*k + j],:)
 *
 * in the order of j, in binary32; weight NULL: 1.  A position outside
 * 0..P-1 adds nothing, so a token without results gets +0.0.
 *
 * Its gradients: dY(position,:) = weight * dout(t,:) and dweight[t*k + j] =
 * the inner product of Y(position,:) and dout(t,:) (0 where the position is
 * out of range).  Positions must differ.  Rows of dY that no position names
 * are left as they were.  dY or dweight may be NULL (not computed); without dweight, Y may be.
 */
GEMM_F32_API int gemm_f32_combine(int type, int T, int k, int N, int P,
                                  const int *position, const float *weight,
                                  const void *Y, int ldy, void *out, int ldo, hipStream_t stream);
GEMM_F32_API int gemm_f32_combine_grad(int type, int T, int k, int N, int P,
                                       const int *position, const float *weight,
                                       const void *Y, int ldy, const void *dout, int lddo,
                                       void *dY, int lddy, float *dweight, hipStream_t stream);

/*
 * A shared product with each row's own low-rank addition:
 *
 *   Y(t,:) = X(t,:) . W + scale[a] * (X(t,:) . A_a) . B_a,   a = adapter[t]
 *
 * X [T x K], W [K x N], A_a [K x R] at A + a * stride_a, B_a [R x N] at
 * B + a * stride_b, a < n; scale NULL: 1.  Rows whose adapter is outside
 * 0..n-1 get the shared product alone.  scale[a] * (X . A_a) is a binary32 sum; calls
 * of many rows keep it in two parts of a 16-bit type, which is off by at most 2^-16 of each
 * value for bfloat16, and for half by 2^-22 of it or 2^-39 of its row's largest.  R = 0 or
 * n = 0: no additions, and A, B, adapter may be NULL.  R is at most
 * GEMM_F32_MAX_RANK.  Any order of adapters is right; rows of one
 * adapter side by side are fastest.
 *
 * The workspace is gemm_f32_adapters_ws_size(type, T, N, K, R) bytes, 16-byte
 * aligned; its contents on return are unspecified.
 */
GEMM_F32_API size_t gemm_f32_adapters_ws_size(int type, int T, int N, int K, int R);
GEMM_F32_API int gemm_f32_adapters(int type, int T, int N, int K, int R, int n,
                                   const void *X, int ldx, const void *W, int ldw,
                                   const void *A, int lda, int64_t stride_a,
                                   const void *B, int ldb, int64_t stride_b,
                                   const int *adapter, const float *scale,
                                   void *Y, int ldy,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F32_ROWS_H */
