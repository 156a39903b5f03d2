/*
 * nvfp4moe_dense.h -- what stands around the dense projections of nvfp4moe.h: the norm in front of them,
 * the projection of 8-bit rows, and the gradients of the norm and of the projections towards their inputs
 * (training around frozen NVFP4 weights). Same library and conventions as nvfp4moe.h (device pointers,
 * caller-owned buffers, calls that only enqueue on the caller's stream and can be captured in a HIP graph,
 * checks that fail closed before anything is enqueued, M = 0 a successful no-op).
 *
 * A row's result does not depend on the other rows, bitwise, with two exceptions that are stated below: a
 * sum over the rows (dweight), and the order of the gradients' sums, which the batch size chooses.
 * None of these operators is on the source pages; every formula is stated here.
 */
#ifndef NVFP4MOE_DENSE_H
#define NVFP4MOE_DENSE_H

#include "nvfp4moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------------------------
 * Root-mean-square norm with the residual's sum in front of it. x, residual fp16 [M][K], weight fp16 [K]:
 *   t[m][k] = x[m][k] + residual[m][k]  (FP32; residual NULL: x),
 *   v[m][k] = t * rstd * weight[k],  rstd = 1 / sqrt(mean over k of t^2 + eps), FP32 throughout
 *   (weight NULL: 1). The outputs, each of them NULL where it is not wanted, but not y and q both:
 *   s        fp16 [M][K]    fp16_rne(t), the residual stream of the next layer
 *   y        fp16 [M][K]    fp16_rne(v)
 *   q        uint8 [M][K]   E4M3FN bytes e4m3_rne(v * (1 / q_scale[m])), for nvfp4_linear_fp8_rows
 *   q_scale  FP32 [M]       max(max over k of |v| / 448, 2^-100); with q, and only with it
 * The norm is taken of t, not of its fp16 rounding. A row of zeros with eps = 0 gives NaN (0 / 0). A NaN or an
 * infinity in t makes v NaN where t is not finite (an infinity makes the rest of its row 0), and with it q_scale
 * and all of the row's q NaN.
 * s may be x or residual; y may be x or residual (in place), but not s. Outputs must not overlap inputs
 * otherwise.
 *
 * nvfp4_add_rms_norm_grad: the gradient. t fp16 [M][K] is the norm's input (the s of the forward call, or its x
 * without a residual), dy fp16 [M][K] the gradient of y; ds fp16 [M][K] the gradient of s from elsewhere (the
 * residual stream; NULL: none). With g = weight * dy:
 *   dx[m][k] = fp16_rne( ds + rstd * (g - t * (rstd^2 * mean over k of g * t)) ), the gradient of x and of residual,
 *   dweight[k] = sum over m of dy[m][k] * t[m][k] * rstd[m]   FP32, in one order fixed by M and K; NULL: not wanted.
 *   dx may be NULL where dweight is given. dx may be dy or ds.
 *   ws  device workspace of at least nvfp4_add_rms_norm_grad_ws_bytes(M, K) bytes, 16-byte aligned (with dweight;
 *       else it may be NULL); contents ignored on entry. Calls that share a ws must not run concurrently.
 *   With M = 0 dweight, where given, is set to zero (the sum over no rows).
 *
 * Requirements: K % 8 == 0, 8 <= K <= 32768; M <= 2^26; eps >= 0; fp16 rows, weight and q 16-byte aligned, FP32
 * 4-byte. Errors: SHAPE for M < 0 or > 2^26, K < 1, eps negative or NaN; UNSUPPORTED for K % 8 or K > 32768; NULL,
 * ALIGN, WORKSPACE. The *_ws_bytes functions return 0 for sizes that the calls reject.
 * --------------------------------------------------------------------------------------------- */
int nvfp4_add_rms_norm(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, int32_t M, int32_t K,
                       float eps, uint16_t *s, uint16_t *y, uint8_t *q, float *q_scale, void *stream);
size_t nvfp4_add_rms_norm_grad_ws_bytes(int32_t M, int32_t K);
int nvfp4_add_rms_norm_grad(const uint16_t *t, const uint16_t *dy, const uint16_t *ds, const uint16_t *weight, int32_t M,
                            int32_t K, float eps, uint16_t *dx, float *dweight, void *ws, size_t ws_bytes,
                            void *stream);

/* ---------------------------------------------------------------------------------------------
 * The channel-FP8 projection of 8-bit rows (nvfp4_linear_fp8 with its activations in 8 bits too):
 *   y[m][n] = fp16_rne( (x_scale[m] * s[n]) * sum_k e4m3(xq[m][k]) * e4m3(W[n][k]) ),  FP32 accumulation,
 *   xq uint8 [M][K] E4M3FN bytes, x_scale FP32 [M], w rows = N, k = K, y fp16 [M][N].
 * The sum is one chain of 128-element steps, in order, at every batch size: a batch is bitwise equal to single-row
 * calls. NaN bytes and infinite or NaN scales follow IEEE rules and stay in their row or column.
 * Requirements: K % 128 == 0 and K <= 16384; N % 16 == 0 and N <= 2^29 - 256; M <= 2^26; xq, y, codes 16-byte aligned,
 * FP32 4-byte. Errors: as nvfp4_linear_fp8.
 * --------------------------------------------------------------------------------------------- */
int nvfp4_linear_fp8_rows(const uint8_t *xq, const float *x_scale, int32_t M, const fp8_channel_weights *w, uint16_t *y,
                          void *stream);

/* ---------------------------------------------------------------------------------------------
 * Gradients through frozen NVFP4 weights.
 * nvfp4_linear_grad: of nvfp4_linear towards its input, w groups = 1, rows = N, k = K:
 *   dx[m][k] = fp16_rne( global * sum_n dy[m][n] * e2m1*e4m3[n][k] ),  dy fp16 [M][N], dx fp16 [M][K].
 *   It serves the gated projection too: w13 with the dz of the call below gives the gradient of its x.
 * nvfp4_linear_swiglu_grad: of nvfp4_linear_swiglu towards its gate and up rows, which it computes again from x:
 *   x fp16 [M][K], dh fp16 [M][I], w13 groups = 1, rows = 2I, k = K in `layout` (as for nvfp4_linear_swiglu),
 *   g and u as there, sig = 1 / (1 + exp(-g)), all FP32:
 *   d gate = fp16_rne( dh * u * sig * (1 + g * (1 - sig)) ),  d up = fp16_rne( dh * g * sig ),
 *   written to dz fp16 [M][2I] in the row order of w13 (layout 0: gates in columns [0, I), ups behind them;
 *   layout 1: gate i in column 2i, up i in column 2i + 1).
 *
 * Sums are FP32. Their order is fixed by N, K and the batch size: a row's result does not depend on what the other
 * rows hold, but may differ in its last bits between batches of different sizes (large ones run other kernels). An
 * infinity or a NaN in a row of dy, x or dh stays in that row.
 *   ws  device workspace of at least nvfp4_linear_grad_ws_bytes(M, N, K) or nvfp4_linear_swiglu_grad_ws_bytes(M, 2I,
 *       K) bytes, 16-byte aligned; contents ignored on entry, overwritten (large batches hold the decoded weight
 *       in it, 2 bytes an element; smaller ones FP32 partial sums; some of the gated ones nothing). Calls that share a ws must not run concurrently.
 * Outputs and ws must not overlap inputs.
 * Requirements: K % 128 == 0, N % 16 == 0 (swiglu: I % 16 == 0), N <= 2^20; K <= 32768 (swiglu: 16384); M <= 2^26;
 * dy, dx, x, dh, dz, codes 16-byte aligned. Errors as in nvfp4moe.h, all before anything is enqueued. The *_ws_bytes
 * functions return 0 for sizes that the calls reject.
 * --------------------------------------------------------------------------------------------- */
size_t nvfp4_linear_grad_ws_bytes(int32_t M, int32_t N, int32_t K);
int nvfp4_linear_grad(const uint16_t *dy, int32_t M, const nvfp4_weights *w, uint16_t *dx, void *ws, size_t ws_bytes,
                      void *stream);
size_t nvfp4_linear_swiglu_grad_ws_bytes(int32_t M, int32_t rows, int32_t K);
int nvfp4_linear_swiglu_grad(const uint16_t *x, const uint16_t *dh, int32_t M, const nvfp4_weights *w13, int32_t layout,
                             uint16_t *dz, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4MOE_DENSE_H */
