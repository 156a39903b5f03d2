/*
 * nvfp4moe_ops.h -- further operators of the library, beside the entry points of nvfp4moe.h and
 * under the same conventions (device pointers, caller-owned buffers, calls that only enqueue on the
 * caller's stream and can be captured in a HIP graph, checks that fail closed before anything is
 * enqueued, M = 0 a successful no-op, a row's result independent of the other rows, bitwise).
 *
 * They are the other readers of the routing plan:
 *   - rows moved by the plan: tokens sorted by expert, expert rows summed back into their tokens
 *     with the routing weights, and the gradient of that sum. With them a caller runs products of
 *     its own between the plan and the combine;
 *   - low-rank adapters of many requests at once (LoRA), beside the dense NVFP4 projections or added
 *     to any finished projection. A batch's adapter ids are planned like expert ids, once for all the
 *     projections that the batch passes through.
 * None of them is on the source pages; every formula is stated here.
 */
#ifndef NVFP4MOE_OPS_H
#define NVFP4MOE_OPS_H

#include "nvfp4moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------------------------
 * Rows moved by the routing plan. Notation: pair p = t*topk + k, pos(p) = its bucket-order row (the
 * plan's pos_of_pair, -1 for a skipped pair), n_valid = the plan's count of valid pairs. `plan`, M,
 * topk and E are those of nvfp4_moe_plan; topk_weights FP32 [M][topk] or NULL (every weight 1).
 *
 * nvfp4_moe_permute: tokens sorted by expert.
 *   x  fp16 [M][K],  xs  fp16 [M*topk][K]:  xs[pos(p)] = fp16_rne( w[p] * x[p / topk] ),
 *   the FP32 product of the weight and the element; without weights the bits of x.
 *   Rows j >= n_valid of xs are not written.
 * nvfp4_moe_unpermute: expert rows back to their tokens.
 *   ys fp16 [M*topk][K] in bucket order,  out fp16 [M][K], every element written:
 *   s = +0; for k = 0..topk-1 with pos(p) >= 0: s = fmaf(w[p], ys[pos(p)], s);  out = fp16_rne(s).
 *   A token without a valid slot gets +0. What rows j >= n_valid of ys hold does not matter. Without weights it
 *   is the gradient of nvfp4_moe_permute without weights (dx from dxs); with them, of the weighted one.
 * nvfp4_moe_unpermute_grad: the gradient of nvfp4_moe_unpermute with weights.
 *   dout fp16 [M][K], ys as above; dys fp16 [M*topk][K], dweights FP32 [M][topk]:
 *   dys[pos(p)] = fp16_rne( w[p] * dout[p / topk] ),
 *   dweights[p] = sum over n of dout[p / topk][n] * ys[pos(p)][n] in FP32, in one order fixed by K;
 *   +0 for a skipped pair. Rows j >= n_valid of dys are not written. dys may be NULL: only dweights
 *   (which also gives the gradient of the weighted nvfp4_moe_permute with respect to its weights:
 *   dout = x, ys = dxs); topk_weights is then not read and may be NULL.
 *
 * Outputs must not overlap inputs. Requirements: those of nvfp4_moe_plan (topk <= 32, E <= 4096,
 * M*topk <= 2^26); K % 8 == 0 and K <= 65536; plan and fp16 rows 16-byte aligned, FP32 4-byte.
 * Errors: SHAPE for M < 0, topk, K < 1 or M*topk out of range, UNSUPPORTED for E > 4096, K % 8 or
 * K > 65536, NULL and ALIGN for the pointers.
 * --------------------------------------------------------------------------------------------- */
int nvfp4_moe_permute(const void *plan, int32_t M, int32_t topk, int32_t E, const uint16_t *x,
                      const float *topk_weights, int32_t K, uint16_t *xs, void *stream);
int nvfp4_moe_unpermute(const void *plan, int32_t M, int32_t topk, int32_t E, const uint16_t *ys,
                        const float *topk_weights, int32_t K, uint16_t *out, void *stream);
int nvfp4_moe_unpermute_grad(const void *plan, int32_t M, int32_t topk, int32_t E, const uint16_t *dout,
                             const uint16_t *ys, const float *topk_weights, int32_t K, uint16_t *dys,
                             float *dweights, void *stream);

/* Low-rank adapters of one projection: `adapters` pairs of A [rank][k] and B [rows][rank]. Adapters of
 * a smaller rank are padded with zero rows of A and zero columns of B. */
typedef struct nvfp4_lora {
    const uint16_t *a;    /* device, fp16 [adapters][rank][k], 16-byte aligned                       */
    const uint16_t *b;    /* device, fp16 [adapters][rows][rank], 16-byte aligned                    */
    const float *scale;   /* device, FP32 [adapters] (alpha / rank), 4-byte aligned                  */
    int32_t adapters, rows, k, rank;
} nvfp4_lora;

/* ---------------------------------------------------------------------------------------------
 * Low-rank adapters. A row with adapter a gets
 *   d[n] = scale[a] * sum_r v[r] * B_a[n][r],   v[r] = sum_k x[k] * A_a[r][k],
 * v in FP32 (one reduction order: 512-element chunks, each one MFMA chain, added in chunk order), and
 * the sum over r in FP32 from v to at least 22 bits of the row's largest |v| (v is scaled by a power
 * of two and split into two fp16 terms). Non-finite values of x and y follow IEEE rules and stay in
 * their row; an infinity in B makes its output column NaN or infinite for the rows of that adapter. A
 * row whose adapter id is skipped (-1, or outside
 * [0, adapters)) gets d = 0 and bitwise the result without adapters.
 *   plan   the routing plan of the adapter ids: nvfp4_moe_plan(ids [M][topk], M, topk, adapters)
 *
 * nvfp4_lora_add: adapters added to a finished result.
 *   x fp16 [M*topk][K], y and out fp16 [M*topk][N] (K = lora->k, N = lora->rows):
 *   out[i] = fp16_rne( y[i] + d ), the sum in FP32. out == y is allowed (in place).
 *   order 0: row i is pair i (with topk = 1, token i); every row of out is written.
 *   order 1: row i is bucket-order row i of the plan, as nvfp4_moe_permute writes them (adapters of
 *            a MoE's experts, with the MoE's own plan); rows i >= n_valid are not written.
 * nvfp4_linear_lora: nvfp4_linear with adapters, one rounding:
 *   y[m][n] = fp16_rne( global * sum_k x[m][k] * e2m1*e4m3 + d[n] ).  topk = 1; lora->rows = w->rows,
 *   lora->k = w->k.
 * nvfp4_linear_swiglu_lora: nvfp4_linear_swiglu with adapters on the gate and up rows:
 *   lora->rows = 2I in the row order of w13 (layout 0 or 1); g and u get their d before silu(g) * u.
 *
 *   ws   device workspace of at least nvfp4_lora_add_ws_bytes(M*topk, K, rank) or
 *        nvfp4_linear_lora_ws_bytes(M, rows, K, rank) bytes, 16-byte aligned; contents ignored on
 *        entry, overwritten. Calls that share a ws must not run concurrently. The projections keep
 *        ceil(K/512) FP32 planes of the whole output in it (0.7 GB for 4096 rows of 4352 x 5120); large
 *        batches may be passed in parts, with the same results.
 * Speed of nvfp4_lora_add: large batches take their faster kernels where M*topk >= 32*adapters, all
 * adapters of the descriptor counted, used or not. A descriptor may cover a part of a larger table
 * (a and b at its first adapter, the ids counted from there).
 * Apart from out == y, outputs and ws must not overlap inputs.
 * Requirements: rank % 8 == 0, 8 <= rank <= 256; K % 128 == 0, K <= 32768 (swiglu: 16384);
 * N % 16 == 0 (swiglu: I % 16 == 0), N <= 2^22; adapters <= 4096; those of nvfp4_moe_plan; plan, x, y, out, h,
 * a, b, codes 16-byte aligned, scale 4-byte. Errors as in nvfp4moe.h (SHAPE also where lora and w
 * disagree), all before anything is enqueued. The *_ws_bytes functions return 0 for sizes that the
 * calls reject as SHAPE.
 * --------------------------------------------------------------------------------------------- */
size_t nvfp4_lora_add_ws_bytes(int32_t P, int32_t K, int32_t rank);
int nvfp4_lora_add(const void *plan, int32_t M, int32_t topk, int32_t order, const uint16_t *x,
                   const nvfp4_lora *lora, const uint16_t *y, uint16_t *out, void *ws, size_t ws_bytes,
                   void *stream);
size_t nvfp4_linear_lora_ws_bytes(int32_t M, int32_t rows, int32_t K, int32_t rank);
int nvfp4_linear_lora(const void *plan, const uint16_t *x, int32_t M, const nvfp4_weights *w,
                      const nvfp4_lora *lora, uint16_t *y, void *ws, size_t ws_bytes, void *stream);
int nvfp4_linear_swiglu_lora(const void *plan, const uint16_t *x, int32_t M, const nvfp4_weights *w13,
                             int32_t layout, const nvfp4_lora *lora, uint16_t *h, void *ws, size_t ws_bytes,
                             void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4MOE_OPS_H */
