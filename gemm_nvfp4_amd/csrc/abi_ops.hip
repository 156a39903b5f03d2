// abi_ops.hip -- the exported entry points of include/nvfp4moe_ops.h: argument checks that fail
// closed, then the launches (moe_rows.hip, lora.hip).
#include <stdint.h>

#include "abi_checks.hpp"
#include "ops.hpp"

#define NVFP4_API extern "C" __attribute__((visibility("default")))

namespace {

using nvfp4::aligned;
using nvfp4::check_weights;
using nvfp4::plan_shape_ok;
using nvfp4::PlanLayout;

// The checks that the row operators share, in the library's order: sizes, limits, then (M > 0) pointers.
int check_rows(const void *plan, int32_t M, int32_t topk, int32_t E, int32_t K)
{
    if (!plan_shape_ok(M, topk, E) || K < 1) return NVFP4_ERR_SHAPE;
    if (E > nvfp4::MAX_EXPERTS || K % 8 != 0 || K > nvfp4::MAX_ROW_K) return NVFP4_ERR_UNSUPPORTED;
    if (M == 0) return NVFP4_OK;
    if (!plan) return NVFP4_ERR_NULL;
    return aligned(plan, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

int move_rows(int (*run)(const nvfp4::PlanView &, int32_t, int32_t, const uint16_t *, const float *, int32_t, uint16_t *,
                         hipStream_t),
              const void *plan, int32_t M, int32_t topk, int32_t E, const uint16_t *in, const float *w, int32_t K,
              uint16_t *out, void *stream)
{
    const int st = check_rows(plan, M, topk, E, K);
    if (st != NVFP4_OK || M == 0) return st;
    if (!in || !out) return NVFP4_ERR_NULL;
    if (!aligned(in, 16) || !aligned(out, 16) || !aligned(w, 4)) return NVFP4_ERR_ALIGN;
    return run(nvfp4::plan_view(plan, nvfp4::plan_layout(M, topk, E)), M, topk, in, w, K, out,
               static_cast<hipStream_t>(stream));
}

bool lora_sizes_ok(int64_t P, int32_t K, int32_t rank)
{
    return P >= 0 && P <= (int64_t(1) << 26) && K >= 1 && rank >= 1;
}

int check_lora(const nvfp4_lora *lora)
{
    if (!lora || !lora->a || !lora->b || !lora->scale) return NVFP4_ERR_NULL;
    if (lora->adapters < 1 || lora->rows < 1 || lora->k < 1 || lora->rank < 1) return NVFP4_ERR_SHAPE;
    if (!aligned(lora->a, 16) || !aligned(lora->b, 16) || !aligned(lora->scale, 4)) return NVFP4_ERR_ALIGN;
    if (lora->adapters > nvfp4::MAX_EXPERTS || lora->rank % 8 != 0 || lora->rank > nvfp4::MAX_LORA_RANK ||
        lora->k % 128 != 0 || lora->k > nvfp4::MAX_LINEAR_K || lora->rows % 16 != 0 || lora->rows > nvfp4::MAX_LORA_ROWS)
        return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

int linear_lora(const void *plan, const uint16_t *x, int32_t M, const nvfp4_weights *w, const nvfp4_lora *lora, bool gated,
                int32_t layout, uint16_t *y, void *ws, size_t ws_bytes, void *stream)
{
    if (M < 0 || M > (1 << 26) || (layout != 0 && layout != 1)) return NVFP4_ERR_SHAPE;
    int st = check_weights(w);
    if (st == NVFP4_OK) st = check_lora(lora);
    if (st != NVFP4_OK) return st;
    if (w->groups != 1 || lora->rows != w->rows || lora->k != w->k || (gated && w->rows % 2 != 0)) return NVFP4_ERR_SHAPE;
    if (gated && (w->k > nvfp4::MAX_LINEAR_SWIGLU_K || (w->rows / 2) % 16 != 0)) return NVFP4_ERR_UNSUPPORTED;
    if (M == 0) return NVFP4_OK;
    if (!plan || !x || !y || !ws) return NVFP4_ERR_NULL;
    if (!aligned(plan, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    if (ws_bytes < nvfp4::linear_lora_ws_bytes(M, w->rows, w->k, lora->rank)) return NVFP4_ERR_WORKSPACE;
    const PlanLayout L = nvfp4::plan_layout(M, 1, lora->adapters);
    return nvfp4::run_linear_lora(nvfp4::plan_view(plan, L), L, x, M, *w, *lora, gated, layout, y, ws,
                                  static_cast<hipStream_t>(stream));
}

}  // namespace

NVFP4_API int nvfp4_moe_permute(const void *plan, int32_t M, int32_t topk, int32_t E, const uint16_t *x,
                                const float *topk_weights, int32_t K, uint16_t *xs, void *stream)
{
    return move_rows(nvfp4::run_permute, plan, M, topk, E, x, topk_weights, K, xs, stream);
}

NVFP4_API int nvfp4_moe_unpermute(const void *plan, int32_t M, int32_t topk, int32_t E, const uint16_t *ys,
                                  const float *topk_weights, int32_t K, uint16_t *out, void *stream)
{
    return move_rows(nvfp4::run_unpermute, plan, M, topk, E, ys, topk_weights, K, out, stream);
}

NVFP4_API int nvfp4_moe_unpermute_grad(const void *plan, int32_t M, int32_t topk, int32_t E, const uint16_t *dout,
                                       const uint16_t *ys, const float *topk_weights, int32_t K, uint16_t *dys,
                                       float *dweights, void *stream)
{
    const int st = check_rows(plan, M, topk, E, K);
    if (st != NVFP4_OK || M == 0) return st;
    if (!dout || !ys || !dweights || (dys && !topk_weights)) return NVFP4_ERR_NULL;
    if (!aligned(dout, 16) || !aligned(ys, 16) || !aligned(dys, 16) || !aligned(dweights, 4) ||
        !aligned(topk_weights, 4))
        return NVFP4_ERR_ALIGN;
    return nvfp4::run_unpermute_grad(nvfp4::plan_view(plan, nvfp4::plan_layout(M, topk, E)), M, topk, dout, ys,
                                     topk_weights, K, dys, dweights, static_cast<hipStream_t>(stream));
}

NVFP4_API size_t nvfp4_lora_add_ws_bytes(int32_t P, int32_t K, int32_t rank)
{
    return lora_sizes_ok(P, K, rank) ? nvfp4::lora_add_ws_bytes(P, K, rank) : 0;
}

NVFP4_API int nvfp4_lora_add(const void *plan, int32_t M, int32_t topk, int32_t order, const uint16_t *x,
                             const nvfp4_lora *lora, const uint16_t *y, uint16_t *out, void *ws, size_t ws_bytes,
                             void *stream)
{
    if (!plan_shape_ok(M, topk, 1) || (order != 0 && order != 1)) return NVFP4_ERR_SHAPE;
    const int st = check_lora(lora);
    if (st != NVFP4_OK || M == 0) return st;
    if (!plan || !x || !y || !out || !ws) return NVFP4_ERR_NULL;
    if (!aligned(plan, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(out, 16) || !aligned(ws, 16))
        return NVFP4_ERR_ALIGN;
    const PlanLayout L = nvfp4::plan_layout(M, topk, lora->adapters);
    if (ws_bytes < nvfp4::lora_add_ws_bytes(L.P, lora->k, lora->rank)) return NVFP4_ERR_WORKSPACE;
    return nvfp4::run_lora_add(nvfp4::plan_view(plan, L), L, order, x, *lora, y, out, ws,
                               static_cast<hipStream_t>(stream));
}

NVFP4_API size_t nvfp4_linear_lora_ws_bytes(int32_t M, int32_t rows, int32_t K, int32_t rank)
{
    return lora_sizes_ok(M, K, rank) && rows >= 1 ? nvfp4::linear_lora_ws_bytes(M, rows, K, rank) : 0;
}

NVFP4_API int nvfp4_linear_lora(const void *plan, const uint16_t *x, int32_t M, const nvfp4_weights *w,
                                const nvfp4_lora *lora, uint16_t *y, void *ws, size_t ws_bytes, void *stream)
{
    return linear_lora(plan, x, M, w, lora, false, 0, y, ws, ws_bytes, stream);
}

NVFP4_API int nvfp4_linear_swiglu_lora(const void *plan, const uint16_t *x, int32_t M, const nvfp4_weights *w13,
                                       int32_t layout, const nvfp4_lora *lora, uint16_t *h, void *ws, size_t ws_bytes,
                                       void *stream)
{
    return linear_lora(plan, x, M, w13, lora, true, layout, h, ws, ws_bytes, stream);
}
