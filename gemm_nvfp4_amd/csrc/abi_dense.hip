// abi_dense.hip -- the exported entry points of include/nvfp4moe_dense.h: argument checks that fail closed,
// then the launches (norm.hip, linear_rows.hip, linear_grad.hip).
#include <stdint.h>

#include "abi_checks.hpp"
#include "dense.hpp"

#define NVFP4_API extern "C" __attribute__((visibility("default")))

namespace {

using nvfp4::aligned;
using nvfp4::check_weights;

bool rows_ok(int32_t M) { return M >= 0 && M <= nvfp4::MAX_DENSE_M; }

// Sizes of the norm and of its gradient (eps: negative or NaN is refused).
int check_norm(int32_t M, int32_t K, float eps)
{
    if (!rows_ok(M) || K < 1 || !(eps >= 0.0f)) return NVFP4_ERR_SHAPE;
    return K % 8 != 0 || K > nvfp4::MAX_NORM_K ? NVFP4_ERR_UNSUPPORTED : NVFP4_OK;
}

// Sizes of a gradient through an NVFP4 weight of `rows` x `k` (gated: gate and up rows).
int check_grad_sizes(int32_t M, int32_t rows, int32_t k, bool gated)
{
    if (!rows_ok(M) || rows < 1 || k < 1 || (gated && rows % 2 != 0)) return NVFP4_ERR_SHAPE;
    if (k % 128 != 0 || k > (gated ? nvfp4::MAX_LINEAR_SWIGLU_K : nvfp4::MAX_LINEAR_K) || rows % (gated ? 32 : 16) != 0 ||
        rows > nvfp4::MAX_GRAD_ROWS)
        return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

int check_grad(int32_t M, const nvfp4_weights *w, bool gated)
{
    const int st = check_weights(w);
    if (st != NVFP4_OK) return st;
    return w->groups != 1 ? NVFP4_ERR_SHAPE : check_grad_sizes(M, w->rows, w->k, gated);
}

}  // namespace

NVFP4_API int nvfp4_add_rms_norm(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, int32_t M, int32_t K,
                                 float eps, uint16_t *s, uint16_t *y, uint8_t *q, float *q_scale, void *stream)
{
    const int st = check_norm(M, K, eps);
    if (st != NVFP4_OK || M == 0) return st;
    if (!x || (!y && !q) || !q != !q_scale) return NVFP4_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(s, 16) || !aligned(y, 16) ||
        !aligned(q, 16) || !aligned(q_scale, 4))
        return NVFP4_ERR_ALIGN;
    return nvfp4::run_norm(x, residual, weight, M, K, eps, s, y, q, q_scale, static_cast<hipStream_t>(stream));
}

NVFP4_API size_t nvfp4_add_rms_norm_grad_ws_bytes(int32_t M, int32_t K)
{
    return check_norm(M, K, 0.0f) == NVFP4_OK ? nvfp4::norm_grad_ws_bytes(M, K) : 0;
}

NVFP4_API int nvfp4_add_rms_norm_grad(const uint16_t *t, const uint16_t *dy, const uint16_t *ds, const uint16_t *weight,
                                      int32_t M, int32_t K, float eps, uint16_t *dx, float *dweight, void *ws,
                                      size_t ws_bytes, void *stream)
{
    const int st = check_norm(M, K, eps);
    if (st != NVFP4_OK || (M == 0 && !dweight)) return st;
    if (M > 0) {
        if (!t || !dy || (!dx && !dweight) || (dweight && !ws)) return NVFP4_ERR_NULL;
        if (!aligned(t, 16) || !aligned(dy, 16) || !aligned(ds, 16) || !aligned(weight, 16) || !aligned(dx, 16) ||
            !aligned(ws, 16))
            return NVFP4_ERR_ALIGN;
    }
    if (!aligned(dweight, 4)) return NVFP4_ERR_ALIGN;
    if (M > 0 && dweight && ws_bytes < nvfp4::norm_grad_ws_bytes(M, K)) return NVFP4_ERR_WORKSPACE;
    return nvfp4::run_norm_grad(t, dy, ds, weight, M, K, eps, dx, dweight, ws, static_cast<hipStream_t>(stream));
}

NVFP4_API int nvfp4_linear_fp8_rows(const uint8_t *xq, const float *x_scale, int32_t M, const fp8_channel_weights *w,
                                    uint16_t *y, void *stream)
{
    if (!rows_ok(M)) return NVFP4_ERR_SHAPE;
    if (!w || !w->codes || !w->channel_scale) return NVFP4_ERR_NULL;
    if (w->rows < 1 || w->k < 16) return NVFP4_ERR_SHAPE;
    if (w->k % 128 != 0 || w->k > nvfp4::MAX_LINEAR_FP8_K || w->rows % 16 != 0 || w->rows > nvfp4::MAX_FP8_ROWS_N)
        return NVFP4_ERR_UNSUPPORTED;
    if (!aligned(w->codes, 16) || !aligned(w->channel_scale, 4)) return NVFP4_ERR_ALIGN;
    if (M == 0) return NVFP4_OK;
    if (!xq || !x_scale || !y) return NVFP4_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(y, 16)) return NVFP4_ERR_ALIGN;
    return nvfp4::run_linear_fp8_rows(xq, x_scale, M, *w, y, static_cast<hipStream_t>(stream));
}

NVFP4_API size_t nvfp4_linear_grad_ws_bytes(int32_t M, int32_t N, int32_t K)
{
    return check_grad_sizes(M, N, K, false) == NVFP4_OK ? nvfp4::linear_grad_ws_bytes(M, N, K) : 0;
}

NVFP4_API int nvfp4_linear_grad(const uint16_t *dy, int32_t M, const nvfp4_weights *w, uint16_t *dx, void *ws,
                                size_t ws_bytes, void *stream)
{
    const int st = check_grad(M, w, false);
    if (st != NVFP4_OK || M == 0) return st;
    if (!dy || !dx || !ws) return NVFP4_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(dx, 16) || !aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    if (ws_bytes < nvfp4::linear_grad_ws_bytes(M, w->rows, w->k)) return NVFP4_ERR_WORKSPACE;
    return nvfp4::run_linear_grad(dy, M, *w, dx, ws, static_cast<hipStream_t>(stream));
}

NVFP4_API size_t nvfp4_linear_swiglu_grad_ws_bytes(int32_t M, int32_t rows, int32_t K)
{
    return check_grad_sizes(M, rows, K, true) == NVFP4_OK ? nvfp4::linear_swiglu_grad_ws_bytes(M, rows, K) : 0;
}

NVFP4_API int nvfp4_linear_swiglu_grad(const uint16_t *x, const uint16_t *dh, int32_t M, const nvfp4_weights *w13,
                                       int32_t layout, uint16_t *dz, void *ws, size_t ws_bytes, void *stream)
{
    if (layout != 0 && layout != 1) return NVFP4_ERR_SHAPE;
    const int st = check_grad(M, w13, true);
    if (st != NVFP4_OK || M == 0) return st;
    if (!x || !dh || !dz || !ws) return NVFP4_ERR_NULL;
    if (!aligned(x, 16) || !aligned(dh, 16) || !aligned(dz, 16) || !aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    if (ws_bytes < nvfp4::linear_swiglu_grad_ws_bytes(M, w13->rows, w13->k)) return NVFP4_ERR_WORKSPACE;
    return nvfp4::run_linear_swiglu_grad(x, dh, M, *w13, layout, dz, ws, static_cast<hipStream_t>(stream));
}
