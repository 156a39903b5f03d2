// abi_checks.hpp -- argument checks shared by the entry points (abi.hip, abi_ops.hip). Host only.
#pragma once

#include "internal.hpp"

namespace nvfp4 {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool plan_shape_ok(int32_t M, int32_t topk, int32_t E)
{
    return M >= 0 && topk >= 1 && topk <= MAX_TOPK && E >= 1 && (int64_t)M * topk <= (int64_t(1) << 26);
}

inline int check_weights(const nvfp4_weights *w)
{
    if (!w || !w->codes || !w->scales || !w->global_scale) return NVFP4_ERR_NULL;
    if (w->groups < 1 || w->rows < 1 || w->k < 16 || w->k % 16 != 0) return NVFP4_ERR_SHAPE;
    if (!aligned(w->codes, 16) || !aligned(w->scales, 8) || !aligned(w->global_scale, 4)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

}  // namespace nvfp4
