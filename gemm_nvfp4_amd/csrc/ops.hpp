// ops.hpp -- launchers behind include/nvfp4moe_ops.h (abi_ops.hip validates their arguments).
#pragma once

#include "../../include/nvfp4moe_ops.h"
#include "internal.hpp"

namespace nvfp4 {

constexpr int MAX_ROW_K = 65536;   // row operators: elements per row
constexpr int MAX_LORA_RANK = 256;
constexpr int MAX_LORA_ROWS = 1 << 22;  // N, within a launch's second axis

// moe_rows.hip
int run_permute(const PlanView &pv, int32_t M, int32_t topk, const uint16_t *x, const float *w, int32_t K, uint16_t *xs,
                hipStream_t s);
int run_unpermute(const PlanView &pv, int32_t M, int32_t topk, const uint16_t *ys, const float *w, int32_t K,
                  uint16_t *out, hipStream_t s);
int run_unpermute_grad(const PlanView &pv, int32_t M, int32_t topk, const uint16_t *dout, const uint16_t *ys,
                       const float *w, int32_t K, uint16_t *dys, float *dw, hipStream_t s);

// lora.hip
size_t lora_add_ws_bytes(int64_t P, int32_t K, int32_t rank);
size_t linear_lora_ws_bytes(int32_t M, int32_t rows, int32_t K, int32_t rank);
int run_lora_add(const PlanView &pv, const PlanLayout &L, int32_t order, const uint16_t *x, const nvfp4_lora &lora,
                 const uint16_t *y, uint16_t *out, void *ws, hipStream_t s);
// gated: y is h [M][rows / 2], lora's and w's rows the gate and up rows in `layout`.
int run_linear_lora(const PlanView &pv, const PlanLayout &L, const uint16_t *x, int32_t M, const nvfp4_weights &w,
                    const nvfp4_lora &lora, bool gated, int32_t layout, uint16_t *y, void *ws, hipStream_t s);

}  // namespace nvfp4
