// dense.hpp -- launchers behind include/nvfp4moe_dense.h (abi_dense.hip validates their arguments).
#pragma once

#include "../../include/nvfp4moe_dense.h"
#include "internal.hpp"

namespace nvfp4 {

constexpr int MAX_NORM_K = 32768;            // 1024 threads of four 8-element pieces
constexpr int MAX_DENSE_M = 1 << 26;
constexpr int MAX_GRAD_ROWS = 1 << 20;       // N: buffer offsets stay below BUF_OOB (asserted in linear_grad.hip)
// N of the 8-bit rows: a launch holds fewer than 2^32 threads along one axis, and up to 32 rows take tiles of 32 x 32, 256
// threads each, dealt out in eights. Larger batches that fit in 288 GB (2 M N bytes of y, 128 N of codes) take fewer.
constexpr int MAX_FP8_ROWS_N = (1 << 29) - 256;

// norm.hip
size_t norm_grad_ws_bytes(int32_t M, int32_t K);
int run_norm(const uint16_t *x, const uint16_t *r, const uint16_t *w, int32_t M, int32_t K, float eps, uint16_t *s,
             uint16_t *y, uint8_t *q, float *q_scale, hipStream_t st);
int run_norm_grad(const uint16_t *t, const uint16_t *dy, const uint16_t *ds, const uint16_t *w, int32_t M, int32_t K,
                  float eps, uint16_t *dx, float *dw, void *ws, hipStream_t st);

// linear_rows.hip
int run_linear_fp8_rows(const uint8_t *xq, const float *xs, int32_t M, const fp8_channel_weights &w, uint16_t *y,
                        hipStream_t s);

// linear_grad.hip
size_t linear_grad_ws_bytes(int32_t M, int32_t N, int32_t K);
int run_linear_grad(const uint16_t *dy, int32_t M, const nvfp4_weights &w, uint16_t *dx, void *ws, hipStream_t s);
size_t linear_swiglu_grad_ws_bytes(int32_t M, int32_t rows, int32_t K);
int run_linear_swiglu_grad(const uint16_t *x, const uint16_t *dh, int32_t M, const nvfp4_weights &w, int32_t layout,
                           uint16_t *dz, void *ws, hipStream_t s);

}  // namespace nvfp4
