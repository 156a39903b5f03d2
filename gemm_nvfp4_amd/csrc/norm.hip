// norm.hip -- the root-mean-square norm with the residual's sum, FP16 or 8-bit rows, and its gradient
// (include/nvfp4moe_dense.h).
//
// Both are bound by memory: a row is read once into registers (8-element pieces, 16 bytes a lane), its sums
// are taken there, and the outputs are written from there. How many threads share a row depends on K alone,
// so a row's sums have one order whatever the batch: thread j takes pieces j, j + T, j + 2T, ...; its elements
// are added in ascending order, then a butterfly over the 64 lanes, then the waves in order.
// Measured, the least of twelve traced calls: one row of 2048 2.6 us (start-up; the call from Python 6.2), 333 rows of 5120 to 8
// bits 5.3 us, 8192 rows of 2048 26.5 us, 5.1 TB/s, a copy's rate; the gradient of 333 rows of 5120 6.9 + 2.3 us, of 8192
// rows of 2048 26.3 + 4.0 us (30.3 a call back to back, 4.4 TB/s).
#include "dense.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {
namespace {

constexpr int WAVE_ROWS = 4;  // rows per block where a wave has a row to itself
// The rows' blocks are split over x and y: a launch holds fewer than 2^32 threads along one axis.
constexpr int GRID_X = 1 << 20;

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;  // the same bits in every lane: each step adds the same pair in both of its lanes
}

// Sums of NS values over the T threads of a row, of which this is number j. T = 64: within the wave. Else over the row's
// waves, in order; `red` holds NS * T / 64 floats and is not written again before another barrier.
template <int T, int NS>
__device__ __forceinline__ void row_sums(float (&v)[NS], float *red, int j)
{
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = wave_sum(v[i]);
    if constexpr (T > 64) {
        constexpr int W = T / 64;
        if ((j & 63) == 0) {
#pragma unroll
            for (int i = 0; i < NS; ++i) red[i * W + (j >> 6)] = v[i];
        }
        lds_barrier();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float s = red[i * W];
#pragma unroll
            for (int w = 1; w < W; ++w) s += red[i * W + w];
            v[i] = s;
        }
    }
}

__device__ __forceinline__ f16x8 load8(const f16 *p) { return *reinterpret_cast<const f16x8 *>(p); }

// The row's |v| maximum as FP32 bits: NaN lies above infinity and that above every number, so an integer
// maximum keeps a NaN, where a floating one drops it.
template <int T>
__device__ __forceinline__ uint32_t row_max_bits(uint32_t v, uint32_t *red)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        lds_barrier();
#pragma unroll
        for (int w = 0; w < T / 64; ++w) v = max(v, red[w]);
    }
    return v;
}

// T threads per row (64: four rows a block, a wave each), V pieces per thread.
template <int T, int V, bool Q>
__global__ __launch_bounds__(T == 64 ? 64 * WAVE_ROWS : T) void norm_kernel(
    const f16 *x, const f16 *r, const f16 *__restrict__ w, int M, int K, float eps, f16 *s, f16 *y, uint8_t *q, float *q_scale)
{
    __shared__ float red[T / 64];
    __shared__ uint32_t red_max[T / 64];
    const int block = (int)blockIdx.y * GRID_X + (int)blockIdx.x;
    const int row = T == 64 ? block * WAVE_ROWS + (threadIdx.x >> 6) : block;
    const int j = T == 64 ? threadIdx.x & 63 : threadIdx.x;
    if (row >= M) return;  // T = 64: wave-uniform, and no barrier follows; else block-uniform
    const size_t base = (size_t)row * K;
    const int pieces = K >> 3;
    f16x8 a[V], b[V], g[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int p = j + v * T;
        a[v] = b[v] = zero8();
        if (p < pieces) {
            a[v] = load8(x + base + 8 * p);
            if (r) b[v] = load8(r + base + 8 * p);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int p = j + v * T;
        g[v] = f16x8{1, 1, 1, 1, 1, 1, 1, 1};
        if (w && p < pieces) g[v] = load8(w + 8 * p);
    }
    float t[V][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t[v][e] = r ? (float)a[v][e] + (float)b[v][e] : (float)a[v][e];
            sum[0] = fmaf(t[v][e], t[v][e], sum[0]);
        }
    }
    row_sums<T, 1>(sum, red, j);
    const float rstd = 1.0f / sqrtf(sum[0] / (float)K + eps);
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int p = j + v * T;
        f16x8 so, yo;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            so[e] = f16_of_f32(t[v][e]);
            t[v][e] = (t[v][e] * rstd) * (float)g[v][e];
            yo[e] = f16_of_f32(t[v][e]);
            if (Q && p < pieces) top = max(top, __float_as_uint(t[v][e]) & 0x7fffffffu);
        }
        if (p < pieces) {
            if (s) *reinterpret_cast<f16x8 *>(s + base + 8 * p) = so;
            if (y) *reinterpret_cast<f16x8 *>(y + base + 8 * p) = yo;
        }
    }
    if constexpr (Q) {
        const float most = __uint_as_float(row_max_bits<T>(top, red_max)) / 448.0f;
        const float scale = most < 0x1p-100f ? 0x1p-100f : most;  // a NaN stays
        const float inv = 1.0f / scale;
        if (j == 0) q_scale[row] = scale;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int p = j + v * T;
            uint32_t o[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float *f = &t[v][4 * h];
                o[h] = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * inv, f[1] * inv, 0, false);
                o[h] = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * inv, f[3] * inv, o[h], true);
            }
            if (p < pieces) *reinterpret_cast<uint2 *>(q + base + 8 * p) = make_uint2(o[0], o[1]);
        }
    }
}

// ---- gradient --------------------------------------------------------------------------------------
// Groups of T threads walk the rows in steps of the number of groups; each thread sums its columns' share of dweight,
// in registers, or in LDS where 1024 threads leave no registers for it. A block's groups meet in LDS in order, and
// the blocks' sums [G][K] are added by a second launch: G, at most one block per CU, decides how much that moves (333
// rows of 5120 took 11.5 us with a block a row and 7 MB of sums). The next row's loads are in flight while a row's sums
// are taken. G depends on M and K alone. With few turns what bounds it is latency: ds is asked for after t and dy have come.
constexpr int GRAD_BLOCKS = 256;

constexpr int grad_groups(int T) { return T == 64 ? 8 : T == 256 ? 2 : 1; }  // 512 threads but for the widest rows
inline int grad_blocks(int M, int T)
{
    const int g = grad_groups(T);
    const int need = (M + g - 1) / g;
    return need < GRAD_BLOCKS ? need : GRAD_BLOCKS;
}

template <int T, int V>
__global__ __launch_bounds__(T * grad_groups(T)) void norm_grad_kernel(const f16 *__restrict__ t, const f16 *dy, const f16 *ds,
                                                                       const f16 *__restrict__ w, int M, int K, float eps,
                                                                       f16 *dx, float *__restrict__ part)
{
    constexpr int GROUPS = grad_groups(T);
    // 1024 threads have 128 registers each: no next row, dweight in LDS, weight and ds read where they are used.
    constexpr bool IN_LDS = T == 1024, AHEAD = T < 1024;
    __shared__ float red[2][GROUPS][2 * (T / 64)];
    __shared__ __attribute__((aligned(16))) f32x4 sums[(IN_LDS || GROUPS > 1) ? 2 * V * T : 1];
    const int j = threadIdx.x % T, group = threadIdx.x / T;
    const int pieces = K >> 3, stride = gridDim.x * GROUPS;
    f32x4 dw[V][2];
    auto weight = [&](int p) { return w && p < pieces ? load8(w + 8 * p) : f16x8{1, 1, 1, 1, 1, 1, 1, 1}; };
    f16x8 g[AHEAD ? V : 1];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (AHEAD) g[v] = weight(j + v * T);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (IN_LDS) sums[(v * 2 + h) * T + j] = f32x4{0.f, 0.f, 0.f, 0.f};
            else dw[v][h] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
    f16x8 a[V], d[V];
    auto load = [&](int row) {
        const size_t base = (size_t)row * K;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int p = j + v * T;
            a[v] = d[v] = zero8();
            if (p < pieces && row < M) {
                a[v] = load8(t + base + 8 * p);
                d[v] = load8(dy + base + 8 * p);
            }
        }
    };
    const int row0 = blockIdx.x * GROUPS + group;
    load(row0);
    int turn = 0;
    // Every group of a block makes the same number of turns, since they share the barriers; rows past the last are zeros.
    for (int first = blockIdx.x * GROUPS; first < M; first += stride, turn ^= 1) {
        const int row = first + group;
        const size_t base = (size_t)row * K;
        const bool in = row < M;
        auto residual = [&](int p) { return ds && in && p < pieces ? load8(ds + base + 8 * p) : zero8(); };
        f16x8 c[AHEAD ? V : 1];
        if (AHEAD) {
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] = residual(j + v * T);
        }
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const f16x8 gv = AHEAD ? g[AHEAD ? v : 0] : weight(j + v * T);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float tv = (float)a[v][e];
                sum[0] = fmaf(tv, tv, sum[0]);
                sum[1] = fmaf((float)gv[e] * (float)d[v][e], tv, sum[1]);
            }
        }
        f16x8 a0[V], d0[V];
        if (AHEAD) {
#pragma unroll
            for (int v = 0; v < V; ++v) a0[v] = a[v], d0[v] = d[v];
            if (first + stride < M) load(row + stride);
        }
        row_sums<T, 2>(sum, red[turn][group], j);
        const float rstd = 1.0f / sqrtf(sum[0] / (float)K + eps);
        const float along = rstd * rstd * (sum[1] / (float)K);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int p = j + v * T;
            const f16x8 &av = AHEAD ? a0[v] : a[v], &dv = AHEAD ? d0[v] : d[v];
            const f16x8 gv = AHEAD ? g[AHEAD ? v : 0] : weight(p), cv = AHEAD ? c[AHEAD ? v : 0] : residual(p);
            f16x8 o;
            f32x4 part_dw[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) part_dw[h] = IN_LDS ? sums[(v * 2 + h) * T + j] : dw[v][h];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float tv = (float)av[e], dy1 = (float)dv[e];
                // a row past the last has rstd = 1 / sqrt(eps), infinite for eps = 0: it must add nothing
                part_dw[e >> 2][e & 3] = fmaf(dy1, in ? tv * rstd : 0.0f, part_dw[e >> 2][e & 3]);
                const float dxv = rstd * ((float)gv[e] * dy1 - tv * along);
                o[e] = f16_of_f32(ds ? (float)cv[e] + dxv : dxv);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (IN_LDS) sums[(v * 2 + h) * T + j] = part_dw[h];
                else dw[v][h] = part_dw[h];
            }
            if (dx && in && p < pieces) *reinterpret_cast<f16x8 *>(dx + base + 8 * p) = o;
        }
        if (!AHEAD && first + stride < M) load(row + stride);
    }
    if (!part) return;  // uniform over the grid
    float *out = part + (size_t)blockIdx.x * K;
    if constexpr (GROUPS > 1) {
        for (int i = 0; i < GROUPS; ++i) {
            if (group == i) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f32x4 &c = sums[(v * 2 + h) * T + j];
                        dw[v][h] = i == 0 ? dw[v][h] : c + dw[v][h];
                        c = dw[v][h];
                    }
            }
            lds_barrier();
        }
        if (group != GROUPS - 1) return;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int p = j + v * T;
        if (p < pieces) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<f32x4 *>(out + 8 * p + 4 * h) = IN_LDS ? sums[(v * 2 + h) * T + j] : dw[v][h];
        }
    }
}

// dweight[k] = sum over the G blocks' sums: thread (i, c) of a block adds planes i, i + 32, ... of column c, then
// the 32 threads of a column meet in LDS, in order.
constexpr int DW_COLS = 32, DW_SPLIT = 32;

__global__ __launch_bounds__(DW_COLS * DW_SPLIT) void norm_dweight_kernel(const float *__restrict__ part, int G, int K,
                                                                         float *__restrict__ dw)
{
    __shared__ float sums[DW_SPLIT][DW_COLS];
    const int c = threadIdx.x & (DW_COLS - 1), i = threadIdx.x / DW_COLS;
    const int k = blockIdx.x * DW_COLS + c;
    float s = 0.0f;
    if (k < K) {
#pragma unroll 4
        for (int g = i; g < G; g += DW_SPLIT) s += part[(size_t)g * K + k];
    }
    sums[i][c] = s;
    lds_barrier();
    if (i == 0 && k < K) {
#pragma unroll
        for (int u = 1; u < DW_SPLIT; ++u) s += sums[u][c];
        dw[k] = s;
    }
}

// Threads per row and pieces per thread, from K: a wave up to 2048, 256 threads up to 8192, 1024 above.
template <typename F>
int by_width(int K, F &&f)
{
    const int pieces = K >> 3;
    auto with = [&](auto T) {
        constexpr int t = decltype(T)::value;
        switch ((pieces + t - 1) / t) {
        case 1: return f(T, std::integral_constant<int, 1>{});
        case 2: return f(T, std::integral_constant<int, 2>{});
        case 3: return f(T, std::integral_constant<int, 3>{});
        default: return f(T, std::integral_constant<int, 4>{});
        }
    };
    if (pieces <= 256) return with(std::integral_constant<int, 64>{});
    if (pieces <= 1024) return with(std::integral_constant<int, 256>{});
    return with(std::integral_constant<int, 1024>{});
}

int row_threads(int K) { return K <= 2048 ? 64 : K <= 8192 ? 256 : 1024; }

}  // namespace

size_t norm_grad_ws_bytes(int32_t M, int32_t K)
{
    return (size_t)grad_blocks(M, row_threads(K)) * (size_t)K * sizeof(float);
}

int run_norm(const uint16_t *x, const uint16_t *r, const uint16_t *w, int32_t M, int32_t K, float eps, uint16_t *s,
             uint16_t *y, uint8_t *q, float *q_scale, hipStream_t st)
{
    return by_width(K, [&](auto T, auto V) {
        constexpr int t = decltype(T)::value, v = decltype(V)::value;
        const int rows = t == 64 ? WAVE_ROWS : 1, blocks = (M + rows - 1) / rows;
        const dim3 grid((unsigned)(blocks < GRID_X ? blocks : GRID_X), (unsigned)((blocks + GRID_X - 1) / GRID_X));
        return launch(q ? norm_kernel<t, v, true> : norm_kernel<t, v, false>, grid, dim3(t * rows), 0, st,
                      reinterpret_cast<const f16 *>(x), reinterpret_cast<const f16 *>(r), reinterpret_cast<const f16 *>(w), M, K,
                      eps, reinterpret_cast<f16 *>(s), reinterpret_cast<f16 *>(y), q, q_scale);
    });
}

int run_norm_grad(const uint16_t *t, const uint16_t *dy, const uint16_t *ds, const uint16_t *w, int32_t M, int32_t K,
                  float eps, uint16_t *dx, float *dw, void *ws, hipStream_t st)
{
    const int G = grad_blocks(M, row_threads(K));
    float *part = dw ? static_cast<float *>(ws) : nullptr;
    if (M > 0) {
        const int r = by_width(K, [&](auto T, auto V) {
            constexpr int tt = decltype(T)::value, v = decltype(V)::value;
            return launch(norm_grad_kernel<tt, v>, dim3((unsigned)G), dim3((unsigned)(tt * grad_groups(tt))), 0, st,
                          reinterpret_cast<const f16 *>(t), reinterpret_cast<const f16 *>(dy),
                          reinterpret_cast<const f16 *>(ds), reinterpret_cast<const f16 *>(w), M, K, eps,
                          reinterpret_cast<f16 *>(dx), part);
        });
        if (r != NVFP4_OK || !dw) return r;
    }
    return launch(norm_dweight_kernel, dim3((unsigned)((K + DW_COLS - 1) / DW_COLS)), dim3(DW_COLS * DW_SPLIT), 0, st,
                  static_cast<const float *>(ws), G, K, dw);
}

}  // namespace nvfp4
