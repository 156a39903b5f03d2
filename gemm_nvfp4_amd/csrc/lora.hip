// lora.hip -- low-rank adapters of many requests at once: d = s_a (x A_a^T) B_a^T for every row's adapter
// a, added to a finished result (lora_add) or to a dense NVFP4 projection before its one rounding
// (linear_lora, linear_swiglu_lora).
//
// The rows come grouped by the routing plan of the adapter ids: a plan tile is up to 16 rows of one
// adapter, one MFMA tile. Two products:
//   shrink  v[r] = sum_k x[k] A[r][k].  A wave takes one (row tile, 512-element chunk): a chain of 16
//           v_mfma_f32_16x16x32_f16 steps from +0, step j covering elements [32j, 32j + 32). Chunk
//           results are added in FP32 in ascending order, so v does not depend on the batch.
//   expand  d[n] = sum_r v[r] B[n][r].  v is FP32 and B fp16: the row of v is scaled by a power of two
//           (largest finite |v| to [2^12, 2^13)) and split into v = hi + lo, two fp16 numbers, so that
//           the matrix pipe sums it to at least 22 bits of the row's largest |v|. One MFMA step takes 16
//           ranks: its lane groups 0 and 1 feed hi, groups 2 and 3 lo, against the same columns of B.
//           B's rows are the MFMA's row operand and the tokens its columns: with rows n0 + 16(i/4) + 4t +
//           i%4 for row i of tile t, a lane holds 16 consecutive outputs of one token after four tiles.
// Rows without an adapter take pseudo tiles behind the plan's (16 consecutive pairs, those with an
// adapter masked) and only copy, or finish, their base result.
#include "nvfp4_device.hpp"
#include "ops.hpp"

namespace nvfp4 {
namespace {

constexpr int TILE = PLAN_TILE_ROWS;  // 16 rows

// Where the rows of a plan tile lie: pair order (row = pair index) or bucket order.
struct TileRows {
    const int32_t *hdr, *tile_expert, *tile_base, *tile_rows, *tile_pair, *pair_expert;
    int bucket;
};

__device__ __forceinline__ int tile_row(const TileRows &tr, int t, int i)
{
    return tr.bucket ? tr.tile_base[t] + i : tr.tile_pair[t * TILE + i];
}

// ---- shrink ---------------------------------------------------------------------------------------
// One wave per (row tile, chunk, group of RT 16-rank tiles): vp[c][row][r] = the chunk's part of v.
constexpr int SHRINK_WAVES = 4;  // consecutive row tiles of one chunk: tiles of one adapter share A in L1

template <int RT>
__global__ __launch_bounds__(SHRINK_WAVES * 64) void shrink_kernel(TileRows tr, const f16 *__restrict__ x, int64_t P,
                                                                   int K, int rank, const f16 *__restrict__ a,
                                                                   float *__restrict__ vp)
{
    const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
    const int t = blockIdx.x * SHRINK_WAVES + (threadIdx.x >> 6);
    const int c = blockIdx.y, r0 = blockIdx.z * RT * 16;
    if (t >= tr.hdr[3]) return;  // wave-uniform
    const int rows = tr.tile_rows[t];
    const int row = tile_row(tr, t, i < rows ? i : 0);
    const f16 *ae = a + (size_t)tr.tile_expert[t] * rank * K;
    const int kb = c * KCHUNK, steps = min(KCHUNK, K - kb) >> 5;
    const f16 *xp = x + (size_t)row * K + kb + 8 * q;
    const f16 *ap[RT];
#pragma unroll
    for (int u = 0; u < RT; ++u) ap[u] = ae + (size_t)min(r0 + 16 * u + i, rank - 1) * K + kb + 8 * q;
    f32x4 acc[RT];
#pragma unroll
    for (int u = 0; u < RT; ++u) acc[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < steps; j0 += 4)  // K % 128 == 0: whole groups of four steps
#pragma unroll
        for (int j = j0; j < j0 + 4; ++j) {
            const f16x8 xf = *reinterpret_cast<const f16x8 *>(xp + 32 * j);
#pragma unroll
            for (int u = 0; u < RT; ++u)
                acc[u] = mfma_step(xf, *reinterpret_cast<const f16x8 *>(ap[u] + 32 * j), acc[u]);
        }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int src = 4 * q + e;
        const int orow = __shfl(row, src, 64);
        if (src < rows) {
#pragma unroll
            for (int u = 0; u < RT; ++u) {
                const int r = r0 + 16 * u + i;
                if (r < rank) vp[((size_t)c * P + orow) * rank + r] = acc[u][e];
            }
        }
    }
}

// ---- expand ---------------------------------------------------------------------------------------
constexpr int EXPAND_WAVES = 4;
constexpr int GROUP_COLS = 64;  // outputs of one token per wave and step

// The 16 consecutive outputs n0 + 16q .. + 15 of the lane's token: d (scaled back), from hi and lo rows in
// LDS.
__device__ __forceinline__ void expand16(float (&d)[16], const f16 *be, int n0, int N, int rank, const f16 *hi,
                                         const f16 *lo, int pitch, int i, int q)
{
    f32x4 acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const f16 *vrow = (q < 2 ? hi : lo) + i * pitch + 8 * (q & 1);
    const bool bv = n0 + 16 * (i >> 2) < N;
    for (int r = 0; r < rank; r += 16) {
        const bool rv = r + 8 * (q & 1) < rank;
        const f16x8 vf = *reinterpret_cast<const f16x8 *>(vrow + r);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int n = n0 + 16 * (i >> 2) + 4 * t + (i & 3);
            f16x8 bf = zero8();
            if (bv && rv) bf = *reinterpret_cast<const f16x8 *>(be + (size_t)n * rank + r + 8 * (q & 1));
            acc[t] = mfma_step(bf, vf, acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[4 * t + e] = acc[t][e];
}

__device__ __forceinline__ void load_base(float (&b)[16], const f16 *y)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f16x8 v = *reinterpret_cast<const f16x8 *>(y + 8 * h);
#pragma unroll
        for (int e = 0; e < 8; ++e) b[8 * h + e] = (float)v[e];
    }
}

__device__ __forceinline__ void load_base(float (&b)[16], const float *y)
{
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const f32x4 v = *reinterpret_cast<const f32x4 *>(y + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[4 * h + e] = v[e];
    }
}

template <int N8>
__device__ __forceinline__ void store_half(f16 *out, const float *v)
{
#pragma unroll
    for (int h = 0; h < N8; ++h) {
        f16x8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = f16_of_f32(v[8 * h + e]);
        *reinterpret_cast<f16x8 *>(out + 8 * h) = o;
    }
}

// GATE 0: plain; 1: gate rows [0, N/2), up rows [N/2, N); 2: row 2i gate i, row 2i + 1 up i.
template <typename BASE, int GATE>
__global__ __launch_bounds__(EXPAND_WAVES * 64) void expand_kernel(TileRows tr, int t_max, int64_t P, int S, int N,
                                                                   int rank, const f16 *__restrict__ b,
                                                                   const float *__restrict__ scale,
                                                                   const float *__restrict__ vp, const BASE *base,
                                                                   f16 *out, int groups_per_wave)
{
    extern __shared__ unsigned char smem[];
    __shared__ int s_row[TILE];
    __shared__ int s_exp[TILE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    const int t = blockIdx.x;
    const bool plain_rows = t >= t_max;  // rows without an adapter
    const int pitch = ((rank + 15) & ~15) + 8;
    float *v32 = reinterpret_cast<float *>(smem);                       // [16][pitch]
    f16 *hi = reinterpret_cast<f16 *>(v32 + TILE * pitch), *lo = hi + TILE * pitch;
    float sc = 0.f;
    const f16 *be = b;
    if (plain_rows) {
        if (threadIdx.x < TILE) {
            const int64_t p = (int64_t)(t - t_max) * TILE + threadIdx.x;
            s_row[threadIdx.x] = p < P && tr.pair_expert[p] < 0 ? (int)p : -1;
        }
        __syncthreads();
    } else {
        if (t >= tr.hdr[3]) return;  // the whole block
        const int rows = tr.tile_rows[t], e = tr.tile_expert[t];
        be = b + (size_t)e * N * rank;
        sc = scale[e];
        if (threadIdx.x < TILE) s_row[threadIdx.x] = (int)threadIdx.x < rows ? tile_row(tr, t, threadIdx.x) : -1;
        __syncthreads();
        for (int o = threadIdx.x; o < TILE * pitch; o += blockDim.x) {
            const int m = o / pitch, r = o - m * pitch;
            float v = 0.f;
            if (s_row[m] >= 0 && r < rank) {
                const float *p = vp + (size_t)s_row[m] * rank + r;
                v = p[0];
                for (int c = 1; c < S; ++c) v += p[(size_t)c * P * rank];
            }
            v32[o] = v;
        }
        __syncthreads();
        // 16 threads per row: the row's largest finite magnitude, then the split of the scaled row.
        const int m = threadIdx.x >> 4, l = threadIdx.x & 15;
        float big = 0.f;
        for (int r = l; r < rank; r += 16) {
            const float f = fabsf(v32[m * pitch + r]);
            if (f < __builtin_inff()) big = fmaxf(big, f);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o, 16));
        const int sh = big > 0.f ? 13 - __builtin_amdgcn_frexp_expf(big) : 0;  // frexp: big = f 2^e, f in [1/2, 1)
        if (l == 0) s_exp[m] = -sh;
        for (int r = l; r < pitch; r += 16) {
            const float f = __builtin_amdgcn_ldexpf(v32[m * pitch + r], sh);
            const f16 h = (f16)f;
            const float rest = f - (float)h;
            hi[m * pitch + r] = h;
            lo[m * pitch + r] = fabsf(f) < __builtin_inff() ? (f16)rest : (f16)0.f;  // infinities and NaN stay in hi
        }
        __syncthreads();
    }
    const int row = s_row[i];
    const int back = plain_rows ? 0 : s_exp[i];
    const int I = N >> 1;
    const int cols = GATE == 1 ? I : N;  // columns that the groups cover
    const int g0 = (blockIdx.y * EXPAND_WAVES + wave) * groups_per_wave;
    for (int g = g0; g < g0 + groups_per_wave && g * GROUP_COLS < cols; ++g) {
        const int n0 = g * GROUP_COLS, n = n0 + 16 * q;
        float d[16], d2[16];
        if (!plain_rows) {
            expand16(d, be, n0, cols, rank, hi, lo, pitch, i, q);
            if (GATE == 1) expand16(d2, be + (size_t)I * rank, n0, cols, rank, hi, lo, pitch, i, q);
        }
        if (row < 0 || n >= cols) continue;
        float y[16], y2[16];
        load_base(y, base + (size_t)row * N + n);
        if (GATE == 1) load_base(y2, base + (size_t)row * N + I + n);
        if (!plain_rows) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                y[e] = fmaf(sc, __builtin_amdgcn_ldexpf(d[e], back), y[e]);
                if (GATE == 1) y2[e] = fmaf(sc, __builtin_amdgcn_ldexpf(d2[e], back), y2[e]);
            }
        }
        if constexpr (GATE == 0) {
            store_half<2>(out + (size_t)row * N + n, y);
        } else if constexpr (GATE == 1) {
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = swiglu(y[e], y2[e]);
            store_half<2>(out + (size_t)row * I + n, y);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = swiglu(y[2 * e], y[2 * e + 1]);
            store_half<1>(out + (size_t)row * I + (n >> 1), y);
        }
    }
}

TileRows tile_rows(const PlanView &pv, int bucket)
{
    return TileRows{pv.hdr, pv.tile_expert, pv.tile_base, pv.tile_rows, pv.tile_pair, pv.pair_expert, bucket};
}

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

int launch_shrink(const TileRows &tr, int64_t t_max, int64_t P, const f16 *x, const nvfp4_lora &lora, float *vp,
                  hipStream_t s)
{
    const int rt = (lora.rank + 15) / 16;
    const dim3 block(SHRINK_WAVES * 64);
    const unsigned gx = (unsigned)((t_max + SHRINK_WAVES - 1) / SHRINK_WAVES), gy = (unsigned)num_chunks(lora.k);
    const f16 *a = reinterpret_cast<const f16 *>(lora.a);
    if (rt == 1) return launch(shrink_kernel<1>, dim3(gx, gy), block, 0, s, tr, x, P, lora.k, lora.rank, a, vp);
    if (rt == 2) return launch(shrink_kernel<2>, dim3(gx, gy), block, 0, s, tr, x, P, lora.k, lora.rank, a, vp);
    return launch(shrink_kernel<4>, dim3(gx, gy, (unsigned)((rt + 3) / 4)), block, 0, s, tr, x, P, lora.k, lora.rank, a, vp);
}

template <typename BASE, int GATE>
int launch_expand(const TileRows &tr, int64_t t_max, int64_t P, bool others, const nvfp4_lora &lora, const float *vp,
                  const BASE *base, f16 *out, hipStream_t s)
{
    const int N = lora.rows, cols = GATE == 1 ? N / 2 : N;
    const int pitch = ((lora.rank + 15) & ~15) + 8;
    const int groups = (cols + GROUP_COLS - 1) / GROUP_COLS;
    const int64_t tiles = t_max + (others ? (P + TILE - 1) / TILE : 0);
    int per_wave = (int)(tiles * groups / (16 * device_cus()));
    if (per_wave < 1) per_wave = 1;
    if (per_wave > 16) per_wave = 16;
    const unsigned gy = (unsigned)((groups + EXPAND_WAVES * per_wave - 1) / (EXPAND_WAVES * per_wave));
    return launch(expand_kernel<BASE, GATE>, dim3((unsigned)tiles, gy), dim3(EXPAND_WAVES * 64),
                  (size_t)TILE * pitch * (sizeof(float) + 2 * sizeof(f16)), s, tr, (int)t_max, P, num_chunks(lora.k), N, lora.rank,
                  reinterpret_cast<const f16 *>(lora.b), lora.scale, vp, base, out, per_wave);
}

}  // namespace

size_t lora_add_ws_bytes(int64_t P, int32_t K, int32_t rank)
{
    return round256((size_t)num_chunks(K) * (size_t)P * rank * sizeof(float));
}

size_t linear_lora_ws_bytes(int32_t M, int32_t rows, int32_t K, int32_t rank)
{
    return round256((size_t)M * rows * sizeof(float)) + lora_add_ws_bytes(M, K, rank);
}

int run_lora_add(const PlanView &pv, const PlanLayout &L, int32_t order, const uint16_t *x, const nvfp4_lora &lora,
                 const uint16_t *y, uint16_t *out, void *ws, hipStream_t s)
{
    const TileRows tr = tile_rows(pv, order);
    float *vp = static_cast<float *>(ws);
    const int st = launch_shrink(tr, L.T, L.P, reinterpret_cast<const f16 *>(x), lora, vp, s);
    if (st != NVFP4_OK) return st;
    return launch_expand<f16, 0>(tr, L.T, L.P, order == 0 && out != y, lora, vp, reinterpret_cast<const f16 *>(y),
                                 reinterpret_cast<f16 *>(out), s);
}

int run_linear_lora(const PlanView &pv, const PlanLayout &L, const uint16_t *x, int32_t M, const nvfp4_weights &w,
                    const nvfp4_lora &lora, bool gated, int32_t layout, uint16_t *y, void *ws, hipStream_t s)
{
    const TileRows tr = tile_rows(pv, 0);
    float *base = static_cast<float *>(ws);
    float *vp = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + round256((size_t)M * w.rows * sizeof(float)));
    int st = run_linear_f32(x, M, w, base, s);
    if (st == NVFP4_OK) st = launch_shrink(tr, L.T, L.P, reinterpret_cast<const f16 *>(x), lora, vp, s);
    if (st != NVFP4_OK) return st;
    f16 *o = reinterpret_cast<f16 *>(y);
    if (!gated) return launch_expand<float, 0>(tr, L.T, L.P, true, lora, vp, base, o, s);
    if (layout == 0) return launch_expand<float, 1>(tr, L.T, L.P, true, lora, vp, base, o, s);
    return launch_expand<float, 2>(tr, L.T, L.P, true, lora, vp, base, o, s);
}

}  // namespace nvfp4
