// linear_rows.hip -- the channel-FP8 projection of 8-bit rows (include/nvfp4moe_dense.h): both operands E4M3, FP32
// sums, a scale per row and one per column.
//
// One reduction order at every batch size: 512-element chunks, each a chain of four 128-element MFMA steps from +0,
// added in chunk order from +0. Few rows stream the weights once: a block per 16 columns whose waves share the chunks
// (all of a wave's weights are requested before the first product) and meet in LDS. More rows take the tiled product of
// tile_gemm.hpp, which adds its accumulators to the sum after every fourth stage.
#include "dense.hpp"
#include "nvfp4_device.hpp"
#include "tile_gemm.hpp"

namespace nvfp4 {
namespace {

constexpr int ROWS_CHUNK = 512, ROWS_STEPS = ROWS_CHUNK / STAGE_BYTES;
constexpr int ROWS_WAVES = 16;
constexpr int ROWS_STREAM_M = 32;
constexpr int LDS_PITCH = 20;  // floats between a partial tile's rows

inline int rows_chunks(int K) { return (K + ROWS_CHUNK - 1) / ROWS_CHUNK; }

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b)
{
    return __builtin_shufflevector(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), 0, 1, 2, 3, 4, 5, 6, 7);
}

// Block b: columns 16 b .. + 15 of all M <= 16 MT rows. LDS: [chunks][MT][16 rows][LDS_PITCH] partial tiles.
template <int MT>
__global__ __launch_bounds__(ROWS_WAVES * 64) void rows_stream_kernel(const uint8_t *__restrict__ xq,
                                                                      const float *__restrict__ xs, int M,
                                                                      const uint8_t *__restrict__ w,
                                                                      const float *__restrict__ cs, int N, int K,
                                                                      f16 *__restrict__ y)
{
    extern __shared__ __attribute__((aligned(16))) float part[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int r = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 16, S = (K + ROWS_CHUNK - 1) / ROWS_CHUNK;
    const rsrc_t rw = make_rsrc(w + (size_t)n0 * K, 16u * K);
    const rsrc_t rx = make_rsrc(xq, (uint32_t)M * K);
    for (int c = wave; c < S; c += waves) {
        const int kb = c * ROWS_CHUNK, steps = min(ROWS_STEPS, (K - kb) / STAGE_BYTES);
        u32x4 b[ROWS_STEPS][2], a[MT][ROWS_STEPS][2];
#pragma unroll
        for (int s = 0; s < ROWS_STEPS; ++s)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                b[s][u] = bload16(rw, s < steps ? (uint32_t)r * K + kb + s * STAGE_BYTES + 64 * u + 16 * q : BUF_OOB, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < ROWS_STEPS; ++s)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    a[m][s][u] = bload16(rx, s < steps && 16 * m + r < M
                                                 ? (uint32_t)(16 * m + r) * K + kb + s * STAGE_BYTES + 64 * u + 16 * q
                                                 : BUF_OOB, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < ROWS_STEPS; ++s)
                if (s < steps) acc = mfma_e4m3(join(b[s][0], b[s][1]), join(a[m][s][0], a[m][s][1]), acc);
            // lane (r, q): columns 4 q .. 4 q + 3 of row r
            *reinterpret_cast<f32x4 *>(part + ((c * MT + m) * 16 + r) * LDS_PITCH + 4 * q) = acc;
        }
    }
    lds_barrier();
    for (int i = threadIdx.x; i < MT * 256; i += blockDim.x) {
        const int m = i >> 4, n = i & 15;
        if (m >= M) break;
        float s = 0.0f;
        for (int c = 0; c < S; ++c) s += part[((size_t)c * MT * 16 + m) * LDS_PITCH + n];
        y[(size_t)m * N + n0 + n] = f16_of_f32((xs[m] * cs[n0 + n]) * s);
    }
}

template <class T>
__global__ __launch_bounds__(T::WAVES * 64) void rows_tile_kernel(const uint8_t *__restrict__ xq,
                                                                  const float *__restrict__ xs, int M,
                                                                  const uint8_t *__restrict__ w,
                                                                  const float *__restrict__ cs, int N, int K,
                                                                  f16 *__restrict__ y)
{
    __shared__ __attribute__((aligned(1024))) unsigned char smem[T::NS * T::BYTES];
    int tm, tn;
    if (!tile_of_block(blockIdx.x, (M + T::BM - 1) / T::BM, (N + T::BN - 1) / T::BN, tm, tn)) return;
    const Place p = place_of<T>();
    const int m0 = tm * T::BM, c0 = tn * T::BN;
    const Operands in = {make_rsrc(xq + (size_t)m0 * K, (uint32_t)min(T::BM, M - m0) * K),
                         make_rsrc(w + (size_t)c0 * K, (uint32_t)min(T::BN, N - c0) * K)};
    uint32_t va[T::LA], vb[T::LB];
#pragma unroll
    for (int i = 0; i < T::LA; ++i) {
        const int r = load_row<T>(p, i);
        va[i] = m0 + r < M ? (uint32_t)r * K + load_byte(r, p.lane) : BUF_OOB;
    }
#pragma unroll
    for (int i = 0; i < T::LB; ++i) {
        const int r = load_row<T>(p, i), c = column_of_row<T>(r);
        vb[i] = c0 + c < N ? (uint32_t)c * K + load_byte(r, p.lane) : BUF_OOB;
    }
    f32x4 acc[T::MT][T::NT];
    tile_product<T, ROWS_STEPS>(smem, p, in, va, vb, 0, K / STAGE_BYTES, STAGE_BYTES, acc);
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int m = 0; m < T::MT; ++m) {
        const int row = m0 + (p.wm * T::MT + m) * 16 + p.r;
        if (row >= M) continue;
        const float sx = xs[row];
#pragma unroll
        for (int t = 0; t < T::NT; ++t) {
            const int c = c0 + p.wn * 16 * T::NT + 4 * T::NT * p.q + 4 * t;
            if (c >= N) continue;
            f16x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = f16_of_f32((sx * cs[c + e]) * acc[m][t][e]);
            *reinterpret_cast<f16x4 *>(y + (size_t)row * N + c) = o;
        }
    }
}

using Large = Tile<true, 6, 4, 2, 4, 2>;   // 192 x 256
using Medium = Tile<true, 4, 4, 2, 2, 2>;  // 128 x 128, two blocks per CU
using Small = Tile<true, 2, 2, 2, 2, 3>;   // 64 x 64, three blocks per CU

}  // namespace

int run_linear_fp8_rows(const uint8_t *xq, const float *xs, int32_t M, const fp8_channel_weights &w, uint16_t *y,
                        hipStream_t s)
{
    const int N = w.rows, K = w.k;
    f16 *o = reinterpret_cast<f16 *>(y);
    if (M <= ROWS_STREAM_M) {
        const int S = rows_chunks(K), waves = S < ROWS_WAVES ? S : ROWS_WAVES, mt = (M + 15) / 16;
        const size_t shmem = (size_t)S * mt * 16 * LDS_PITCH * sizeof(float);
        return launch(mt == 1 ? rows_stream_kernel<1> : rows_stream_kernel<2>, dim3((unsigned)(N / 16)),
                      dim3((unsigned)(waves * 64)), shmem, s, xq, xs, M, w.codes, w.channel_scale, N, K, o);
    }
    auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
    auto tiled = [&](auto tile) {
        using T = decltype(tile);
        return launch(rows_tile_kernel<T>, dim3(tile_grid(tiles(T::BM, T::BN))), dim3(T::WAVES * 64), 0, s, xq, xs, M, w.codes,
                      w.channel_scale, N, K, o);
    };
    if (tiles(Large::BM, Large::BN) >= 256) return tiled(Large{});
    if (tiles(Medium::BM, Medium::BN) >= 256) return tiled(Medium{});
    return tiled(Small{});
}

}  // namespace nvfp4
