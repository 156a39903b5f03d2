// linear_rows.hip -- the channel-FP8 projection of 8-bit rows (include/nvfp4moe_dense.h): both operands E4M3, FP32
// sums, a scale per row and one per column.
//
// One reduction order at every batch size: a single chain of 128-element MFMA steps from +0, in the order of the
// reduction axis. Few rows stream the weights once: a block for every 16 columns, whose waves hold the whole axis in
// flight and hand the chain on from one to the next. More rows take the tiled product of tile_gemm.hpp, whose shape the
// batch chooses.
//
// Measured at 4352 x 5120, calls back to back: one row 9.1 us (2.4 TB/s of 22.3 MB: 82 KB a block at what a CU has in flight,
// start-up, and 1.2 us of the chain's hand-overs), 13 rows 9.5, 333 rows 18.9 (780 TFLOP/s), 8192 rows 164 (2.2 PFLOP/s; the
// library's product of 8192^3 reaches 2.27). Sums in 512-element chunks, each closed by FP32 additions, reached 1.75 to 2.1
// PFLOP/s where the one chain reaches 2.3 to 2.65 in whole rounds.
#include "dense.hpp"
#include "nvfp4_device.hpp"
#include "tile_gemm.hpp"

namespace nvfp4 {
namespace {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int ROWS_STREAM_M = 32;  // most rows of the streaming kernel
constexpr int ROWS_GROUP = 5;  // steps whose operands a wave holds at once

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b)
{
    return __builtin_shufflevector(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), 0, 1, 2, 3, 4, 5, 6, 7);
}

// Four neighbouring scales, which are 4-byte aligned.
__device__ __forceinline__ f32x4 load_scales(const float *p)
{
    f32x4 v;
    __builtin_memcpy(&v, p, sizeof(v));
    return v;
}

// Block b: columns 16 b .. + 15 of all M <= 16 MT rows. The waves share the steps in groups of ROWS_GROUP, in turn. All
// of a group's loads are in flight before the wave's turn comes, so the block has the whole reduction axis in flight
// (up to ROWS_GROUP steps a wave) and yet computes one chain: a wave takes the accumulators over from the one before,
// through LDS, and asks for its next group as soon as it has passed them on.
template <int MT>
__global__ __launch_bounds__(MT == 1 ? 1024 : 512) void rows_stream_kernel(const uint8_t *__restrict__ xq,
                                                                           const float *__restrict__ xs, int M,
                                                                           const uint8_t *__restrict__ w,
                                                                           const float *__restrict__ cs, int N, int K,
                                                                           f16 *__restrict__ y)
{
    constexpr int G = ROWS_GROUP;
    __shared__ f32x4 handed[MT][64];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * 16, S = K / STAGE_BYTES;
    const rsrc_t rw = make_rsrc(w + (size_t)n0 * K, 16u * K);
    const rsrc_t rx = make_rsrc(xq, (uint32_t)M * K);
    const uint32_t wo = (uint32_t)r * K + 16 * q;
    uint32_t xo[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xo[m] = 16 * m + r < M ? (uint32_t)(16 * m + r) * K + 16 * q : BUF_OOB;
    u32x4 b[G][2], a[MT][G][2];
    auto load = [&](int s0) {
#pragma unroll
        for (int s = 0; s < G; ++s)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // steps past the end re-read the last one; they are not used
                const uint32_t at = (uint32_t)min(s0 + s, S - 1) * STAGE_BYTES + 64 * u;
                b[s][u] = bload16(rw, wo, at);
#pragma unroll
                for (int m = 0; m < MT; ++m) a[m][s][u] = bload16(rx, xo[m], at);
            }
    };
    load(wave * G);
    for (int g0 = 0; g0 * G < S; g0 += waves) {
        for (int turn = 0; turn < waves; ++turn) {
            const int s0 = (g0 + turn) * G;
            if (turn == wave && s0 < S) {
                f32x4 acc[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[m] = s0 == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : handed[m][lane];
#pragma unroll
                for (int s = 0; s < G; ++s)
                    if (s0 + s < S) {
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            acc[m] = mfma_e4m3(join(b[s][0], b[s][1]), join(a[m][s][0], a[m][s][1]), acc[m]);
                    }
#pragma unroll
                for (int m = 0; m < MT; ++m) handed[m][lane] = acc[m];
                if (s0 + waves * G < S) load(s0 + waves * G);
            }
            lds_barrier();
        }
    }
    // lane (r, q) of row tile m: columns 4 q .. 4 q + 3 of row r; a wave a row tile
    const f32x4 sc = load_scales(cs + n0 + 4 * q);
    for (int m = wave; m < MT; m += waves) {
        const int row = 16 * m + r;
        if (row >= M) continue;
        const f32x4 acc = handed[m][lane];
        const float sx = xs[row];
        f16x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = f16_of_f32((sx * sc[e]) * acc[e]);
        *reinterpret_cast<f16x4 *>(y + (size_t)row * N + n0 + 4 * q) = o;
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
    Rows<T::LA> ra;
    Rows<T::LB> rb;
    ra.buf = make_rsrc(xq + (size_t)m0 * K, (uint32_t)min(T::BM, M - m0) * K);
    rb.buf = make_rsrc(w + (size_t)c0 * K, (uint32_t)min(T::BN, N - c0) * K);
#pragma unroll
    for (int i = 0; i < T::LA; ++i) {
        const int r = load_row<T>(p, i);
        ra.off[i] = m0 + r < M ? (uint32_t)r * K + load_byte(r, p.lane) : BUF_OOB;
    }
#pragma unroll
    for (int i = 0; i < T::LB; ++i) {
        const int r = load_row<T>(p, i), c = column_of_row<T>(r);
        rb.off[i] = c0 + c < N ? (uint32_t)c * K + load_byte(r, p.lane) : BUF_OOB;
    }
    f32x4 acc[T::MT][T::NT];
    tile_product<T>(smem, p, ra, rb, 0, K / STAGE_BYTES, STAGE_BYTES, acc);
    // all scales at once: asked for one by one between the stores, each waited for its own way to memory and back
    const int row0 = m0 + p.wm * T::MT * 16 + p.r, col0 = c0 + p.wn * 16 * T::NT + 4 * T::NT * p.q;
    f32x4 sc[T::NT];
    float sx[T::MT];
#pragma unroll
    for (int t = 0; t < T::NT; ++t) sc[t] = load_scales(cs + min(col0 + 4 * t, N - 4));
#pragma unroll
    for (int m = 0; m < T::MT; ++m) sx[m] = xs[min(row0 + 16 * m, M - 1)];
#pragma unroll
    for (int m = 0; m < T::MT; ++m) {
        const int row = row0 + 16 * m;
        if (row >= M) continue;
#pragma unroll
        for (int t = 0; t < T::NT; ++t) {
            const int c = col0 + 4 * t;
            if (c >= N) continue;
            f16x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = f16_of_f32((sx[m] * sc[t][e]) * acc[m][t][e]);
            *reinterpret_cast<f16x4 *>(y + (size_t)row * N + c) = o;
        }
    }
}

// The stream has the whole reduction axis in flight, which the tiles walk, but a block for every 16 columns, so it wins at
// few rows where the blocks have a CU each, us by the stream and in tiles: 2048 x 8192 8.4 and 14.5 at one row, 11.2 and
// 14.7 at 16, 15.0 and 15.0 at 32; 2048 x 2048 4.0 and 5.4 at one row, 4.9 and 5.6 at 16, 6.0 and 5.6 at 24. With more
// blocks than CUs it holds at a few rows for a while: 4352 x 5120 9.4 and 10.3 at one, 10.4 and 10.4 at 8, 11.9 and 10.5
// at 16; 8192 x 8192 16.8 and 15.8 at one.
bool use_stream(int M, int N, int K)
{
    if (N <= 16 * TILE_CUS) return M <= 16 || (M <= ROWS_STREAM_M && K >= 4096);
    return M <= 4 && N <= 20 * TILE_CUS;
}

// The tile shapes; their times (Shape) are measured at 40 stages (K = 5120). The shape of the least estimated time is
// taken. Many tiles: whole rounds over the CUs decide, at 1.0 to 2.65 PFLOP/s; 8192 x 4352 outputs of K = 5120 take 167 us
// in the two rounds of 384 x 192, 216 in the four of 192 x 256. What bounds the large shapes is the way from the
// L2s into LDS (64 KB a stage for 256 x 256, 12 to 15 TB/s over the chip) and the matrix pipes, each a little
// more than half busy. Few tiles: the fewer bytes a CU has to bring in, the better, so small tiles on all CUs win, with
// rings as deep as two or more blocks to a CU allow: 64 x 4352 outputs take 11.4 us with 32 x 32 and five stages, 12.5 with
// 64 x 32 and three (20.2 with two), 14.9 with 64 x 64 and three (22.5 with two); 333 x 4352 take 19.6 with 64 x 64, 25.7
// with 64 x 32, 26.6 with 32 x 32. 128 x 128 comes with two stages and two blocks to a CU, and with three and one: 1000 x 4352
// 36.1 and 56.2, 512 x 8192 of K = 8192 61.1 and 46.8.
using T384x192 = Tile<true, 6, 6, 4, 2, 2>;
using T256x256 = Tile<true, 8, 4, 2, 4, 2>;
using T192x256 = Tile<true, 6, 4, 2, 4, 2>;
using T192x192 = Tile<true, 6, 3, 2, 4, 3>;
using T128x128 = Tile<true, 4, 4, 2, 2, 2>;
using D128x128 = Tile<true, 4, 4, 2, 2, 3>;
using T64x64 = Tile<true, 2, 2, 2, 2, 3>;
using T64x32 = Tile<true, 2, 1, 2, 2, 3>;
using T32x32 = Tile<true, 1, 1, 2, 2, 5>;
constexpr Shape SHAPES[] = {{384, 192, 1, 1950, 1950}, {256, 256, 1, 1620, 1620}, {192, 256, 1, 1300, 1300},
                            {192, 192, 1, 1075, 1075}, {128, 128, 2, 780, 450},   {128, 128, 1, 640, 640},
                            {64, 64, 3, 300, 215},     {64, 32, 4, 230, 135},     {32, 32, 4, 190, 103}};

template <class F>
int with_shape(int i, F &&f)
{
    switch (i) {  // the order of SHAPES
    case 0: return f(T384x192{});
    case 1: return f(T256x256{});
    case 2: return f(T192x256{});
    case 3: return f(T192x192{});
    case 4: return f(T128x128{});
    case 5: return f(D128x128{});
    case 6: return f(T64x64{});
    case 7: return f(T64x32{});
    default: return f(T32x32{});
    }
}

}  // namespace

int run_linear_fp8_rows(const uint8_t *xq, const float *xs, int32_t M, const fp8_channel_weights &w, uint16_t *y,
                        hipStream_t s)
{
    const int N = w.rows, K = w.k;
    f16 *o = reinterpret_cast<f16 *>(y);
    if (use_stream(M, N, K)) {
        const int groups = (K / STAGE_BYTES + ROWS_GROUP - 1) / ROWS_GROUP, most = M <= 16 ? 16 : 8;
        auto *kernel = M <= 16 ? rows_stream_kernel<1> : rows_stream_kernel<2>;
        return launch(kernel, dim3((unsigned)(N / 16)), dim3((unsigned)(64 * (groups < most ? groups : most))), 0, s, xq, xs, M,
                      w.codes, w.channel_scale, N, K, o);
    }
    int best = 0;
    int64_t least = INT64_MAX;
    for (int i = 0; i < (int)(sizeof(SHAPES) / sizeof(SHAPES[0])); ++i) {
        const int64_t ns = SHAPES[i].ns(SHAPES[i].tiles(M, N), K / STAGE_BYTES);
        if (ns < least) least = ns, best = i;
    }
    return with_shape(best, [&](auto tile) {
        using T = decltype(tile);
        return launch(rows_tile_kernel<T>, dim3(tile_grid(SHAPES[best].tiles(M, N))), dim3(T::WAVES * 64), 0, s, xq, xs, M,
                      w.codes, w.channel_scale, N, K, o);
    });
}

}  // namespace nvfp4
