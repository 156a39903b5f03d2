// linear_grad.hip -- gradients through frozen NVFP4 weights (include/nvfp4moe_dense.h): of the dense projection
// towards its input, dx = dy W, and of the gated projection towards its gate and up rows, which are computed again.
//
// Three regimes by the batch size:
//   * few rows: the packed weights are streamed once. dx: the reduction axis is the weight's rows, the packed axis the
//     output's columns, so a lane takes eight rows' dwords (eight codes each) and transposes them in registers into
//     eight B fragments, one per code position; no value crosses a lane. A block's waves share 512 rows of the weight,
//     hold them decoded while the rows of dy pass by in sixteens, add their tiles in LDS in order and store one FP32
//     plane; a second launch adds the planes in order. Gated: the chunk products of the split-K projection
//     (linear.hip), then a fold with the gradient's epilogue;
//   * some hundred rows, gated: tiles on the packed weights, decoded in registers (packed_gemm.hpp), in one launch;
//   * many rows: the weight is decoded once into the workspace (for dx transposed), exactly, as fp16, and the tiled
//     product of tile_gemm.hpp runs on it, with the gradient in its epilogue. Where the output has too few tiles for
//     the CUs the reduction axis is split too, and the same folds add the planes.
#include "dense.hpp"
#include "nvfp4_device.hpp"
#include "packed_gemm.hpp"
#include "tile_gemm.hpp"

namespace nvfp4 {
namespace {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int FOLD_THREADS = 256;

// ---- few rows: dx from the packed weights ------------------------------------------------------------
constexpr int ST_WAVES = 8, ST_ROWS = 64;            // waves per block, weight rows per wave
constexpr int ST_CHUNK = ST_WAVES * ST_ROWS;         // weight rows per plane
constexpr int ST_COLS = 128;                         // output columns per block
constexpr int FEW_ROWS = 64, ST_MAX_M = 512;  // always, and at most
// One buffer holds all of dy, and the offset that feeds zeros has to lie past it: with 512 rows of 2^20 it begins right there.
static_assert((uint64_t)ST_MAX_M * MAX_GRAD_ROWS * sizeof(f16) <= BUF_OOB, "dy's rows within a buffer");

__host__ __device__ inline int grad_planes(int N) { return (N + ST_CHUNK - 1) / ST_CHUNK; }

// Eight rows' dwords, and their block scales' bytes, to the fragments of the eight code positions:
// b[c][i] = code c of row i times row i's scale.
__device__ __forceinline__ void decode_columns(f16x8 (&b)[8], const uint32_t (&codes)[8], const uint32_t (&scales)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const f16x2 s = e4m3_pair<false>(scales[i] | scales[i + 1] << 8);
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
            uint32_t lo, hi;  // codes c and c + 1 of rows i and i + 1
            switch (c) {      // the byte of the dword is an immediate
            case 0:
                lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[i], 1.0f, 0));
                hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[i + 1], 1.0f, 0));
                break;
            case 2:
                lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[i], 1.0f, 1));
                hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[i + 1], 1.0f, 1));
                break;
            case 4:
                lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[i], 1.0f, 2));
                hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[i + 1], 1.0f, 2));
                break;
            default:
                lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[i], 1.0f, 3));
                hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[i + 1], 1.0f, 3));
            }
            const f16x2 even = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(hi, lo, 0x05040100u)) * s;
            const f16x2 odd = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(hi, lo, 0x07060302u)) * s;
            b[c][i] = even[0], b[c][i + 1] = even[1];
            b[c + 1][i] = odd[0], b[c + 1][i + 1] = odd[1];
        }
    }
}

// Block (column group g, chunk c): plane c, columns 128 g .. + 127, of all rows. Lane (r, q) of a wave holds columns
// 128 g + 8 r .. + 7 and, per 32-row step, weight rows 8 q .. + 7: it decodes them once, and the rows of dy pass by in
// sixteens. Weight rows at or past N read as zeros (codes and scales), so do dy's elements there and its rows at or past M.
// 24 rows of 4352 x 5120: 8.9 us and 1.8 for the fold (10.7 a call). What bounds it: 4-byte loads of 64-byte pieces of the rows,
// whose lines and whose scales' lines the neighbouring columns' blocks share, so that neighbours on different XCDs cost
// 10 to 30% (8192 x 8192, 24 rows: 24.8 us dealt out in turn, 20.0 with neighbours on one XCD); from 48 rows on the
// planes, 1.2 us for 16 rows.
__global__ __launch_bounds__(ST_WAVES * 64, 4) void grad_stream_kernel(const f16 *__restrict__ dy, int M,
                                                                       const uint8_t *__restrict__ codes,
                                                                       const uint8_t *__restrict__ scales, int N, int K,
                                                                       float *__restrict__ part)
{
    __shared__ __attribute__((aligned(16))) float tiles[ST_WAVES][16][ST_COLS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    // neighbouring columns, which share cache lines of codes and scales, go to one XCD
    const int groups = K / ST_COLS, blocks = groups * grad_planes(N);
    const int block = (int)(blockIdx.x & 7) * ((blocks + 7) >> 3) + (int)(blockIdx.x >> 3);
    if (block >= blocks) return;
    const int g = block % groups, c = block / groups;
    const int n0 = c * ST_CHUNK, rows = min(ST_CHUNK, N - n0);
    const int col = g * ST_COLS + 8 * r;
    const rsrc_t rc = make_rsrc(codes + (size_t)n0 * (K >> 1), (uint32_t)rows * (K >> 1));
    const rsrc_t rs = make_rsrc(scales + (size_t)n0 * (K >> 4), (uint32_t)rows * (K >> 4));
    const rsrc_t rd = make_rsrc(dy, (uint32_t)M * N * 2u);
    uint32_t w[2][8], sc[2][8];
    f16x8 a[2], b[2][8];
    auto load_a = [&](int m0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = wave * ST_ROWS + h * 32 + 8 * q;
            a[h] = __builtin_bit_cast(f16x8, bload16(rd, n < rows && m0 + r < M ? ((uint32_t)(m0 + r) * N + n0 + n) * 2u : BUF_OOB, 0));
        }
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int n = wave * ST_ROWS + h * 32 + 8 * q;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[h][i] = bload4(rc, (uint32_t)(n + i) * (K >> 1) + (col >> 1), 0);
            sc[h][i] = __builtin_amdgcn_raw_buffer_load_b8(rs, (uint32_t)(n + i) * (K >> 4) + (col >> 4), 0, 0);
        }
    }
    load_a(0);
#pragma unroll
    for (int h = 0; h < 2; ++h) decode_columns(b[h], w[h], sc[h]);
    // 512 threads: one float4 of the 16 x 128 tile each. In LDS a row's first halves of eight columns lie in front of the
    // second halves, 16 bytes from lane to lane (at their own places, 32, half of the writes' cycles were conflicts).
    const int om = threadIdx.x >> 5, slot = threadIdx.x & 31, oc = 8 * (slot & 15) + 4 * (slot >> 4);
#pragma unroll 1
    for (int m0 = 0; m0 < M; m0 += 16) {
        f32x4 acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = mfma_step(a[h], b[h][e], acc[e]);
        if (m0 + 16 < M) load_a(m0 + 16);
        if (m0 > 0) lds_barrier();  // the previous tile's sums have been read
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 *o = reinterpret_cast<f32x4 *>(&tiles[wave][4 * q + j][4 * r]);
            o[0] = f32x4{acc[0][j], acc[1][j], acc[2][j], acc[3][j]};
            o[16] = f32x4{acc[4][j], acc[5][j], acc[6][j], acc[7][j]};
        }
        lds_barrier();
        f32x4 s = *reinterpret_cast<const f32x4 *>(&tiles[0][om][4 * slot]);
#pragma unroll
        for (int v = 1; v < ST_WAVES; ++v) s += *reinterpret_cast<const f32x4 *>(&tiles[v][om][4 * slot]);
        if (m0 + om < M) *reinterpret_cast<f32x4 *>(part + ((size_t)c * M + m0 + om) * K + g * ST_COLS + oc) = s;
    }
}

// ---- folds -------------------------------------------------------------------------------------------
// The sum of S planes at one float4, in plane order.
__device__ __forceinline__ f32x4 plane_sum(const float *p, size_t plane, int S)
{
    f32x4 s = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll 8
    for (int i = 1; i < S; ++i) s += *reinterpret_cast<const f32x4 *>(p + i * plane);
    return s;
}

// out[i] = fp16(global * sum of the planes), four elements per thread.
__global__ __launch_bounds__(FOLD_THREADS) void grad_fold_kernel(const float *__restrict__ part, int S, size_t plane,
                                                                 const float *__restrict__ gscale, f16 *__restrict__ out)
{
    const size_t i = ((size_t)blockIdx.x * FOLD_THREADS + threadIdx.x) * 4;
    if (i >= plane) return;
    const f32x4 s = plane_sum(part + i, plane, S);
    const float gs = gscale[0];
    f16x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = f16_of_f32(s[e] * gs);
    *reinterpret_cast<f16x4 *>(out + i) = o;
}

// The gradient of silu(g) * u: sig = 1 / (1 + e^-g) by the hardware's base-2 exponential and reciprocal, as
// swiglu() takes it. g = -inf gives 0 * inf = NaN, as the formula does.
__device__ __forceinline__ void swiglu_grad(float g, float u, float dh, float &dg, float &du)
{
    const float e = __builtin_amdgcn_exp2f(-g * 1.44269504088896341f);
    const float sig = __builtin_amdgcn_rcpf(1.0f + e);
    du = dh * (g * sig);
    dg = dh * u * (sig * (1.0f + g * (1.0f - sig)));
}

// dz of four gate/up pairs i .. i + 3 of row m, from their sums before the global scale.
__device__ __forceinline__ void store_dz(f16 *dz, size_t row, int I, int i, int layout, const f32x4 &g, const f32x4 &u, float gs,
                                         const f16x4 &dh)
{
    f16x4 a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float dg, du;
        swiglu_grad(g[e] * gs, u[e] * gs, (float)dh[e], dg, du);
        a[e] = f16_of_f32(dg), b[e] = f16_of_f32(du);
    }
    f16 *o = dz + row * 2 * I;
    if (layout) {
        *reinterpret_cast<f16x8 *>(o + 2 * i) = f16x8{a[0], b[0], a[1], b[1], a[2], b[2], a[3], b[3]};
    } else {
        *reinterpret_cast<f16x4 *>(o + i) = a;
        *reinterpret_cast<f16x4 *>(o + I + i) = b;
    }
}

// dz from S planes [M][2I] of the gate and up rows' sums, four pairs per thread.
__global__ __launch_bounds__(FOLD_THREADS) void swiglu_grad_fold_kernel(const float *__restrict__ part, int S, int M, int I,
                                                                        const float *__restrict__ gscale, int layout,
                                                                        const f16 *__restrict__ dh, f16 *__restrict__ dz)
{
    const size_t at = ((size_t)blockIdx.x * FOLD_THREADS + threadIdx.x) * 4;
    if (at >= (size_t)M * I) return;
    const size_t m = at / I, plane = (size_t)M * 2 * I;
    const int i = (int)(at % I);
    const float *p = part + m * 2 * I;
    const f32x4 a = plane_sum(p + (layout ? 2 * i : i), plane, S);
    const f32x4 b = plane_sum(p + (layout ? 2 * i + 4 : I + i), plane, S);
    const f16x4 d = *reinterpret_cast<const f16x4 *>(dh + at);
    const f32x4 g = layout ? f32x4{a[0], a[2], b[0], b[2]} : a;
    const f32x4 u = layout ? f32x4{a[1], a[3], b[1], b[3]} : b;
    store_dz(dz, m, I, i, layout, g, u, gscale[0], d);
}

// ---- many rows: decoded weights ------------------------------------------------------------------------
// w [N][K] to fp16 wt [K][ld], ld = N rounded up to 64, zeros in the padding. A thread takes eight rows' dwords; a
// block 64 rows by 256 columns, so a wave reads 32-byte pieces of 64 rows whose lines the block's other waves share,
// and eight neighbouring lanes store 128 contiguous bytes of a row of wt.
__global__ __launch_bounds__(256) void decode_transposed_kernel(const uint8_t *__restrict__ codes,
                                                                const uint8_t *__restrict__ scales, int N, int K, int ld,
                                                                f16 *__restrict__ wt)
{
    const int groups = (K + 255) / 256;
    const int n = (int)(blockIdx.x / groups) * 64 + 8 * (threadIdx.x & 7);
    const int k = (int)(blockIdx.x % groups) * 256 + 8 * (threadIdx.x >> 3);
    if (k >= K) return;
    uint32_t w[8], sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool in = n + i < N;  // N % 16 == 0: all eight rows or none
        const size_t row = in ? n + i : 0;
        w[i] = *reinterpret_cast<const uint32_t *>(codes + row * (K >> 1) + (k >> 1));
        sc[i] = in ? scales[row * (K >> 4) + (k >> 4)] : 0;
        if (!in) w[i] = 0;
    }
    f16x8 b[8];
    decode_columns(b, w, sc);
#pragma unroll
    for (int c = 0; c < 8; ++c) *reinterpret_cast<f16x8 *>(wt + (size_t)(k + c) * ld + n) = b[c];
}

// w [N][K] to fp16 in the same order, eight elements per thread. 4352 x 5120: 12.0 us (57 MB, 4.7 TB/s).
__global__ __launch_bounds__(256) void decode_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                     size_t eights, f16 *__restrict__ w)
{
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= eights) return;
    const f16 s = e4m3_pair<false>(scales[i >> 1])[0];
    reinterpret_cast<f16x8 *>(w)[i] = decode8(reinterpret_cast<const uint32_t *>(codes)[i], s);
}

// A [M][red] times B [cols][ld] over all stages or one of `splits` runs of them. 4096 x 2176 outputs of 5120: 87 us in the
// steady state, 99 traced (920 to 1050 TFLOP/s; 198 tiles on 256 CUs). PLANE: FP32 sums to plane
// blockIdx.y of `out`; else fp16(global * sum).
template <class T, bool PLANE>
__global__ __launch_bounds__(T::WAVES * 64) void grad_tile_kernel(const f16 *__restrict__ a, int M, int red,
                                                                  const f16 *__restrict__ b, int ld, int cols,
                                                                  const float *__restrict__ gscale, void *__restrict__ out)
{
    static_assert((uint64_t)(T::BM > T::BN ? T::BM : T::BN) * MAX_GRAD_ROWS * sizeof(f16) <= BUF_OOB, "a tile's rows within a buffer");
    __shared__ __attribute__((aligned(1024))) unsigned char smem[T::NS * T::BYTES];
    int tm, tn;
    if (!tile_of_block(blockIdx.x, (M + T::BM - 1) / T::BM, (cols + T::BN - 1) / T::BN, tm, tn)) return;
    const Place p = place_of<T>();
    const int m0 = tm * T::BM, c0 = tn * T::BN;
    Rows<T::LA> ra;
    Rows<T::LB> rb;
    ra.buf = make_rsrc(a + (size_t)m0 * red, (uint32_t)min(T::BM, M - m0) * red * 2u);
    rb.buf = make_rsrc(b + (size_t)c0 * ld, (uint32_t)min(T::BN, cols - c0) * ld * 2u);
#pragma unroll
    for (int i = 0; i < T::LA; ++i) {
        const int r = load_row<T>(p, i);
        ra.off[i] = m0 + r < M ? (uint32_t)r * red * 2u + load_byte(r, p.lane) : BUF_OOB;
    }
#pragma unroll
    for (int i = 0; i < T::LB; ++i) {
        const int r = load_row<T>(p, i), c = column_of_row<T>(r);
        rb.off[i] = c0 + c < cols ? (uint32_t)c * ld * 2u + load_byte(r, p.lane) : BUF_OOB;
    }
    const int stages = (red + 63) / 64, per = (stages + gridDim.y - 1) / gridDim.y;
    const int first = min(stages, (int)blockIdx.y * per), last = min(stages, first + per);
    const int tail = last == stages && red % 64 ? red % 64 * 2 : STAGE_BYTES;
    f32x4 acc[T::MT][T::NT];
    tile_product<T>(smem, p, ra, rb, first, last, tail, acc);
    const float gs = PLANE ? 1.0f : gscale[0];
#pragma unroll
    for (int m = 0; m < T::MT; ++m) {
        const int row = m0 + (p.wm * T::MT + m) * 16 + p.r;
        if (row >= M) continue;
#pragma unroll
        for (int t = 0; t < T::NT; ++t) {
            const int c = c0 + p.wn * 16 * T::NT + 4 * T::NT * p.q + 4 * t;
            if (c >= cols) continue;
            if constexpr (PLANE) {
                *reinterpret_cast<f32x4 *>(static_cast<float *>(out) + ((size_t)blockIdx.y * M + row) * cols + c) = acc[m][t];
            } else {
                f16x4 o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = f16_of_f32(acc[m][t][e] * gs);
                *reinterpret_cast<f16x4 *>(static_cast<f16 *>(out) + (size_t)row * cols + c) = o;
            }
        }
    }
}

// x [M][K] times the decoded gate and up rows, and the gradient of SwiGLU on them. Even tiles of a wave hold gate
// rows and odd ones the up rows of the same i, so that a lane has both: staged row 16 t + 4 q + j of wave column w
// is pair i0 + 8 NT w + 2 NT q + 4 (t / 2) + j, gate (t even) or up. 4096 rows of 4352 x 5120: 158 us behind the decoding
// (1155 TFLOP/s, 253 tiles in one round). Each load brings rows of one 16-row tile, and a
// wave's loads are all gates or all ups (the waves number a multiple of four).
template <class T>
__global__ __launch_bounds__(T::WAVES * 64) void swiglu_grad_tile_kernel(const f16 *__restrict__ x, int M, int K,
                                                                         const f16 *__restrict__ w, int I, int layout,
                                                                         const float *__restrict__ gscale,
                                                                         const f16 *__restrict__ dh, f16 *__restrict__ dz)
{
    static_assert(T::NT % 2 == 0 && T::WAVES % 4 == 0, "gates and ups in turn");
    constexpr int BI = T::BN / 2;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[T::NS * T::BYTES];
    int tm, tn;
    if (!tile_of_block(blockIdx.x, (M + T::BM - 1) / T::BM, (I + BI - 1) / BI, tm, tn)) return;
    const Place p = place_of<T>();
    const int m0 = tm * T::BM, i0 = tn * BI;
    const int up = (p.wave >> 1) & 1;  // load rows 8 (wave + WAVES i): tile (wave + WAVES i) / 2
    const f16 *wb = w + (layout ? (size_t)2 * i0 + up : (size_t)up * I + i0) * K;
    const uint32_t step = (uint32_t)K * (layout ? 4u : 2u);  // bytes from pair to pair
    Rows<T::LA> ra;
    Rows<T::LB> rb;
    ra.buf = make_rsrc(x + (size_t)m0 * K, (uint32_t)min(T::BM, M - m0) * K * 2u);
    rb.buf = make_rsrc(wb, (uint32_t)(min(BI, I - i0) - 1) * step + K * 2u);
#pragma unroll
    for (int i = 0; i < T::LA; ++i) {
        const int r = load_row<T>(p, i);
        ra.off[i] = m0 + r < M ? (uint32_t)r * K * 2u + load_byte(r, p.lane) : BUF_OOB;
    }
#pragma unroll
    for (int i = 0; i < T::LB; ++i) {
        const int r = load_row<T>(p, i);
        const int t = (r >> 4) % T::NT, wc = r / (16 * T::NT);
        const int pair = wc * 8 * T::NT + ((r >> 2) & 3) * 2 * T::NT + 4 * (t >> 1) + (r & 3);
        rb.off[i] = i0 + pair < I ? (uint32_t)pair * step + load_byte(r, p.lane) : BUF_OOB;
    }
    f32x4 acc[T::MT][T::NT];
    tile_product<T>(smem, p, ra, rb, 0, K / 64, STAGE_BYTES, acc);
    const float gs = gscale[0];
    const int pair0 = i0 + p.wn * 8 * T::NT + 2 * T::NT * p.q;
#pragma unroll
    for (int m = 0; m < T::MT; ++m) {
        const int row = m0 + (p.wm * T::MT + m) * 16 + p.r;
        f16x4 d[T::NT / 2];  // a row's loads at once
#pragma unroll
        for (int t = 0; t < T::NT; t += 2)
            d[t / 2] = *reinterpret_cast<const f16x4 *>(dh + (size_t)min(row, M - 1) * I + min(pair0 + 2 * t, I - 4));
        if (row >= M) continue;
#pragma unroll
        for (int t = 0; t < T::NT; t += 2) {
            const int i = pair0 + 2 * t;
            if (i < I) store_dz(dz, row, I, i, layout, acc[m][t], acc[m][t + 1], gs, d[t / 2]);
        }
    }
}

// ---- some hundred rows, gated: packed weights ----------------------------------------------------------------
// The gated gradient from the packed rows in one launch. Weight row 4 q + j of a wave's tile t is pair
// i0 + 8 NT w + 2 NT q + 2 t + j % 2, gate (j < 2) or up: a lane has both of 2 NT neighbouring pairs of a row.
// 4352 x 5120: 333 rows take 34 us (440 TFLOP/s; 55 us by chunk products, 46 decoded), 700 rows 53 us (590; 74 decoded), 1900
// rows 88 us (960; 115 decoded). A block alone on its CU is bound by a stage's latency (0.8 us: the way into LDS, which as
// compiled no product overlaps (packed_gemm.hpp), sixteen fragment reads, four decodes in a row), several by the LDS reads of
// A, which NT tiles of a wave share.
template <class T>
__global__ __launch_bounds__(T::THREADS, T::OCC) void swiglu_grad_packed_kernel(const f16 *__restrict__ x, int M, int K,
                                                                        const uint8_t *codes,
                                                                        const uint8_t *scales, int I, int layout,
                                                                        const float *__restrict__ gscale,
                                                                        const f16 *__restrict__ dh, f16 *__restrict__ dz)
{
    constexpr int BI = T::BN / 2, NP = 2 * T::NT;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[T::LDS];
    int tm, tn;
    if (!tile_of_block(blockIdx.x, (M + T::BM - 1) / T::BM, (I + BI - 1) / BI, tm, tn)) return;
    const PackedPlace p = packed_place<T>();
    const int m0 = tm * T::BM, i0 = tn * BI + p.wave * 8 * T::NT;
    PackedRows<T> b;
#pragma unroll
    for (int t = 0; t < T::NT; ++t) {
        const int i = min(i0 + NP * (p.r >> 2) + 2 * t + (p.r & 1), I - 1), up = (p.r >> 1) & 1;
        const size_t row = layout ? 2 * (size_t)i + up : (size_t)up * I + i;
        b.codes[t] = codes + row * (K >> 1) + 16 * p.q;
        b.scales[t] = scales + row * (K >> 4) + 2 * p.q;
    }
    f32x4 acc[T::MT][T::NT];
    if (!packed_product<T>(smem, p, x + (size_t)m0 * K, min(T::BM, M - m0), K, b, acc)) return;
    const float gs = gscale[0];
    const int i = i0 + NP * p.q;  // I % 16 == 0: all of a lane's pairs or none
    if (i >= I) return;
    typedef _Float16 pairs_t __attribute__((ext_vector_type(NP)));
    typedef _Float16 both_t __attribute__((ext_vector_type(2 * NP)));
    pairs_t dhs[T::MT];
#pragma unroll
    for (int m = 0; m < T::MT; ++m)
        dhs[m] = *reinterpret_cast<const pairs_t *>(dh + (size_t)min(m0 + 16 * m + p.r, M - 1) * I + i);
#pragma unroll
    for (int m = 0; m < T::MT; ++m) {
        const int row = m0 + 16 * m + p.r;
        if (row >= M) continue;
        const pairs_t d = dhs[m];
        pairs_t g, u;
        both_t z;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            const f32x4 &s = acc[m][e >> 1];
            float dg, du;
            swiglu_grad(s[e & 1] * gs, s[2 + (e & 1)] * gs, (float)d[e], dg, du);
            g[e] = z[2 * e] = f16_of_f32(dg), u[e] = z[2 * e + 1] = f16_of_f32(du);
        }
        f16 *o = dz + (size_t)row * 2 * I;
        if (layout) {
            *reinterpret_cast<both_t *>(o + 2 * i) = z;
        } else {
            *reinterpret_cast<pairs_t *>(o + i) = g;
            *reinterpret_cast<pairs_t *>(o + I + i) = u;
        }
    }
}

// ---- host --------------------------------------------------------------------------------------------
// The tile shapes; their times (Shape) are measured at 4352 x 5120 and 5120 x 2176 (1.0 to 1.35 PFLOP/s in whole rounds
// of tiles). Rounds decide at many rows: 4096 x 4352 outputs take 167 us in the one round of 384 x 192, 254 in the two of
// 256 x 256 (272 tiles on 256 CUs), 200 in the two of 192 x 192; 4096 x 2176 outputs 116 us with 192 x 256, 143 with
// 128 x 128. At some hundred rows small tiles fill the CUs: 333 x 5120 outputs of 4352 rows take 42 us with 64 x 64, 56 with
// 128 x 128. Three stages where a CU holds two blocks of them, two of 128 x 128 where its tiles are
// more than the CUs (1000 x 5120: 83 us, 102 with three stages and one block to a CU; 512 x 5120: 66 against 58).
using T384x192 = Tile<false, 6, 6, 4, 2, 2>;
using T256x256 = Tile<false, 8, 4, 2, 4, 2>;
using T192x256 = Tile<false, 6, 4, 2, 4, 2>;
using T192x192 = Tile<false, 3, 6, 4, 2, 2>;
using T128x128 = Tile<false, 4, 4, 2, 2, 2>;
using D128x128 = Tile<false, 4, 4, 2, 2, 3>;
using T64x64 = Tile<false, 2, 2, 2, 2, 3>;
constexpr Shape SHAPES[] = {{384, 192, 1, 1940, 1940}, {256, 256, 1, 1510, 1510}, {192, 256, 1, 1320, 1320},
                            {192, 192, 1, 1170, 1170}, {128, 128, 2, 800, 470},   {128, 128, 1, 690, 690},
                            {64, 64, 3, 345, 225}};

struct Choice {
    int shape, splits;
    int64_t ns;
};

// The shape, and the number of runs that the reduction axis is cut into, with the least estimated time: rounds of
// blocks over the CUs, and for more than one run the planes' way to memory and back and the fold's launch.
Choice choose(int64_t M, int64_t cols, int64_t red)
{
    const int64_t stages = (red + 63) / 64;
    Choice best = {0, 1, INT64_MAX};
    for (int i = 0; i < (int)(sizeof(SHAPES) / sizeof(SHAPES[0])); ++i) {
        const Shape &h = SHAPES[i];
        const int64_t tiles = h.tiles(M, cols);
        for (int s = 1; s <= 8 && (s == 1 || s * 8 <= stages); ++s) {
            int64_t ns = h.ns(tiles * s, (stages + s - 1) / s);
            if (s > 1) ns += 4000 + M * cols * 8 * s / 2500;  // there and back, with the fold's launch
            if (ns < best.ns) best = {i, s, ns};
        }
    }
    return best;
}

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
    default: return f(T64x64{});
    }
}

// Whether dx of M rows takes the packed weights in one stream, or decodes them for tiles. Estimates in ns fitted to
// measurements; us by the stream and the tiles: 4352 x 5120 22.7 and 33.7 at 100 rows, 34.5 and 44.1 at 200, 41.3 and
// 41.2 at 256, 53.2 and 44.4 at 333; 2048 x 2048 13.4 and 13.5 at 100, 20.0 and 17.0 at 200; 512 x 8192 12.5 and 10.9 at 100,
// 23.4 and 12.2 at 256.
bool grad_streams(int64_t M, int64_t N, int64_t K)
{
    if (M <= FEW_ROWS) return true;
    if (M > ST_MAX_M) return false;
    const int64_t elements = N * K;
    const int64_t stream = 5000 + elements / 6000 + (M + 15) / 16 * (900 + grad_planes((int)N) * K * 16 * 8 / 5000);
    return stream < choose(M, K, N).ns + 2500 + elements / 2000;
}

// The tiles on packed weights, for the gated gradient. Times of a stage of 128 elements (of two with KS = 2, whose groups
// walk them together), measured at 4352 x 5120.
using P64x64x2 = PackedTile<4, 1, 4, 2, 4>;
using P64x64 = PackedTile<4, 1, 4, 1, 4>;
using P128x128 = PackedTile<8, 2, 4, 1, 2>;
constexpr Shape PACKED[] = {{64, 64, 2, 1050, 800}, {64, 64, 4, 820, 400}, {128, 128, 2, 1450, 925}};

// How the gated gradient of M rows is computed: by the chunk products of linear.hip in passes of 64 rows and their fold
// (CHUNKS), in tiles on the packed weights (the number of the shape), or in tiles on decoded ones (DECODED). Estimates in
// ns fitted to measurements; 4352 x 5120, us by the three: 128 rows 23, 24, 34; 333 rows 55, 35, 46; 512 rows 81, 50, 61;
// 1000 rows 74 packed, 89 decoded; 1900 rows packed 88, 2000 rows 121 decoded; 4096 rows 215 packed, 166 decoded.
enum { CHUNKS = -2, DECODED = -1 };
int swiglu_way(int64_t M, int64_t rows, int64_t K)
{
    if (M <= FEW_ROWS) return CHUNKS;
    const int64_t elements = rows * K, stages = K / PACKED_STAGE;
    int way = CHUNKS;
    int64_t least = 7000 + elements / 4000 + M * (31 + num_chunks((int)K) * rows * 8 / 5000);  // the planes, there and back
    for (int i = 0; i < 3; ++i) {
        const int64_t ns = 2000 + PACKED[i].ns(PACKED[i].tiles(M, rows), i == 0 ? (stages + 1) / 2 : stages);
        if (ns < least) least = ns, way = i;
    }
    const int64_t decoded = choose(M, rows, K).ns + 2000 + elements * 53 / 100000;
    return decoded < least ? DECODED : way;
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
int padded(int n) { return (n + 63) & ~63; }

int launch_plain(const Choice &c, const f16 *a, int M, int red, const f16 *b, int ld, int cols, const float *gscale, void *out,
                 hipStream_t s)
{
    return with_shape(c.shape, [&](auto tile) {
        using T = decltype(tile);
        const int64_t tiles = SHAPES[c.shape].tiles(M, cols);
        return launch(c.splits > 1 ? grad_tile_kernel<T, true> : grad_tile_kernel<T, false>,
                      dim3(tile_grid(tiles), (unsigned)c.splits), dim3(T::WAVES * 64), 0, s, a, M, red, b, ld, cols, gscale, out);
    });
}

int launch_swiglu_fold(const float *part, int S, int M, int I, const nvfp4_weights &w, int layout, const f16 *dh, f16 *dz,
                       hipStream_t s)
{
    const size_t quads = (size_t)M * I / 4;
    return launch(swiglu_grad_fold_kernel, dim3((unsigned)((quads + FOLD_THREADS - 1) / FOLD_THREADS)), dim3(FOLD_THREADS), 0, s,
                  part, S, M, I, w.global_scale, layout, dh, dz);
}

}  // namespace

size_t linear_grad_ws_bytes(int32_t M, int32_t N, int32_t K)
{
    if (grad_streams(M, N, K)) return up256((size_t)grad_planes(N) * M * K * sizeof(float));
    const Choice c = choose(M, K, N);
    const size_t planes = c.splits > 1 ? (size_t)c.splits * M * K * sizeof(float) : 0;
    return up256((size_t)K * padded(N) * 2) + up256(planes);
}

int run_linear_grad(const uint16_t *dy, int32_t M, const nvfp4_weights &w, uint16_t *dx, void *ws, hipStream_t s)
{
    const int N = w.rows, K = w.k;
    const f16 *d = reinterpret_cast<const f16 *>(dy);
    f16 *o = reinterpret_cast<f16 *>(dx);
    const size_t plane = (size_t)M * K;
    auto fold = [&](const float *part, int S) {
        return launch(grad_fold_kernel, dim3((unsigned)((plane / 4 + FOLD_THREADS - 1) / FOLD_THREADS)), dim3(FOLD_THREADS), 0, s,
                      part, S, plane, w.global_scale, o);
    };
    if (grad_streams(M, N, K)) {
        float *part = static_cast<float *>(ws);
        const int S = grad_planes(N);
        const int st = launch(grad_stream_kernel, dim3(tile_grid((int64_t)K / ST_COLS * S)), dim3(ST_WAVES * 64), 0, s, d, M,
                              w.codes, w.scales, N, K, part);
        return st != NVFP4_OK ? st : fold(part, S);
    }
    const int ld = padded(N);
    f16 *wt = static_cast<f16 *>(ws);
    int st = launch(decode_transposed_kernel, dim3((unsigned)((ld / 64) * ((K + 255) / 256))), dim3(256), 0, s, w.codes, w.scales, N,
                    K, ld, wt);
    if (st != NVFP4_OK) return st;
    const Choice c = choose(M, K, N);
    if (c.splits == 1) return launch_plain(c, d, M, N, wt, ld, K, w.global_scale, o, s);
    float *part = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + up256((size_t)K * ld * 2));
    st = launch_plain(c, d, M, N, wt, ld, K, w.global_scale, part, s);
    return st != NVFP4_OK ? st : fold(part, c.splits);
}

size_t linear_swiglu_grad_ws_bytes(int32_t M, int32_t rows, int32_t K)
{
    const int way = swiglu_way(M, rows, K);
    if (way == CHUNKS) return up256(linear_ws_bytes(M, rows, K));
    if (way != DECODED) return 256;  // nothing is kept there; 0 means sizes that are rejected
    const Choice c = choose(M, rows, K);
    const size_t planes = c.splits > 1 ? (size_t)c.splits * M * rows * sizeof(float) : 0;
    return up256((size_t)rows * K * 2) + up256(planes);
}

int run_linear_swiglu_grad(const uint16_t *x, const uint16_t *dh, int32_t M, const nvfp4_weights &w, int32_t layout,
                           uint16_t *dz, void *ws, hipStream_t s)
{
    const int K = w.k, I = w.rows / 2;
    const f16 *xf = reinterpret_cast<const f16 *>(x), *df = reinterpret_cast<const f16 *>(dh);
    f16 *o = reinterpret_cast<f16 *>(dz);
    const int way = swiglu_way(M, w.rows, K);
    if (way == CHUNKS) {
        float *part = static_cast<float *>(ws);
        const int st = run_linear_partials(x, M, w, part, s);
        return st != NVFP4_OK ? st : launch_swiglu_fold(part, num_chunks(K), M, I, w, layout, df, o, s);
    }
    if (way != DECODED) {
        auto tiles = [&](auto tile) {
            using T = decltype(tile);
            return launch(swiglu_grad_packed_kernel<T>, dim3(tile_grid(PACKED[way].tiles(M, w.rows))), dim3(T::THREADS), 0, s, xf, M,
                          K, w.codes, w.scales, I, layout, w.global_scale, df, o);
        };
        return way == 0 ? tiles(P64x64x2{}) : way == 1 ? tiles(P64x64{}) : tiles(P128x128{});
    }
    f16 *wd = static_cast<f16 *>(ws);
    const size_t eights = (size_t)w.rows * K / 8;
    int st = launch(decode_kernel, dim3((unsigned)((eights + 255) / 256)), dim3(256), 0, s, w.codes, w.scales, eights, wd);
    if (st != NVFP4_OK) return st;
    const Choice c = choose(M, w.rows, K);
    if (c.splits == 1)
        return with_shape(c.shape, [&](auto tile) {
            using T = decltype(tile);
            const int64_t tiles = SHAPES[c.shape].tiles(M, w.rows);
            return launch(swiglu_grad_tile_kernel<T>, dim3(tile_grid(tiles)), dim3(T::WAVES * 64), 0, s, xf, M, K, wd, I, layout,
                          w.global_scale, df, o);
        });
    float *part = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + up256((size_t)w.rows * K * 2));
    st = launch_plain(c, xf, M, K, wd, K, w.rows, w.global_scale, part, s);
    return st != NVFP4_OK ? st : launch_swiglu_fold(part, c.splits, M, I, w, layout, df, o, s);
}

}  // namespace nvfp4
