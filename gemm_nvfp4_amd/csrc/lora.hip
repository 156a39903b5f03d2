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
#include "linear_device.hpp"
#include "nvfp4_device.hpp"
#include "ops.hpp"

namespace nvfp4 {
namespace {

constexpr int TILE = PLAN_TILE_ROWS;  // 16 rows

// Where the rows of a plan tile lie: pair order (row = pair index) or bucket order.
struct TileRows {
    const int32_t *hdr, *tile_expert, *tile_base, *tile_rows, *tile_pair, *pair_expert;
    int t_max, bucket;  // t_max: bound of the number of tiles
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

// ---- batches of many rows per adapter -------------------------------------------------------------
// A block takes a quad: four consecutive row tiles, one per wave. Tiles lie in adapter order, so a quad holds
// one adapter or a few, and goes through them one after the other (nearly always one), staging that
// adapter's matrix in LDS for the waves whose tile it is.
constexpr int QUAD = 4;

struct Quad {
    int e0, e1, e2, e3;  // adapters of its tiles; -1 behind the last tile
    __device__ __forceinline__ int adapter(int p) const { return p == 0 ? e0 : p == 1 ? e1 : p == 2 ? e2 : e3; }
    // whether tile p is the first one of its adapter
    __device__ __forceinline__ bool starts(int p) const
    {
        return adapter(p) >= 0 && (p == 0 || adapter(p) != adapter(p - 1));
    }
};

// The quad's adapters and, for this lane, row i of the wave's tile (-1 past its rows). All loads are issued
// together: what the plan holds behind its last tile is some word, and is dropped.
__device__ __forceinline__ Quad load_quad(const TileRows &tr, int quad, int &te, int &row)
{
    const int wave = threadIdx.x >> 6, i = threadIdx.x & 15, t0 = QUAD * quad, last = tr.t_max - 1;
    const int n = tr.hdr[3], t = min(t0 + wave, last);
    const int rows = tr.tile_rows[t], base = tr.bucket ? tr.tile_base[t] + i : tr.tile_pair[t * TILE + i];
    Quad r{tr.tile_expert[t0], tr.tile_expert[min(t0 + 1, last)], tr.tile_expert[min(t0 + 2, last)],
           tr.tile_expert[min(t0 + 3, last)]};
    if (t0 >= n) r.e0 = -1;
    if (t0 + 1 >= n) r.e1 = -1;
    if (t0 + 2 >= n) r.e2 = -1;
    if (t0 + 3 >= n) r.e3 = -1;
    te = __builtin_amdgcn_readfirstlane(r.adapter(wave));
    row = te >= 0 && i < rows ? base : -1;
    return r;
}

// Waits until at most `newest` of this wave's memory operations (the last ones issued) are outstanding.
__device__ __forceinline__ void wait_all_but(int newest)
{
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    if (newest == 2) __builtin_amdgcn_s_waitcnt(0x0F72);       // vmcnt(2); expcnt and lgkmcnt at their maxima
    else if (newest == 1) __builtin_amdgcn_s_waitcnt(0x0F71);
    else __builtin_amdgcn_s_waitcnt(0x0F70);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Shrink: one block per (quad, chunk, group of RT 16-rank tiles). A wave's rows of x go straight to
// registers, all 16 fragments in flight while A arrives by direct-to-LDS loads in two halves of the chunk (a
// whole chunk of 64 ranks would leave two blocks per CU). Half rows are 512 bytes without padding; the
// 16-byte piece at place p of rank r is piece p ^ (r & 15), so that the fragment reads of 16 ranks fall into
// distinct banks.
constexpr int HALF = KCHUNK / 2;

template <int RT>
__global__ __launch_bounds__(256, 3) void shrink_quad_kernel(TileRows tr, const f16 *__restrict__ x, int64_t P, int K, int rank,
                                                          const f16 *__restrict__ a, float *__restrict__ vp)
{
    __shared__ __attribute__((aligned(16))) unsigned char as[RT * 16 * HALF * 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    int te, row;
    const Quad quad = load_quad(tr, blockIdx.x, te, row);
    if (quad.e0 < 0) return;  // the whole block
    const int c = blockIdx.y, r0 = blockIdx.z * RT * 16;
    const int kb = c * KCHUNK, steps = min(KCHUNK, K - kb) >> 5;
    f16x8 xf[16];
    if (row >= 0) {  // lanes past the tile's rows feed whatever their registers hold into rows that are not stored
        const f16 *xp = x + (size_t)row * K + kb + 8 * q;
#pragma unroll
        for (int j = 0; j < 16; ++j) xf[j] = *reinterpret_cast<const f16x8 *>(xp + 32 * (j < steps ? j : 0));
    }
    typedef const __attribute__((address_space(3))) f16x8 lds_f16x8;
#pragma unroll 1
    for (int p = 0; p < QUAD; ++p) {
        if (!quad.starts(p)) continue;  // the whole block
        const unsigned char *ae = reinterpret_cast<const unsigned char *>(a + (size_t)quad.adapter(p) * rank * K);
        // Two half rows per instruction: lanes 0-31 rank 2v, lanes 32-63 rank 2v + 1 of pair v. Pieces past K
        // and ranks past the last one load their neighbours' bytes, which no result reads.
        auto stage = [&](int half) {
#pragma unroll
            for (int v = 0; v < RT * 2; ++v) {
                const int r = 2 * (wave + 4 * v) + (lane >> 5);
                const int k = kb + half * HALF + 8 * ((lane & 31) ^ (r & 15));
                const uint32_t off = 2u * ((uint32_t)min(r0 + r, rank - 1) * (uint32_t)K + (uint32_t)(k < K ? k : 0));
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(ae + off),
                                                 (__attribute__((address_space(3))) void *)(as + (wave + 4 * v) * 1024), 16, 0, 0);
            }
        };
        f32x4 acc[RT];
#pragma unroll
        for (int u = 0; u < RT; ++u) acc[u] = f32x4{0.f, 0.f, 0.f, 0.f};
        const bool mine = te == quad.adapter(p);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (half == 1 && steps <= 8) break;
            if (p + half > 0) lds_barrier();  // the staged fragments have been read
            stage(half);
            wait_all_but(0);  // this wave's direct-to-LDS loads have landed
            lds_barrier();    // and every other wave's
            if (mine) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (8 * half + (j & ~3) < steps) {  // K % 128 == 0: whole groups of four steps
#pragma unroll
                        for (int u = 0; u < RT; ++u)
                            acc[u] = mfma_step(xf[8 * half + j],
                                               *(lds_f16x8 *)(as + (16 * u + i) * HALF * 2 + 16 * ((4 * j + q) ^ i)), acc[u]);
                    }
            }
        }
        if (!mine) continue;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int orow = __shfl(row, 4 * q + n, 64);
            if (orow >= 0) {
#pragma unroll
                for (int u = 0; u < RT; ++u) {
                    const int r = r0 + 16 * u + i;
                    if (r < rank) vp[((size_t)c * P + orow) * rank + r] = acc[u][n];
                }
            }
        }
    }
}

// ---- expand ---------------------------------------------------------------------------------------
// One wave per (row tile, range of column groups), no barriers: a lane folds the 8 ranks of its token that it
// feeds (lane groups 0 and 2 the same ones, hi and lo), keeps the fragments of v in registers and streams B
// and the base result past them.
constexpr int EXPAND_WAVES = 4;
constexpr int GROUP_COLS = 64;  // outputs of one token per wave and step

// The lane's 8 ranks of step s of its token's v: chunk partials added in ascending order.
__device__ __forceinline__ void fold_v(float (&v)[8], const float *p, size_t plane, int S, bool valid)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (!valid) return;
    constexpr int CB = 8;  // chunks whose loads are issued before their adds
    for (int c0 = 0; c0 < S; c0 += CB) {
        f32x4 l[CB][2];
#pragma unroll
        for (int c = 0; c < CB; ++c)
            if (c0 + c < S) {
                l[c][0] = *reinterpret_cast<const f32x4 *>(p + (c0 + c) * plane);
                l[c][1] = *reinterpret_cast<const f32x4 *>(p + (c0 + c) * plane + 4);
            }
#pragma unroll
        for (int c = 0; c < CB; ++c)
            if (c0 + c < S) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = c0 + c ? v[e] + l[c][0][e] : l[c][0][e];
                    v[4 + e] = c0 + c ? v[4 + e] + l[c][1][e] : l[c][1][e];
                }
            }
    }
}

// The power of two that brings a row's largest finite |v| to [2^12, 2^13), and the two fp16 terms of a
// value scaled by it. Infinities and NaN stay in hi alone.
__device__ __forceinline__ int shift_of(float big)
{
    return big > 0.f ? 13 - __builtin_amdgcn_frexp_expf(big) : 0;  // frexp: big = f 2^e, f in [1/2, 1)
}
__device__ __forceinline__ void split(float v, int sh, f16 &hi, f16 &lo)
{
    const float f = __builtin_amdgcn_ldexpf(v, sh);
    hi = (f16)f;
    lo = fabsf(f) < __builtin_inff() ? (f16)(f - (float)hi) : (f16)0.f;
}

// The 16 consecutive outputs n0 + 16q .. + 15 of the lane's token, still scaled.
template <int RS>
__device__ __forceinline__ void expand16(float (&d)[16], const f16x8 (&vf)[RS], const f16 *be, int n0, int N, int rank, int i,
                                         int q)
{
    constexpr int SB = RS < 4 ? RS : 4;  // steps whose loads are issued together
    f32x4 acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bool bv = n0 + 16 * (i >> 2) < N;
    const f16 *bp = be + (size_t)(n0 + 16 * (i >> 2) + (i & 3)) * rank + 8 * (q & 1);
#pragma unroll
    for (int s0 = 0; s0 < RS; s0 += SB) {
        f16x8 bf[SB][4];
#pragma unroll
        for (int s = 0; s < SB; ++s) {
            const bool v = bv && 16 * (s0 + s) + 8 * (q & 1) < rank;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                bf[s][t] = zero8();
                if (v) bf[s][t] = *reinterpret_cast<const f16x8 *>(bp + (size_t)(4 * t) * rank + 16 * (s0 + s));
            }
        }
#pragma unroll
        for (int s = 0; s < SB; ++s)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[t] = mfma_step(bf[s][t], vf[s0 + s], acc[t]);
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

// GATE 0: plain; 1: gate rows [0, N/2), up rows [N/2, N); 2: row 2i gate i, row 2i + 1 up i. The waves of a
// block take consecutive column ranges of one tile.
template <typename BASE, int GATE, int RS>
__global__ __launch_bounds__(EXPAND_WAVES * 64) void expand_kernel(TileRows tr, int t_max, int t_all, int64_t P, int S, int N,
                                                                   int rank, const f16 *__restrict__ b,
                                                                   const float *__restrict__ scale,
                                                                   const float *__restrict__ vp, const BASE *base,
                                                                   f16 *out, int groups_per_wave)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    const int t = blockIdx.x, g0 = (blockIdx.y * EXPAND_WAVES + wave) * groups_per_wave;
    if (t >= t_all) return;
    const bool plain_rows = t >= t_max;  // rows without an adapter
    int row = -1, back = 0;
    float sc = 0.f;
    const f16 *be = b;
    f16x8 vf[RS];
    if (plain_rows) {
        const int64_t p = (int64_t)(t - t_max) * TILE + i;
        if (p < P && tr.pair_expert[p] < 0) row = (int)p;
    } else {
        if (t >= tr.hdr[3]) return;
        const int rows = tr.tile_rows[t], e = tr.tile_expert[t];
        if (i < rows) row = tile_row(tr, t, i);
        be = b + (size_t)e * N * rank;
        sc = scale[e];
        float v[RS][8], big = 0.f;
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            const int r = 16 * s + 8 * (q & 1);
            fold_v(v[s], vp + (size_t)(row < 0 ? 0 : row) * rank + r, (size_t)P * rank, S, row >= 0 && r < rank);
        }
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float f = fabsf(v[s][k]);
                if (f < __builtin_inff()) big = fmaxf(big, f);
            }
        big = fmaxf(big, __shfl_xor(big, 16, 64));  // the token's other eight ranks of each step
        const int sh = shift_of(big);
        back = -sh;
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                f16 hi, lo;
                split(v[s][k], sh, hi, lo);
                vf[s][k] = q < 2 ? hi : lo;
            }
    }
    const int I = N >> 1;
    const int cols = GATE == 1 ? I : N;  // columns that the groups cover
    for (int g = g0; g < g0 + groups_per_wave && g * GROUP_COLS < cols; ++g) {
        const int n0 = g * GROUP_COLS, n = n0 + 16 * q;
        const bool live = row >= 0 && n < cols;
        float y[16], y2[16], d[16], d2[16];
        if (live) {
            load_base(y, base + (size_t)row * N + n);
            if (GATE == 1) load_base(y2, base + (size_t)row * N + I + n);
        }
        if (!plain_rows) {
            expand16<RS>(d, vf, be, n0, cols, rank, i, q);
            if (GATE == 1) expand16<RS>(d2, vf, be + (size_t)I * rank, n0, cols, rank, i, q);
        }
        if (!live) continue;
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

// ---- expand of quads (lora_add) -------------------------------------------------------------------
// v folded and split once per row, in the order of the expand kernels' fragments: vs[row][r / 8] holds 8 hi
// then 8 lo terms, shifts[row] the row's power of two. Rows without an adapter are folded too (whatever the
// workspace holds) and never read. The blocks behind the folding ones copy those rows of y to out.
constexpr int FOLD_THREADS = 256;

__global__ __launch_bounds__(FOLD_THREADS) void fold_split_kernel(const float *__restrict__ vp, int64_t P, int S, int rank,
                                                                  int lg, f16 *__restrict__ vs, int *__restrict__ shifts,
                                                                  int64_t fold_blocks, const int32_t *__restrict__ pair_expert,
                                                                  const f16 *__restrict__ y, int N, f16 *__restrict__ out)
{
    if ((int64_t)blockIdx.x >= fold_blocks) {  // one block per row to copy (y and out are different buffers)
        const int64_t p = (int64_t)blockIdx.x - fold_blocks;
        if (pair_expert[p] >= 0) return;
        const f16x8 *src = reinterpret_cast<const f16x8 *>(y + p * N);
        f16x8 *dst = reinterpret_cast<f16x8 *>(out + p * N);
#pragma unroll 4
        for (int n = threadIdx.x; n < N / 8; n += FOLD_THREADS) dst[n] = src[n];
        return;
    }
    const int64_t row = (int64_t)blockIdx.x * (FOLD_THREADS >> lg) + (threadIdx.x >> lg);  // 2^lg lanes per row
    const int r = 8 * (threadIdx.x & ((1 << lg) - 1));
    const bool valid = row < P && r < rank;
    float v[8], big = 0.f;
    fold_v(v, vp + (valid ? row * rank + r : 0), (size_t)P * rank, S, valid);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f = fabsf(v[e]);
        if (f < __builtin_inff()) big = fmaxf(big, f);
    }
    for (int o = 1 << lg >> 1; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o, 64));
    if (!valid) return;
    const int sh = shift_of(big);
    f16x8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f16 h, l;
        split(v[e], sh, h, l);
        hi[e] = h, lo[e] = l;
    }
    f16 *o = vs + (row * rank + r) * 2;
    *reinterpret_cast<f16x8 *>(o) = hi;
    *reinterpret_cast<f16x8 *>(o + 8) = lo;
    if (r == 0) shifts[row] = sh;
}

// out = y + d for a quad's rows and a range of column groups. A group's B (64 rows of `rank` elements, one
// contiguous piece of memory) is staged in LDS by direct-to-LDS loads, the next group's while this one is
// computed; the accumulators go through LDS, so that y and out are read and written in whole 128-byte lines.
// Fragments of v stay in registers. The MFMA's row operand is B (rows 16u + i of the group in tile u), so a
// lane's accumulators are four neighbouring outputs of one token. What bounds it is the traffic of y; fragment loads of B and y straight
// from memory (a lane a row: one 16-byte piece per cycle and CU) took twice the time.
// LDS: B pieces of 8 ranks, piece p of row n at place p ^ swizzle(n); then 16 x D_PITCH floats per wave.
constexpr int D_PITCH = GROUP_COLS + 4;

template <int RS>
struct BStage {
    static constexpr int PIECES = 2 * RS;                 // 16-byte pieces per row, rank padded to 16 RS
    static constexpr int BYTES = GROUP_COLS * PIECES * 16;
    static constexpr int BUFFERS = RS <= 8 ? 2 : 1;
    static constexpr size_t LDS = (size_t)BUFFERS * BYTES + (size_t)QUAD * TILE * D_PITCH * sizeof(float);
    // rows of fewer than 16 pieces: row n of the 16 that a fragment read takes, by the bank slots they share
    __device__ static __forceinline__ int place(int n, int p)
    {
        return PIECES >= 16 ? (p & ~15) | ((p ^ n) & 15) : p ^ ((n / (16 / PIECES)) & (PIECES - 1));
    }
};

template <int RS>
__global__ __launch_bounds__(256) void expand_quad_kernel(TileRows tr, int N, int rank, const f16 *__restrict__ b,
                                                          const float *__restrict__ scale, const f16 *__restrict__ vs,
                                                          const int *__restrict__ shifts, const f16 *y, f16 *out,
                                                          int groups_per_block)
{
    typedef BStage<RS> B;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    int te, row;
    const Quad quad = load_quad(tr, blockIdx.x, te, row);
    if (quad.e0 < 0) return;  // the whole block
    const int g0 = blockIdx.y * groups_per_block, g_end = min(g0 + groups_per_block, (N + GROUP_COLS - 1) / GROUP_COLS);
    // This lane's two pieces of a group's y and out: rows 8h + lane / 8, columns 8 (lane % 8) .. + 7.
    const int c8 = 8 * (lane & 7);
    int yrow[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) yrow[h] = __shfl(row, 8 * h + (lane >> 3), 64);
    float *dw = reinterpret_cast<float *>(smem + B::BUFFERS * B::BYTES) + wave * TILE * D_PITCH;
    typedef __attribute__((address_space(3))) unsigned char lds_byte;
    typedef const __attribute__((address_space(3))) f16x8 lds_f16x8;
    f16x8 yv[2];
    auto load_y = [&](int g) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (yrow[h] >= 0 && g < g_end && g * GROUP_COLS + c8 < N)
                yv[h] = *reinterpret_cast<const f16x8 *>(y + (size_t)yrow[h] * N + g * GROUP_COLS + c8);
    };
    f16x8 vf[RS];
    float sc = 0.f;
    int back = 0;
#pragma unroll 1
    for (int p = 0; p < QUAD; ++p) {
        if (!quad.starts(p)) continue;  // the whole block
        const bool mine = te == quad.adapter(p);
        const unsigned char *be = reinterpret_cast<const unsigned char *>(b + (size_t)quad.adapter(p) * N * rank);
        // Place l of the group's pieces (row n = l / PIECES) is filled with the piece that belongs there; pieces
        // past the rank and rows past N are read as some other piece, and only ever meet zeros of v or columns
        // that are not stored.
        auto stage = [&](int g) {
            const unsigned char *bg = be + (size_t)g * GROUP_COLS * rank * 2;
            const int cols = N - g * GROUP_COLS;
#pragma unroll
            for (int v = 0; v < GROUP_COLS * B::PIECES / 256 || v == 0; ++v) {
                const int first = (wave + QUAD * v) * 64, l = first + lane, n = l / B::PIECES;
                if (B::PIECES == 2 && wave >= 2) break;  // 64 rows of two pieces: two waves' loads
                const int piece = B::place(n, l % B::PIECES);  // its own inverse
                const uint32_t off = 2u * ((uint32_t)min(n, cols - 1) * (uint32_t)rank + (uint32_t)(8 * piece < rank ? 8 * piece : 0));
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(bg + off),
                                                 (__attribute__((address_space(3))) void *)(smem + (B::BUFFERS == 2 ? (g & 1) * B::BYTES : 0) +
                                                                                            first * 16),
                                                 16, 0, 0);
            }
        };
        if (p > 0) lds_barrier();  // the staged fragments have been read
        stage(g0);
        if (mine) {
            load_y(g0);
            sc = scale[te];
            back = row >= 0 ? -shifts[row] : 0;
#pragma unroll
            for (int s = 0; s < RS; ++s) {
                const int r = 16 * s + 8 * (q & 1);
                vf[s] = zero8();
                if (row >= 0 && r < rank) vf[s] = *reinterpret_cast<const f16x8 *>(vs + ((size_t)row * rank + r) * 2 + 8 * (q >> 1));
            }
        }
        int stores = 0;  // this wave's newest memory operations, wave-uniform
        for (int g = g0; g < g_end; ++g) {
            const int n0 = g * GROUP_COLS;
            wait_all_but(stores);  // this wave's part of the group's B has landed
            lds_barrier();         // and every other wave's; the other buffer has been read
            f16x8 yc[2] = {yv[0], yv[1]};
            if (B::BUFFERS == 2 && g + 1 < g_end) stage(g + 1);
            if (mine) {
                load_y(g + 1);
                __builtin_amdgcn_sched_barrier(0);  // loads before the stores below, which the next wait leaves out
                const unsigned char *bs = smem + (B::BUFFERS == 2 ? (g & 1) * B::BYTES : 0);
                f32x4 acc[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < RS; ++s)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int n = 16 * u + i;
                        acc[u] = mfma_step(*(lds_f16x8 *)(lds_byte *)(bs + (n * B::PIECES + B::place(n, 2 * s + (q & 1))) * 16), vf[s],
                                           acc[u]);
                    }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    f32x4 d;
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = __builtin_amdgcn_ldexpf(acc[u][e], back);
                    *reinterpret_cast<f32x4 *>(dw + i * D_PITCH + 16 * u + 4 * q) = d;
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
                stores = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float *sp = dw + (8 * h + (lane >> 3)) * D_PITCH + c8;
                    const f32x4 lo = *reinterpret_cast<const f32x4 *>(sp), hi = *reinterpret_cast<const f32x4 *>(sp + 4);
                    f16x8 o;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = f16_of_f32(fmaf(sc, e < 4 ? lo[e & 3] : hi[e & 3], (float)yc[h][e]));
                    const bool live = yrow[h] >= 0 && n0 + c8 < N;
                    if (live) *reinterpret_cast<f16x8 *>(out + (size_t)yrow[h] * N + n0 + c8) = o;
                    stores += __ballot(live) != 0;
                }
                __builtin_amdgcn_wave_barrier();
            }
            if (B::BUFFERS == 1 && g + 1 < g_end) {
                lds_barrier();  // the staged fragments have been read
                stage(g + 1);
                stores = 0;     // the staging loads are newer than the stores
            }
        }
    }
}

TileRows tile_rows(const PlanView &pv, const PlanLayout &L, int bucket)
{
    return TileRows{pv.hdr, pv.tile_expert, pv.tile_base, pv.tile_rows, pv.tile_pair, pv.pair_expert, (int)L.T, bucket};
}

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// The quad kernels, once adapters average at least 16 rows and the batch is not small.
bool use_quads(int64_t P, int adapters) { return P >= 512 && P >= 16 * (int64_t)adapters; }

template <int RT>
int launch_shrink(const TileRows &tr, int64_t t_max, int64_t P, const f16 *x, const nvfp4_lora &lora, float *vp,
                  hipStream_t s)
{
    const unsigned gy = (unsigned)num_chunks(lora.k), gz = (unsigned)((lora.rank + 16 * RT - 1) / (16 * RT));
    return launch(shrink_kernel<RT>, dim3((unsigned)((t_max + SHRINK_WAVES - 1) / SHRINK_WAVES), gy, gz),
                  dim3(SHRINK_WAVES * 64), 0, s, tr, x, P, lora.k, lora.rank, reinterpret_cast<const f16 *>(lora.a), vp);
}

int launch_shrink(const TileRows &tr, int64_t t_max, int64_t P, const f16 *x, const nvfp4_lora &lora, float *vp,
                  hipStream_t s)
{
    if (lora.rank <= 16) return launch_shrink<1>(tr, t_max, P, x, lora, vp, s);
    if (lora.rank <= 32) return launch_shrink<2>(tr, t_max, P, x, lora, vp, s);
    return launch_shrink<4>(tr, t_max, P, x, lora, vp, s);
}

template <typename BASE, int GATE, int RS>
int launch_expand_rs(const TileRows &tr, int64_t t_max, int64_t P, bool others, const nvfp4_lora &lora, const float *vp,
                     const BASE *base, f16 *out, hipStream_t s)
{
    const int N = lora.rows, cols = GATE == 1 ? N / 2 : N;
    const int groups = (cols + GROUP_COLS - 1) / GROUP_COLS;
    const int64_t tiles = t_max + (others ? (P + TILE - 1) / TILE : 0);
    // about sixteen waves per CU of the device, at most 17 column groups each
    int per_wave = (int)(tiles * groups / (16 * (int64_t)device_cus()));
    per_wave = per_wave < 1 ? 1 : per_wave > 17 ? 17 : per_wave;
    const int per_block = per_wave * EXPAND_WAVES;
    return launch(expand_kernel<BASE, GATE, RS>, dim3((unsigned)tiles, (unsigned)((groups + per_block - 1) / per_block)),
                  dim3(EXPAND_WAVES * 64), 0, s, tr, (int)t_max, (int)tiles, P, num_chunks(lora.k), N, lora.rank,
                  reinterpret_cast<const f16 *>(lora.b), lora.scale, vp, base, out, per_wave);
}

template <typename BASE, int GATE>
int launch_expand(const TileRows &tr, int64_t t_max, int64_t P, bool others, const nvfp4_lora &lora, const float *vp,
                  const BASE *base, f16 *out, hipStream_t s)
{
    const int rs = (lora.rank + 15) / 16;
    if (rs <= 1) return launch_expand_rs<BASE, GATE, 1>(tr, t_max, P, others, lora, vp, base, out, s);
    if (rs <= 2) return launch_expand_rs<BASE, GATE, 2>(tr, t_max, P, others, lora, vp, base, out, s);
    if (rs <= 4) return launch_expand_rs<BASE, GATE, 4>(tr, t_max, P, others, lora, vp, base, out, s);
    if (rs <= 8) return launch_expand_rs<BASE, GATE, 8>(tr, t_max, P, others, lora, vp, base, out, s);
    return launch_expand_rs<BASE, GATE, 16>(tr, t_max, P, others, lora, vp, base, out, s);
}

constexpr int QUAD_BLOCKS_PER_CU = 3;

template <int RS>
int launch_expand_quad(const TileRows &tr, const nvfp4_lora &lora, const f16 *vs, const int *shifts, const f16 *y, f16 *out,
                       hipStream_t s)
{
    const int groups = (lora.rows + GROUP_COLS - 1) / GROUP_COLS, quads = (tr.t_max + QUAD - 1) / QUAD;
    int per_block = (int)((int64_t)quads * groups / (QUAD_BLOCKS_PER_CU * (int64_t)device_cus()));
    per_block = per_block < 1 ? 1 : per_block;
    const size_t lds = BStage<RS>::LDS;
    static_assert(BStage<RS>::LDS <= 64 * 1024, "within the LDS that a launch may use without an opt-in");
    return launch(expand_quad_kernel<RS>, dim3((unsigned)quads, (unsigned)((groups + per_block - 1) / per_block)), dim3(256), lds,
                  s, tr, lora.rows, lora.rank, reinterpret_cast<const f16 *>(lora.b), lora.scale, vs, shifts, y, out, per_block);
}

// lora_add of a batch of quads: shrink, fold + split (and the rows without an adapter), expand.
int add_quads(const TileRows &tr, int64_t P, const f16 *x, const nvfp4_lora &lora, const f16 *y, f16 *out, uint8_t *ws,
              hipStream_t s)
{
    const int rank = lora.rank, S = num_chunks(lora.k);
    const size_t vp_bytes = round256((size_t)S * P * rank * sizeof(float));
    float *vp = reinterpret_cast<float *>(ws);
    f16 *vs = reinterpret_cast<f16 *>(ws + vp_bytes);
    int *shifts = reinterpret_cast<int *>(ws + vp_bytes + round256((size_t)P * rank * 4));
    const unsigned quads = (unsigned)((tr.t_max + QUAD - 1) / QUAD);
    const f16 *a = reinterpret_cast<const f16 *>(lora.a);
    int st;
    if (rank <= 16) st = launch(shrink_quad_kernel<1>, dim3(quads, S), dim3(256), 0, s, tr, x, P, lora.k, rank, a, vp);
    else if (rank <= 32) st = launch(shrink_quad_kernel<2>, dim3(quads, S), dim3(256), 0, s, tr, x, P, lora.k, rank, a, vp);
    else st = launch(shrink_quad_kernel<4>, dim3(quads, S, (rank + 63) / 64), dim3(256), 0, s, tr, x, P, lora.k, rank, a, vp);
    if (st != NVFP4_OK) return st;
    int lg = 0;
    while ((8 << lg) < rank) ++lg;
    const int64_t fold_blocks = (P + (FOLD_THREADS >> lg) - 1) / (FOLD_THREADS >> lg);
    const int64_t copy_blocks = !tr.bucket && out != y ? P : 0;
    st = launch(fold_split_kernel, dim3((unsigned)(fold_blocks + copy_blocks)), dim3(FOLD_THREADS), 0, s, vp, P, S, rank, lg,
                vs, shifts, fold_blocks, tr.pair_expert, y, lora.rows, out);
    if (st != NVFP4_OK) return st;
    const int rs = (rank + 15) / 16;
    return rs <= 1 ? launch_expand_quad<1>(tr, lora, vs, shifts, y, out, s)
         : rs <= 2 ? launch_expand_quad<2>(tr, lora, vs, shifts, y, out, s)
         : rs <= 4 ? launch_expand_quad<4>(tr, lora, vs, shifts, y, out, s)
         : rs <= 8 ? launch_expand_quad<8>(tr, lora, vs, shifts, y, out, s)
                   : launch_expand_quad<16>(tr, lora, vs, shifts, y, out, s);
}

}  // namespace

size_t lora_add_ws_bytes(int64_t P, int32_t K, int32_t rank)
{
    // chunk partials of v; v folded and split; its shifts
    return round256((size_t)num_chunks(K) * (size_t)P * rank * sizeof(float)) + round256((size_t)P * rank * 4) +
           round256((size_t)P * 4);
}

size_t linear_lora_ws_bytes(int32_t M, int32_t rows, int32_t K, int32_t rank)
{
    return round256((size_t)M * rows * sizeof(float)) + lora_add_ws_bytes(M, K, rank);
}

int run_lora_add(const PlanView &pv, const PlanLayout &L, int32_t order, const uint16_t *x, const nvfp4_lora &lora,
                 const uint16_t *y, uint16_t *out, void *ws, hipStream_t s)
{
    const TileRows tr = tile_rows(pv, L, order);
    if (use_quads(L.P, lora.adapters))
        return add_quads(tr, L.P, reinterpret_cast<const f16 *>(x), lora, reinterpret_cast<const f16 *>(y),
                         reinterpret_cast<f16 *>(out), static_cast<uint8_t *>(ws), s);
    float *vp = static_cast<float *>(ws);
    const int st = launch_shrink(tr, L.T, L.P, reinterpret_cast<const f16 *>(x), lora, vp, s);
    if (st != NVFP4_OK) return st;
    return launch_expand<f16, 0>(tr, L.T, L.P, order == 0 && out != y, lora, vp, reinterpret_cast<const f16 *>(y),
                                 reinterpret_cast<f16 *>(out), s);
}

int run_linear_lora(const PlanView &pv, const PlanLayout &L, const uint16_t *x, int32_t M, const nvfp4_weights &w,
                    const nvfp4_lora &lora, bool gated, int32_t layout, uint16_t *y, void *ws, hipStream_t s)
{
    const TileRows tr = tile_rows(pv, L, 0);
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
