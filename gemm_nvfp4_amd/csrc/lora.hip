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
//           B's rows are the MFMA's row operand and the tokens its columns, so a lane ends with four
//           neighbouring outputs of one token.
// Three forms of it, with the same results bitwise:
//   beside a projection   the projection's chunk products and the shrink in one launch, their sums, the expand
//                         and the epilogue in a second. Bound by the weight stream and the latency of two launches.
//   lora_add by tiles     shrink, then expand by row tiles: small batches, where latency counts.
//   lora_add by quads     shrink and expand by four row tiles with A and B staged in LDS, v folded and split by a
//                         launch between them: bound by the traffic of x and y.
// Fragment loads straight from memory (16 lanes read 16 rows) cost the address unit a cycle per lane, so that
// large batches bring matrices and results through LDS in whole lines.
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

// Waits until at most `newest` of this wave's memory operations (the last ones issued) are outstanding.
__device__ __forceinline__ void wait_all_but(int newest)
{
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    if (newest == 2) __builtin_amdgcn_s_waitcnt(0x0F72);       // vmcnt(2); expcnt and lgkmcnt at their maxima
    else if (newest == 1) __builtin_amdgcn_s_waitcnt(0x0F71);
    else __builtin_amdgcn_s_waitcnt(0x0F70);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// ---- shrink ---------------------------------------------------------------------------------------
// One wave per unit: (row tile t, 16-rank tile u, chunk c), chunks fastest; vp[c][row][r] = the chunk's
// part of v. Lanes of rows past the tile's load nothing (a tile of a decode batch is often one row).
__device__ __forceinline__ void shrink_unit(const TileRows &tr, int64_t unit, const f16 *x, int64_t P, int K, int rank,
                                            const f16 *a, float *vp)
{
    const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
    const int S = num_chunks(K), U = (rank + 15) >> 4;
    const int c = (int)(unit % S), tu = (int)(unit / S), r0 = 16 * (tu % U), t = tu / U;
    if (t >= tr.t_max) return;  // wave-uniform, as all below but the row
    const int n = tr.hdr[3], e = tr.tile_expert[t], rows = tr.tile_rows[t];
    const int at = tr.bucket ? tr.tile_base[t] + i : tr.tile_pair[t * TILE + i];
    if (t >= n) return;
    const int row = i < rows ? at : -1;
    const int kb = c * KCHUNK, steps = min(KCHUNK, K - kb) >> 5;
    const f16 *ap = a + ((size_t)e * rank + min(r0 + i, rank - 1)) * K + kb + 8 * q;
    const f16 *xp = x + (size_t)(row < 0 ? 0 : row) * K + kb + 8 * q;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 16; h += 8) {  // eight steps' loads in flight at once
        f16x8 af[8], xf[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // K % 128 == 0: whole groups of four steps
            af[j] = xf[j] = zero8();
            if (((h + j) & ~3) < steps) {
                af[j] = *reinterpret_cast<const f16x8 *>(ap + 32 * (h + j));
                if (row >= 0) xf[j] = *reinterpret_cast<const f16x8 *>(xp + 32 * (h + j));
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (((h + j) & ~3) < steps) acc = mfma_step(xf[j], af[j], acc);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int orow = __shfl(row, 4 * q + k, 64);
        if (orow >= 0 && r0 + i < rank) vp[((size_t)c * P + orow) * rank + r0 + i] = acc[k];
    }
}

constexpr int SHRINK_WAVES = 4;
__global__ __launch_bounds__(SHRINK_WAVES * 64) void shrink_kernel(TileRows tr, const f16 *__restrict__ x, int64_t P, int K,
                                                                   int rank, const f16 *__restrict__ a,
                                                                   float *__restrict__ vp)
{
    shrink_unit(tr, (int64_t)blockIdx.x * SHRINK_WAVES + (threadIdx.x >> 6), x, P, K, rank, a, vp);
}

int64_t shrink_units(const TileRows &tr, const nvfp4_lora &lora)
{
    return (int64_t)tr.t_max * ((lora.rank + 15) / 16) * num_chunks(lora.k);
}

// ---- the projection's chunk products and the shrink in one launch ---------------------------------
// Blocks [0, shrink_blocks) take shrink units. Each of the others takes one chunk and one 16-row weight tile
// per wave, as the split-K form of the projection (linear.hip): part[c][m][n] is the library's chunk result,
// so the sum over c is bitwise nvfp4_linear's. Small batches decode the weights
// anew for every 16 rows of x: the 100 registers of a wave then let all blocks of a launch be resident at once,
// several to a CU, so that the shrink's, whose first loads wait for the plan, run beside the weight stream. KEEP,
// for larger ones: decoded weights kept for all rows, one block per CU, 64 rows of x staged at once (whole call in a
// captured graph, 4352 x 5120, rank 16, KEEP off and on: 15.8 and 18.3 us at 32 rows, 18.2 and 18.3 at 33, 22.1 and
// 20.5 at 64, 30.6 and 24.5 at 128, 242 and 125 at 1024, 819 and 506 at 4096). The partials are S = K / 512 planes of
// the whole output, written here and read by the second launch: at 4096 rows 713 MB each way, 280 us of the call at the
// rate of a copy.
constexpr int FUSED_WAVES = 12;  // most waves per block
// A launch holds fewer than 2^32 threads along one axis. WIDE, for grids past that: FUSED_GRID_X blocks along x, then y. (In
// its own instance: the index in every grid cost the kernel that keeps the weights two spilled registers, 25.9 instead of
// 24.5 us at 128 rows of 4352 x 5120.)
constexpr int FUSED_GRID_X = 1 << 20;

template <bool KEEP, bool WIDE>
__global__ __launch_bounds__(FUSED_WAVES * 64, KEEP ? 3 : 4) void linear_shrink_kernel(const f16 *__restrict__ x, int M,
                                                                            const uint8_t *__restrict__ codes,
                                                                            const uint8_t *__restrict__ scales, int N, int K,
                                                                            float *__restrict__ part, TileRows tr, int rank,
                                                                            const f16 *__restrict__ a, float *__restrict__ vp,
                                                                            int shrink_blocks)
{
    constexpr int ROWS = KEEP ? 64 : 32;  // activation rows staged in LDS per pass
    __shared__ __attribute__((aligned(16))) unsigned char xs[ROWS * XS_PITCH];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nwaves = blockDim.x >> 6;
    const int block = (WIDE ? (int)blockIdx.y * FUSED_GRID_X : 0) + (int)blockIdx.x;
    if (block < shrink_blocks) {
        shrink_unit(tr, (int64_t)block * nwaves + wave, x, M, K, rank, a, vp);
        return;
    }
    const int S = num_chunks(K), blk = block - shrink_blocks, c = blk % S;
    if (WIDE && (blk / S) * nwaves >= N >> 4) return;  // the whole block: behind the last one
    const int n = lane & 15, q = lane >> 4;
    const int t = (blk / S) * nwaves + wave;  // this wave's weight tile
    const bool tv = t < (N >> 4);             // wave-uniform
    const int kb = c * KCHUNK;
    const bool qv = q < (min(KCHUNK, K - kb) >> 7);
    RawChunk w = RawChunk{};
    if (tv && qv) {
        const size_t row = (size_t)t * 16 + n;
        w = load_chunk(codes + row * ((size_t)K >> 1), scales + row * ((size_t)K >> 4), kb, q);
    }
    f16x8 bf[4][4];
    const int k = kb + 8 * lane;
    for (int m0 = 0; m0 < M; m0 += ROWS) {
        const int gm = min(M - m0, ROWS);
        if (m0 > 0) lds_barrier();  // the previous pass's fragment reads are done
        for (int r = wave; r < gm; r += nwaves) {
            const f16 *src = x + (size_t)(m0 + r) * K + (k < K ? k : 0);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                             (__attribute__((address_space(3))) void *)(xs + r * XS_PITCH), 16, 0, 0);
        }
        wait_all_but(0);  // this wave's direct-to-LDS loads (and weights) are done
        lds_barrier();    // and every other wave's
        if (!tv) continue;
        auto decode = [&]() {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const f16x2 sc = chunk_scales(w, b);
#pragma unroll
                for (int s = 0; s < 4; ++s) bf[b][s] = decode8(w.codes[b][s], sc[s >> 1]);
            }
        };
        if (KEEP && m0 == 0) decode();
#pragma unroll 1
        for (int rt = 0; rt * 16 < gm; ++rt) {
            f16x8 af[4][4];
            load_a_tile<A_STAGED>(af, x, make_rsrc(x, 0), xs, rt * 16 + n, gm, K, kb, q, qv);
            if (!KEEP) {
                keep_in_loop(w);
                decode();
            }
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int s = 0; s < 4; ++s) acc = mfma_step(af[b][s], bf[b][s], acc);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = m0 + rt * 16 + 4 * q + j;
                if (m < M) part[((size_t)c * M + m) * N + (size_t)t * 16 + n] = acc[j];
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

// Shrink: one block per (quad, chunk, group of RT 16-rank tiles). A wave's rows of x go straight to
// registers, all 16 fragments in flight while A arrives by direct-to-LDS loads: for 64 ranks in two halves of
// the chunk (a whole one would leave two blocks per CU: 22.4 instead of 18.6 us at 4096 rows, rank 64, K =
// 5120), else at once. Staged rows have no padding; the 16-byte piece at place p of rank r is piece
// p ^ (r & 15), so that the fragment reads of 16 ranks fall into distinct banks.
template <int RT>
__global__ __launch_bounds__(256, 3) void shrink_quad_kernel(TileRows tr, const f16 *__restrict__ x, int64_t P, int K, int rank,
                                                          const f16 *__restrict__ a, float *__restrict__ vp)
{
    constexpr int PHASES = RT == 4 ? 2 : 1, PART = KCHUNK / PHASES;  // elements of a rank staged at once
    constexpr int RPI = 512 / PART;                                  // ranks per 1 KB instruction
    __shared__ __attribute__((aligned(16))) unsigned char as[RT * 16 * PART * 2];
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
        // Pieces past K and ranks past the last one load other bytes of the matrix, which no result reads.
        auto stage = [&](int phase) {
#pragma unroll
            for (int v = 0; v < RT * 4 / RPI; ++v) {
                const int r = RPI * (wave + QUAD * v) + lane / (64 / RPI);
                const int k = kb + phase * PART + 8 * ((lane % (64 / RPI)) ^ (r & 15));
                const uint32_t off = 2u * ((uint32_t)min(r0 + r, rank - 1) * (uint32_t)K + (uint32_t)(k < K ? k : 0));
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(ae + off),
                                                 (__attribute__((address_space(3))) void *)(as + (wave + QUAD * v) * 1024),
                                                 16, 0, 0);
            }
        };
        f32x4 acc[RT];
#pragma unroll
        for (int u = 0; u < RT; ++u) acc[u] = f32x4{0.f, 0.f, 0.f, 0.f};
        const bool mine = te == quad.adapter(p);
#pragma unroll
        for (int ph = 0; ph < PHASES; ++ph) {
            constexpr int STEPS = 16 / PHASES;
            if (ph > 0 && steps <= STEPS) break;
            if (p + ph > 0) lds_barrier();  // the staged fragments have been read
            stage(ph);
            wait_all_but(0);  // this wave's direct-to-LDS loads have landed
            lds_barrier();    // and every other wave's
            if (mine) {
#pragma unroll
                for (int j = 0; j < STEPS; ++j)
                    if (STEPS * ph + (j & ~3) < steps) {  // K % 128 == 0: whole groups of four steps
#pragma unroll
                        for (int u = 0; u < RT; ++u)
                            acc[u] = mfma_step(xf[STEPS * ph + j],
                                               *(lds_f16x8 *)(as + (16 * u + i) * PART * 2 + 16 * ((4 * j + q) ^ i)), acc[u]);
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

// ---- expand of tiles ------------------------------------------------------------------------------
// One block per (row tile, 128 columns), one wave per 64 columns. After the plan's words come the chunk partials of
// v (folded by the block into LDS), B and the base result. Behind the plan's tiles lie pseudo tiles of 16
// consecutive rows each, for the rows without an adapter. EARLY: B and the base result are asked for before the
// partials are waited for, and held in registers meanwhile (launch_expand says when).
constexpr int GROUP_COLS = 64;   // outputs of one token per wave
constexpr int TILE_WAVES = 2;   // (4: 7.3 instead of 6.4 us at 32 rows of 4352 x 5120, rank 16, an adapter each)

// Four ranks of a row's v: its chunk partials added in ascending order, the loads of ten chunks in flight at
// once.
struct Fold4 {
    f32x4 v;
    __device__ __forceinline__ void run(const float *p, size_t plane, int S)
    {
        constexpr int CB = 10;
        v = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int c0 = 0; c0 < S; c0 += CB) {
            f32x4 l[CB];
#pragma unroll
            for (int c = 0; c < CB; ++c)
                if (c0 + c < S) l[c] = *reinterpret_cast<const f32x4 *>(p + (c0 + c) * plane);
#pragma unroll
            for (int c = 0; c < CB; ++c)
                if (c0 + c < S) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = c0 + c ? v[e] + l[c][e] : l[c][e];
                }
        }
    }
};

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

// The fragments of a token's v from its row in LDS: the lane's 8 ranks of each step, scaled and split (hi in lane
// groups 0 and 1, lo in 2 and 3); zeros past `rank`. Returns the power of two.
template <int RS>
__device__ __forceinline__ int split_row(f16x8 (&vf)[RS], const float *v32, int rank, int q)
{
    float v[RS][8], big = 0.f;
#pragma unroll
    for (int s = 0; s < RS; ++s) {
        const int r = 16 * s + 8 * (q & 1);
        const f32x4 v0 = *reinterpret_cast<const f32x4 *>(v32 + r), v1 = *reinterpret_cast<const f32x4 *>(v32 + r + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[s][k] = r < rank ? (k < 4 ? v0[k & 3] : v1[k & 3]) : 0.f;
            const float f = fabsf(v[s][k]);
            if (f < __builtin_inff()) big = fmaxf(big, f);
        }
    }
    big = fmaxf(big, __shfl_xor(big, 16, 64));  // the token's other eight ranks of each step
    const int sh = shift_of(big);
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            f16 hi, lo;
            split(v[s][k], sh, hi, lo);
            vf[s][k] = q < 2 ? hi : lo;
        }
    return sh;
}

// The fragments of B for ranks 16s0 .. + 16SB - 1 of a group of 64 outputs: rows n0 + 16u + i in MFMA tile u, so
// that a lane ends with the outputs n0 + 16u + 4q .. + 3 of token i.
template <int SB>
__device__ __forceinline__ void load_b(f16x8 (&bf)[SB][4], const f16 *be, int n0, int N, int rank, int s0, int i, int q)
{
    const f16 *bp = be + (size_t)(n0 + i) * rank + 8 * (q & 1);
#pragma unroll
    for (int s = 0; s < SB; ++s)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            bf[s][u] = zero8();
            if (n0 + 16 * u < N && 16 * (s0 + s) + 8 * (q & 1) < rank)  // N % 16 == 0
                bf[s][u] = *reinterpret_cast<const f16x8 *>(bp + (size_t)(16 * u) * rank + 16 * (s0 + s));
        }
}

// The base result of eight consecutive outputs, in two steps: start() issues its loads (of the first CB chunks,
// for chunk partials), finish() returns it in FP32.
template <typename T, int CB>
struct BaseLoads;

template <int CB>
struct BaseLoads<f16, CB> {
    f16x8 v;
    __device__ __forceinline__ void start(const f16 *p, size_t, int) { v = *reinterpret_cast<const f16x8 *>(p); }
    __device__ __forceinline__ void finish(float (&y)[8], const f16 *, size_t, int, float)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (float)v[e];
    }
};

template <int CB>
struct BaseLoads<float, CB> {
    f32x4 v[CB][2];
    __device__ __forceinline__ void load(const float *p, size_t plane, int c0, int S)
    {
#pragma unroll
        for (int c = 0; c < CB; ++c)
            if (c0 + c < S) {
                v[c][0] = *reinterpret_cast<const f32x4 *>(p + (c0 + c) * plane);
                v[c][1] = *reinterpret_cast<const f32x4 *>(p + (c0 + c) * plane + 4);
            }
    }
    __device__ __forceinline__ void start(const float *p, size_t plane, int S) { load(p, plane, 0, S); }
    __device__ __forceinline__ void finish(float (&y)[8], const float *p, size_t plane, int S, float gs)
    {
        for (int c0 = 0; c0 < S; c0 += CB) {
            if (c0 > 0) load(p, plane, c0, S);
#pragma unroll
            for (int c = 0; c < CB; ++c)
                if (c0 + c < S) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = c0 + c ? y[e] + v[c][e >> 2][e & 3] : v[c][e >> 2][e & 3];
                }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= gs;
    }
};

// Base: y fp16 [P][N] (T = f16), or Sb planes of FP32 [P][N] that are added in order and scaled by gscale[0].
// GATE 0: plain; 1: gate rows [0, N/2), up rows [N/2, N); 2: row 2i gate i, row 2i + 1 up i.
// The accumulators go through LDS, so that the base result is read and the output written in row segments: lane
// l finishes columns 8 (l % 8) .. + 7 of the wave's 64, of rows l / 8 and l / 8 + 8 of the tile.
constexpr int D_PITCH = GROUP_COLS + 4;

template <typename T, int GATE, int RS, bool EARLY>
__global__ __launch_bounds__(TILE_WAVES * 64) void expand_tile_kernel(TileRows tr, int64_t P, int S, int N, int rank,
                                                                      const f16 *__restrict__ b,
                                                                      const float *__restrict__ scale,
                                                                      const float *__restrict__ vp, const T *base, int Sb,
                                                                      const float *__restrict__ gscale, f16 *out)
{
    constexpr int SETS = GATE == 1 ? 2 : 1;      // column sets: gate and up rows apart
    constexpr int SB = RS < 4 ? RS : 4;          // steps of B whose loads are issued together
    constexpr int CB = 10 / SETS;                // chunk planes whose loads are issued together
    constexpr int V_PITCH = 16 * RS + 4;
    __shared__ float v32[TILE * V_PITCH];
    __shared__ float dw[TILE_WAVES][SETS][TILE][D_PITCH];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    const int t = blockIdx.x, n0 = (blockIdx.y * TILE_WAVES + wave) * GROUP_COLS, n = n0 + 8 * (lane & 7);
    const bool plain_rows = t >= tr.t_max;  // rows without an adapter
    int row = -1, e = 0, rows = TILE;
    if (plain_rows) {
        const int64_t p = (int64_t)(t - tr.t_max) * TILE + i;
        if (p < P && tr.pair_expert[p] < 0) row = (int)p;
    } else {
        const int nt = tr.hdr[3], at = tr.bucket ? tr.tile_base[t] + i : tr.tile_pair[t * TILE + i];
        rows = tr.tile_rows[t];
        e = tr.tile_expert[t];
        if (t >= nt) return;  // the whole block
        if (i < rows) row = at;
    }
    const int I = N >> 1, cols = GATE == 1 ? I : N;
    const size_t plane = (size_t)P * N;
    const float gs = gscale ? gscale[0] : 1.0f;
    BaseLoads<T, CB> bl[SETS];
    auto start = [&](int r) {
        if (r < 0 || n >= cols) return;
#pragma unroll
        for (int z = 0; z < SETS; ++z) bl[z].start(base + (size_t)r * N + z * I + n, plane, Sb);
    };
    auto finish = [&](int m, int r, float sc) {
        if (r < 0 || n >= cols) return;
        float y[SETS][8];
#pragma unroll
        for (int z = 0; z < SETS; ++z) {
            bl[z].finish(y[z], base + (size_t)r * N + z * I + n, plane, Sb, gs);
            if (!plain_rows) {
                const float *dp = &dw[wave][z][m][8 * (lane & 7)];
                const f32x4 d0 = *reinterpret_cast<const f32x4 *>(dp), d1 = *reinterpret_cast<const f32x4 *>(dp + 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    y[z][k] = fmaf(sc, d0[k], y[z][k]);
                    y[z][4 + k] = fmaf(sc, d1[k], y[z][4 + k]);
                }
            }
        }
        if constexpr (GATE == 2) {
            typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
            f16x4 o;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = f16_of_f32(swiglu(y[0][2 * k], y[0][2 * k + 1]));
            *reinterpret_cast<f16x4 *>(out + (size_t)r * I + (n >> 1)) = o;
        } else {
            f16x8 o;
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = f16_of_f32(GATE == 1 ? swiglu(y[0][k], y[SETS - 1][k]) : y[0][k]);
            *reinterpret_cast<f16x8 *>(out + (size_t)r * cols + n) = o;
        }
    };
    const int m0 = lane >> 3, r_first = __shfl(row, m0, 64), r_second = __shfl(row, m0 + 8, 64);
    if (plain_rows) {
        if constexpr (sizeof(T) == sizeof(f16)) {  // y's bits: a conversion would change signalling NaN
            start(r_first);
            if (r_first >= 0 && n < cols) *reinterpret_cast<f16x8 *>(out + (size_t)r_first * cols + n) = bl[0].v;
            start(r_second);
            if (r_second >= 0 && n < cols) *reinterpret_cast<f16x8 *>(out + (size_t)r_second * cols + n) = bl[0].v;
        } else {
            start(r_first);
            finish(m0, r_first, 0.f);
            start(r_second);
            finish(m0 + 8, r_second, 0.f);
        }
        return;
    }
    const f16 *be = b + (size_t)e * N * rank;
    f16x8 bf[SETS][SB][4];
    auto start_rest = [&]() {
#pragma unroll
        for (int z = 0; z < SETS; ++z) load_b<SB>(bf[z], be + (size_t)z * I * rank, n0, cols, rank, 0, i, q);
        start(r_first);
    };
    if (EARLY) start_rest();
    // v: one thread per four ranks of a row, all chunks in flight.
    const int r4 = rank >> 2, tasks = rows * r4;
    for (int t0 = 0; t0 < tasks; t0 += TILE_WAVES * 64) {
        const int task = t0 + threadIdx.x, m = task / r4, r = 4 * (task - m * r4);
        const int vrow = __shfl(row, m & 15, 64);  // lane m holds row m
        if (task < tasks) {
            Fold4 f;
            f.run(vp + (size_t)vrow * rank + r, (size_t)P * rank, S);
            *reinterpret_cast<f32x4 *>(&v32[m * V_PITCH + r]) = f.v;
        }
    }
    if (!EARLY) start_rest();
    lds_barrier();
    f16x8 vf[RS];
    const int sh = split_row<RS>(vf, &v32[i * V_PITCH], row >= 0 ? rank : 0, q);
    f32x4 acc[SETS][4];
#pragma unroll
    for (int z = 0; z < SETS; ++z)
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[z][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < RS; ++s) {
        if (s > 0 && s % SB == 0) {
#pragma unroll
            for (int z = 0; z < SETS; ++z) load_b<SB>(bf[z], be + (size_t)z * I * rank, n0, cols, rank, s, i, q);
        }
#pragma unroll
        for (int z = 0; z < SETS; ++z)
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[z][u] = mfma_step(bf[z][s % SB][u], vf[s], acc[z][u]);
    }
#pragma unroll
    for (int z = 0; z < SETS; ++z)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            f32x4 d;
#pragma unroll
            for (int k = 0; k < 4; ++k) d[k] = __builtin_amdgcn_ldexpf(acc[z][u][k], -sh);
            *reinterpret_cast<f32x4 *>(&dw[wave][z][i][16 * u + 4 * q]) = d;
        }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    const float sc = scale[e];
    finish(m0, r_first, sc);
    if (rows > 8) {  // wave-uniform
        start(r_second);
        finish(m0 + 8, r_second, sc);
    }
}

// ---- expand of quads (lora_add) -------------------------------------------------------------------
// v folded and split once per row, in the order of the expand kernel's fragments: vs[row][r / 8] holds 8 hi
// then 8 lo terms, shifts[row] the row's power of two. Rows without an adapter are folded too (whatever the
// workspace holds) and never read. The blocks behind the folding ones copy those rows of y to out.
// (Folding in the expand blocks instead, once per column range, saves this launch but was slower: 25.0 instead
// of 23.0 us at 6000 rows, rank 16, four chunks; copying there too: 51 instead of 46 us at 4096 rows, rank 64.)
constexpr int FOLD_THREADS = 64;  // small blocks: the few threads spread over all CUs (256: 7.1 instead of 6.0 us)

__global__ __launch_bounds__(FOLD_THREADS) void fold_split_kernel(const float *__restrict__ vp, int64_t P, int S, int rank,
                                                                  int lg, f16 *__restrict__ vs, int *__restrict__ shifts,
                                                                  int64_t fold_blocks, const int32_t *__restrict__ pair_expert,
                                                                  const f16 *__restrict__ y, int N, f16 *__restrict__ out)
{
    if ((int64_t)blockIdx.x >= fold_blocks) {  // a block copies row after row (y and out are different buffers)
        for (int64_t p = (int64_t)blockIdx.x - fold_blocks; p < P; p += (int64_t)gridDim.x - fold_blocks) {
            if (pair_expert[p] >= 0) continue;
            const f16x8 *src = reinterpret_cast<const f16x8 *>(y + p * N);
            f16x8 *dst = reinterpret_cast<f16x8 *>(out + p * N);
#pragma unroll 4
            for (int n = threadIdx.x; n < N / 8; n += FOLD_THREADS) dst[n] = src[n];
        }
        return;
    }
    const int64_t row = (int64_t)blockIdx.x * (FOLD_THREADS >> lg) + (threadIdx.x >> lg);  // 2^lg lanes per row
    const int r = 8 * (threadIdx.x & ((1 << lg) - 1));
    const bool valid = row < P && r < rank;
    Fold4 v[2];
    v[0].v = v[1].v = f32x4{0.f, 0.f, 0.f, 0.f};
    float big = 0.f;
    if (valid) {
        v[0].run(vp + row * rank + r, (size_t)P * rank, S);
        v[1].run(vp + row * rank + r + 4, (size_t)P * rank, S);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f = fabsf(v[e >> 2].v[e & 3]);
        if (f < __builtin_inff()) big = fmaxf(big, f);
    }
    for (int o = 1 << lg >> 1; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o, 64));
    if (!valid) return;
    const int sh = shift_of(big);
    f16x8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f16 h, l;
        split(v[e >> 2].v[e & 3], sh, h, l);
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
// lane's accumulators are four neighbouring outputs of one token. What bounds it is the traffic of y (71 MB in 20 us
// at 4096 rows, rank 64, N = 4352). NT: y and out past the caches. Fragment loads of B and y straight from memory took 87 us.
// LDS: B pieces of 8 ranks, piece p of row n at place p ^ swizzle(n); then 16 x D_PITCH floats per wave.
__device__ __attribute__((aligned(16))) const uint32_t zero_piece[4] = {0, 0, 0, 0};

template <int RS>
struct BStage {
    static constexpr int PIECES = 2 * RS;                 // 16-byte pieces per row, rank padded to 16 RS
    static constexpr int BYTES = GROUP_COLS * PIECES * 16;
    static constexpr int BUFFERS = RS <= 8 ? 2 : 1;
    static constexpr size_t LDS = (size_t)BUFFERS * BYTES + (size_t)QUAD * TILE * D_PITCH * sizeof(float);
    // rows of fewer than 16 pieces: row n of the 16 that a fragment read takes, by the bank slots they share
    __device__ static __forceinline__ int place(int n, int p)
    {
        if constexpr (PIECES >= 16) return (p & ~15) | ((p ^ n) & 15);
        else return p ^ ((n / (16 / PIECES)) & (PIECES - 1));
    }
};

template <int RS, bool NT>
__global__ __launch_bounds__(256) void expand_quad_kernel(TileRows tr, int N, int rank, const f16 *__restrict__ b,
                                                          const float *__restrict__ scale, const f16 *__restrict__ vs,
                                                          const int *__restrict__ shifts, const f16 *y, f16 *out,
                                                          int groups_per_block)
{
    typedef BStage<RS> B;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    const int g0 = blockIdx.y * groups_per_block, g_end = min(g0 + groups_per_block, (N + GROUP_COLS - 1) / GROUP_COLS);
    int te, row;
    const Quad quad = load_quad(tr, blockIdx.x, te, row);
    if (quad.e0 < 0) return;  // the whole block
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
            if (yrow[h] >= 0 && g < g_end && g * GROUP_COLS + c8 < N) {
                const f16x8 *p = reinterpret_cast<const f16x8 *>(y + (size_t)yrow[h] * N + g * GROUP_COLS + c8);
                yv[h] = NT ? __builtin_nontemporal_load(p) : *p;
            }
    };
    f16x8 vf[RS];
    float sc = 0.f;
    int back = 0;
#pragma unroll 1
    for (int p = 0; p < QUAD; ++p) {
        if (!quad.starts(p)) continue;  // the whole block
        const bool mine = te == quad.adapter(p);
        const unsigned char *be = reinterpret_cast<const unsigned char *>(b + (size_t)quad.adapter(p) * N * rank);
        // Place l of the group's pieces (row n = l / PIECES) is filled with the piece that belongs there, zeros past
        // the rank; rows past N are read as the last row, for columns that are not stored.
        auto stage = [&](int g) {
            const unsigned char *bg = be + (size_t)g * GROUP_COLS * rank * 2;
            const int cols = N - g * GROUP_COLS;
#pragma unroll
            for (int v = 0; v < GROUP_COLS * B::PIECES / 256 || v == 0; ++v) {
                const int first = (wave + QUAD * v) * 64, l = first + lane, n = l / B::PIECES;
                if (B::PIECES == 2 && wave >= 2) break;  // 64 rows of two pieces: two waves' loads
                const int piece = B::place(n, l % B::PIECES);  // its own inverse
                const uint32_t off = 2u * ((uint32_t)min(n, cols - 1) * (uint32_t)rank + 8u * (uint32_t)piece);
                const void *src = 8 * piece < rank ? static_cast<const void *>(bg + off) : zero_piece;
                unsigned char *dst = smem + (B::BUFFERS == 2 ? (g & 1) * B::BYTES : 0) + first * 16;
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                                 (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
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
                if (row >= 0 && r < rank)
                    vf[s] = *reinterpret_cast<const f16x8 *>(vs + ((size_t)row * rank + r) * 2 + 8 * (q >> 1));
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
                        const unsigned char *bp = bs + (n * B::PIECES + B::place(n, 2 * s + (q & 1))) * 16;
                        acc[u] = mfma_step(*(lds_f16x8 *)(lds_byte *)bp, vf[s], acc[u]);
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
                    if (live) {
                        f16x8 *p = reinterpret_cast<f16x8 *>(out + (size_t)yrow[h] * N + n0 + c8);
                        if (NT) __builtin_nontemporal_store(o, p);
                        else *p = o;
                    }
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

// The quad kernels take batches of enough work, with at least two row tiles for each adapter of the table. Measured in a
// captured graph with x, y and out of three calls in turn, tile against quad kernels (us): rank 16, K = 5120, N = 4352,
// one adapter: 15.3 / 16.1 at 1024 rows, 18.1 / 17.9 at 1536, 23.3 / 21.1 at 2048, 46.8 / 33.0 at 4096; rank 16, K = 2048,
// N = 1024: 15.4 / 17.8 at 4096, 22.9 / 23.4 at 8192, 46.8 / 42.3 at 16384; with 64 adapters there 15.8 / 17.8 at 4096,
// 23.2 / 22.7 at 6000; rank 8, K = N = 4096: 18.6 / 20.5 at 2048, 35.7 / 33.2 at 4096; rank 64, K = 5120, N = 4352: 16.1 /
// 15.4 at 256, 23.4 / 17.7 at 512, 34.3 / 20.1 at 1024; with 64 adapters there 35.8 / 49.6 at 1024 (16 rows each, four
// adapters to a quad), 59.2 / 35.0 at 2048. The host knows the table, not how many of its adapters a batch uses: 4096 rows of 8
// adapters out of more than 128 take the tile kernels, 107 us at 256 where the quad kernels take 47.
bool use_quads(int64_t P, const nvfp4_lora &lora)
{
    return P * lora.rank * ((int64_t)lora.k + lora.rows) >= 250000000 && P >= 32 * (int64_t)lora.adapters;
}

int launch_shrink(const TileRows &tr, int64_t P, const f16 *x, const nvfp4_lora &lora, float *vp, hipStream_t s)
{
    const int64_t blocks = (shrink_units(tr, lora) + SHRINK_WAVES - 1) / SHRINK_WAVES;
    return launch(shrink_kernel, dim3((unsigned)blocks), dim3(SHRINK_WAVES * 64), 0, s, tr, x, P, lora.k, lora.rank,
                  reinterpret_cast<const f16 *>(lora.a), vp);
}

// Base result of the expand kernels: a finished y, or Sb planes with their scale.
template <typename T>
struct BaseOf {
    const T *y;
    int Sb;
    const float *gscale;
    bool others;  // rows without an adapter are written too
};

template <typename T, int GATE>
int launch_expand(const TileRows &tr, int64_t P, const nvfp4_lora &lora, const float *vp, const BaseOf<T> &base, f16 *out,
                  hipStream_t s)
{
    const int N = lora.rows, cols = GATE == 1 ? N / 2 : N, rs = (lora.rank + 15) / 16;
    const int64_t tiles = tr.t_max + (base.others ? (P + TILE - 1) / TILE : 0);
    const int64_t groups = (cols + TILE_WAVES * GROUP_COLS - 1) / (TILE_WAVES * GROUP_COLS);
    // EARLY for chunk partials (an fp16 base is one load and only pays for the registers: lora_add of 64 rows of 32
    // adapters, rank 64, 17.5 us without and 19.4 with), but for rank 16 only in up to three blocks per CU, since it
    // leaves two waves per SIMD instead of three. Measured without and with (whole linear_lora, 4352 x 5120): rank 64
    // 12.6 and 10.4 us at one row, 34.5 and 30.0 at 64 rows of 32 adapters; rank 16 9.4 and 9.1 at one row, 12.0 and
    // 11.8 at 16, 24.8 and 26.3 at 64.
    const bool early = rs > 1 || tiles * groups <= 3 * (int64_t)device_cus();
    auto go = [&](auto *kernel) {
        return launch(kernel, dim3((unsigned)tiles, (unsigned)groups), dim3(TILE_WAVES * 64), 0, s, tr, P,
                      num_chunks(lora.k), N, lora.rank, reinterpret_cast<const f16 *>(lora.b), lora.scale, vp, base.y, base.Sb,
                      base.gscale, out);
    };
    constexpr bool E = sizeof(T) == 4;
    return rs <= 1 ? (early ? go(expand_tile_kernel<T, GATE, 1, E>) : go(expand_tile_kernel<T, GATE, 1, false>))
         : rs <= 2 ? go(expand_tile_kernel<T, GATE, 2, E>) : rs <= 4 ? go(expand_tile_kernel<T, GATE, 4, E>)
         : rs <= 8 ? go(expand_tile_kernel<T, GATE, 8, E>) : go(expand_tile_kernel<T, GATE, 16, E>);
}

template <int RS>
int launch_expand_quad(const TileRows &tr, int64_t P, const nvfp4_lora &lora, const f16 *vs, const int *shifts, const f16 *y,
                       f16 *out, hipStream_t s)
{
    const int groups = (lora.rows + GROUP_COLS - 1) / GROUP_COLS, quads = (tr.t_max + QUAD - 1) / QUAD;
    // About four blocks per CU, of two column groups at least. Measured with 1, 2, 3, 4 and 6 per CU: 24.9, 21.2,
    // 21.6, 20.1 and 23.3 us at 4096 rows, rank 64, N = 4352.
    const int per_cu = (int)((int64_t)quads * groups / (4 * (int64_t)device_cus()));
    const int per_block = per_cu < 2 ? 2 : per_cu;
    static_assert(BStage<RS>::LDS <= 64 * 1024, "within the LDS that a launch may use without an opt-in");
    // y and out together past 64 MiB, in whole lines: non-temporal, so that they leave the caches to x and v. Measured
    // without and with (whole lora_add, rows over 4352 x 5120, rank 64, with x, y and out of three calls in turn): 54.4
    // and 51.0 us at 4096 rows, 79.4 and 74.8 at 8192; but 49.0 and 50.8 at 4096 in place, 35.3 and 36.9 at 2048; 8192
    // rows of 2048, 31.8 and 33.0; 16384 rows of 1040, 63.0 and 64.4.
    const bool nt = lora.rows % 64 == 0 && (out == y ? 1 : 2) * P * lora.rows * (int64_t)sizeof(f16) > (int64_t(64) << 20);
    return launch(nt ? expand_quad_kernel<RS, true> : expand_quad_kernel<RS, false>,
                  dim3((unsigned)quads, (unsigned)((groups + per_block - 1) / per_block)), dim3(256), BStage<RS>::LDS, s, tr,
                  lora.rows, lora.rank, reinterpret_cast<const f16 *>(lora.b), lora.scale, vs, shifts, y, out, per_block);
}

constexpr int64_t MAX_COPY_BLOCKS = 1 << 20;  // a launch holds fewer than 2^32 threads

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
    const int64_t copy_blocks = tr.bucket || out == y ? 0 : P < MAX_COPY_BLOCKS ? P : MAX_COPY_BLOCKS;
    st = launch(fold_split_kernel, dim3((unsigned)(fold_blocks + copy_blocks)), dim3(FOLD_THREADS), 0, s, vp, P, S, rank, lg,
                vs, shifts, fold_blocks, tr.pair_expert, y, lora.rows, out);
    if (st != NVFP4_OK) return st;
    const int rs = (rank + 15) / 16;
    return rs <= 1 ? launch_expand_quad<1>(tr, P, lora, vs, shifts, y, out, s)
         : rs <= 2 ? launch_expand_quad<2>(tr, P, lora, vs, shifts, y, out, s)
         : rs <= 4 ? launch_expand_quad<4>(tr, P, lora, vs, shifts, y, out, s)
         : rs <= 8 ? launch_expand_quad<8>(tr, P, lora, vs, shifts, y, out, s)
                   : launch_expand_quad<16>(tr, P, lora, vs, shifts, y, out, s);
}

}  // namespace

size_t lora_add_ws_bytes(int64_t P, int32_t K, int32_t rank)
{
    // chunk partials of v; v folded and split; its shifts
    return round256((size_t)num_chunks(K) * (size_t)P * rank * sizeof(float)) + round256((size_t)P * rank * 4) +
           round256((size_t)P * 4);
}

// The projection's chunk products (as many as nvfp4_linear_ws keeps), then the chunk partials of v.
size_t linear_lora_ws_bytes(int32_t M, int32_t rows, int32_t K, int32_t rank)
{
    return round256(linear_ws_bytes(M, rows, K)) + round256((size_t)num_chunks(K) * (size_t)M * rank * sizeof(float));
}

int run_lora_add(const PlanView &pv, const PlanLayout &L, int32_t order, const uint16_t *x, const nvfp4_lora &lora,
                 const uint16_t *y, uint16_t *out, void *ws, hipStream_t s)
{
    const TileRows tr = tile_rows(pv, L, order);
    const f16 *xh = reinterpret_cast<const f16 *>(x), *yh = reinterpret_cast<const f16 *>(y);
    f16 *oh = reinterpret_cast<f16 *>(out);
    if (use_quads(L.P, lora)) return add_quads(tr, L.P, xh, lora, yh, oh, static_cast<uint8_t *>(ws), s);
    float *vp = static_cast<float *>(ws);
    const int st = launch_shrink(tr, L.P, xh, lora, vp, s);
    if (st != NVFP4_OK) return st;
    return launch_expand<f16, 0>(tr, L.P, lora, vp, BaseOf<f16>{yh, 1, nullptr, order == 0 && out != y}, oh, s);
}

int run_linear_lora(const PlanView &pv, const PlanLayout &L, const uint16_t *x, int32_t M, const nvfp4_weights &w,
                    const nvfp4_lora &lora, bool gated, int32_t layout, uint16_t *y, void *ws, hipStream_t s)
{
    const TileRows tr = tile_rows(pv, L, 0);
    const f16 *xh = reinterpret_cast<const f16 *>(x);
    const int N = w.rows, K = w.k, S = num_chunks(K);
    float *part = static_cast<float *>(ws);
    float *vp = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + round256(linear_ws_bytes(M, N, K)));
    // One unit (weight tile and chunk, or shrink unit) per wave: T waves per block for so many blocks per CU. Four
    // up to 16 rows, three above: measured for this launch (4352 x 5120) with 1, 2, 3, 4 and 6 per CU 8.8, 6.9, 6.8,
    // 6.6 and 7.6 us at one row, 12.2, 12.0, 10.8, 11.1 and 13.9 at 32. One, with the weights kept, beyond 64 rows,
    // and from 33 where its blocks all fit at once (15.1 and 14.6 us at 64 rows).
    const int64_t shrinks = shrink_units(tr, lora), units = (int64_t)(N / 16) * S + shrinks, cus = device_cus();
    auto waves = [&](int64_t slots) {
        const int64_t t = (units + slots - 1) / slots;
        return (int)(t < 1 ? 1 : t > FUSED_WAVES ? FUSED_WAVES : t);
    };
    auto blocks_of = [&](int T) { return (shrinks + T - 1) / T + (int64_t)S * ((N / 16 + T - 1) / T); };
    const bool keep = M > 64 || (M > 32 && blocks_of(waves(cus)) <= cus);
    const int T = waves(keep ? cus : (M > 16 ? 3 : 4) * cus);
    const int64_t blocks = blocks_of(T);
    const bool wide = blocks * T * 64 >= (int64_t(1) << 32);  // then M is far beyond 64
    const dim3 grid = wide ? dim3(FUSED_GRID_X, (unsigned)((blocks + FUSED_GRID_X - 1) / FUSED_GRID_X)) : dim3((unsigned)blocks);
    const int st = launch(wide ? linear_shrink_kernel<true, true> : keep ? linear_shrink_kernel<true, false>
                                                                         : linear_shrink_kernel<false, false>,
                          grid, dim3((unsigned)(T * 64)), 0, s, xh, M, w.codes, w.scales, N, K, part, tr, lora.rank,
                          reinterpret_cast<const f16 *>(lora.a), vp, (int)((shrinks + T - 1) / T));
    if (st != NVFP4_OK) return st;
    const BaseOf<float> base{part, S, w.global_scale, true};
    f16 *o = reinterpret_cast<f16 *>(y);
    if (!gated) return launch_expand<float, 0>(tr, L.P, lora, vp, base, o, s);
    if (layout == 0) return launch_expand<float, 1>(tr, L.P, lora, vp, base, o, s);
    return launch_expand<float, 2>(tr, L.P, lora, vp, base, o, s);
}

}  // namespace nvfp4
