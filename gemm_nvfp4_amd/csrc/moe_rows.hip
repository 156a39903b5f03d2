// moe_rows.hip -- rows moved by the routing plan: tokens sorted by expert (permute), expert rows summed
// back into their tokens with the routing weights (unpermute), and that sum's gradient.
//
//   permute         xs[pos(p)] = w[p] x[t]                            p = t*topk + k, pos = pos_of_pair
//   unpermute       out[t]     = sum_k w[p] ys[pos(p)]                in slot order, one fp16 rounding
//   unpermute_grad  dys[pos(p)] = w[p] dout[t],  dw[p] = dout[t] . ys[pos(p)]
//
// All three only move rows, so HBM bounds them; the work is split by token (never by bucket row), so
// that a token's own row is read or written once whatever topk is, and every bucket row once. A thread
// holds one 16-byte piece (8 elements) of the token's row and walks the token's slots: the stores (or
// loads) of all slots are in flight together. Elements are FP32 between the load and the one rounding.
#include "nvfp4_device.hpp"
#include "ops.hpp"

namespace nvfp4 {
namespace {

constexpr int ROW_THREADS = 256;
constexpr int SEG_THREADS = 256;  // most pieces of a row per block
constexpr int SLOTS = 16;  // slots of permute and unpermute whose rows are in flight at once

__device__ __forceinline__ f16x8 round8(const float (&v)[8])
{
    f16x8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = f16_of_f32(v[e]);
    return r;
}

// Index of this block along the token axis, which is split over x and z: a launch holds fewer than
// 2^32 threads along one axis.
constexpr int GRID_X = 1 << 20;
__device__ __forceinline__ int token_block() { return (int)blockIdx.z * GRID_X + (int)blockIdx.x; }

// This thread's token and piece. UNI: a block takes one token (and one of blockIdx.y segments of its row), whose
// positions and weights are then scalar loads. Else rows are shorter than a wave and a block takes
// ROW_THREADS >> lg tokens, 2^lg lanes each.
template <bool UNI>
__device__ __forceinline__ bool row_piece(int lg, int M, int pieces, int &t, int &pc)
{
    if (UNI) {
        t = token_block();
        pc = blockIdx.y * blockDim.x + threadIdx.x;
    } else {
        t = token_block() * (ROW_THREADS >> lg) + (int)(threadIdx.x >> lg);
        pc = threadIdx.x & ((1 << lg) - 1);
    }
    return t < M && pc < pieces;
}

// A bucket row's piece. NT: non-temporal, for row buffers larger than the L2s (each row is touched once).
template <bool NT>
__device__ __forceinline__ f16x8 load_row(const f16 *p)
{
    const f16x8 *q = reinterpret_cast<const f16x8 *>(p);
    return NT ? __builtin_nontemporal_load(q) : *q;
}

template <bool NT>
__device__ __forceinline__ void store_row(f16 *p, f16x8 v)
{
    f16x8 *q = reinterpret_cast<f16x8 *>(p);
    if (NT) __builtin_nontemporal_store(v, q);
    else *q = v;
}

template <bool UNI, bool NT>
__global__ __launch_bounds__(SEG_THREADS) void permute_kernel(const int32_t *__restrict__ pos_of_pair,
                                                              const f16 *__restrict__ x, const float *__restrict__ w,
                                                              int M, int topk, int pieces, int lg, f16 *__restrict__ xs)
{
    int t, pc;
    if (!row_piece<UNI>(lg, M, pieces, t, pc)) return;
    const f16x8 v = *reinterpret_cast<const f16x8 *>(x + ((size_t)t * pieces + pc) * 8);
    const int32_t *pos = pos_of_pair + (size_t)t * topk;
    for (int k0 = 0; k0 < topk; k0 += SLOTS) {
        int j[SLOTS];
        float wk[SLOTS];
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            j[i] = k0 + i < topk ? pos[k0 + i] : -1;
            wk[i] = w && k0 + i < topk ? w[(size_t)t * topk + k0 + i] : 1.0f;
        }
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            if (j[i] < 0) continue;
            f16x8 o = v;
            if (w) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = wk[i] * (float)v[e];
                o = round8(f);
            }
            store_row<NT>(xs + ((size_t)j[i] * pieces + pc) * 8, o);
        }
    }
}

template <bool UNI, bool NT>
__global__ __launch_bounds__(SEG_THREADS) void unpermute_kernel(const int32_t *__restrict__ pos_of_pair,
                                                                const f16 *__restrict__ ys, const float *__restrict__ w,
                                                                int M, int topk, int pieces, int lg,
                                                                f16 *__restrict__ out)
{
    int t, pc;
    if (!row_piece<UNI>(lg, M, pieces, t, pc)) return;
    const int32_t *pos = pos_of_pair + (size_t)t * topk;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < topk; k0 += SLOTS) {
        f16x8 v[SLOTS];
        int j[SLOTS];
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) j[i] = k0 + i < topk ? pos[k0 + i] : -1;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            if (j[i] >= 0) v[i] = load_row<NT>(ys + ((size_t)j[i] * pieces + pc) * 8);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            if (j[i] >= 0) {
                const float wk = w ? w[(size_t)t * topk + k0 + i] : 1.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = fmaf(wk, (float)v[i][e], s[e]);
            }
    }
    *reinterpret_cast<f16x8 *>(out + ((size_t)t * pieces + pc) * 8) = round8(s);
}

// Sums of SL values (a power of two, at most 16) over the wave's 64 lanes: in each of the first log2(SL) steps
// a lane hands over half of its values and keeps the sums of the other half (17 exchanges for 16 values
// instead of 96), then the remaining lanes' sums are added. Lane l ends with the sum of value l / (64 / SL).
template <int SL>
__device__ __forceinline__ float wave_sums(float (&a)[SL])
{
    const int lane = threadIdx.x & 63;
    int o = 32;
#pragma unroll
    for (int h = SL / 2; h >= 1; h >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float give = up ? a[i] : a[i + h];
            const float keep = up ? a[i + h] : a[i];
            a[i] = keep + __shfl_xor(give, o, 64);
        }
    }
    float s = a[0];
#pragma unroll
    for (int r = 32 / SL; r > 0; r >>= 1) s += __shfl_xor(s, r, 64);
    return s;
}

// One block per (token, NS of its slots); its waves share the row's pieces, hold each slot's partial dot product in a
// register and add them across the wave and, through LDS, across the waves in ascending order: an order that depends
// on K alone. NS is at most GRAD_SLOTS (16 slots at once are straight-line code of 10 KB, whose fetch took longer than
// its loads: 7.7 us for one token of 128 elements), and less where there are few tokens; a thread has about GRAD_SLOTS
// bucket-row pieces in flight.
constexpr int GRAD_SLOTS = 8;

template <int NS, bool NT>
__global__ __launch_bounds__(ROW_THREADS) void unpermute_grad_kernel(const int32_t *__restrict__ pos_of_pair,
                                                                     const f16 *__restrict__ dout,
                                                                     const f16 *__restrict__ ys,
                                                                     const float *__restrict__ w, int M, int topk,
                                                                     int pieces,
                                                                     f16 *__restrict__ dys, float *__restrict__ dw)
{
    constexpr int SL = NS <= 1 ? 1 : NS <= 2 ? 2 : NS <= 4 ? 4 : 8;  // NS as wave_sums takes it
    constexpr int PB = GRAD_SLOTS / NS;
    __shared__ float part[ROW_THREADS / 64][SL];
    const int t = token_block(), k0 = blockIdx.y * NS, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (t >= M) return;  // the whole block
    const int32_t *pos = pos_of_pair + (size_t)t * topk;
    int j[NS];
    float wk[NS], acc[SL];
#pragma unroll
    for (int i = 0; i < SL; ++i) acc[i] = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        j[i] = k0 + i < topk ? pos[k0 + i] : -1;
        wk[i] = dys && k0 + i < topk ? w[(size_t)t * topk + k0 + i] : 0.f;
    }
    for (int p0 = threadIdx.x; p0 < pieces; p0 += PB * blockDim.x) {
        f16x8 d[PB], v[PB][NS];
#pragma unroll
        for (int b = 0; b < PB; ++b) {
            const int pc = p0 + b * blockDim.x;
            if (pc >= pieces) continue;
            d[b] = *reinterpret_cast<const f16x8 *>(dout + ((size_t)t * pieces + pc) * 8);
#pragma unroll
            for (int i = 0; i < NS; ++i)  // a skipped slot reads row 0 and drops it: no branch parts the loads
                v[b][i] = load_row<NT>(ys + ((size_t)max(j[i], 0) * pieces + pc) * 8);
        }
#pragma unroll
        for (int b = 0; b < PB; ++b) {
            const int pc = p0 + b * blockDim.x;
            if (pc >= pieces) continue;
#pragma unroll
            for (int i = 0; i < NS; ++i)
                if (j[i] >= 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[i] = fmaf((float)d[b][e], (float)v[b][i][e], acc[i]);
                    if (dys) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = wk[i] * (float)d[b][e];
                        store_row<NT>(dys + ((size_t)j[i] * pieces + pc) * 8, round8(f));
                    }
                }
        }
    }
    const float sum = wave_sums<SL>(acc);
    if (lane % (64 / SL) == 0) part[wave][lane / (64 / SL)] = sum;
    __syncthreads();
    const int i = threadIdx.x;
    if (i < NS && k0 + i < topk) {
        float s = part[0][i];
        for (int v = 1; v < (int)(blockDim.x >> 6); ++v) s += part[v][i];
        dw[(size_t)t * topk + k0 + i] = s;  // a skipped pair's partial sums are all +0
    }
}

dim3 token_grid(int64_t blocks, int segments)
{
    return dim3((unsigned)(blocks < GRID_X ? blocks : GRID_X), (unsigned)segments,
                (unsigned)((blocks + GRID_X - 1) / GRID_X));
}

// How a row operator is launched. Rows of at least a wave: one block per row and segment, as many whole waves as
// the segment needs, so that a row's lines are touched together (rows of 129 pieces in 16-lane segments spread over
// blocks took three times the floor). Shorter rows: the power of two that holds them.
struct RowLaunch {
    bool uni;
    int lg;
    dim3 grid, block;
};

RowLaunch row_launch(int M, int pieces)
{
    RowLaunch r;
    r.uni = pieces >= 64;
    r.lg = 0;
    while ((1 << r.lg) < pieces && !r.uni) ++r.lg;
    if (r.uni) {
        int segments = 0, threads = 0;
        for (int n = (pieces + SEG_THREADS - 1) / SEG_THREADS, end = n + 3; n <= end; ++n) {  // fewest idle lanes
            const int waves = ((pieces + n - 1) / n + 63) / 64 * 64;
            if (segments == 0 || (int64_t)n * waves < (int64_t)segments * threads) segments = n, threads = waves;
        }
        r.block = dim3((unsigned)threads);
        r.grid = token_grid(M, segments);
    } else {
        const int rows = ROW_THREADS >> r.lg;
        r.block = dim3(ROW_THREADS);
        r.grid = token_grid(((int64_t)M + rows - 1) / rows, 1);
    }
    return r;
}

// Whether the bucket rows exceed what the L2s of the eight XCDs hold (4 MB each) and are whole 128-byte lines (lines
// shared by two rows would go to memory twice). Measured on MI355X without / with non-temporal rows (us): permute,
// unpermute and unpermute_grad of rows of 2048 elements, top-10, buffers changing from call to call: 16 MiB of bucket
// rows 5.7 / 4.6, 6.4 / 8.4, 12.6 / 11.1; 32 MiB 8.6 / 7.7, 11.1 / 10.0, 20.5 / 18.0; 64 MiB 14.6 / 14.1, 20.9 / 18.3, 34.3 / 31.2;
// 128 MiB 29.6 / 27.3, 35.1 / 31.0, 62 / 58; 320 MiB 74 / 66, 76 / 69, 152 / 137. (The same buffers again and again, which the
// 256 MB behind the L2s hold: 64 MiB 12.5 / 13.6, 15.4 / 16.0, 26.1 / 29.4; 128 MiB 23.0 / 26.6, 24.6 / 28.5, 49 / 57.) 131072 rows
// of 1032: permute 49.8 / 100.2, unpermute 56.2 / 65.0.
bool streams(int64_t P, int K) { return K % 64 == 0 && P * K * 2 > (int64_t(32) << 20); }

const f16 *half(const uint16_t *p) { return reinterpret_cast<const f16 *>(p); }
f16 *half(uint16_t *p) { return reinterpret_cast<f16 *>(p); }

}  // namespace

int run_permute(const PlanView &pv, int32_t M, int32_t topk, const uint16_t *x, const float *w, int32_t K, uint16_t *xs,
                hipStream_t s)
{
    const int pieces = K / 8;
    const RowLaunch r = row_launch(M, pieces);
    auto go = [&](auto *kernel) {
        return launch(kernel, r.grid, r.block, 0, s, pv.pos_of_pair, half(x), w, M, topk, pieces, r.lg,
                      half(xs));
    };
    if (streams((int64_t)M * topk, K)) return r.uni ? go(permute_kernel<true, true>) : go(permute_kernel<false, true>);
    return r.uni ? go(permute_kernel<true, false>) : go(permute_kernel<false, false>);
}

int run_unpermute(const PlanView &pv, int32_t M, int32_t topk, const uint16_t *ys, const float *w, int32_t K,
                  uint16_t *out, hipStream_t s)
{
    const int pieces = K / 8;
    const RowLaunch r = row_launch(M, pieces);
    auto go = [&](auto *kernel) {
        return launch(kernel, r.grid, r.block, 0, s, pv.pos_of_pair, half(ys), w, M, topk, pieces, r.lg,
                      half(out));
    };
    if (streams((int64_t)M * topk, K)) return r.uni ? go(unpermute_kernel<true, true>) : go(unpermute_kernel<false, true>);
    return r.uni ? go(unpermute_kernel<true, false>) : go(unpermute_kernel<false, false>);
}

int run_unpermute_grad(const PlanView &pv, int32_t M, int32_t topk, const uint16_t *dout, const uint16_t *ys,
                       const float *w, int32_t K, uint16_t *dys, float *dw, hipStream_t s)
{
    const int pieces = K / 8;
    const int threads = pieces >= ROW_THREADS ? ROW_THREADS : (pieces + 63) / 64 * 64;
    // Rounds of at most GRAD_SLOTS slots; more of fewer while there are under two blocks per CU.
    int rounds = (topk + GRAD_SLOTS - 1) / GRAD_SLOTS;
    while (rounds < topk && (int64_t)M * rounds < 2 * (int64_t)device_cus()) rounds = 2 * rounds < topk ? 2 * rounds : topk;
    const int ns = (topk + rounds - 1) / rounds;
    auto go = [&](auto *kernel) {
        return launch(kernel, token_grid(M, (topk + ns - 1) / ns), dim3((unsigned)threads), 0, s, pv.pos_of_pair, half(dout),
                      half(ys), w, M, topk, pieces, half(dys), dw);
    };
    if (streams((int64_t)M * topk, K)) {
        switch (ns) {
        case 1: return go(unpermute_grad_kernel<1, true>);
        case 2: return go(unpermute_grad_kernel<2, true>);
        case 3: return go(unpermute_grad_kernel<3, true>);
        case 4: return go(unpermute_grad_kernel<4, true>);
        case 5: return go(unpermute_grad_kernel<5, true>);
        case 6: return go(unpermute_grad_kernel<6, true>);
        case 7: return go(unpermute_grad_kernel<7, true>);
        default: return go(unpermute_grad_kernel<8, true>);
        }
    }
    switch (ns) {
    case 1: return go(unpermute_grad_kernel<1, false>);
    case 2: return go(unpermute_grad_kernel<2, false>);
    case 3: return go(unpermute_grad_kernel<3, false>);
    case 4: return go(unpermute_grad_kernel<4, false>);
    case 5: return go(unpermute_grad_kernel<5, false>);
    case 6: return go(unpermute_grad_kernel<6, false>);
    case 7: return go(unpermute_grad_kernel<7, false>);
    default: return go(unpermute_grad_kernel<8, false>);
    }
}

}  // namespace nvfp4
