// tile_gemm.hpp -- C = A B^T over two row-major operands of one type (fp16, or E4M3 bytes), both contiguous along the
// reduction axis: the tiled product behind the gradients through decoded weights (linear_grad.hip) and the
// projection of 8-bit rows (linear_rows.hip).
//
// A block of WM x WN waves owns BM x BN outputs; a wave MT x NT tiles of 16 x 16. The reduction axis is walked in
// stages of 128 bytes (64 fp16 or 128 E4M3 elements): both operands' rows come into LDS by direct-to-LDS loads,
// one 1 KB instruction for eight rows, NS - 1 stages ahead, with one block barrier per stage.
//
// LDS: a row is 128 bytes, its eight 16-byte units XOR-ed with (row / 2) % 8. A 16-byte read is conflict-free where 16
// neighbouring lanes fall on the 16 units of 256 bytes (two rows). A fragment read takes unit q or q + 4 of rows
// 0..15 in lanes 0..15 of group q: two rows of a parity and their neighbours differ in (row / 2) % 8, so the sixteen
// rows take each unit of both parities once (counted: no conflicts; XOR-ed with 2 * ((row / 4) % 4) half of
// all LDS cycles went to them). A direct-to-LDS load writes 16 bytes a lane in lane order, so the swizzle stands in
// the lane's global address instead; it stays within the row's 128 bytes.
//
// The weight rows feed MFMA's first operand and the batch's rows the second, so a lane's four results of a tile are
// four neighbouring columns of one row. Weight row 16 t + 4 q + j of a wave's tiles holds column 4 NT q + 4 t + j:
// over its NT tiles a lane then has 4 NT neighbouring columns, which it stores without a transposition.
//
// fp16: two v_mfma_f32_16x16x32_f16 per stage and tile; E4M3: one v_mfma_f32_16x16x128_f8f6f4, the form that runs at
// twice the fp16 rate. The element order inside a stage is the same in both operands, and any such order is as
// good as another.
#pragma once

#include "nvfp4_device.hpp"

namespace nvfp4 {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int STAGE_BYTES = 128;

__host__ __device__ constexpr int unit_swizzle(int row) { return (row >> 1) & 7; }

// One 16 x 16 x 128 product of E4M3 operands. Zeros for both operands' scales, as constants, select the instruction without
// scales (as E8M0 bytes they would be 2^-127).
__device__ __forceinline__ f32x4 mfma_e4m3(i32x8 a, i32x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Waits until at most N of this wave's vector memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    static_assert(N < 64, "vmcnt has six bits");
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Block barrier between stages: this wave's LDS reads are done, its loads into LDS stay in flight (a release fence would
// wait for them all, which made every ring one stage deep); wait_loads() in front says which of them have to be there.
__device__ __forceinline__ void stage_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16 bytes a lane from a buffer to LDS: lane i's bytes land at `to` + 16 i. Offsets past the buffer give zeros.
__device__ __forceinline__ void load_to_lds(rsrc_t from, unsigned char *to, uint32_t voff, uint32_t soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 16, voff, soff, 0, 0);
}

template <bool FP8_, int MT_, int NT_, int WM_, int WN_, int NS_>
struct Tile {
    static constexpr bool FP8 = FP8_;
    static constexpr int MT = MT_, NT = NT_, WM = WM_, WN = WN_, NS = NS_;
    // products of one fragment of A with NT of B in a stage, and how many of these a fragment is read ahead (four are 3%
    // faster than two with 256 x 256)
    static constexpr int STEPS = FP8 ? MT : 2 * MT, AHEAD = STEPS < 4 ? STEPS : 4;
    static constexpr int WAVES = WM * WN, BM = WM * MT * 16, BN = WN * NT * 16;
    static constexpr int LA = BM / 8 / WAVES, LB = BN / 8 / WAVES;  // loads per wave and stage
    static constexpr int BYTES = (BM + BN) * STAGE_BYTES;           // one stage
    static_assert(LA * 8 * WAVES == BM && LB * 8 * WAVES == BN, "whole loads per wave");
    static_assert(NS * BYTES <= 160 * 1024, "LDS of a CU");
};

// This wave's and lane's place in a block.
struct Place {
    int wave, lane, wm, wn, r, q;
};
template <class T>
__device__ __forceinline__ Place place_of()
{
    Place p;
    p.lane = threadIdx.x & 63;
    p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    p.wm = p.wave / T::WN, p.wn = p.wave % T::WN;
    p.r = p.lane & 15, p.q = p.lane >> 4;
    return p;
}

// The row of a tile that load i of this wave brings for this lane, and the lane's byte within the row.
template <class T>
__device__ __forceinline__ int load_row(const Place &p, int i)
{
    return (p.wave + T::WAVES * i) * 8 + (p.lane >> 3);
}
__device__ __forceinline__ uint32_t load_byte(int row, int lane) { return 16u * ((lane & 7) ^ unit_swizzle(row)); }

// The column (of the block's BN) that row `row` of the staged weight tile holds.
template <class T>
__device__ __forceinline__ int column_of_row(int row)
{
    const int w = row / (16 * T::NT), t = (row / 16) % T::NT, q = (row / 4) & 3, j = row & 3;
    return w * 16 * T::NT + 4 * T::NT * q + 4 * t + j;
}

// What one stage adds to a wave's tiles: acc += A B^T over the 128 bytes of the rows staged at `ar` (the block's rows of
// A) and `br` (of B). A step is the products of one fragment of A with NT of B; fragments are read ahead of their
// products: A's AHEAD steps, B's second half during the first.
template <class T>
__device__ __forceinline__ void stage_products(const unsigned char *ar, const unsigned char *br, const Place &p,
                                               f32x4 (&acc)[T::MT][T::NT])
{
    constexpr int MT = T::MT, NT = T::NT, D = T::AHEAD;
    // This lane's rows, and its two units of a row: q and q + 4, swizzled (a tile's rows start at multiples of 16).
    const int sw = unit_swizzle(p.r);
    const int u0 = 16 * (p.q ^ sw), u1 = 16 * ((p.q + 4) ^ sw);
    ar += (p.wm * MT * 16 + p.r) * STAGE_BYTES;
    br += (p.wn * NT * 16 + p.r) * STAGE_BYTES;
    auto unit = [](const unsigned char *rows, int tile, int u) {
        return *reinterpret_cast<const f16x8 *>(rows + tile * 16 * STAGE_BYTES + u);
    };
    if constexpr (T::FP8) {
        auto frag = [&](const unsigned char *rows, int tile) {
            return __builtin_shufflevector(__builtin_bit_cast(i32x4, unit(rows, tile, u0)),
                                           __builtin_bit_cast(i32x4, unit(rows, tile, u1)), 0, 1, 2, 3, 4, 5, 6, 7);
        };
        i32x8 bf[NT], af[MT];
#pragma unroll
        for (int t = 0; t < NT; ++t) bf[t] = frag(br, t);
#pragma unroll
        for (int m = 0; m < D; ++m) af[m] = frag(ar, m);
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * (NT + D), 0);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (m + D < MT) {
                af[m + D] = frag(ar, m + D);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[m][t] = mfma_e4m3(bf[t], af[m], acc[m][t]);
            __builtin_amdgcn_sched_group_barrier(0x008, NT, 0);
        }
    } else {
        f16x8 bf[2][NT], af[2 * MT];
#pragma unroll
        for (int t = 0; t < NT; ++t) bf[0][t] = unit(br, t, u0);
#pragma unroll
        for (int s = 0; s < D; ++s) af[s] = unit(ar, s % MT, s < MT ? u0 : u1);
        __builtin_amdgcn_sched_group_barrier(0x100, NT + D, 0);
#pragma unroll
        for (int s = 0; s < 2 * MT; ++s) {
            if (s + D < 2 * MT) {
                af[s + D] = unit(ar, (s + D) % MT, s + D < MT ? u0 : u1);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            if (s < MT) {  // B's second half, spread over the first half's steps
#pragma unroll
                for (int t = s * NT / MT; t < (s + 1) * NT / MT; ++t) {
                    bf[1][t] = unit(br, t, u1);
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[s % MT][t] = mfma_step(bf[s / MT][t], af[s], acc[s % MT][t]);
            __builtin_amdgcn_sched_group_barrier(0x008, NT, 0);
        }
    }
}

// Rows of one operand: a buffer from the block's first row on, and each load's byte offset at stage 0 (BUF_OOB: zeros).
template <int L>
struct Rows {
    rsrc_t buf;
    uint32_t off[L];
};

// acc = A B^T over stages [first, last): one chain of products for each output, in the order of the stages. tail: bytes of
// the last stage of A's rows that exist (128: all); later units are fed as zeros (B's must exist and be finite).
template <class T>
__device__ __forceinline__ void tile_product(unsigned char *smem, const Place &p, const Rows<T::LA> &a, const Rows<T::LB> &b,
                                             int first, int last, int tail, f32x4 (&acc)[T::MT][T::NT])
{
    constexpr int NS = T::NS;
    auto load = [&](int k, int buf) {
        unsigned char *to = smem + buf * T::BYTES + p.wave * 1024;
        const uint32_t so = (uint32_t)k * STAGE_BYTES;
        const bool cut = tail < STAGE_BYTES && k == last - 1;  // uniform
#pragma unroll
        for (int i = 0; i < T::LA; ++i) {
            uint32_t v = a.off[i];
            if (cut) v = (int)load_byte(load_row<T>(p, i), p.lane) < tail ? v : BUF_OOB;
            load_to_lds(a.buf, to + T::WAVES * i * 1024, v, so);
        }
        to += T::BM * STAGE_BYTES;
#pragma unroll
        for (int i = 0; i < T::LB; ++i) load_to_lds(b.buf, to + T::WAVES * i * 1024, b.off[i], so);
    };
#pragma unroll
    for (int m = 0; m < T::MT; ++m)
#pragma unroll
        for (int t = 0; t < T::NT; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
        if (first + s < last) load(first + s, s);
    int buf = 0;
    for (int k = first; k < last; ++k) {
        // stage k has landed: at most the NS - 2 stages behind it are still in flight (with two stages none)
        if (NS > 2 && k + NS - 2 < last) wait_loads<(NS - 2) * (T::LA + T::LB)>();
        else wait_loads<0>();
        stage_barrier();  // every wave's part of it, and every wave is done with the buffer that is filled next
        if (k + NS - 1 < last) load(k + NS - 1, buf == 0 ? NS - 1 : buf - 1);
        const unsigned char *at = smem + buf * T::BYTES;
        stage_products<T>(at, at + T::BM * STAGE_BYTES, p, acc);
        buf = buf == NS - 1 ? 0 : buf + 1;
    }
}

// Tile (m, n) of block `b` of `mt` x `nt` tiles. The hardware deals block ids to the 8 XCDs in turn: consecutive tiles
// are given to one XCD, in groups of four tile rows, so that the blocks that run at once on an XCD share their operands'
// rows in its L2. False for the padding ids of the last XCD.
__device__ __forceinline__ bool tile_of_block(int b, int mt, int nt, int &m, int &n)
{
    const int tiles = mt * nt, per = (tiles + 7) >> 3;
    const int i = (b & 7) * per + (b >> 3);
    if (i >= tiles) return false;
    constexpr int GROUP = 4;
    const int g = i / (GROUP * nt), in = i - g * GROUP * nt;
    const int rows = min(GROUP, mt - g * GROUP);
    m = g * GROUP + in % rows;
    n = in / rows;
    return true;
}
inline unsigned tile_grid(int64_t tiles) { return (unsigned)(8 * ((tiles + 7) / 8)); }

// A tile shape as the host weighs it: its sizes, the blocks that a CU holds at once, and what a stage takes, in ns: of a
// block alone on its CU (bound by the way of its own loads), and per block where a CU holds several (bound by what
// the CU loads or multiplies). The CUs are counted as an MI355X has them, without asking the device: sizes alone decide
// which kernel runs.
constexpr int TILE_CUS = 256;
struct Shape {
    int bm, bn, per_cu, alone, each;
    int64_t tiles(int64_t rows, int64_t cols) const { return ((rows + bm - 1) / bm) * ((cols + bn - 1) / bn); }
    int64_t ns(int64_t blocks, int64_t stages) const
    {
        const int64_t full = blocks / (TILE_CUS * per_cu), rest = blocks % (TILE_CUS * per_cu);
        const int64_t last = (rest + TILE_CUS - 1) / TILE_CUS * each;
        return stages * (full * per_cu * each + (rest == 0 ? 0 : last > alone ? last : alone));
    }
};

}  // namespace nvfp4
