// packed_gemm.hpp -- C = A B^T with A fp16 [M][K] and B NVFP4 rows, decoded in registers: the tiled product of the gated
// projection's gradient at a few hundred rows (linear_grad.hip), where the product over decoded weights (tile_gemm.hpp)
// would spend as long on writing and reading them: they take 3.6 times the packed bytes.
//
// A block owns BM x BN outputs; its waves stand side by side along B, a wave has MT x NT tiles of 16 x 16. The
// reduction axis is walked in stages of 128 elements:
//   * A's rows, 256 bytes each, come into LDS by direct-to-LDS loads a stage ahead, one block barrier a stage. A
//     row's sixteen 16-byte units are XOR-ed with row_key(row), in the lane's global address. A 16-byte read serves 16 lanes
//     at a time, rows 0..3 and 12..15 of one lane group with rows 4..11 of the next and so on: the key's upper bits
//     make those fall on the 16 units of 256 bytes too (the row's number itself gave conflicts in half of the cycles);
//   * each wave loads its own codes two stages ahead, 16 bytes a lane and tile: lane group q owns elements 32 q .. + 31 of
//     the stage, MFMA step d takes elements 32 q + 8 d .. + 7 of them, and A's fragment of that step is unit 4 q + d of
//     the row. A step's weights are decoded while the products of the step before run.
// KS wave groups of a block share the reduction axis in runs of stages, and the first group adds the others' sums in
// order: a stage is mostly waiting, 0.8 us of it, and few blocks are bound by the number of stages.
//
// The weight rows feed MFMA's first operand, the batch's rows the second: a lane's four results of a tile belong to one
// row of A, and the kernel chooses which weight rows they are.
#pragma once

#include "tile_gemm.hpp"

namespace nvfp4 {

constexpr int PACKED_STAGE = 128;  // elements

// Rows 4 b .. + 3 of sixteen take 4 (0, 2, 3, 1)[b] + 0..3.
__device__ __forceinline__ int row_key(int row)
{
    const int b = (row >> 2) & 3;
    return ((b ^ b >> 1) & 1) << 3 | (b >> 1) << 2 | (row & 3);
}

template <int MT_, int NT_, int WN_, int KS_, int OCC_>
struct PackedTile {
    static constexpr int MT = MT_, NT = NT_, WN = WN_, KS = KS_, OCC = OCC_;  // OCC: waves of a SIMD that have registers
    static constexpr int BM = MT * 16, BN = WN * NT * 16, THREADS = 64 * WN * KS;
    static constexpr int LA = BM / 4 / WN;                // A's loads per wave and stage
    static constexpr int BYTES = BM * PACKED_STAGE * 2;   // one stage of A
    static constexpr int LDS = KS * 2 * BYTES;
    static_assert(LA * 4 * WN == BM && WN % 4 == 0, "whole loads per wave, all of one unit per lane");
    static_assert(KS == 1 || MT * NT * WN * 1024 <= 2 * BYTES, "a group's sums fit its stages");
};

// This wave's and lane's place: lane 16 q + r of wave `wave` of group `group`.
struct PackedPlace {
    int group, wave, lane, r, q;
};
template <class T>
__device__ __forceinline__ PackedPlace packed_place()
{
    PackedPlace p;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    p.group = w / T::WN, p.wave = w % T::WN;
    p.lane = threadIdx.x & 63, p.r = p.lane & 15, p.q = p.lane >> 4;
    return p;
}

// The lane's codes and block scales of its weight row in each of its tiles, at its first element of the row. The kernel must
// not declare them __restrict__: loads from memory that nothing may write could pass loads_apart().
template <class T>
struct PackedRows {
    const uint8_t *codes[T::NT], *scales[T::NT];
};

// Plain loads behind this stay behind the loads into LDS in front of it, which a count of loads in flight relies on: the
// compiler has to take it for a write to all memory.
__device__ __forceinline__ void loads_apart() { asm volatile("" ::: "memory"); }

// acc = A B^T, A's rows from `a` on (`rows` of them, at most BM; the others count as zeros), K % 128 == 0. The result is in
// the first group's waves; the others return false.
template <class T>
__device__ __forceinline__ bool packed_product(unsigned char *smem_all, const PackedPlace &p, const f16 *a, int rows, int K,
                                               const PackedRows<T> &b, f32x4 (&acc)[T::MT][T::NT])
{
    constexpr int MT = T::MT, NT = T::NT, ROW = PACKED_STAGE * 2;
    const int stages = K / PACKED_STAGE, per = (stages + T::KS - 1) / T::KS;
    const int first = min(stages, p.group * per), last = min(stages, first + per);
    unsigned char *const smem = smem_all + p.group * 2 * T::BYTES;
    const rsrc_t from = make_rsrc(a, (uint32_t)rows * K * 2u);
    const int row0 = 4 * p.wave + (p.lane >> 4);  // load i of a wave: rows 4 (wave + WN i) .. + 3, whole sixteens apart
    uint32_t off[T::LA];
#pragma unroll
    for (int i = 0; i < T::LA; ++i) {
        const int row = row0 + 4 * T::WN * i;
        off[i] = row < rows ? (uint32_t)row * K * 2u + 16u * ((p.lane & 15) ^ row_key(row0)) : BUF_OOB;
    }
    auto load_a = [&](int k, int buf) {
        unsigned char *to = smem + buf * T::BYTES + p.wave * 1024;
#pragma unroll
        for (int i = 0; i < T::LA; ++i) load_to_lds(from, to + T::WN * i * 1024, off[i], (uint32_t)k * ROW);
    };
    u32x4 codes[2][NT];
    uint16_t scales[2][NT];
    auto load_b = [&](int k, int set) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            codes[set][t] = *reinterpret_cast<const u32x4 *>(b.codes[t] + (size_t)k * (PACKED_STAGE / 2));
            scales[set][t] = *reinterpret_cast<const uint16_t *>(b.scales[t] + (size_t)k * (PACKED_STAGE / 16));
        }
    };
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // In the steady state a stage asks for A of the next and, behind loads_apart(), for the weights of the one after, 2 NT
    // loads, which the next stage's start leaves in flight. The first stage and the last wait for all. As compiled, A is
    // waited for behind its loads all the same: over the paths through these conditions the compiler cannot tell which
    // loads of the codes are still out, and waits for all before the first decode.
    if (first < last) load_b(first, 0), load_a(first, 0), load_b(min(first + 1, last - 1), 1);
    int buf = 0;
    const int a0 = p.r * ROW;
    int unit[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) unit[d] = a0 + 16 * ((4 * p.q + d) ^ row_key(p.r));
    for (int k0 = first; k0 < first + per; k0 += 2) {  // every group passes every barrier
#pragma unroll
        for (int set = 0; set < 2; ++set) {
            const int k = k0 + set;
            if (k >= first + per) break;
            // this wave's part of stage k, and its weights
            if (k > first && k + 1 < last) wait_loads<2 * NT>();
            else wait_loads<0>();
            stage_barrier();  // everyone's part, and everyone is done with the buffer that is filled next
            if (k >= last) continue;
            const unsigned char *const at = smem + buf * T::BYTES;
            f16x8 af[4][MT], bf[2][NT];
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int m = 0; m < MT; ++m) af[d][m] = *reinterpret_cast<const f16x8 *>(at + unit[d] + m * 16 * ROW);
            if (k + 1 < last) load_a(k + 1, buf ^ 1);
            buf ^= 1;
            auto decode = [&](int d) {
#pragma unroll
                for (int t = 0; t < NT; ++t) bf[d & 1][t] = decode8(codes[set][t][d], e4m3_pair<false>(scales[set][t])[d >> 1]);
            };
            decode(0);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if (d < 3) {
                    decode(d + 1);
                } else {
                    loads_apart();
                    load_b(min(k + 2, last - 1), set);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[m][t] = mfma_step(bf[d & 1][t], af[d][m], acc[m][t]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    if constexpr (T::KS > 1) {
        lds_barrier();  // the last stages have been read
        f32x4 *sums = reinterpret_cast<f32x4 *>(smem) + p.wave * MT * NT * 64 + p.lane;
        if (p.group > 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) sums[(m * NT + t) * 64] = acc[m][t];
        }
        lds_barrier();
        if (p.group > 0) return false;
#pragma unroll
        for (int g = 1; g < T::KS; ++g)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[m][t] += sums[g * 2 * (T::BYTES / 16) + (m * NT + t) * 64];
    }
    return true;
}

}  // namespace nvfp4
