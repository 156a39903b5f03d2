// linear_device.hpp -- device pieces shared by the dense projections (linear.hip) and the projections with
// low-rank adapters (lora.hip).
#pragma once

#include "nvfp4_device.hpp"

namespace nvfp4 {

constexpr int XS_PITCH = 1040;  // bytes between staged chunk rows of x in LDS (see linear.hip)

// An empty asm that the compiler must treat as changing the weight registers: placed inside the
// row-tile loop, it keeps the decode there. Hoisted out of the loop, the decoded fragments would hold
// 128 registers across it (spills) and the decode would wait for the weights before the A loads of
// the first row tile are issued. No instruction is emitted.
__device__ __forceinline__ void keep_in_loop(RawChunk &w)
{
#pragma unroll
    for (int b = 0; b < 4; ++b) asm volatile("" : "+v"(w.codes[b]));
    asm volatile("" : "+v"(w.scales[0]), "+v"(w.scales[1]));
}

// Where a kernel's A fragments come from.
enum AFrom { A_GLOBAL, A_BUFFER, A_STAGED };

// The A fragments of one 16-row tile, row m of the pass's M rows (xg: the pass's first row): from
// this wave's staged LDS rows (A_STAGED: the pass is rows 0..M-1 of x), or from x by loads that only
// valid lanes issue (A_GLOBAL) or by buffer loads that all lanes issue, at an out-of-range offset for
// the others (A_BUFFER: no branch, so no wait for the earlier loads at the merge; measured faster
// for the channel-FP8 kernel, slower for the NVFP4 one). Rows at or past M, and lane groups past the
// chunk end, are zeros.
template <AFrom AF>
__device__ __forceinline__ void load_a_tile(f16x8 (&af)[4][4], const f16 *xg, rsrc_t xr, const unsigned char *xw,
                                            int m, int M, int K, int kb, int q, bool qv)
{
    const bool v = m < M && qv;
    if constexpr (AF == A_STAGED) {
        // The compiler does not order LDS reads after the direct-to-LDS loads that fill them: wait
        // for every load of this wave (vmcnt(0); expcnt and lgkmcnt left at their maxima).
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        // an LDS-typed pointer, so that the reads are ds_read_b128 and not flat loads
        typedef const __attribute__((address_space(3))) f16x8 lds_f16x8;
        lds_f16x8 *p = (lds_f16x8 *)(xw + (v ? m : 0) * XS_PITCH + 256 * q);
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int s = 0; s < 4; ++s) af[b][s] = v ? p[4 * b + s] : zero8();
    } else if constexpr (AF == A_BUFFER) {
        const uint32_t o = v ? (uint32_t)(m * K + kb + 128 * q) * 2u : BUF_OOB;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int s = 0; s < 4; ++s) af[b][s] = __builtin_bit_cast(f16x8, bload16(xr, o + 64 * b + 16 * s, 0));
    } else {
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int s = 0; s < 4; ++s) af[b][s] = zero8();
        if (v) {
            const f16 *xp = xg + (size_t)m * K;
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int s = 0; s < 4; ++s) af[b][s] = a_frag(xp, kb, q, b, s);
        }
    }
}

}  // namespace nvfp4
