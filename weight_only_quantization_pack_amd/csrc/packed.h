// Device helpers shared by the kernels that read packed tiles straight into
// registers: one lane slot of a tile, its group parameters, and the exact fp16
// operands (q - z) of v_mfma_f32_16x16x32_f16.
#pragma once

#include "awq_internal.h"

namespace awq {

template <int WQ>
struct TileSlot { uint32_t w[WQ]; };

template <int WQ, int POLICY>
__device__ __forceinline__ TileSlot<WQ> load_tile_slot(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    TileSlot<WQ> s;
    if constexpr (WQ == 4) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, POLICY);
        s.w[0] = v[0]; s.w[1] = v[1]; s.w[2] = v[2]; s.w[3] = v[3];
    } else {
        const auto v = __builtin_amdgcn_raw_buffer_load_b96(r, off, 0, POLICY);
        s.w[0] = v[0]; s.w[1] = v[1]; s.w[2] = v[2];
    }
    return s;
}

// the four exact fp16 operands (q - z) of a lane slot: operand i holds the
// lane's k = 8 i .. 8 i + 7 (of its 32)
template <int BITS, int WQ>
__device__ __forceinline__ void exact_operands(const TileSlot<WQ>& w, _Float16 z, half8_t* b) {
    const _Float16 zb = (_Float16)1024.0f + z, zb16 = (_Float16)64.0f + z;
    const half2_t zz = {zb, zb}, zz16 = {zb16, zb16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t pr[4];
        if constexpr (BITS == 4) {
            int4_word_pairs(w.w[i], pr);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) pr[t] = int3_pair_bits(w.w, 4 * i + t);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const half2_t p = __builtin_bit_cast(half2_t, pr[t]) - (BITS == 4 && (t & 1) ? zz16 : zz);
            b[i][2 * t] = p[0];
            b[i][2 * t + 1] = p[1];
        }
    }
}

}  // namespace awq
