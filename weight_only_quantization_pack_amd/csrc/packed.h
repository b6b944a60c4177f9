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

// The four exact fp16 operands (q - z) of a lane slot: operand i holds the
// lane's k = 8 i .. 8 i + 7 (of its 32).  A code goes under an exponent whose
// mantissa step puts it at its place in the word, so that a word needs one
// shift:
//   int4: nibbles at bits 0..3 and 4..7 (and 16 above) of w and of w >> 8,
//         under 2^10 (1024 + q) and 2^6 (64 + q)
//   int3: fields at bits 0, 3 and 6 of w, 0 and 3 of w >> 9, under 2^10, 2^7
//         (128 + q) and 2^4 (16 + q); the last pair's bits are gathered from the
//         three words' bits 15 and 31
// and subtracting the exponent's value plus z is exact.
template <int BITS, int WQ>
__device__ __forceinline__ void exact_operands(const TileSlot<WQ>& w, _Float16 z, half8_t* b) {
    auto pair = [](_Float16 v) { return (half2_t){v, v}; };
    const half2_t z10 = pair((_Float16)1024.0f + z);
    auto put = [&](int p, uint32_t bits, half2_t zz) {      // pair p of the slot's 16
        const half2_t v = __builtin_bit_cast(half2_t, bits) - zz;
        b[p / 4][2 * (p % 4)] = v[0];
        b[p / 4][2 * (p % 4) + 1] = v[1];
    };
    if constexpr (BITS == 4) {
        const half2_t z6 = pair((_Float16)64.0f + z);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t pr[4];
            int4_word_pairs(w.w[i], pr);
#pragma unroll
            for (int t = 0; t < 4; ++t) put(4 * i + t, pr[t], t & 1 ? z6 : z10);
        }
    } else {
        const half2_t z7 = pair((_Float16)128.0f + z), z4 = pair((_Float16)16.0f + z);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uint32_t v = w.w[i], v9 = v >> 9;
            put(5 * i, and_or(v, 0x00070007u, 0x64006400u), z10);
            put(5 * i + 1, and_or(v, 0x00380038u, 0x58005800u), z7);
            put(5 * i + 2, and_or(v, 0x01C001C0u, 0x4C004C00u), z4);
            put(5 * i + 3, and_or(v9, 0x00070007u, 0x64006400u), z10);
            put(5 * i + 4, and_or(v9, 0x00380038u, 0x58005800u), z7);
        }
        put(15, int3_pair_bits(w.w, 15), z10);
    }
}

}  // namespace awq
