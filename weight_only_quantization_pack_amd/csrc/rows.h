// Device helpers of the row-wise operators (norms, row quantization and the
// 8-bit products): 16-bit element types, reductions over a wave and a
// workgroup, and the 8-bit code of a row element.
#pragma once

#include "awq_internal.h"

namespace awq {

typedef int int4_t __attribute__((ext_vector_type(4)));

// 16-bit element types: 8 elements travel as one 16-byte chunk
struct F16 {
    static __device__ __forceinline__ float load(uint16_t b) { return (float)bits_half(b); }
    static __device__ __forceinline__ uint16_t store(float f) { return half_bits((_Float16)f); }
};
struct BF16 {
    static __device__ __forceinline__ float load(uint16_t b) {
        return __builtin_bit_cast(float, (uint32_t)b << 16);
    }
    static __device__ __forceinline__ uint16_t store(float f) {      // round to nearest even
        return __builtin_bit_cast(uint16_t, (__bf16)f);
    }
};

template <class E>
__device__ __forceinline__ void unpack8(uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = E::load((uint16_t)(w[i] & 0xFFFFu));
        f[2 * i + 1] = E::load((uint16_t)(w[i] >> 16));
    }
}

template <class E>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return (uint32_t)E::store(lo) | (uint32_t)E::store(hi) << 16;
}

template <class E>
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack2<E>(f[0], f[1]), pack2<E>(f[2], f[3]), pack2<E>(f[4], f[5]), pack2<E>(f[6], f[7]));
}

// v combined over the 64 lanes in a fixed order, the result in every lane.
// Prefix steps inside each row of 16 lanes, then the row ends are passed on
// (DPP: no LDS round trip); lanes a step does not reach add the identity 0.
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op) {
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true));   // row_shr:1
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, true));   // row_shr:2
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, true));   // row_shr:4
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, true));   // row_shr:8
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));  // row_bcast:15
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

struct SumF32 {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }
};
struct MaxU32 {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};

// The same over the W waves of a workgroup: each wave leaves its value in
// `slots` (W words, not used by the reduction before this one), every thread
// adds them up in the same order.  One barrier.
template <int W, class Op>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, uint32_t* slots, Op op) {
    v = wave_reduce(v, op);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
        __syncthreads();
        v = slots[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v = op(v, slots[w]);
    }
    return v;
}

// |f| as bits: their order as integers is the order of the magnitudes, with
// infinity and then NaN on top, so a maximum over them carries a NaN along
__device__ __forceinline__ uint32_t abs_bits(float f) { return __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu; }

// Codes of the elements of one row, q = rint(127 v / top), top = max |v|, held
// in 8 bits (|q| <= 127).  The division runs only where it can matter: v * inv
// (inv = fp32(127 / top)) is within 127 * 2^-23 of the quotient, so a product
// further than 2^-14 from half way between two integers has its code already.
// Where it runs, fp32 gives the code of the exact quotient for 16-bit v, ties
// to even: with v = a 2^i and top = b 2^(i + d), a and b in [2^10, 2^11) and
// d >= -1, the quotient is a half-integer or misses it by at least
// 2^-(12 + max(d, 0)), and its rounding (127 v is exact) moves it by at most
// 2^-(16 + d).  127 v would overflow in rows whose top is near the largest
// fp32: from 2^120 on both are brought down by 2^64 first, exactly but for
// values below 2^-62, whose code is 0 either way.
struct RowScale {
    float top, inv;          // max |v|; 127 / top
    float down;              // what v and top are multiplied by for the division
    bool tiny;               // 127 / top would overflow: always divide
    __device__ __forceinline__ explicit RowScale(uint32_t top_bits) {
        top = __builtin_bit_cast(float, top_bits);
        inv = 127.0f / top;
        down = top >= 0x1p120f ? 0x1p-64f : 1.0f;
        tiny = top < 0x1p-100f;
    }
    __device__ __forceinline__ float scale() const { return top / 127.0f; }
};

// Adding 1.5 * 2^23 rounds t (|t| <= 127) to an integer, ties to even, and leaves
// it in the sum's low byte.
__device__ __forceinline__ uint2 pack_codes8(const float* v, const RowScale& s) {
    constexpr float kRound = 0x1.8p23f;
    uint32_t k[8];
    float far = 0.0f;                              // largest distance from an integer
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = v[i] * s.inv, r = t + kRound;
        k[i] = __builtin_bit_cast(uint32_t, r);
        far = fmaxf(far, fabsf(t - (r - kRound)));
    }
    const bool slow = far > 0.5f - 0x1p-14f || s.tiny;
    if (__builtin_amdgcn_ballot_w64(slow)) {
        if (slow) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                k[i] = s.top == 0.0f ? 0u : __builtin_bit_cast(uint32_t, v[i] * s.down * 127.0f / (s.top * s.down) + kRound);
        }
    }
    auto bytes = [](const uint32_t* q) {           // the low bytes of four words
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(q[3], q[2], 0x0C0C0400u),
                                     __builtin_amdgcn_perm(q[1], q[0], 0x0C0C0400u), 0x05040100u);
    };
    return make_uint2(bytes(k), bytes(k + 4));
}

}  // namespace awq
