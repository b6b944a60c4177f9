// What the two attention kernels (attend.hip, attend_tile.hip) share: the
// arguments and the line of work that a call's sequences make up.
#pragma once

#include "cache.h"

namespace awq {

constexpr int kStep = 32;                // keys of a step
constexpr float kLow = -1e30f;           // below every score: the maximum before the first key
constexpr float kSlack = 8.0f;           // the maximum may lag by 2^8: weights stay far below fp16's maximum
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct AttendArgs {
    const uint16_t* q;
    long long q_stride;
    uint16_t* out;
    float* lse;
    Cache cache;
    Sequences seqs;
    float scale, softcap;                // |scale| 2^24, for the operands' unit; its sign goes into q
    float sign;
    int heads, group, window, bf16;
    int split;                           // stretches may end inside a tile
    int groups;                          // workgroups of the first launch
    float* parts;                        // [groups][2][rows * (dim + 2)]
};

// the steps of a sequence: the same for all its tiles of rows (their own first and
// last keys lie inside)
struct Line {
    int rows, tiles, step0, steps;
    int len, n;
    __device__ __forceinline__ Line(const AttendArgs& a, int b, int tile_rows) {
        const Sequences& s = a.seqs;
        n = s.rows(b);
        len = s.len(b);
        rows = n * a.group;
        tiles = (rows + tile_rows - 1) / tile_rows;
        const int span = s.span(b, a.cache.page_log2);
        int first = 0;
        if (a.window > 0) first = max((int)max((long long)len - n + 1 - a.window, 0LL), 0);
        step0 = first / kStep;
        steps = max((span + kStep - 1) / kStep - step0, 1);
    }
    __device__ __forceinline__ long long units(int kv) const { return (long long)tiles * kv * steps; }
};

// all units (or tiles), and those before sequence b_stop; by one wave
__device__ __forceinline__ void count_units(const AttendArgs& a, int tile_rows, bool tiles, int b_stop, long long& total,
                                            long long& before) {
    const int lane = threadIdx.x & 63;
    total = before = 0;
    for (int b0 = 0; b0 < a.seqs.B; b0 += 64) {
        const int b = b0 + lane;
        long long u = 0;
        if (b < a.seqs.B) {
            const Line l(a, b, tile_rows);
            u = tiles ? (long long)l.tiles * a.cache.kv : l.units(a.cache.kv);
        }
        long long v = b < b_stop ? u : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            u += __shfl_xor(u, d);
            v += __shfl_xor(v, d);
        }
        total += u;
        before += v;
    }
}

// the sequence that holds the unit at `at` (or, unsplit, the tile at `at`) and the
// units (tiles) before it; -1 past the last.  By one wave.
__device__ __forceinline__ int find_line(const AttendArgs& a, int tile_rows, bool tiles, long long at, long long& before) {
    const int lane = threadIdx.x & 63;
    before = 0;
    for (int b0 = 0; b0 < a.seqs.B; b0 += 64) {
        const int b = b0 + lane;
        long long u = 0;
        if (b < a.seqs.B) {
            const Line l(a, b, tile_rows);
            u = tiles ? (long long)l.tiles * a.cache.kv : l.units(a.cache.kv);
        }
        long long sum = u;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const long long o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        const long long all = __shfl(sum, 63);
        if (at < before + all) {
            const uint64_t hit = __builtin_amdgcn_ballot_w64(at < before + sum);
            const int f = __builtin_ctzll(hit);
            before += __shfl(sum - u, f);
            return b0 + f;
        }
        before += all;
    }
    return -1;
}

__device__ __forceinline__ float lane_value(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

union Half8 {
    uint32_t w[4];
    half8_t h;
};

// bytes i, i + 1 of w (biased codes) as two fp16 numbers of 2^-24 steps
__device__ __forceinline__ uint32_t key_pair(uint32_t w, int i) {
    return __builtin_amdgcn_perm(0u, w, i ? 0x0C030C02u : 0x0C010C00u);
}

// The power of two that brings a row's largest channel, `top`, to 2^13: fp16 then holds
// all of its channels' bits (bf16 has 8) down to 2^-27 of the largest.
__device__ __forceinline__ int query_exponent(float top) {
    const int e = top > 0.0f ? 13 - ((int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127) : 0;
    return min(max(e, -120), 120);
}
__device__ __forceinline__ float power_of_two(int e) { return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23); }

// rows of a tile, and into how many parts its keys are split
struct TilePlan {
    int rows, parts;
};
// the kernel for tiles of many rows; a.groups = its workgroups, a.split = parts > 1
TilePlan tile_plan(int T, int B, int group, int kv, int dim, int max_new, int max_len, int cus);
int launch_attend_tile(const AttendArgs& a, const TilePlan& p, hipStream_t st);

}  // namespace awq
