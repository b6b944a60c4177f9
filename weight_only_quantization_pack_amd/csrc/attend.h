// What the two attention kernels (attend.hip, attend_tile.hip) share: the
// arguments and the line of work that a call's sequences make up.
#pragma once

#include "cache.h"

namespace awq {

constexpr int kStep = 32;                // keys of a step
// Steps that a tile's start and end take as long as.  64 ragged sequences of 200 to 8000
// tokens, 8 kv heads: 90 us of a workgroup's longest stretch without, 76 with 8, 71 with 16.
constexpr int kFixed = 16;
constexpr float kLow = -3e38f;           // below every finite score: the maximum before the first key
// A weight is exp2(t - M).  M is set 2^7 below the largest score met and may lag by 2^8 more, so the row's largest
// weight is 2^7 .. 2^15: below fp16's maximum, and with all the room below that fp16 has.  Weights keep their 11
// bits down to 2^-21 of the largest and are lost from 2^-32 on (with M at the maximum itself 2^-14 and 2^-25, which the tail of
// a softmax passes where one key, or one page's values, are far above the others).
constexpr float kRoom = 7.0f, kSlack = 8.0f;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct AttendArgs {
    const uint16_t* q;
    long long q_stride;
    uint16_t* out;
    float* lse;
    Cache cache;
    Sequences seqs;
    int piece;                           // of tiles of many rows: tiles of keys that a part takes (more where keys are)
    float scale, softcap;                // |scale| 2^24, for the operands' unit; its sign goes into q
    float sign;
    int heads, group, window, bf16;
    int split;                           // stretches may end inside a tile
    int groups;                          // workgroups of the first launch
    float* parts;                        // [groups][2][rows * (dim + 2)]
    long long* line;                     // [B + 1]: units before each sequence; units of a stretch (split, attend.hip)
};

// the steps of a sequence: the same for all its tiles of rows (their own first and
// last keys lie inside)
struct Line {
    int rows, tiles, step0, steps;
    int start, n, len;                   // first row, rows, tokens
    __device__ __forceinline__ Line(const AttendArgs& a, int b, int tile_rows)
        : Line(a, a.seqs.start(b), a.seqs.rows(b), a.seqs.len(b), tile_rows) {}
    __device__ __forceinline__ Line(const AttendArgs& a, int start_, int n_, int len_, int tile_rows)
        : start(start_), n(n_), len(len_) {
        rows = n * a.group;
        tiles = (rows + tile_rows - 1) / tile_rows;
        const int span = a.seqs.span(len, a.cache.page_log2);
        int first = 0;
        if (a.window > 0) first = max((int)max((long long)len - n + 1 - a.window, 0LL), 0);
        step0 = first / kStep;
        steps = max((int)(((uint32_t)span + (kStep - 1)) / kStep) - step0, 1);       // a span may end at 2^31 - 1
    }
    // a tile's units: its steps behind a few that stand for its start and end
    __device__ __forceinline__ int tile_units() const { return kFixed + steps; }
    __device__ __forceinline__ long long units(int kv) const { return (long long)tiles * kv * tile_units(); }
};

// Inclusive prefix of v >= 0 over the lanes, in two parts of 26 and 32 bits: 32-bit adds
// between lanes instead of 64-bit ones through LDS.
__device__ __forceinline__ long long lane_prefix(long long v) {
    constexpr int kBits = 26;            // 64 values of 26 bits stay in 32
    const uint32_t lo = lane_prefix((uint32_t)v & ((1u << kBits) - 1)), hi = lane_prefix((uint32_t)(v >> kBits));
    return ((long long)hi << kBits) + lo;
}
__device__ __forceinline__ long long lane_value(long long v, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return (long long)((uint64_t)hi << 32 | lo);
}

// a / b for a >= 0, b > 0: mostly in 32 bits
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((uint64_t)a | (uint64_t)b) >> 32) return a / b;
    return (uint32_t)a / (uint32_t)b;
}

// The line of steps, read by every wave for itself: sequence b in lane b % 64, the first
// 64 kept in registers.
class LineWalk {
    struct Block {
        int start, n, len;
        long long u;
    };
    const AttendArgs& a;
    const int tile_rows;
    Block first;
    __device__ __forceinline__ Block block(int b) const {
        Block k{0, 0, 0, 0};
        if (b < a.seqs.B) {
            const Line l(a, b, tile_rows);
            k = {l.start, l.n, l.len, l.units(a.cache.kv)};
        }
        return k;
    }

public:
    struct Place {
        int b;                           // or -1
        long long before;                // units before the sequence, or all
        Line line;
    };
    __device__ __forceinline__ LineWalk(const AttendArgs& a_, int tile_rows_)
        : a(a_), tile_rows(tile_rows_), first(block(threadIdx.x & 63)) {}
    // Calls f(b, units, before) for the sequences, 64 at a time, until it is true for
    // one, and gives the first such.
    template <class F>
    __device__ __forceinline__ Place operator()(F f) const {
        const int lane = threadIdx.x & 63;
        long long before = 0;
        for (int b0 = 0; b0 < a.seqs.B; b0 += 64) {
            const Block k = b0 == 0 ? first : block(b0 + lane);
            const long long sum = before + lane_prefix(k.u);
            const uint64_t hit = __builtin_amdgcn_ballot_w64(f(b0 + lane, k.u, sum - k.u));
            if (hit) {
                const int i = __builtin_ctzll(hit);
                return {b0 + i, lane_value(sum - k.u, i), line(k, i)};
            }
            before = lane_value(sum, 63);
        }
        return {-1, before, Line(a, 0, 0, 0, tile_rows)};
    }
    __device__ __forceinline__ Line line(int b) const { return b < 64 ? line(first, b) : Line(a, b, tile_rows); }

private:
    __device__ __forceinline__ Line line(const Block& k, int i) const {
        return Line(a, __builtin_amdgcn_readlane(k.start, i), __builtin_amdgcn_readlane(k.n, i),
                    __builtin_amdgcn_readlane(k.len, i), tile_rows);
    }
};

// Tiles without a line: sequence b has the places from start(b) * group / tile_rows + b on,
// enough for its tiles, and finding it takes the starts alone.  The sequence and the
// tile (counted from the place) of `place`; b = -1 where there is none.  By a wave.
__device__ __forceinline__ long long first_place(const AttendArgs& a, int tile_rows, int b, int start) {
    return (uint32_t)(start * a.group) / (uint32_t)tile_rows + b;
}
// The tiles of keys [t0, t1) that some of a tile's rows see, and into how many parts they go.
constexpr int kTileKeys = 64;
struct TileSpan {
    int pos_lo, pos_hi, t0, t1, parts;             // positions of the first and last row
    __device__ __forceinline__ TileSpan(const AttendArgs& a, const Line& l, int tile_rows, int tile, int most) {
        const int pos0 = l.len - l.n;
        pos_lo = pos0 + tile * tile_rows / a.group;
        pos_hi = pos0 + min(tile * tile_rows + tile_rows - 1, l.rows - 1) / a.group;
        const int span = a.seqs.span(l.len, a.cache.page_log2);
        const int first = a.window > 0 ? max((int)max((long long)pos_lo + 1 - a.window, 0LL), 0) : 0;
        const int last = min(pos_hi, span - 1);                      // -1: nothing
        t0 = first / kTileKeys;
        t1 = last >= first ? last / kTileKeys + 1 : t0;
        parts = min(max((t1 - t0 + a.piece - 1) / a.piece, 1), most);
    }
};

struct TilePlace {
    int b, tile;
    Line line;
};
__device__ __forceinline__ TilePlace find_tile(const AttendArgs& a, int tile_rows, long long place) {
    const Sequences& s = a.seqs;
    const int b = first_by_wave(s.B, [&](int k) { return first_place(a, tile_rows, k + 1, s.start(k + 1)) > place; });
    if (b < 0) return {-1, 0, Line(a, 0, 0, 0, tile_rows)};
    const Line l(a, b, tile_rows);
    const long long tile = place - first_place(a, tile_rows, b, l.start);
    return {tile >= 0 && tile < l.tiles ? b : -1, (int)tile, l};
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
// What a block's scales make of a score's product (>= 0), and of its values.  A block whose
// scale is not finite (a key or value was not) has a factor of NaN, which stands for it:
// the value's scale is kept within what logarithm and reciprocal have: from 2^-80, so that the sum of 2^31 weights of
// up to 2^15 over it is below 2^127.
__device__ __forceinline__ float key_factor(float ks, float vs, float scale) {
    return __builtin_fmaf(0.0f, ks + vs, ks * scale);
}
__device__ __forceinline__ float value_scale(float vs) { return fminf(fmaxf(vs, 0x1p-80f), 0x1p126f); }

__device__ __forceinline__ float power_of_two(int e) { return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23); }

// rows of a tile, into how many parts at most its keys are split
struct TilePlan {
    int rows, parts;
};
// the kernel for tiles of many rows; a.groups = its workgroups, a.split = parts > 1
TilePlan tile_plan(int T, int B, int group, int kv, int dim, int max_new, int max_len, int cus);
int launch_attend_tile(const AttendArgs& a, const TilePlan& p, hipStream_t st);

}  // namespace awq
