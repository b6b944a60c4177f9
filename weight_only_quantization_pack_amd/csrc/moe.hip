// A mixture-of-experts layer for a few tokens over packed experts:
//   l = x Wr^T;  the top_k largest l of each token (ties to the lowest index)
//   p = softmax(l) over the chosen ones, or over all experts
//   y = sum_j p_j down_j(SiLU(gate_j x') * up_j x'),  x' = x * inv_s or x
//
// HBM-bound: the packed bytes of an expert are read once for up to 16, 32 or 64
// rows of its tokens' operands (launch_experts; 64-wide groups and an operand in
// two planes take 2 rows a token each, so 64 rows are 16 to 64 tokens), and once
// more for every further pass; an expert that no token takes is not read.  The
// launches:
//   k_moe_route   one workgroup per token: its logits, choices and weights
//   gate and up   h = SiLU(g) * u of every (token, choice)
//   down          the projections of h
//   k_moe_join    y = the weighted sum of a token's choices; with one token the
//                 down product's workgroup that ends last on a block of columns
//                 does it there, and this launch is saved
// Both expert products run as k_moe_token (one token) or k_moe_tile (more).
//
// The weights are the B operand of v_mfma_f32_16x16x32_f16 (lane slot =
// operand, as packed), always the exact (q - z), and the group scale
// multiplies the fp32 group sums, so the only roundings on the way are those
// of fp32 sums.  The 16 rows of the A operand hold more than one row per token
// where that keeps the products exact:
//   - an operand that is not an fp16 number (h, and x' = x * inv_s) is split
//     into hi = fp16(v) and lo = fp16((v - hi) * 2^11), two rows whose sums
//     are added as hi + lo / 2^11: 22 bits of v (from 2^-14 up; steps of 2^-35
//     below; past 65504 hi is infinite and the sums NaN), for matrix time that
//     is free while the weights are what is waited for;
//   - with 64-wide groups a k32 product mixes both groups of a tile (lane
//     quarters 0, 1 and 2, 3), so rows 0..7 hold the tokens with quarters 2, 3
//     zeroed and rows 8..15 the same tokens with quarters 0, 1 zeroed: the
//     group sums come out in different rows.
#include <climits>
#include <type_traits>

#include "packed.h"
#include "rows.h"

namespace awq {
namespace {

constexpr int kMaxAssign = kMoeMaxTokens * kMoeMaxTopK;
constexpr uint32_t kOutOfRange = 0x80000000u;      // > every buffer's size: loads return zero
constexpr float kLoScale = 2048.0f;                // of the lo plane
constexpr int kNonTemporal = 2;                    // weights: each byte is read once

__device__ __forceinline__ __amdgpu_buffer_rsrc_t moe_rsrc(const void* p, size_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ void load16_lds(__amdgpu_buffer_rsrc_t r, unsigned char* lds, uint32_t voff,
                                           uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)lds, 16, voff, soff, 0, 0);
}

__device__ __forceinline__ void split_hi_lo(float v, _Float16& hi, _Float16& lo) {
    hi = (_Float16)v;
    lo = (_Float16)((v - (float)hi) * kLoScale);
}

// Values that another workgroup of the same launch reads: written through to
// and read from the point where all compute units see the same memory.
__device__ __forceinline__ void store_shared(float* p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_shared(const float* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------------------
// router and choices: one workgroup of 16 waves per token, bound by what one
// compute unit reads (64 experts x 2048: 8 us; 8 experts x 4096: 4 to 5 us)
// ---------------------------------------------------------------------------
struct RouteArgs {
    const _Float16 *x, *router;
    const float* inv_s;                            // or nullptr
    int* ids;                                      // [M][top_k]
    float* weights;
    _Float16* scaled;                              // x' hi plane [M][K], then the lo plane (inv_s only)
    int* arrived;                                  // the down product's counters, cleared here
    int n_arrived;
    int M, E, K, top_k, renorm;
};

// One wave picks a token's experts from its logits (the sums of their parts, in
// order).  The keys order the logits
// as integers; a NaN comes below every number and a taken expert below a NaN,
// so every pick is a valid expert that was not picked before.
__device__ void route_token(const float* partial, int slabs, int E, int top_k, bool renorm, int* ids,
                            float* weights) {
    const int lane = threadIdx.x & 63;
    constexpr int PER = kMoeMaxExperts / 64;
    uint32_t key[PER];
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < E ? partial[e] : 0.0f;
        for (int p = 1; p < slabs && 64 * i < E; ++p) v[i] += e < E ? partial[p * E + e] : 0.0f;
        const uint32_t b = __builtin_bit_cast(uint32_t, v[i] + 0.0f);      // -0 as 0: they tie
        key[i] = e >= E ? 0u : v[i] != v[i] ? 1u : b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
    }
    float mine = 0.0f;                             // lane c keeps choice c
    int id = 0;
    for (int c = 0; c < top_k; ++c) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (64 * i < E) best = max(best, key[i]);
        best = wave_reduce(best, MaxU32());
        bool found = false;                        // lowest index with that key
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (64 * i >= E || found) continue;    // wave-uniform
            const uint64_t on = __builtin_amdgcn_ballot_w64(key[i] == best);
            if (on) {
                found = true;
                const int at = __ffsll((unsigned long long)on) - 1;
                const float l = __builtin_bit_cast(
                    float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v[i]), at));
                if (lane == c) { mine = l; id = 64 * i + at; }
                if (lane == at) key[i] = 0u;
            }
        }
    }
    const float top = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mine), 0));
    const float p = lane < top_k ? expf(mine - top) : 0.0f;
    float s = p;
    if (!renorm) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i < E) s += expf(v[i] - top);
    }
    const float sum = __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(uint32_t, s), SumF32()));
    if (lane < top_k) {
        ids[lane] = id;
        weights[lane] = p / sum;
    }
}

// The logits are units of RB experts by kSlab k, taken by the 16 waves in turn:
// a lane holds 8 k of every 512 of x and of RB router rows, all of them loaded
// at once.  RB = 4 where that still gives every wave a unit, else 1.  The layer with
// RB = 4 / 1, one token, 4 experts of 256 channels, router of 128 x 2048 18.5 / 21.4 us, 64 x
// 2048 15.4 / 16.9, 32 x 4096 15.7 / 17.2 (64 units each or more); below, where the
// rule takes 1, 32 x 2048 14.2 / 14.8, 16 x 4096 14.6 / 15.2, 8 x 4096 14.0 / 14.3:
// 4 is no slower there either.
constexpr int kSlab = 2048;

template <int RB>
__global__ __launch_bounds__(1024) void k_moe_route(RouteArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    float* partial = reinterpret_cast<float*>(smem);          // [slabs][E]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const size_t m = blockIdx.x;
    const int slabs = (a.K + kSlab - 1) / kSlab, groups = (a.E + RB - 1) / RB;
    const _Float16* x = a.x + m * a.K;
    const __amdgpu_buffer_rsrc_t rx = moe_rsrc(x, (size_t)a.K * 2);
    const __amdgpu_buffer_rsrc_t rr = moe_rsrc(a.router, (size_t)a.E * a.K * 2);
    auto load = [&](const __amdgpu_buffer_rsrc_t& r, uint32_t row, int k) {
        return __builtin_bit_cast(half8_t, __builtin_amdgcn_raw_buffer_load_b128(
            r, k < a.K ? (row * (uint32_t)a.K + (uint32_t)k) * 2u : kOutOfRange, 0, 0));
    };
    for (int unit = wave; unit < slabs * groups; unit += 16) {
        const int slab = unit / groups, e0 = unit % groups * RB;
        half8_t xv[4], rv[4][RB];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = slab * kSlab + 512 * i + 8 * lane;
            xv[i] = load(rx, 0, k);
#pragma unroll
            for (int q = 0; q < RB; ++q) rv[i][q] = load(rr, (uint32_t)min(e0 + q, a.E - 1), k);
        }
        float sum[RB] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < RB; ++q)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    sum[q] = __builtin_amdgcn_fdot2((half2_t){xv[i][2 * w], xv[i][2 * w + 1]},
                                                    (half2_t){rv[i][q][2 * w], rv[i][q][2 * w + 1]}, sum[q], false);
#pragma unroll
        for (int q = 0; q < RB; ++q) {
            const float l = __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(uint32_t, sum[q]), SumF32()));
            if (lane == 0 && e0 + q < a.E) partial[slab * a.E + e0 + q] = l;
        }
    }
    if (m == 0)
        for (int i = tid; i < a.n_arrived; i += 1024) a.arrived[i] = 0;
    if (a.inv_s) {
        const size_t at = m * a.K, plane = (size_t)a.M * a.K;
        for (int k = tid; k < a.K; k += 1024)
            split_hi_lo((float)x[k] * a.inv_s[k], a.scaled[at + k], a.scaled[plane + at + k]);
    }
    __syncthreads();
    if (wave == 0)
        route_token(partial, slabs, a.E, a.top_k, a.renorm, a.ids + m * a.top_k, a.weights + m * a.top_k);
}

// ---------------------------------------------------------------------------
// expert products
// ---------------------------------------------------------------------------
struct ExpertArgs {
    const uint32_t* q[2];                          // gate and up, or down alone
    const _Float16 *s[2], *z[2];
    const _Float16* in;                            // operand: hi plane [rows][K], then (split) the lo plane
    int split;                                     // the operand has a lo plane
    int rows;                                      // M (gate/up) or M * top_k (down)
    const int* ids;                                // [M * top_k]
    const float* weights;
    _Float16* h;                                   // gate/up out: hi plane [M * top_k][N], then lo
    float* part;                                   // down: fp32 [splits][M * top_k][N]
    int splits, split_tiles;                       // down, more tokens: K in splits of so many tiles
    int* arrived;                                  // down: workgroups done with a block of columns
    _Float16* y;                                   // down out [M][N]
    int M, E, top_k;
    int N, K;                                      // of one expert's layer
};

// How the 16 operand rows of a tile are shared out (see the top of the file)
template <int GS>
struct RowMap {
    static constexpr int HR = GS == 64 ? 8 : 16;   // rows that differ (the rest: the other group)
    int per_tile;                                  // tokens of a tile
    bool low;                                      // this lane's row: the lo plane?
    int slot;                                      // its token
    bool mine;                                     // its quarter is in the row's group
    __device__ __forceinline__ RowMap(int split, int j, int hq) {
        per_tile = split ? HR / 2 : HR;
        const int jr = j % HR;
        low = jr >= per_tile;
        slot = jr % per_tile;
        mine = GS == 128 || (j >> 3) == (hq >> 1);
    }
    // the sums of a lane's four rows with those of the rows that belong to the
    // same tokens: valid in the lanes whose row 4 hq is below per_tile
    __device__ __forceinline__ float4_t join(float4_t v) const {
        if constexpr (GS == 64) v = add(v, 32, 1.0f);
        if (per_tile < HR) v = add(v, GS == 64 ? 16 : 32, 1.0f / kLoScale);
        return v;
    }
    static __device__ __forceinline__ float4_t add(float4_t v, int lanes, float f) {
        float4_t o;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = __builtin_fmaf(__shfl_down(v[r], lanes), f, v[r]);
        return o;
    }
};

// one expert's buffers
template <int BITS, int GS, int NL>
struct Weights {
    static constexpr int WQ = BITS == 4 ? 4 : 3;
    __amdgpu_buffer_rsrc_t q[NL], s[NL], z[NL];
    __device__ __forceinline__ Weights(const ExpertArgs& a, int e) {
        const uint32_t tiles = (uint32_t)((a.N + 15) / 16) * (uint32_t)(a.K / kGroup);
        const size_t params = (size_t)tiles * (16 * kGroup / GS);
#pragma unroll
        for (int l = 0; l < NL; ++l) {
            q[l] = moe_rsrc(a.q[l] + (size_t)e * tiles * 64 * WQ, (size_t)tiles * 64 * WQ * 4);
            s[l] = moe_rsrc(a.s[l] + (size_t)e * params, params * 2);
            z[l] = moe_rsrc(a.z[l] + (size_t)e * params, params * 2);
        }
    }
};

template <int WQ, int NL>
struct TileRegs {
    TileSlot<WQ> w[NL];
    uint32_t d[NL], z[NL];
};

// tile t of an expert (all layers); tiles that are not there give zero codes
// and a zero scale
template <int BITS, int GS, int NL>
__device__ __forceinline__ void load_tile(const Weights<BITS, GS, NL>& r, uint32_t t, bool ok, int lane,
                                          TileRegs<(BITS == 4 ? 4 : 3), NL>& o) {
    constexpr int WQ = BITS == 4 ? 4 : 3;
    const uint32_t j = lane & 15, pgrp = GS == 64 ? (uint32_t)(lane >> 5) : 0u;
    const uint32_t oq = ok ? (t * 64u + (uint32_t)lane) * (WQ * 4u) : kOutOfRange;
    const uint32_t op = ok ? ((t * (kGroup / GS) + pgrp) * 16u + (j & ~1u)) * 2u : kOutOfRange;
#pragma unroll
    for (int l = 0; l < NL; ++l) {
        o.w[l] = load_tile_slot<WQ, kNonTemporal>(r.q[l], oq);
        o.d[l] = __builtin_amdgcn_raw_buffer_load_b32(r.s[l], op, 0, 0);
        o.z[l] = __builtin_amdgcn_raw_buffer_load_b32(r.z[l], op, 0, 0);
    }
}

// acc += d * (x . (q - z)) of one tile and layer for MT operand tiles
template <int BITS, int WQ, int MT>
__device__ __forceinline__ void tile_product(const TileSlot<WQ>& w, uint32_t d, uint32_t z, uint32_t psh,
                                             const half8_t (*x)[MT], float4_t* acc) {
    half8_t b[4];
    exact_operands<BITS, WQ>(w, bits_half((uint16_t)(z >> psh)), b);
    const float df = (float)bits_half((uint16_t)(d >> psh));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        float4_t g = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) g = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[q][m], b[q], g, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[m][r] = __builtin_fmaf(df, g[r], acc[m][r]);
    }
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// ---------------------------------------------------------------------------
// One token.  A work item is a block of 16 output rows of one choice; WK waves
// take its tiles in turn, each with U tiles in flight, and their sums meet in
// LDS.  A workgroup is 8 / WK items and ends with them: with several
// workgroups on a compute unit, one waits for its first tiles while others
// compute.  2 of 8 experts of 14336 x 4096, int4 g128: gate and up 22.9 us (5.4
// TB/s), down 14.0 us (4.4 TB/s; every workgroup reads its operand, two planes of
// 28 KB).  With the operand through registers behind the weights 23.9 and 16.2 us.
// Registers hold it to 3 workgroups a compute unit, LDS to 2 in that down product
// (its operand planes of 56 KB and the waves' sums of 8 KB).
// ---------------------------------------------------------------------------
// LDS of an item's operand planes, in whole 1 KB loads
__host__ __device__ __forceinline__ int token_lds(int split, int K) { return ((K * 2 << split) + 1023) / 1024 * 1024; }

template <int BITS, int GS, int WK, bool GATEUP>
__global__ __launch_bounds__(512, 6) void k_moe_token(ExpertArgs a) {
    constexpr int WQ = BITS == 4 ? 4 : 3;
    constexpr int NL = GATEUP ? 2 : 1;
    constexpr int SUB = 8 / WK;
    constexpr int U = GATEUP ? 2 : 4;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    __shared__ float4_t red[8][NL][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, hq = lane >> 4;
    const int sub = wave / WK, wk = wave % WK;
    const int G = a.K / kGroup, NB = (a.N + 15) / 16;
    const int total = a.top_k * NB;
    const int item = (int)blockIdx.x * SUB + sub;
    const bool live = item < total;
    const int c = live ? item / NB : 0, b = live ? item % NB : 0;
    const int nw = live && wk < G ? (G - wk + WK - 1) / WK : 0;

    // The operand planes of this item (gate/up: one token's for all items) go
    // direct to LDS, asked for before the weights, since loads return in order
    const int row_bytes = a.K * 2;
    unsigned char* xs = smem + (GATEUP ? 0 : sub * token_lds(a.split, a.K));
    {
        const int n = row_bytes / 16 << a.split;             // 16-byte chunks
        const __amdgpu_buffer_rsrc_t rx =
            moe_rsrc(a.in, (size_t)__builtin_amdgcn_readfirstlane(a.rows * row_bytes << a.split));
        for (int i0 = GATEUP ? wave : wk; i0 * 64 < n; i0 += GATEUP ? 8 : WK) {
            const int i = i0 * 64 + lane, p = i >= row_bytes / 16;
            const uint32_t at = (uint32_t)(p * a.rows + (GATEUP ? 0 : c) - p) * (uint32_t)row_bytes + 16u * (uint32_t)i;
            load16_lds(rx, xs + i0 * 1024, i < n ? at : kOutOfRange, 0);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    const Weights<BITS, GS, NL> rw(a, __builtin_amdgcn_readfirstlane(a.ids[c]));
    TileRegs<WQ, NL> ring[U];
    auto load = [&](int i, int u) {
        load_tile<BITS, GS, NL>(rw, (uint32_t)b * (uint32_t)G + (uint32_t)(wk + WK * i), i < nw, lane, ring[u]);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
        __builtin_amdgcn_sched_barrier(0);
        load(u, u);
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(3 * NL * U));       // the weights need not have landed
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const RowMap<GS> map(a.split, j, hq);
    const unsigned char* xl = xs + (map.low ? row_bytes : 0) + 64 * hq;
    const uint32_t psh = 16u * (uint32_t)(j & 1);

    float4_t acc[NL][1];
#pragma unroll
    for (int l = 0; l < NL; ++l) acc[l][0] = (float4_t){0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < nw; i0 += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u < nw) {                     // wave-uniform
                const unsigned char* xt = xl + (wk + WK * (i0 + u)) * (2 * kGroup);
                half8_t x[4][1];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    x[q][0] = *reinterpret_cast<const half8_t*>(xt + 16 * q);
                    if (!map.mine) x[q][0] = (half8_t){};
                }
#pragma unroll
                for (int l = 0; l < NL; ++l)
                    tile_product<BITS, WQ, 1>(ring[u].w[l], ring[u].d[l], ring[u].z[l], psh, x, acc[l]);
            }
            load(i0 + u + U, u);
        }
    }
#pragma unroll
    for (int l = 0; l < NL; ++l) red[wave][l][lane] = acc[l][0];
    __syncthreads();
    if (wk != 0 || !live) return;
    float4_t v[NL];
#pragma unroll
    for (int l = 0; l < NL; ++l) {
        v[l] = red[wave][l][lane];
#pragma unroll
        for (int q = 1; q < WK; ++q) {
            const float4_t o = red[wave + q][l][lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[l][r] += o[r];
        }
        v[l] = map.join(v[l]);
    }
    const int n = 16 * b + j;                      // row 0 is the token: lanes 0..15
    if constexpr (GATEUP) {
        if (lane < 16) {
            const size_t at = (size_t)c * a.N + n;
            split_hi_lo(silu_mul(v[0][0], v[NL - 1][0]), a.h[at], a.h[(size_t)a.top_k * a.N + at]);
        }
    } else {
        if (lane < 16) store_shared(a.part + (size_t)c * a.N + n, v[0][0]);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        int before = 0;
        if (lane == 0) before = __hip_atomic_fetch_add(a.arrived + b, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (__builtin_amdgcn_readfirstlane(before) != a.top_k - 1) return;
        // the last one: lane quarter hq sums choices hq, hq + 4, .., and the
        // quarters are added in a fixed order
        float sum = 0.0f;
        for (int q = hq; q < a.top_k; q += 4)
            sum = __builtin_fmaf(a.weights[q], load_shared(a.part + (size_t)q * a.N + n), sum);
        sum += __shfl_down(sum, 32);
        sum += __shfl_down(sum, 16);
        if (lane < 16) a.y[n] = (_Float16)sum;
    }
}

// ---------------------------------------------------------------------------
// More tokens.  A workgroup of WV waves owns one expert and WV / KW blocks of 16
// output rows, each of KW waves over the whole K; the operand rows of the expert's
// tokens go through LDS for all of them.  S steps of KT tiles are in flight:
// operand rows direct to LDS, weights (whole 1 KB or 768-byte tiles) to registers.
// 64 tokens, 2 of 8 experts of 14336 x 4096, int4 g128: gate and up 103 us (4.8
// TB/s), down 92 us (2.7 TB/s: two operand rows a token, so twice the products
// and fragment reads for a byte); an expert of more than 32 of the tokens takes a
// second pass (the layer 239 to 252 us, 202 to 214 without one).  13 tokens, 6 of
// 64 experts of 1408 x 2048, int3 g64, x' = x * inv_s: the layer 56.5 us, 51.4 in
// a build that multiplies the words without unpacking them, and 58.0 with int4:
// the unpacking is a tenth of it, not what bounds it.
// ---------------------------------------------------------------------------
struct Lists {
    int ids[kMaxAssign];                           // every choice
    uint32_t present[kMoeMaxExperts / 32];         // experts that some token takes
    int mine[kMoeMaxTokens];                       // this expert's assignments, ascending
};

// The expert number `which` (ascending) of those that tokens take and how many
// assignments it has (listed in L.mine), or -1 for the expert where fewer are
// taken.  A token takes an expert at most once.
struct Share { int expert, count; };

template <int NT>
__device__ __forceinline__ Share find_share(Lists& L, const int* ids, int assigned, int which) {
    constexpr int WORDS = kMoeMaxExperts / 32;
    const int tid = threadIdx.x, lane = tid & 63;
    if (tid < WORDS) L.present[tid] = 0;
    __syncthreads();
    for (int i = tid; i < assigned; i += NT) {
        const int e = ids[i];
        L.ids[i] = e;
        atomicOr(&L.present[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    // lanes 0..15 hold 32 experts each; the word that holds number `which`
    const uint32_t word = lane < WORDS ? L.present[lane] : 0u;
    int upto = __builtin_popcount(word);           // experts taken in the words up to this lane's
#pragma unroll
    for (int d = 1; d < WORDS; d <<= 1) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    const uint64_t past = __builtin_amdgcn_ballot_w64(lane < WORDS && upto > which);
    if (past == 0) return Share{-1, 0};
    const int at = __builtin_ctzll(past);
    uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)word, at);
    for (int skip = which - (__builtin_amdgcn_readlane(upto, at) - __builtin_popcount(bits)); skip > 0; --skip)
        bits &= bits - 1;
    Share s{__builtin_amdgcn_readfirstlane(32 * at + __builtin_ctz(bits)), 0};
    for (int i0 = 0; i0 < assigned; i0 += 64) {    // every wave counts, the first one writes
        const bool is = i0 + lane < assigned && L.ids[i0 + lane] == s.expert;
        const uint64_t on = __builtin_amdgcn_ballot_w64(is);
        if (tid < 64 && is) L.mine[s.count + __popcll(on & ((1ull << lane) - 1))] = i0 + lane;
        s.count += __popcll(on);
    }
    s.count = __builtin_amdgcn_readfirstlane(s.count);
    __syncthreads();
    return s;
}

// The 16-byte chunk of a 256-byte operand row that LDS position p of row r (of
// its tile) holds is p ^ row_swizzle(r): fragment reads then take distinct banks (the
// prefill kernel's activation rows, measured there)
__device__ __forceinline__ int row_swizzle(int r) { return (r & 0xA) | ((r & 1) << 2) | ((r >> 2) & 1); }

// waves per SIMD that k_moe_tile's registers are held to
constexpr int tile_waves(int GS, int MT, int WV, bool gate_up) {
    return MT >= 4 ? (WV == 8 && !gate_up ? 4 : 2) : MT == 2 && gate_up && GS == 64 ? 2 : 3;
}

template <int BITS, int GS, int MT, int WV, int KW, bool GATEUP>
struct TileShape {
    static constexpr int NL = GATEUP ? 2 : 1;
    static constexpr int HR = RowMap<GS>::HR;
    static constexpr int XR = MT * HR;             // operand rows in LDS
    // tiles per step: at least one 4-row load for every wave, and KW
    static constexpr int KL = XR / 4 >= WV ? 1 : WV / (XR / 4), KT = KL > KW ? KL : KW;
    static constexpr int KI = KT / KW;             // a wave's
    static constexpr int XW = XR / 4 * KT / WV;    // its loads per wave
    static constexpr int TB = (XR + (GS == 64)) * 256;     // a tile's rows (and a row of zeros)
    static constexpr int BUF = TB * KT;
    static constexpr int LPS = XW + 3 * NL * KI;   // loads per step and wave
    static constexpr int S = KT * NL >= 4 ? 3 : XR >= 64 ? 4 : KT * NL == 2 ? 4 : 6;
    static constexpr int SUMS = KW > 1 ? WV * NL * MT * 1024 : 0;      // the waves' sums
    static constexpr size_t LDS = (size_t)S * BUF + SUMS;
    static_assert(XW * WV == XR / 4 * KT, "every wave loads the same number of row groups");
    static_assert(LPS * (S - 2) <= 63, "vmcnt counts to 63");
};

template <int BITS, int GS, int MT, int WV, int KW, bool GATEUP>
__global__ __launch_bounds__(64 * WV, tile_waves(GS, MT, WV, GATEUP)) void k_moe_tile(ExpertArgs a) {
    using T = TileShape<BITS, GS, MT, WV, KW, GATEUP>;
    constexpr int WQ = BITS == 4 ? 4 : 3, NL = T::NL, S = T::S, KT = T::KT, KI = T::KI;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    __shared__ Lists L;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, hq = lane >> 4;
    const int G = a.K / kGroup, NB = (a.N + 15) / 16, NG = (NB + WV / KW - 1) / (WV / KW);
    const int assigned = a.M * a.top_k;
    const int b = (int)blockIdx.x % NG * (WV / KW) + wave / KW;         // this wave's row block,
    const int kw = wave % KW;                      // and which of each step's KW tiles
    const Share share = find_share<64 * WV>(L, a.ids, assigned, (int)blockIdx.x / NG);
    if (share.expert < 0) return;
    const int cnt = share.count;
    const Weights<BITS, GS, NL> rw(a, share.expert);
    const RowMap<GS> map(a.split, j, hq);
    const uint32_t psh = 16u * (uint32_t)(j & 1);
    const size_t plane = (size_t)a.rows * a.K * 2;
    // the size through a scalar register: a descriptor held in vector registers
    // would cost a loop around every load
    const __amdgpu_buffer_rsrc_t rx =
        moe_rsrc(a.in, (size_t)__builtin_amdgcn_readfirstlane((int)(plane << a.split)));
    // this workgroup's tiles of every row: all, or (down) one split of them
    const int g0 = GATEUP ? 0 : (int)blockIdx.y * a.split_tiles;
    const int g1 = GATEUP ? G : min(G, g0 + a.split_tiles);
    const int steps = (g1 - g0 + KT - 1) / KT;
    const uint32_t tile0 = (uint32_t)min(b, NB - 1) * (uint32_t)G;

    if constexpr (GS == 64) {                      // the rows of zeros
        for (int i = tid; i < S * KT * 64; i += 64 * WV)
            *reinterpret_cast<uint32_t*>(smem + i / 64 * T::TB + T::XR * 256 + i % 64 * 4) = 0;
    }
    for (int s0 = 0; s0 < cnt; s0 += MT * map.per_tile) {
        // row group ii = wave * XW + i: tile ii / (XR / 4) of the step, LDS rows 4 rg ..
        uint32_t xoff[T::XW];
#pragma unroll
        for (int i = 0; i < T::XW; ++i) {
            const int rg = (wave * T::XW + i) % (T::XR / 4);
            const int r = 4 * rg + (lane >> 4);
            const int jr = r % T::HR;
            const int s = s0 + r / T::HR * map.per_tile + jr % map.per_tile;
            const int as = s < cnt ? L.mine[s] : 0;
            const int row = GATEUP ? as / a.top_k : as;
            xoff[i] = s < cnt ? (uint32_t)((jr >= map.per_tile ? plane : 0) + (size_t)row * a.K * 2) +
                                    16u * (uint32_t)((lane & 15) ^ row_swizzle(jr))
                              : kOutOfRange;
        }
        TileRegs<WQ, NL> ring[S][KI];
        auto issue = [&](int step, int slot) {
#pragma unroll
            for (int i = 0; i < T::XW; ++i) {
                const int ii = wave * T::XW + i;
                // stated uniform: a scalar offset of the load
                const int g = __builtin_amdgcn_readfirstlane(g0 + step * KT + ii / (T::XR / 4));
                load16_lds(rx, smem + slot * T::BUF + ii / (T::XR / 4) * T::TB + ii % (T::XR / 4) * 1024,
                           g < g1 ? xoff[i] : kOutOfRange, (uint32_t)g * 256u);
            }
#pragma unroll
            for (int t = 0; t < KI; ++t) {
                const int g = g0 + step * KT + kw + KW * t;
                load_tile<BITS, GS, NL>(rw, tile0 + (uint32_t)g, g < g1, lane, ring[slot][t]);
            }
        };
        float4_t acc[NL][MT];
#pragma unroll
        for (int l = 0; l < NL; ++l)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[l][m] = (float4_t){0.f, 0.f, 0.f, 0.f};
        const int live = min(MT, (cnt - s0 + map.per_tile - 1) / map.per_tile);
        // this lane's chunks of its operand row, or (64-wide groups, a row of the
        // other group) of the row of zeros
        int xat[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            xat[q] = map.mine ? (j % T::HR) * 256 + (((4 * hq + q) ^ row_swizzle(j % T::HR)) << 4) : T::XR * 256;
        const int mstep = map.mine ? T::HR * 256 : 0;
        auto compute = [&](int slot, const TileRegs<WQ, NL>* regs, auto tiles) {
            constexpr int LM = decltype(tiles)::value;
            const unsigned char* xb = smem + slot * T::BUF + kw * T::TB;
#pragma unroll
            for (int t = 0; t < KI; ++t) {
                half8_t x[4][LM];
#pragma unroll
                for (int m = 0; m < LM; ++m)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        x[q][m] = *reinterpret_cast<const half8_t*>(xb + KW * t * T::TB + m * mstep + xat[q]);
#pragma unroll
                for (int l = 0; l < NL; ++l)
                    tile_product<BITS, WQ, LM>(regs[t].w[l], regs[t].d[l], regs[t].z[l], psh, x, acc[l]);
            }
        };
#pragma unroll
        for (int s = 0; s < S - 1; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            issue(s, s);
        }
        __builtin_amdgcn_sched_barrier(0);
        int step0 = 0;
        do {
#pragma unroll
            for (int st = 0; st < S; ++st) {
                const int step = step0 + st;
                // this wave's part of the step has landed; then everybody's, and
                // everybody is done with the buffer that is loaded next (a bare
                // barrier: a fence would also drain the later steps' loads)
                __builtin_amdgcn_s_waitcnt(vmcnt_imm(T::LPS * (S - 2)));
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
                issue(step + S - 1, (st + S - 1) % S);
                __builtin_amdgcn_sched_barrier(0);
                if (step < steps) {
                    // the operand tiles that hold tokens (wave-uniform)
                    if (MT >= 4 && live > 3) compute(st, ring[st], std::integral_constant<int, MT>());
                    else if (MT >= 4 && live > 2) compute(st, ring[st], std::integral_constant<int, MT >= 4 ? 3 : MT>());
                    else if (MT >= 2 && live > 1) compute(st, ring[st], std::integral_constant<int, MT >= 2 ? 2 : MT>());
                    else compute(st, ring[st], std::integral_constant<int, 1>());
                }
            }
            step0 += S;
        } while (step0 < steps);

        if constexpr (KW > 1) {                    // the first wave of a row block adds the others' sums
            float4_t* sums = reinterpret_cast<float4_t*>(smem + S * T::BUF) + wave * (NL * MT * 64) + lane;
#pragma unroll
            for (int l = 0; l < NL; ++l)
#pragma unroll
                for (int m = 0; m < MT; ++m) sums[(l * MT + m) * 64] = acc[l][m];
            __syncthreads();
            if (kw == 0) {
#pragma unroll
                for (int l = 0; l < NL; ++l)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int q = 1; q < KW; ++q) {
                            const float4_t o = sums[((q * NL + l) * MT + m) * 64];
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[l][m][r] += o[r];
                        }
            }
        }
        const int n = 16 * b + j;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (m >= live || kw != 0) continue;
            float4_t v[NL];
#pragma unroll
            for (int l = 0; l < NL; ++l) v[l] = map.join(acc[l][m]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int slot = 4 * hq + r, s = s0 + m * map.per_tile + slot;
                if (slot < map.per_tile && s < cnt && b < NB) {
                    const size_t at = (size_t)L.mine[s] * a.N + n;
                    if constexpr (GATEUP)
                        split_hi_lo(silu_mul(v[0][r], v[NL - 1][r]), a.h[at], a.h[(size_t)assigned * a.N + at]);
                    else
                        a.part[(size_t)blockIdx.y * assigned * a.N + at] = v[0][r];
                }
            }
        }
        // the pass's loads have landed and its LDS reads are done
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
}

// y[m] = the choices' rows (the sums of their splits), weighted, in their order;
// 4 columns a thread (64 x 4096, 2 choices: 5 us, of which the launch is half)
__global__ __launch_bounds__(256) void k_moe_join(const float* part, const float* weights, _Float16* y, int top_k,
                                                  int K, int splits) {
    const int k = (blockIdx.x * 256 + threadIdx.x) * 4;
    const size_t m = blockIdx.y;
    if (k >= K) return;
    float4_t sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int c = 0; c < top_k; ++c) {
        const float w = weights[m * top_k + c];
        const float* p = part + (m * top_k + c) * K + k;
        float4_t v = *reinterpret_cast<const float4_t*>(p);
        for (int s = 1; s < splits; ++s) {
            const float4_t o = *reinterpret_cast<const float4_t*>(p + (size_t)s * gridDim.y * top_k * K);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += o[r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] = __builtin_fmaf(w, v[r], sum[r]);
    }
    *reinterpret_cast<uint2*>(y + m * K + k) = make_uint2(pack2<F16>(sum[0], sum[1]), pack2<F16>(sum[2], sum[3]));
}

using ExpertFn = void (*)(ExpertArgs);

int set_lds(ExpertFn kern, size_t lds) {
    if (lds <= 48 * 1024) return 0;
    return (int)hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
}

// one token: waves of an item by the K tiles, so that a workgroup is one item of
// long rows or several of short ones.  The layer at 2 / 4 / 8 waves, int4 g128:
// 8 of 64 experts, 512 x 512 15.6 / 15.0 / 14.8 us, 896 x 896 18.2 / 17.0 / 17.2,
// 1024 x 1024 18.7 / 17.6 / 17.9; 4 of 32, 2048 x 2048 20.2 / 18.3 / 18.2, 3968 x
// 3968 31.6 / 31.5 / 32.5, 4096 x 4096 30.5 / 30.4 / 32.4; 1 of 4, 8192 x 4096 - /
// 21.5 / 20.1.  So 2 waves are a few per cent behind 4 in short rows, and 8 ahead
// of 4 only where items are fewer than the card holds.
template <int BITS, int GS, bool GATEUP>
int launch_token(const ExpertArgs& a, hipStream_t st) {
    const int G = a.K / kGroup, NB = (a.N + 15) / 16;
    const int wk = G >= 32 ? 8 : G >= 8 ? 4 : 2;
    ExpertFn kern = wk == 8 ? k_moe_token<BITS, GS, 8, GATEUP>
                            : wk == 4 ? k_moe_token<BITS, GS, 4, GATEUP> : k_moe_token<BITS, GS, 2, GATEUP>;
    const int sub = 8 / wk;
    const size_t lds = (size_t)(GATEUP ? 1 : sub) * token_lds(a.split, a.K);
    if (int e = set_lds(kern, lds)) return e;
    hipLaunchKernelGGL(kern, dim3((a.top_k * NB + sub - 1) / sub), dim3(512), lds, st, a);
    return (int)hipGetLastError();
}

template <int BITS, int GS, bool GATEUP, int MT, int WV, int KW>
int launch_tile_waves(const ExpertArgs& a, hipStream_t st) {
    using T = TileShape<BITS, GS, MT, WV, KW, GATEUP>;
    auto kern = k_moe_tile<BITS, GS, MT, WV, KW, GATEUP>;
    if (T::LDS > 48 * 1024)
        if (int e = (int)hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)T::LDS))
            return e;
    const int NG = ((a.N + 15) / 16 + WV / KW - 1) / (WV / KW);
    const int experts = min(a.M * a.top_k, a.E);
    hipLaunchKernelGGL(kern, dim3(experts * NG, GATEUP ? 1 : a.splits), dim3(64 * WV), T::LDS, st, a);
    return (int)hipGetLastError();
}

// 8 waves share the operand rows of 64-row steps, unless that leaves more than
// half of the compute units without a workgroup (23 tokens, 6 of 16 experts, 512 x
// 2944: 50.6 us, 43.6 with 4 waves; 54 tokens, 3 of 11, 640 x 2048: 31.7 and 35.8).
// Gate and up of few row blocks: KW waves take each step's KW tiles in turn, one
// block of rows for all of them, and the first adds their sums (36 tokens, 4 of 6
// experts, 256 x 1920: 39.3 us, 35.3 so; 64 tokens, 2 of 8, 1024 x 4096: 52.4 and
// 44.0).  KW = 4 where the steps' operand rows then leave LDS for two workgroups.
// From 8 K tiles on (36 tokens, 2 of 8, 512 x 1024: 19.9 us, 21.0 without; 8 tokens
// 15.8 and 17.4; of 6 tiles 19.5 and 20.5, of 4 18.1 and 18.2).
template <int BITS, int GS, bool GATEUP, int MT>
int launch_tile(const ExpertArgs& a, hipStream_t st) {
    const int cus = device_cu_count(), experts = min(a.M * a.top_k, a.E);
    if constexpr (MT * RowMap<GS>::HR >= 64)
        if (experts * ((a.N + 127) / 128) * (GATEUP ? 1 : a.splits) >= cus / 2)
            return launch_tile_waves<BITS, GS, GATEUP, MT, 8, 1>(a, st);
    if constexpr (GATEUP)
        if (experts * ((a.N + 63) / 64) < cus && a.K / kGroup >= 8)
            return launch_tile_waves<BITS, GS, GATEUP, MT, 4, (MT * RowMap<GS>::HR >= 32 ? 2 : 4)>(a, st);
    return launch_tile_waves<BITS, GS, GATEUP, MT, 4, 1>(a, st);
}

template <int BITS, int GS, bool GATEUP>
int launch_experts(const ExpertArgs& a, hipStream_t st) {
    if (a.M == 1) return launch_token<BITS, GS, GATEUP>(a, st);
    // operand tiles: an expert with more tokens than they hold takes further
    // passes over its weights, one with fewer skips the empty ones.  The shares
    // are uneven: one tile where it holds three even shares (59 tokens, 5 of 40
    // experts: 169 us at one tile for two shares, 153 at two tiles), two where
    // they hold two (64 tokens, 2 of 8 experts: 191 us, 223 at four tiles).
    const int rows_per_token = (a.split ? 2 : 1) * (GS == 64 ? 2 : 1);
    const int even = (a.M * a.top_k + a.E - 1) / a.E;
    if (min(a.M, 3 * even) * rows_per_token <= 16) return launch_tile<BITS, GS, GATEUP, 1>(a, st);
    if (min(a.M, 2 * even) * rows_per_token <= 32) return launch_tile<BITS, GS, GATEUP, 2>(a, st);
    return launch_tile<BITS, GS, GATEUP, 4>(a, st);
}

template <bool GATEUP>
int launch_experts_any(const ExpertArgs& a, int bits, int group_size, hipStream_t st) {
    if (group_size == 64)
        return bits == 4 ? launch_experts<4, 64, GATEUP>(a, st) : launch_experts<3, 64, GATEUP>(a, st);
    return bits == 4 ? launch_experts<4, 128, GATEUP>(a, st) : launch_experts<3, 128, GATEUP>(a, st);
}

// K splits of the down projections of more than one token: as many as bring the
// expert workgroups (of 4 row blocks) to 6 per compute unit while a split
// keeps 16 tiles, or to one while it keeps 8 (31 tokens, 4 of 7 experts, 3712 x
// 640: 66 us without the second, 52 with it).  The layer with 2 of 8 experts of
// 14336 x 4096 and 64 tokens: 217 us at 6 a compute unit, 252 at 3, 215 at 12; of
// 4096 x 4096 93, 98, 93, with 8 tiles a split 91, with 32 98; but 16 tokens of
// 8192 x 4096 91 us at 6, 87 at 3, 94 at 12.
int down_splits(int M, int K, int I, int E, int top_k) {
    if (M == 1) return 1;
    const int wgs = min(M * top_k, E) * ((K / 16 + 3) / 4);
    const int cus = device_cu_count();
    return max(1, max(min((I / kGroup) / 16, 6 * cus / max(wgs, 1)), min((I / kGroup) / 8, cus / max(wgs, 1))));
}

// the workspace's parts, each 256-byte aligned
struct Workspace {
    size_t ids, weights, arrived, h, part, scaled, bytes;
    Workspace(int M, int K, int I, int E, int top_k) {
        size_t at = 0;
        auto take = [&](size_t n) {
            const size_t here = at;
            at += (n + 255) / 256 * 256;
            return here;
        };
        const size_t as = (size_t)M * top_k;
        ids = take(as * 4);
        weights = take(as * 4);
        arrived = take((size_t)(K / 16) * 4);
        h = take(as * I * 4);
        part = take(as * K * 4 * down_splits(M, K, I, E, top_k));
        scaled = take((size_t)M * K * 4);
        bytes = at;
    }
};

}  // namespace

size_t moe_workspace_bytes(int M, int K, int I, int E, int top_k) { return Workspace(M, K, I, E, top_k).bytes; }

int launch_moe(const MoeProblem& p, void* workspace, hipStream_t st) {
    const Workspace w(p.M, p.K, p.I, p.E, p.top_k);
    unsigned char* ws = (unsigned char*)workspace;
    _Float16* scaled = (_Float16*)(ws + w.scaled);
    ExpertArgs a{};
    a.ids = (int*)(ws + w.ids);
    a.weights = (float*)(ws + w.weights);
    a.arrived = (int*)(ws + w.arrived);
    a.h = (_Float16*)(ws + w.h);
    a.part = (float*)(ws + w.part);
    a.y = (_Float16*)p.y;
    a.M = p.M; a.E = p.E; a.top_k = p.top_k;

    const RouteArgs r{(const _Float16*)p.x, (const _Float16*)p.router, p.inv_s, (int*)(ws + w.ids),
                      (float*)(ws + w.weights), scaled, a.arrived, p.K / 16, p.M, p.E, p.K, p.top_k, p.renormalize};
    const int slabs = (p.K + kSlab - 1) / kSlab;
    auto route = p.E * slabs >= 64 ? k_moe_route<4> : k_moe_route<1>;
    hipLaunchKernelGGL(route, dim3(p.M), dim3(1024), (size_t)slabs * p.E * 4, st, r);
    if (int e = (int)hipGetLastError()) return e;

    for (int l = 0; l < 2; ++l) {
        a.q[l] = (const uint32_t*)p.qweight[l];
        a.s[l] = (const _Float16*)p.scales[l];
        a.z[l] = (const _Float16*)p.zeros[l];
    }
    a.in = p.inv_s ? scaled : (const _Float16*)p.x;
    a.split = p.inv_s != nullptr;
    a.rows = p.M;
    a.N = p.I; a.K = p.K;
    if (int e = launch_experts_any<true>(a, p.bits, p.group_size, st)) return e;

    a.q[0] = (const uint32_t*)p.qweight[2];
    a.s[0] = (const _Float16*)p.scales[2];
    a.z[0] = (const _Float16*)p.zeros[2];
    a.in = a.h;
    a.split = 1;
    a.rows = p.M * p.top_k;
    a.N = p.K; a.K = p.I;
    const int tiles = p.I / kGroup, splits = down_splits(p.M, p.K, p.I, p.E, p.top_k);
    a.split_tiles = (tiles + splits - 1) / splits;
    a.splits = (tiles + a.split_tiles - 1) / a.split_tiles;
    if (int e = launch_experts_any<false>(a, p.bits, p.group_size, st)) return e;
    if (p.M == 1) return 0;
    hipLaunchKernelGGL(k_moe_join, dim3((p.K / 4 + 255) / 256, p.M), dim3(256), 0, st, a.part, a.weights, a.y,
                       p.top_k, p.K, a.splits);
    return (int)hipGetLastError();
}

}  // namespace awq
