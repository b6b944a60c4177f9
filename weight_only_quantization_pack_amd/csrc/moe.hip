// A mixture-of-experts layer for a few tokens over packed experts:
//   l = x Wr^T;  the top_k largest l of each token (ties to the lowest index)
//   p = softmax(l) over the chosen ones, or over all experts
//   y = sum_j p_j down_j(SiLU(gate_j x') * up_j x'),  x' = x * inv_s or x
//
// HBM-bound: every packed byte of an expert that some token takes is read
// once, by whichever tokens take it.  Launches:
//   k_moe_router  the logits (fp16 MFMA, fp32 sums); x' where there is a scale
//   k_moe_experts the chosen experts and, for each, its gate and up
//                 projections over its tokens: h = SiLU(g) * u
//   k_moe_experts the down projections of h, one fp32 row per (token, choice)
//   k_moe_join    y = sum over the choices, in their order, rounded once
//
// One kernel serves both expert products.  A work item is a block of 16 output
// rows of one chosen expert; WK waves take its k tiles in turn.  The weights
// are the B operand of v_mfma_f32_16x16x32_f16 (lane slot = operand, as
// packed), always the exact (q - z), and the group scale multiplies the fp32
// group sums, so the only roundings on the way are those of fp32 sums.  The
// 16 operand rows of A hold more than one row per token where that keeps the
// products exact:
//   - an operand that is not an fp16 number (h, and x' = x * inv_s) is split
//     into hi = fp16(v) and lo = fp16((v - hi) * 2^11), two rows whose sums
//     are added as hi + lo / 2^11: 22 bits of v, for matrix time that is free
//     while the weights are what is waited for;
//   - with 64-wide groups a k32 product mixes both groups of a tile (lane
//     quarters 0, 1 and 2, 3), so rows 0..7 hold the tokens with quarters 2, 3
//     zeroed and rows 8..15 the same tokens with quarters 0, 1 zeroed: the
//     group sums come out in different rows.
#include "packed.h"
#include "rows.h"

namespace awq {
namespace {

constexpr int kMoeWaves = 8;                       // waves of an expert workgroup
constexpr int kMaxAssign = kMoeMaxTokens * kMoeMaxTopK;
constexpr uint32_t kOutOfRange = 0x80000000u;      // > every buffer's size: loads return zero
constexpr float kLoScale = 2048.0f;                // of the lo plane

__device__ __forceinline__ __amdgpu_buffer_rsrc_t moe_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ half8_t load_half8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(half8_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

__device__ __forceinline__ void split_hi_lo(float v, _Float16& hi, _Float16& lo) {
    hi = (_Float16)v;
    lo = (_Float16)((v - (float)hi) * kLoScale);
}

// ---------------------------------------------------------------------------
// router: one workgroup per 16 experts x 16 tokens, its 16 waves take the k32
// steps in turn
// ---------------------------------------------------------------------------
struct RouterArgs {
    const _Float16 *x, *router;
    const float* inv_s;                            // or nullptr
    float* logits;                                 // [M][E]
    _Float16* scaled;                              // x' hi plane [M][K], then the lo plane (inv_s only)
    int M, E, K;
};

__global__ __launch_bounds__(1024) void k_moe_router(RouterArgs a) {
    __shared__ float4_t red[16][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int j = lane & 15, h = lane >> 4;
    const int e0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
    const int mrows = min(16, a.M - m0);
    const uint32_t row = (uint32_t)a.K * 2u;
    const __amdgpu_buffer_rsrc_t rx = moe_rsrc(a.x + (size_t)m0 * a.K, (uint32_t)mrows * row);
    const __amdgpu_buffer_rsrc_t rr = moe_rsrc(a.router + (size_t)e0 * a.K, (uint32_t)min(16, a.E - e0) * row);
    float4_t acc = {0.f, 0.f, 0.f, 0.f};
    const int steps = a.K / 32;
    for (int s = wave; s < steps; s += 16) {
        const uint32_t off = (uint32_t)j * row + (uint32_t)s * 64u + 16u * h;
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(load_half8(rx, off), load_half8(rr, off), acc, 0, 0, 0);
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
        float4_t sum = red[0][lane];
        for (int w = 1; w < 16; ++w) {
            const float4_t o = red[w][lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[r] += o[r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (4 * h + r < mrows && e0 + j < a.E) a.logits[(size_t)(m0 + 4 * h + r) * a.E + e0 + j] = sum[r];
    }
    if (a.inv_s && blockIdx.x == 0) {
        const size_t plane = (size_t)a.M * a.K;
        for (int i = tid; i < mrows * a.K; i += 1024) {
            const int m = i / a.K, k = i - m * a.K;
            const size_t at = (size_t)(m0 + m) * a.K + k;
            split_hi_lo((float)a.x[at] * a.inv_s[k], a.scaled[at], a.scaled[plane + at]);
        }
    }
}

// ---------------------------------------------------------------------------
// routing of all tokens, by every expert workgroup for itself
// ---------------------------------------------------------------------------
struct Lists {
    int ids[kMaxAssign];                           // expert of assignment token * top_k + choice
    int order[kMaxAssign];                         // assignments grouped by expert (any order within one)
    int count[kMoeMaxExperts], start[kMoeMaxExperts], cursor[kMoeMaxExperts];
    int active[kMoeMaxExperts];                    // experts with tokens, ascending
    int n_active, most;                            // how many, and the largest count
};

// From ids: counts, starts, the grouped order and the active experts.  Called
// by a whole workgroup after ids are written and visible.
__device__ void build_lists(Lists& L, int assigned, int E) {
    const int tid = threadIdx.x, lane = tid & 63;
    for (int e = tid; e < E; e += 64 * kMoeWaves) L.count[e] = 0;
    __syncthreads();
    for (int i = tid; i < assigned; i += 64 * kMoeWaves) atomicAdd(&L.count[L.ids[i]], 1);
    __syncthreads();
    if (tid < 64) {                                // wave 0: prefix over the experts, 64 at a time
        int base = 0, act = 0, most = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            const int c = e < E ? L.count[e] : 0;
            int incl = c;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(incl, d);
                if (lane >= d) incl += o;
            }
            const uint64_t on = __builtin_amdgcn_ballot_w64(c > 0);
            if (e < E) {
                L.start[e] = L.cursor[e] = base + incl - c;
                if (c > 0) L.active[act + __popcll(on & ((1ull << lane) - 1))] = e;
            }
            base += __shfl(incl, 63);
            act += __popcll(on);
            most = max(most, (int)wave_reduce((uint32_t)c, MaxU32()));
        }
        if (lane == 0) { L.n_active = act; L.most = most; }
    }
    __syncthreads();
    for (int i = tid; i < assigned; i += 64 * kMoeWaves) L.order[atomicAdd(&L.cursor[L.ids[i]], 1)] = i;
    __syncthreads();
}

// One wave picks a token's experts from its logits.  The keys order the logits
// as integers; a NaN comes below every number and a taken expert below a NaN,
// so every pick is a valid expert that was not picked before.
__device__ void route_token(const float* logits, int E, int top_k, bool renorm, int* ids, float* weights) {
    const int lane = threadIdx.x & 63;
    constexpr int PER = kMoeMaxExperts / 64;
    uint32_t key[PER];
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < E ? logits[e] : 0.0f;
        const uint32_t b = __builtin_bit_cast(uint32_t, v[i] + 0.0f);      // -0 as 0: they tie
        key[i] = e >= E ? 0u : v[i] != v[i] ? 1u : b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
    }
    float top = 0.0f, chosen = 0.0f, mine = 0.0f;  // mine: lane j keeps choice j's exp
    for (int c = 0; c < top_k; ++c) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) best = max(best, key[i]);
        best = wave_reduce(best, MaxU32());
        int pick = -1;                             // lowest index with that key
        float l = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint64_t on = __builtin_amdgcn_ballot_w64(key[i] == best);
            if (pick < 0 && on) {
                const int at = __ffsll((unsigned long long)on) - 1;
                pick = 64 * i + at;
                l = __shfl(v[i], at);
                if (lane == at) key[i] = 0u;
            }
        }
        if (c == 0) top = l;
        const float p = expf(l - top);
        chosen += p;
        if (lane == c) { mine = p; ids[c] = pick; }
    }
    float sum = chosen;
    if (!renorm) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i < E) s += expf(v[i] - top);
        sum = __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(uint32_t, s), SumF32()));
    }
    if (lane < top_k) weights[lane] = mine / sum;
}

// ---------------------------------------------------------------------------
// expert products
// ---------------------------------------------------------------------------
struct ExpertArgs {
    const uint32_t* q[2];                          // gate and up, or down alone
    const _Float16 *s[2], *z[2];
    const _Float16 *hi, *lo;                       // operand planes [rows][K]; lo nullptr: hi is exact
    const float* logits;                           // gate/up
    int* ids;                                      // [M * top_k]: written by gate/up, read by down
    float* weights;
    _Float16* h;                                   // gate/up out: hi plane [assignments][N], then lo
    float* part;                                   // down out: fp32 [assignments][N]
    int M, E, top_k, renorm;
    int N, K;                                      // of one expert's layer
};

template <int BITS, int GS, int WK, int MT, bool GATEUP>
__global__ __launch_bounds__(64 * kMoeWaves, 2) void k_moe_experts(ExpertArgs a) {
    constexpr int WQ = BITS == 4 ? 4 : 3;
    constexpr int NL = GATEUP ? 2 : 1;             // layers per item
    constexpr int SUB = kMoeWaves / WK;            // items of a workgroup at a time
    constexpr int U = MT == 1 ? 4 : MT == 2 ? 2 : 1;
    constexpr int HR = GS == 64 ? 8 : 16;          // operand rows that differ (the rest: the other group)
    __shared__ Lists L;
    __shared__ float4_t red[SUB][WK][NL][MT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, hq = lane >> 4;
    const int sub = wave / WK, wk = wave % WK;
    const int assigned = a.M * a.top_k;

    if constexpr (GATEUP) {
        float* weights = reinterpret_cast<float*>(L.order);       // until the lists are built
        for (int m = wave; m < a.M; m += kMoeWaves)
            route_token(a.logits + (size_t)m * a.E, a.E, a.top_k, a.renorm, L.ids + m * a.top_k,
                        weights + m * a.top_k);
        __syncthreads();
        if (blockIdx.x == 0)
            for (int i = tid; i < assigned; i += 64 * kMoeWaves) {
                a.ids[i] = L.ids[i];
                a.weights[i] = weights[i];
            }
        __syncthreads();
    } else {
        for (int i = tid; i < assigned; i += 64 * kMoeWaves) L.ids[i] = a.ids[i];
        __syncthreads();
    }
    build_lists(L, assigned, a.E);

    const int G = a.K / kGroup, NB = (a.N + 15) / 16;
    const int hilo = a.lo ? 2 : 1;
    const int per_tile = HR / hilo;                // tokens of an operand tile
    const int nw = wk < G ? (G - wk + WK - 1) / WK : 0;
    const uint32_t tiles = (uint32_t)NB * (uint32_t)G;
    const uint32_t psh = 16u * (uint32_t)(j & 1);
    const uint32_t pgrp = GS == 64 ? (uint32_t)(hq >> 1) : 0u;
    // this lane's operand row: token slot, plane, and whether its quarter is the row's group
    const int jr = j % HR, slot = jr % per_tile;
    const bool low = jr >= per_tile;
    const bool mine = GS == 128 || (j >> 3) == (hq >> 1);
    const int total = L.n_active * NB;
    const int passes = (L.most + MT * per_tile - 1) / (MT * per_tile);

    for (int base = blockIdx.x * SUB; base < total; base += gridDim.x * SUB) {
        const int item = base + sub;
        const bool live = item < total;
        const int e = __builtin_amdgcn_readfirstlane(L.active[live ? item / NB : 0]);
        const int b = live ? item % NB : 0;
        const int cnt = __builtin_amdgcn_readfirstlane(L.count[e]), first = L.start[e];
        __amdgpu_buffer_rsrc_t rq[NL], rs[NL], rz[NL];
#pragma unroll
        for (int l = 0; l < NL; ++l) {
            const size_t params = (size_t)tiles * (16 * kGroup / GS);
            rq[l] = moe_rsrc(a.q[l] + (size_t)e * tiles * 64 * WQ, tiles * 64u * WQ * 4u);
            rs[l] = moe_rsrc(a.s[l] + (size_t)e * params, (uint32_t)(params * 2));
            rz[l] = moe_rsrc(a.z[l] + (size_t)e * params, (uint32_t)(params * 2));
        }
        for (int pass = 0; pass < passes; ++pass) {
            const int s0 = pass * MT * per_tile;   // first token slot of this pass
            const bool work = live && s0 < cnt;    // wave-uniform
            const _Float16* src[MT];
            bool on[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int s = s0 + t * per_tile + slot;
                on[t] = work && mine && s < cnt;
                const int as = L.order[first + (s < cnt ? s : 0)];
                const int row = GATEUP ? as / a.top_k : as;
                src[t] = (low ? a.lo : a.hi) + (size_t)row * a.K + 32 * hq;
            }
            TileSlot<WQ> w[U][NL];
            uint32_t pd[U][NL], pz[U][NL];
            half8_t x[U][MT][4];
            auto load = [&](int i, int u) {
                const bool ok = work && i < nw;
                const int g = wk + WK * i;
                const uint32_t t = (uint32_t)b * (uint32_t)G + (uint32_t)g;
                const uint32_t oq = ok ? (t * 64u + (uint32_t)lane) * (WQ * 4u) : kOutOfRange;
                const uint32_t op = ok ? ((t * (kGroup / GS) + pgrp) * 16u + (uint32_t)(j & ~1)) * 2u : kOutOfRange;
#pragma unroll
                for (int l = 0; l < NL; ++l) {
                    w[u][l] = load_tile_slot<WQ, 2>(rq[l], oq);
                    pd[u][l] = __builtin_amdgcn_raw_buffer_load_b32(rs[l], op, 0, 0);
                    pz[u][l] = __builtin_amdgcn_raw_buffer_load_b32(rz[l], op, 0, 0);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        half8_t v = {};
                        if (ok && on[m]) v = *reinterpret_cast<const half8_t*>(src[m] + (size_t)g * kGroup + 8 * q);
                        x[u][m][q] = v;
                    }
            };
            float4_t acc[NL][MT];
#pragma unroll
            for (int l = 0; l < NL; ++l)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[l][m] = (float4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < U; ++u) load(u, u);
            for (int i0 = 0; i0 < nw; i0 += U) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (i0 + u < nw) {             // wave-uniform
#pragma unroll
                        for (int l = 0; l < NL; ++l) {
                            half8_t bop[4];
                            exact_operands<BITS, WQ>(w[u][l], bits_half((uint16_t)(pz[u][l] >> psh)), bop);
                            const float d = (float)bits_half((uint16_t)(pd[u][l] >> psh));
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                float4_t g = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    g = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[u][m][q], bop[q], g, 0, 0, 0);
#pragma unroll
                                for (int r = 0; r < 4; ++r) acc[l][m][r] = __builtin_fmaf(d, g[r], acc[l][m][r]);
                            }
                        }
                    }
                    load(i0 + u + U, u);
                }
            }
#pragma unroll
            for (int l = 0; l < NL; ++l)
#pragma unroll
                for (int m = 0; m < MT; ++m) red[sub][wk][l][m][lane] = acc[l][m];
            __syncthreads();
            // token slot ts, column c: its operand rows over the WK waves, in a fixed order
            if (work) {
                const int n_here = min(MT * per_tile, cnt - s0);
                for (int i = wk * 64 + lane; i < n_here * 16; i += 64 * WK) {
                    const int ts = i >> 4, c = i & 15;
                    const int m = ts / per_tile, r0 = ts % per_tile;
                    float v[NL];
#pragma unroll
                    for (int l = 0; l < NL; ++l) {
                        float part[2] = {0.f, 0.f};                // hi, lo
                        for (int p = 0; p < hilo; ++p)
                            for (int g = 0; g < kGroup / GS; ++g) {
                                const int row = g * HR + p * per_tile + r0;
                                for (int q = 0; q < WK; ++q)
                                    part[p] += red[sub][q][l][m][(row >> 2) * 16 + c][row & 3];
                            }
                        v[l] = part[0] + part[1] * (1.0f / kLoScale);
                    }
                    const int n = 16 * b + c;
                    const size_t at = (size_t)L.order[first + s0 + ts] * a.N + n;
                    if constexpr (GATEUP) {
                        const float hv = v[0] / (1.0f + expf(-v[0])) * v[1];
                        split_hi_lo(hv, a.h[at], a.h[(size_t)assigned * a.N + at]);
                    } else {
                        a.part[at] = v[0];
                    }
                }
            }
            __syncthreads();
        }
    }
}

__global__ __launch_bounds__(256) void k_moe_join(const float* part, const float* weights, _Float16* y, int top_k,
                                                  int K) {
    const int k = blockIdx.x * 256 + threadIdx.x;
    const size_t m = blockIdx.y;
    if (k >= K) return;
    float sum = 0.0f;
    for (int c = 0; c < top_k; ++c)
        sum = __builtin_fmaf(weights[m * top_k + c], part[(m * top_k + c) * K + k], sum);
    y[m * K + k] = (_Float16)sum;
}

using ExpertFn = void (*)(ExpertArgs);

template <int BITS, int GS, bool GATEUP, int WK>
ExpertFn pick_mt(int mt) {
    return mt == 1 ? k_moe_experts<BITS, GS, WK, 1, GATEUP>
                   : mt == 2 ? k_moe_experts<BITS, GS, WK, 2, GATEUP> : k_moe_experts<BITS, GS, WK, 4, GATEUP>;
}

template <int BITS, int GS, bool GATEUP>
int launch_experts(const ExpertArgs& a, hipStream_t st) {
    const int G = a.K / kGroup, NB = (a.N + 15) / 16;
    const int most_active = min(a.M * a.top_k, a.E);
    const int cus = device_cu_count();
    // waves of an item: 8 where a wave still has 4 tiles, else fewer
    const int wk = G >= 32 ? 8 : G >= 8 ? 4 : 1;
    // operand tiles: of an even share of the tokens per expert, twice over
    const int rows_per_token = (a.lo ? 2 : 1) * (GS == 64 ? 2 : 1);
    const int share = min(a.M, 2 * ((a.M * a.top_k + a.E - 1) / a.E));
    const int mt = share * rows_per_token <= 16 ? 1 : share * rows_per_token <= 32 ? 2 : 4;
    ExpertFn kern = wk == 8 ? pick_mt<BITS, GS, GATEUP, 8>(mt)
                            : wk == 4 ? pick_mt<BITS, GS, GATEUP, 4>(mt) : pick_mt<BITS, GS, GATEUP, 1>(mt);
    const int sub = kMoeWaves / wk;
    const int grid = min(2 * cus, (most_active * NB + sub - 1) / sub);
    hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * kMoeWaves), 0, st, a);
    return (int)hipGetLastError();
}

template <bool GATEUP>
int launch_experts_any(const ExpertArgs& a, int bits, int group_size, hipStream_t st) {
    if (group_size == 64)
        return bits == 4 ? launch_experts<4, 64, GATEUP>(a, st) : launch_experts<3, 64, GATEUP>(a, st);
    return bits == 4 ? launch_experts<4, 128, GATEUP>(a, st) : launch_experts<3, 128, GATEUP>(a, st);
}

// the workspace's parts, each 256-byte aligned
struct Workspace {
    size_t logits, ids, weights, h, part, scaled, bytes;
    Workspace(int M, int K, int I, int E, int top_k) {
        size_t at = 0;
        auto take = [&](size_t n) {
            const size_t here = at;
            at += (n + 255) / 256 * 256;
            return here;
        };
        const size_t as = (size_t)M * top_k;
        logits = take((size_t)M * E * 4);
        ids = take(as * 4);
        weights = take(as * 4);
        h = take(as * I * 4);
        part = take(as * K * 4);
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
    const RouterArgs r{(const _Float16*)p.x, (const _Float16*)p.router, p.inv_s, (float*)(ws + w.logits), scaled,
                       p.M, p.E, p.K};
    hipLaunchKernelGGL(k_moe_router, dim3((p.E + 15) / 16, (p.M + 15) / 16), dim3(1024), 0, st, r);
    if (int e = (int)hipGetLastError()) return e;

    ExpertArgs a{};
    for (int l = 0; l < 2; ++l) {
        a.q[l] = (const uint32_t*)p.qweight[l];
        a.s[l] = (const _Float16*)p.scales[l];
        a.z[l] = (const _Float16*)p.zeros[l];
    }
    a.hi = p.inv_s ? scaled : (const _Float16*)p.x;
    a.lo = p.inv_s ? scaled + (size_t)p.M * p.K : nullptr;
    a.logits = r.logits;
    a.ids = (int*)(ws + w.ids);
    a.weights = (float*)(ws + w.weights);
    a.h = (_Float16*)(ws + w.h);
    a.M = p.M; a.E = p.E; a.top_k = p.top_k; a.renorm = p.renormalize;
    a.N = p.I; a.K = p.K;
    if (int e = launch_experts_any<true>(a, p.bits, p.group_size, st)) return e;

    a.q[0] = (const uint32_t*)p.qweight[2];
    a.s[0] = (const _Float16*)p.scales[2];
    a.z[0] = (const _Float16*)p.zeros[2];
    a.hi = a.h;
    a.lo = a.h + (size_t)p.M * p.top_k * p.I;
    a.part = (float*)(ws + w.part);
    a.N = p.K; a.K = p.I;
    if (int e = launch_experts_any<false>(a, p.bits, p.group_size, st)) return e;
    hipLaunchKernelGGL(k_moe_join, dim3((p.K + 255) / 256, p.M), dim3(256), 0, st, a.part, a.weights,
                       (_Float16*)p.y, p.top_k, p.K);
    return (int)hipGetLastError();
}

}  // namespace awq
