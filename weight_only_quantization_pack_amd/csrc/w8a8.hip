// Products in 8-bit integers with one scale for each token and each channel:
//   y[m][n] = sx[m] * sw[n] * sum_k x[m][k] * w[n][k]  (+ bias[n])
// x int8 [M][K] (codes of the row quantizer), w int8 [N][K], both row-major;
// the sum is exact in int32 (K < 2^17), the scales and the bias are fp32, and
// y is rounded once to fp16 or bf16.
//
// v_mfma_i32_16x16x64_i8 takes 16 k of 16 rows per lane quarter: lane (j, h)
// holds row j, k = 16 h .. 16 h + 15 -- one aligned 16-byte chunk of a
// row-major row, so neither operand needs repacking.  The weights are the A
// operand: accumulator register r of lane (j, h) is then row m = j and column
// n = 4 h + r, four consecutive outputs.
#include "rows.h"

namespace awq {
namespace {

constexpr int kStep = 128;                         // k per step: one 128-byte line of every row
constexpr uint32_t kOutOfRange = 0x80000000u;      // > every buffer's size: loads return zero

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p, size_t bytes) {
    const uint32_t n = bytes < 0x7FFFFFFFull ? (uint32_t)bytes : 0x7FFFFFFFu;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)n, 0x00020000);
}

__device__ __forceinline__ int4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(int4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
// weights of a product with few rows are read once: non-temporal
__device__ __forceinline__ int4_t load16_nt(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(int4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 2));
}

// 16 bytes per lane from buffer offset voff + soff to LDS at lds + 16 * lane
__device__ __forceinline__ void load16_lds(__amdgpu_buffer_rsrc_t r, unsigned char* lds, uint32_t voff,
                                           uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)lds, 16, voff, soff, 0, 0);
}

struct Args {
    const int8_t* x;                               // codes, or (FUSED) nullptr
    const uint4* rows;                             // FUSED: 16-bit rows [M][K / 8] chunks
    const float* sx;
    const int8_t* w;
    const float *sw, *bias;
    uint16_t* y;
    int* part;                                     // split K: int32 [splits][M][N], else nullptr
    int M, N, K, steps;                            // steps of this split (blockIdx.y)
};

// four consecutive outputs n .. n + 3 of row m
template <class E>
__device__ __forceinline__ void store4(const Args& a, int m, int n, int4_t acc, float sx) {
    if (a.part) {
        int* p = a.part + ((size_t)blockIdx.y * a.M + m) * a.N + n;
        if (n + 3 < a.N && (a.N & 3) == 0) {
            *reinterpret_cast<int4_t*>(p) = acc;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < a.N) p[r] = acc[r];
        }
        return;
    }
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int c = min(n + r, a.N - 1);
        v[r] = (float)acc[r] * (sx * a.sw[c]) + (a.bias ? a.bias[c] : 0.0f);
    }
    uint16_t* p = a.y + (size_t)m * a.N + n;
    if (n + 3 < a.N && (a.N & 3) == 0) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2<E>(v[0], v[1]), pack2<E>(v[2], v[3]));
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < a.N) p[r] = E::store(v[r]);
    }
}

// ---------------------------------------------------------------------------
// Few rows (M <= 64): HBM-bound on the weights, each read once.  A workgroup
// of 8 waves owns 16 NBW columns and all rows; its waves take the K steps in
// turn, each through a ring of U steps in flight, and their exact int32 sums
// meet in LDS.
//
// FUSED (few 16-bit rows that fit in registers): the workgroup quantizes the
// rows itself, behind its first weight loads, and keeps the codes in LDS.
// ---------------------------------------------------------------------------
constexpr int kWaves = 8;
constexpr int kFusedChunks = 8;                    // 16-byte chunks of x a thread quantizes at most

template <class E, int MT, int NBW, int U, bool FUSED>
__global__ __launch_bounds__(64 * kWaves, 2) void k_w8a8_few(Args a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    __shared__ uint32_t slots[kWaves];
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = tid >> 6;
    const int j = lane & 15, h = lane >> 4;
    const int n0 = blockIdx.x * 16 * NBW;
    const int total = (a.K + kStep - 1) / kStep;
    const int k0 = blockIdx.y * a.steps;
    const int mine = min(total - k0, a.steps);     // steps of this split
    const int nw = wave < mine ? (mine - wave + kWaves - 1) / kWaves : 0;
    const size_t K = (size_t)a.K;

    const __amdgpu_buffer_rsrc_t rw =
        make_rsrc(a.w + (size_t)n0 * K, (size_t)min(16 * NBW, a.N - n0) * K);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, FUSED ? 0 : (size_t)a.M * K);

    int4_t w[U][NBW][2], x[FUSED ? 1 : U][MT][2];
    auto load = [&](int i, int u) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = (k0 + wave + kWaves * i) * kStep + 64 * s + 16 * h;
            const bool ok = i < nw && k < a.K;
#pragma unroll
            for (int b = 0; b < NBW; ++b)          // rows past N are past the buffer's end
                w[u][b][s] = load16_nt(rw, ok ? (uint32_t)(16 * b + j) * (uint32_t)a.K + (uint32_t)k : kOutOfRange);
            if constexpr (!FUSED) {
#pragma unroll
                for (int t = 0; t < MT; ++t)       // as are rows past M
                    x[u][t][s] = load16(rx, ok ? (uint32_t)(16 * t + j) * (uint32_t)a.K + (uint32_t)k : kOutOfRange);
            }
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, u);

    // FUSED: 1, 2 or 4 rows (MP), 8 / MP waves a row
    float* sxs = reinterpret_cast<float*>(slots);
    const int xstride = (a.K + kStep - 1) / kStep * kStep + 16;
    if constexpr (FUSED) {
        const int MP = a.M > 2 ? 4 : a.M;
        const int per = 64 * kWaves / MP;          // threads per row
        const int row = tid / per, t = tid - row * per;
        const int chunks = a.K / 8;
        uint4 r[kFusedChunks];
#pragma unroll
        for (int c = 0; c < kFusedChunks; ++c) {
            const int i = t + per * c;
            r[c] = row < a.M && i < chunks ? a.rows[(size_t)row * chunks + i] : make_uint4(0, 0, 0, 0);
        }
        float v[8];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < kFusedChunks; ++c) {
            unpack8<E>(r[c], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[e]));
        }
        top = wave_reduce(top, MaxU32());
        if (lane == 0) slots[wave] = top;
        __syncthreads();
        const int wpr = kWaves / MP;
        top = 0;
        for (int q = 0; q < wpr; ++q) top = max(top, slots[row * wpr + q]);
        const RowScale s(top);
        unsigned char* xr = smem + row * xstride;
#pragma unroll
        for (int c = 0; c < kFusedChunks; ++c) {
            const int i = t + per * c;
            // steps end past K: the chunks there are zero
            if (row < a.M && i < (xstride - 16) / 8) {
                unpack8<E>(r[c], v);
                *reinterpret_cast<uint2*>(xr + 8 * i) = pack_codes8(v, s);
            }
        }
        __syncthreads();                           // codes complete, slots read
        if (t == 0) sxs[row] = s.scale();
    }

    int4_t acc[MT][NBW];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int b = 0; b < NBW; ++b) acc[t][b] = (int4_t){0, 0, 0, 0};

    for (int i0 = 0; i0 < nw; i0 += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u < nw) {                     // wave-uniform
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        int4_t xv;
                        if constexpr (FUSED)
                            xv = *reinterpret_cast<const int4_t*>(
                                smem + (j < a.M ? j : 0) * xstride + (k0 + wave + kWaves * (i0 + u)) * kStep +
                                64 * s + 16 * h);
                        else
                            xv = x[u][t][s];
#pragma unroll
                        for (int b = 0; b < NBW; ++b)
                            acc[t][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][b][s], xv, acc[t][b], 0, 0, 0);
                    }
            }
            load(i0 + u + U, u);
        }
    }

    // the waves' sums, [wave][tile][lane]
    float sx[MT];
    __syncthreads();                               // every read of the codes is done
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int m = 16 * t + j;
        sx[t] = a.part || m >= a.M ? 0.0f : FUSED ? sxs[m] : a.sx[m];
    }
    int4_t* red = reinterpret_cast<int4_t*>(smem);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int b = 0; b < NBW; ++b) red[(wave * MT * NBW + t * NBW + b) * 64 + lane] = acc[t][b];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int b = 0; b < NBW; ++b) {
            const int tile = t * NBW + b;
            if (tile % kWaves != wave) continue;
            int4_t sum = red[tile * 64 + lane];
#pragma unroll
            for (int q = 1; q < kWaves; ++q) sum += red[(q * MT * NBW + tile) * 64 + lane];
            const int m = 16 * t + j, n = n0 + 16 * b + 4 * h;
            if (m < a.M && n < a.N) store4<E>(a, m, n, sum, sx[t]);
        }
}

// ---------------------------------------------------------------------------
// Many rows: both operands through LDS, TM x TN output tiles.
// ---------------------------------------------------------------------------
template <class E, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_w8a8_tile(Args a) {
    constexpr int WV = WM * WN;
    constexpr int FM = TM / WM / 16, FN = TN / WN / 16;      // 16-row fragments of a wave
    constexpr int XI = TM / 8 / WV, WI = TN / 8 / WV;        // 8-row loads of a wave per step
    constexpr int XB = TM * kStep, BUF = (TM + TN) * kStep;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, h = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const int nTn = (a.N + TN - 1) / TN;
    const int m0 = (int)blockIdx.x / nTn * TM, n0 = (int)blockIdx.x % nTn * TN;
    const int total = (a.K + kStep - 1) / kStep;
    const int k0 = blockIdx.y * a.steps;
    const int steps = min(total - k0, a.steps);
    const size_t K = (size_t)a.K;

    const int mrows = min(TM, a.M - m0), nrows = min(TN, a.N - n0);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (size_t)m0 * K, (size_t)mrows * K);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (size_t)n0 * K, (size_t)nrows * K);

    // A load instruction fills 8 rows: lane l writes chunk l & 7 of row
    // l >> 3, which holds the row's global chunk (l & 7) ^ (l >> 3), so that
    // the fragment reads of 16 rows spread over the banks
    const int lr = lane >> 3, kc = (lane & 7) ^ lr;
    uint32_t xoff[XI], woff[WI];
#pragma unroll
    for (int i = 0; i < XI; ++i)
        xoff[i] = (uint32_t)min(8 * (wave * XI + i) + lr, mrows - 1) * (uint32_t)a.K + 16u * kc;
#pragma unroll
    for (int i = 0; i < WI; ++i)
        woff[i] = (uint32_t)min(8 * (wave * WI + i) + lr, nrows - 1) * (uint32_t)a.K + 16u * kc;
    auto issue = [&](int kt, int buf) {
        const uint32_t at = (uint32_t)(k0 + kt) * kStep;
        const bool ok = (int)at + 16 * kc < a.K;
        unsigned char* xb = smem + buf * BUF;
#pragma unroll
        for (int i = 0; i < XI; ++i)
            load16_lds(rx, xb + (wave * XI + i) * 1024, ok ? xoff[i] : kOutOfRange, at);
#pragma unroll
        for (int i = 0; i < WI; ++i)
            load16_lds(rw, xb + XB + (wave * WI + i) * 1024, ok ? woff[i] : kOutOfRange, at);
    };

    int4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int c = 0; c < FN; ++c) acc[i][c] = (int4_t){0, 0, 0, 0};

    issue(0, 0);
    for (int kt = 0; kt < steps; ++kt) {
        const int buf = kt & 1;
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();                           // step kt is in LDS; the other buffer is free
        if (kt + 1 < steps) issue(kt + 1, buf ^ 1);
        const unsigned char* xb = smem + buf * BUF + (wm * FM * 16 + j) * kStep;
        const unsigned char* wb = smem + buf * BUF + XB + (wn * FN * 16 + j) * kStep;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int p = ((4 * s + h) ^ (j & 7)) * 16;
            int4_t wv[FN];
#pragma unroll
            for (int c = 0; c < FN; ++c) wv[c] = *reinterpret_cast<const int4_t*>(wb + c * 16 * kStep + p);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int4_t xv = *reinterpret_cast<const int4_t*>(xb + i * 16 * kStep + p);
#pragma unroll
                for (int c = 0; c < FN; ++c)
                    acc[i][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[c], xv, acc[i][c], 0, 0, 0);
            }
        }
    }

#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + (wm * FM + i) * 16 + j;
        if (m >= a.M) continue;
        const float sx = a.part ? 0.0f : a.sx[m];
#pragma unroll
        for (int c = 0; c < FN; ++c) {
            const int n = n0 + (wn * FN + c) * 16 + 4 * h;
            if (n < a.N) store4<E>(a, m, n, acc[i][c], sx);
        }
    }
}

// split K: the splits' exact sums, then the scales
template <class E>
__global__ __launch_bounds__(256) void k_w8a8_join(Args a, int splits) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, total = (size_t)a.M * a.N;
    if (i >= total) return;
    int sum = 0;
    for (int s = 0; s < splits; ++s) sum += a.part[(size_t)s * total + i];
    const int m = (int)(i / a.N), n = (int)(i - (size_t)m * a.N);
    const float v = (float)sum * (a.sx[m] * a.sw[n]) + (a.bias ? a.bias[n] : 0.0f);
    a.y[i] = E::store(v);
}

// how a product is cut: the tile kernel and the K splits
struct Plan {
    int few;                                       // k_w8a8_few
    int mt, nbw;                                   // its row tiles and column blocks
    int blocks, splits, steps;                     // workgroups per split, splits, steps of each
};

Plan plan(int M, int N, int K) {
    Plan p{};
    const int cus = device_cu_count();
    const int total = (K + kStep - 1) / kStep;
    p.few = M <= 64;
    if (p.few) {
        p.mt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
        p.nbw = 1;
        p.blocks = (N + 16 * p.nbw - 1) / (16 * p.nbw);
    } else {
        p.blocks = ((M + 255) / 256) * ((N + 255) / 256);
    }
    p.splits = 1;
    p.steps = total;
    // fewer workgroups than compute units: cut K while a split keeps 16 steps
    if (p.blocks < cus) {
        int s = cus / p.blocks;
        s = min(s, total / 16);
        if (s > 1) {
            p.steps = (total + s - 1) / s;
            p.splits = (total + p.steps - 1) / p.steps;
        }
    }
    return p;
}

template <class E, int MT, int NBW, int U, bool FUSED>
int launch_few(const Args& a, const Plan& p, hipStream_t st) {
    const size_t red = (size_t)kWaves * MT * NBW * 64 * 16;
    const size_t codes = FUSED ? (size_t)a.M * ((size_t)(a.K + kStep - 1) / kStep * kStep + 16) : 0;
    const size_t lds = max(red, codes);
    auto kern = k_w8a8_few<E, MT, NBW, U, FUSED>;
    if (lds > 64 * 1024)
        if (int e = (int)hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds))
            return e;
    hipLaunchKernelGGL(kern, dim3(p.blocks, p.splits), dim3(64 * kWaves), lds, st, a);
    return (int)hipGetLastError();
}

template <class E, int TM, int TN, int WM, int WN>
int launch_tile(const Args& a, const Plan& p, hipStream_t st) {
    constexpr size_t lds = 2 * (TM + TN) * kStep;
    auto kern = k_w8a8_tile<E, TM, TN, WM, WN>;
    if (int e = (int)hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                         hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds))
        return e;
    hipLaunchKernelGGL(kern, dim3(p.blocks, p.splits), dim3(64 * WM * WN), lds, st, a);
    return (int)hipGetLastError();
}

template <class E>
int launch_t(Args a, const Plan& p, hipStream_t st) {
    int e;
    if (a.rows) e = launch_few<E, 1, 1, 4, true>(a, p, st);
    else if (p.few && p.mt == 1) e = launch_few<E, 1, 1, 4, false>(a, p, st);
    else if (p.few && p.mt == 2) e = launch_few<E, 2, 1, 4, false>(a, p, st);
    else if (p.few) e = launch_few<E, 4, 1, 2, false>(a, p, st);
    else e = launch_tile<E, 256, 256, 2, 4>(a, p, st);
    if (e || !a.part) return e;
    const size_t total = (size_t)a.M * a.N;
    hipLaunchKernelGGL((k_w8a8_join<E>), dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, a, p.splits);
    return (int)hipGetLastError();
}

// the decode product quantizes its rows itself
bool fused_rows(const Plan& p, int M, int K) {
    return p.few && p.splits == 1 && M <= 4 && (M == 3 ? 4 : M) * (K / 8) <= kFusedChunks * 64 * kWaves;
}

size_t align16(size_t v) { return (v + 15) & ~(size_t)15; }

}  // namespace

size_t w8a8_workspace_bytes(int M, int N, int K) {
    const Plan p = plan(M, N, K);
    return p.splits > 1 ? (size_t)p.splits * M * N * 4 : 0;
}

size_t linear_w8a8_workspace_bytes(int M, int N, int K) {
    if (fused_rows(plan(M, N, K), M, K)) return 0;
    return align16((size_t)M * K) + align16((size_t)M * 4) + w8a8_workspace_bytes(M, N, K);
}

int launch_w8a8(const W8a8Problem& p, void* workspace, hipStream_t st) {
    const Plan pl = plan(p.M, p.N, p.K);
    Args a{};
    a.w = (const int8_t*)p.weight;
    a.sw = p.weight_scales;
    a.bias = p.bias;
    a.y = (uint16_t*)p.y;
    a.M = p.M; a.N = p.N; a.K = p.K;
    a.steps = pl.steps;
    unsigned char* ws = (unsigned char*)workspace;
    if (p.rows && fused_rows(pl, p.M, p.K)) {
        a.rows = (const uint4*)p.rows;
    } else if (p.rows) {
        float* sx = (float*)(ws + align16((size_t)p.M * p.K));
        if (int e = launch_quantize_rows(p.rows, p.M, p.K, p.dtype, ws, sx, st)) return e;
        a.x = (const int8_t*)ws;
        a.sx = sx;
        ws = (unsigned char*)sx + align16((size_t)p.M * 4);
    } else {
        a.x = (const int8_t*)p.x;
        a.sx = p.x_scales;
    }
    a.part = pl.splits > 1 ? (int*)ws : nullptr;
    return p.dtype == AWQ_BF16 ? launch_t<BF16>(a, pl, st) : launch_t<F16>(a, pl, st);
}

}  // namespace awq
