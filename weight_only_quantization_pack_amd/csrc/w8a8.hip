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
//
// Sizes below are M x N x K, or N x K of the weights.
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

// p[n .. n + 3], entries past the last one repeated
__device__ __forceinline__ float4_t load4(const float* p, int n, int N) {
    if (n + 3 < N) return (float4_t){p[n], p[n + 1], p[n + 2], p[n + 3]};
    return (float4_t){p[min(n, N - 1)], p[min(n + 1, N - 1)], p[min(n + 2, N - 1)], p[min(n + 3, N - 1)]};
}

// four consecutive outputs n .. n + 3 of row m
template <class E>
__device__ __forceinline__ void store4(const Args& a, int m, int n, int4_t acc, float sx, float4_t sw, float4_t bias) {
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
    for (int r = 0; r < 4; ++r) v[r] = (float)acc[r] * (sx * sw[r]) + bias[r];
    uint16_t* p = a.y + (size_t)m * a.N + n;
    if (n + 3 < a.N && (a.N & 3) == 0) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2<E>(v[0], v[1]), pack2<E>(v[2], v[3]));
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < a.N) p[r] = E::store(v[r]);
    }
}

// Outputs leave through LDS: a wave turns ROWS rows of COLS columns there (row
// r at stage + r * 2 COLS, its 16-byte chunks XOR-ed by row_xor(r)) and stores
// them from row m0, column n0 on -- 16 bytes a lane where the rows of y are
// 16-byte aligned (N a multiple of 8), else two bytes a lane along a row
// (1123 x 768 x 20369: 74 us with four scattered two-byte stores a lane).
template <int COLS>
__device__ __forceinline__ int row_xor(int r) { return COLS == 64 ? r & 7 : (r >> 1) & 3; }

template <class E, int COLS>
__device__ __forceinline__ void stage4(unsigned char* stage, int r, int col, int4_t acc, float sx, float4_t sw,
                                       float4_t bias) {
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = (float)acc[q] * (sx * sw[q]) + bias[q];
    *reinterpret_cast<uint2*>(stage + r * (2 * COLS) + (((col >> 3) ^ row_xor<COLS>(r)) << 4) + (col & 4) * 2) =
        make_uint2(pack2<E>(v[0], v[1]), pack2<E>(v[2], v[3]));
}

template <int ROWS, int COLS>
__device__ __forceinline__ void store_rows(const Args& a, const unsigned char* stage, int m0, int n0) {
    const int lane = threadIdx.x & 63;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");       // the wave's own writes
    if ((a.N & 7) == 0) {
        constexpr int CH = COLS / 8, RI = 64 / CH;           // chunks of a row, rows of a store
#pragma unroll
        for (int g = 0; g < ROWS / RI; ++g) {
            const int r = RI * g + lane / CH, c = lane % CH;
            const uint4 o = *reinterpret_cast<const uint4*>(stage + r * (2 * COLS) + ((c ^ row_xor<COLS>(r)) << 4));
            if (m0 + r < a.M && n0 + 8 * c < a.N)
                *reinterpret_cast<uint4*>(a.y + (size_t)(m0 + r) * a.N + n0 + 8 * c) = o;
        }
    } else {
        constexpr int RI = 64 / COLS, AT = 8;                // rows of a store, stores at a time
        const int c = lane % COLS;
        uint16_t* y = a.y + (size_t)(m0 + lane / COLS) * a.N + n0 + c;
        const bool in = n0 + c < a.N;
#pragma unroll
        for (int g0 = 0; g0 < ROWS / RI; g0 += AT) {
            uint16_t o[AT];
#pragma unroll
            for (int g = 0; g < AT; ++g) {
                const int r = RI * (g0 + g) + lane / COLS;
                o[g] = *reinterpret_cast<const uint16_t*>(stage + r * (2 * COLS) +
                                                          (((c >> 3) ^ row_xor<COLS>(r)) << 4) + (c & 7) * 2);
            }
#pragma unroll
            for (int g = 0; g < AT; ++g) {
                if (in && m0 + RI * (g0 + g) + lane / COLS < a.M) *y = o[g];
                y += (size_t)RI * a.N;
            }
        }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");       // read before the next rows are written
}

// Workgroup id -> output tile.  Ids go round-robin over the 8 XCDs: XCD x takes
// a contiguous run of the tile sequence, which walks column by column through
// bands of 8 tile rows, so that the tiles an XCD runs at once share operand
// rows and columns in its L2.
__device__ __forceinline__ void tile_of(int id, int nTm, int nTn, int& tm, int& tn) {
    const int nT = nTm * nTn, q = nT / 8, r = nT % 8, xcd = id & 7;
    const int t = xcd * q + min(xcd, r) + (id >> 3);
    constexpr int BAND = 8;
    const int band = t / (BAND * nTn), in = t - band * (BAND * nTn);
    const int rows = min(BAND, nTm - band * BAND);
    tm = band * BAND + in % rows;
    tn = in / rows;
}

// ---------------------------------------------------------------------------
// Up to 4 rows: HBM-bound on the weights, each read once.  No matrix
// instruction: a lane multiplies 16 codes of a weight row with four
// v_dot4_i32_i8, so a wave reads 1 KB of one row at a time (the matrix operand
// takes 64 bytes of 16 rows: 4096 x 11008 at M = 1 / 4 14.5 / 14.8 us).  A wave
// owns R columns, whose steps of 1024 k share each read of x from LDS, U steps
// in flight; the lanes' exact sums are added at the end.
//
// What a workgroup does before its first product counts: the codes go direct to
// LDS, asked for before the weights, since loads return in order (4096 x 11008
// at M = 1 / 4: 12.3 us, 3.7 TB/s / 13.4 us, 13.2 / 17.9 with codes through
// registers behind the weights).  R = 2 keeps two workgroups on a compute unit
// there (R = 4: 14.5 at M = 4).  Codes of more than 64 KB are split along K
// (28672 x 20480 at M = 4: 110 us, 119 on 16-row operands).
//
// FUSED (one or two 16-bit rows that fit in registers): the workgroup quantizes
// the rows itself (4096 x 11008 at M = 1: 12.2 us, 15.7 with a launch of its own;
// 4 rows of 4096 x 4096: 9.1 and 9.4, so only up to two).
// ---------------------------------------------------------------------------
constexpr int kWaves = 4;
constexpr int kRowStep = 1024;                     // k of a wave's load
constexpr int kRowLds = 64 * 1024;                 // codes of a split, at most
constexpr int kFusedRows = 2;
constexpr int kFusedChunks = 8;                    // 16-byte chunks of x a thread quantizes at most
constexpr int kRowColumns = 2;                     // of a wave

__device__ __forceinline__ int sum_lanes(int v) {
    struct Add {
        __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a + b; }
    };
    return (int)wave_reduce((uint32_t)v, Add());
}

template <class E, int MR, bool FUSED>
__global__ __launch_bounds__(64 * kWaves, 4) void k_w8a8_row(Args a) {
    constexpr int R = kRowColumns, U = 4;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    __shared__ uint32_t slots[kWaves];
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = ((int)blockIdx.x * kWaves + wave) * R;
    const int kb = blockIdx.y * a.steps * kStep, ke = min(a.K, kb + a.steps * kStep);      // of this split
    const int steps = (ke - kb + kRowStep - 1) / kRowStep, stride = steps * kRowStep;
    const size_t K = (size_t)a.K;
    // the size in a scalar register: a descriptor in vector registers costs every load a loop
    const int columns = __builtin_amdgcn_readfirstlane(max(0, min(R, a.N - n0)));
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (size_t)min(n0, a.N - 1) * K, (size_t)columns * K);
    int4_t w[U][R];
    auto load = [&](int step, int u) {
        const int k = kb + step * kRowStep + 16 * lane;
#pragma unroll
        for (int r = 0; r < R; ++r) w[u][r] = load16(rw, k < ke ? (uint32_t)r * (uint32_t)a.K + (uint32_t)k : kOutOfRange);
    };
    // The codes [MR][stride], first: loads return in order, and the weights take
    // longer.  What lies past the split's end meets zero weights.
    constexpr int WPR = kWaves / MR, per = 64 * WPR;         // waves and threads of a row
    const int row = wave / WPR, t = tid - row * per;
    const int chunks = a.K / 8;
    uint4 x[kFusedChunks];
    if constexpr (FUSED) {
#pragma unroll
        for (int c = 0; c < kFusedChunks; ++c) {
            const int i = t + per * c;
            x[c] = row < a.M && i < chunks ? a.rows[(size_t)row * chunks + i] : make_uint4(0, 0, 0, 0);
        }
    } else {
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, (size_t)a.M * K);
#pragma unroll
        for (int m = 0; m < MR; ++m)
            for (int i = wave; i < steps; i += kWaves) {
                const int k = kb + i * kRowStep + 16 * lane;
                load16_lds(rx, smem + m * stride + i * kRowStep,
                           k < ke ? (uint32_t)m * (uint32_t)a.K + (uint32_t)k : kOutOfRange, 0);
            }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, u);
    __builtin_amdgcn_sched_barrier(0);
    float sx[MR];
    if constexpr (FUSED) {
        float v[8];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < kFusedChunks; ++c) {
            if (per * c >= chunks) continue;       // uniform
            unpack8<E>(x[c], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[e]));
        }
        top = wave_reduce(top, MaxU32());
        if (lane == 0) slots[wave] = top;
        __syncthreads();
        uint32_t tops[MR];
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            tops[m] = slots[m * WPR];
#pragma unroll
            for (int q = 1; q < WPR; ++q) tops[m] = max(tops[m], slots[m * WPR + q]);
            sx[m] = RowScale(tops[m]).scale();
            if (m == row) top = tops[m];
        }
        const RowScale s(top);
#pragma unroll
        for (int c = 0; c < kFusedChunks; ++c) {
            const int i = t + per * c;
            if (per * c < chunks && i < chunks) {
                unpack8<E>(x[c], v);
                *reinterpret_cast<uint2*>(smem + row * stride + 8 * i) = pack_codes8(v, s);
            }
        }
        __syncthreads();
    } else {
        // the codes have landed, the weights need not have
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(U * R));
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MR; ++m) sx[m] = a.part ? 0.0f : a.sx[min(m, a.M - 1)];
    }

    int acc[MR][R] = {};
    for (int i0 = 0; i0 < steps; i0 += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u < steps) {                  // wave-uniform
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    const int4_t x = *reinterpret_cast<const int4_t*>(smem + m * stride + (i0 + u) * kRowStep + 16 * lane);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[m][r] = __builtin_amdgcn_sdot4(w[u][r][q], x[q], acc[m][r], false);
                }
            }
            load(i0 + u + U, u);
        }
    }
    // lane R m + r keeps the sum of row m and column n0 + r
    int sum = 0;
    float scale = 0.0f;
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int v = sum_lanes(acc[m][r]);
            if (lane == R * m + r) { sum = v; scale = sx[m]; }
        }
    const int m = lane / R, n = n0 + lane % R;
    if (m >= a.M || lane >= MR * R || n >= a.N) return;
    if (a.part) {
        a.part[((size_t)blockIdx.y * a.M + m) * a.N + n] = sum;
    } else {
        const float v = (float)sum * (scale * a.sw[n]) + (a.bias ? a.bias[n] : 0.0f);
        a.y[(size_t)m * a.N + n] = E::store(v);
    }
}

// ---------------------------------------------------------------------------
// 5 to 16 rows of a short product (4096 x 4096 at M = 16: 7.5 us, 2.2 TB/s): a
// workgroup of 4 waves owns 16 columns; its waves take the K steps in turn, each
// through a ring of U steps in flight with the codes straight from L2, and their
// exact int32 sums meet in LDS.
// ---------------------------------------------------------------------------
template <class E, int U>
__global__ __launch_bounds__(64 * kWaves, 4) void k_w8a8_few(Args a) {
    __shared__ int4_t red[kWaves][64];
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = tid >> 6;
    const int j = lane & 15, h = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int total = (a.K + kStep - 1) / kStep;
    const int k0 = blockIdx.y * a.steps;
    const int mine = min(total - k0, a.steps);     // steps of this split
    const int nw = wave < mine ? (mine - wave + kWaves - 1) / kWaves : 0;
    const size_t K = (size_t)a.K;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (size_t)n0 * K, (size_t)min(16, a.N - n0) * K);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, (size_t)a.M * K);

    int4_t w[U][2], x[U][2];
    auto load = [&](int i, int u) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = (k0 + wave + kWaves * i) * kStep + 64 * s + 16 * h;
            // rows past N or M are past the buffers' ends
            const uint32_t off = i < nw && k < a.K ? (uint32_t)j * (uint32_t)a.K + (uint32_t)k : kOutOfRange;
            w[u][s] = load16(rw, off);
            x[u][s] = load16(rx, off);
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, u);
    int4_t acc = {0, 0, 0, 0};
    for (int i0 = 0; i0 < nw; i0 += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u < nw) {                     // wave-uniform
#pragma unroll
                for (int s = 0; s < 2; ++s) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][s], x[u][s], acc, 0, 0, 0);
            }
            load(i0 + u + U, u);
        }
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int q = 1; q < kWaves; ++q) acc += red[q][lane];
    const int n = n0 + 4 * h;
    if (j < a.M && n < a.N)
        store4<E>(a, j, n, acc, a.part ? 0.0f : a.sx[j], load4(a.sw, n, a.N),
                  a.bias ? load4(a.bias, n, a.N) : (float4_t){0.f, 0.f, 0.f, 0.f});
}

// ---------------------------------------------------------------------------
// A decode batch (up to 64 rows): HBM-bound on the weights.  A workgroup of WV
// waves owns 16 WV columns, one block of 16 per wave over the whole K (or one
// split of it).  Both operands go direct to LDS in whole 128-byte lines, S steps
// of 256 k in flight; a wave waits for its own weights, and for everybody's part
// of the codes, which all waves share (without sharing them a workgroup moves as
// many bytes from L2 as from HBM: 8192 x 28672 at M = 16 65 us).  Weights loaded
// straight into fragments, 64 bytes of 16 rows at a time, take longer: 8192 x
// 28672 at M = 64 63.8 against 54.4 us, 4096 x 11008 19.1 and 17.0.
//
// 8 waves where their workgroups keep most compute units (20480 x 8192 at M = 64:
// 41.7 us, 4.0 TB/s, 48.7 with 4 waves), else 4 (16384 x 4096: 17.3 us, 21.7 with
// 8; 11008 x 4096 at M = 16: 11.3 and 14.9).
// ---------------------------------------------------------------------------
constexpr int kBatchSteps = 2;                     // 128-k steps at a time

template <int MT, int WV>
struct BatchShape {
    static constexpr int KT = kBatchSteps;
    static constexpr int XG = MT * 2 * KT;         // 8-row loads of the codes per step
    static constexpr int XW = XG < WV ? 1 : XG / WV;         // of a wave
    static constexpr int XB = XG * 1024, BUF = XB + WV * KT * 2048;
    static constexpr int LPS = XW + 2 * KT;
    static constexpr int S = 160 * 1024 / BUF < 4 ? 160 * 1024 / BUF : 4;
    static constexpr size_t LDS = (size_t)S * BUF;
    static_assert(XG % WV == 0 || WV % XG == 0, "every wave loads the same number of row groups");
};

template <class E, int MT, int WV>
__global__ __launch_bounds__(64 * WV, WV == 8 ? 2 : 4) void k_w8a8_batch(Args a) {
    using T = BatchShape<MT, WV>;
    constexpr int KT = T::KT, S = T::S;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, h = lane >> 4;
    const int n0 = ((int)blockIdx.x * WV + wave) * 16;
    const int total = (a.K + kStep - 1) / kStep;
    const int k0 = blockIdx.y * a.steps;           // a.steps: 128-k steps of a split, a multiple of KT
    const int steps = (min(total - k0, a.steps) + KT - 1) / KT;
    const size_t K = (size_t)a.K;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, (size_t)a.M * K);
    const int columns = __builtin_amdgcn_readfirstlane(max(0, min(16, a.N - n0)));      // in a scalar register
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (size_t)min(n0, a.N - 1) * K, (size_t)columns * K);

    // a load fills 8 rows of 128 bytes, chunk l & 7 of row l >> 3 from the row's
    // chunk (l & 7) ^ (row & 6); rows past M are past the buffer's end
    const int lr = lane >> 3, kc = (lane & 7) ^ (lr & 6);
    uint32_t xoff[T::XW];
#pragma unroll
    for (int i = 0; i < T::XW; ++i)
        xoff[i] = (uint32_t)((wave * T::XW + i) % T::XG % (MT * 2) * 8 + lr) * (uint32_t)a.K + 16u * kc;
    uint32_t woff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) woff[i] = (uint32_t)(8 * i + lr) * (uint32_t)a.K + 16u * kc;
    // Rows lie K bytes apart: with K a power of two, workgroups at the same k
    // would ask a few memory channels for all of their lines.  The sums are exact
    // in any order, so each of an XCD's workgroups begins at a step of its own
    // (28672 x 8192 at M = 16 / 64: 43.5 / 45 us, 52.6 / 56.4 from step 0).
    const int first = (int)((blockIdx.x >> 3) % (unsigned)steps);
    auto issue = [&](int i0, int slot) {
        const int step = i0 >= steps ? steps : i0 + first < steps ? i0 + first : i0 + first - steps;
#pragma unroll
        for (int i = 0; i < T::XW; ++i) {
            const int ii = (wave * T::XW + i) % T::XG;
            const uint32_t at = (uint32_t)__builtin_amdgcn_readfirstlane((k0 + step * KT + ii / (MT * 2)) * kStep);
            // chunks past K, and all of the steps past the last one, load zeros
            const bool ok = step < steps && (int)at + 16 * kc < a.K;
            load16_lds(rx, smem + slot * T::BUF + ii * 1024, ok ? xoff[i] : kOutOfRange, at);
        }
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t at = (uint32_t)(k0 + step * KT + t) * kStep;
                const bool ok = step < steps && (int)at + 16 * kc < a.K;
                load16_lds(rw, smem + slot * T::BUF + T::XB + (wave * KT + t) * 2048 + i * 1024, ok ? woff[i] : kOutOfRange, at);
            }
    };
    int4_t acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = (int4_t){0, 0, 0, 0};
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
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int4_t wv = *reinterpret_cast<const int4_t*>(
                            smem + st * T::BUF + T::XB + (wave * KT + t) * 2048 + j * kStep + (((4 * q + h) ^ (j & 6)) << 4));
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const int4_t xv = *reinterpret_cast<const int4_t*>(
                                smem + st * T::BUF + (t * MT + m) * 2048 + j * kStep + (((4 * q + h) ^ (j & 6)) << 4));
                            acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, xv, acc[m], 0, 0, 0);
                        }
                    }
            }
        }
        step0 += S;
    } while (step0 < steps);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    const int n = n0 + 4 * h;
    if (n >= a.N) return;
    const float4_t sw = load4(a.sw, n, a.N);
    const float4_t bias = a.bias ? load4(a.bias, n, a.N) : (float4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = 16 * m + j;
        if (row < a.M) store4<E>(a, row, n, acc[m], a.part ? 0.0f : a.sx[row], sw, bias);
    }
}

// XOR of the eight 16-byte chunks of row r in LDS (rows of 128 bytes).  A
// ds_read_b128 serves lanes 0-3, 12-15, 20-23, 24-27 together (then 4-11, 16-19,
// 28-31, and the same of the upper half); with this XOR each such group of a
// fragment read (lane (j, h): row j, chunk c + h) takes 16 distinct bank
// quadruples (no SQ_LDS_BANK_CONFLICT).
__device__ __forceinline__ int chunk_swizzle(int r) { return r & 6; }

// ---------------------------------------------------------------------------
// Many rows, too few for 256 x 256 tiles on every compute unit: TM x TN output
// tiles, WM x WN waves.  Both operands go through LDS in steps of 128 k, S steps
// in flight as direct-to-LDS loads; a wave reads the fragments of step t + 1
// while the MFMAs of step t run.
//
// 512 x 6144 x 4096: 19 to 23 us (1100 to 1340 TOP/s) for 192 tiles on 256 compute
// units.  A step takes 0.58 us against 0.22 of MFMA: the loads are what is waited
// for (0.49 us when all of them hit L2, 0.41 without the weights'; without the
// fragment reads still 0.57), since a 128 x 128 tile reads twice the bytes of a
// 256 x 256 tile for each product.  Two workgroups of 4 waves on a compute unit,
// 4 waves in place of 8, 64 columns, and steps of 64 k were no faster.
// ---------------------------------------------------------------------------
template <class E, int TM, int TN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN, WM * WN / 4) void k_w8a8_tile(Args a) {
    constexpr int WV = WM * WN;
    constexpr int FM = TM / WM / 16, FN = TN / WN / 16;      // 16-row fragments of a wave
    constexpr int XI = TM / 8 / WV, WI = TN / 8 / WV;        // 8-row loads of a wave per step
    constexpr int XB = TM * kStep, BUF = (TM + TN) * kStep;
    constexpr int LPS = XI + WI;
    static_assert(XI * WV * 8 == TM && WI * WV * 8 == TN, "every wave loads the same number of row groups");
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, h = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    int tm, tn;
    tile_of(blockIdx.x, (a.M + TM - 1) / TM, (a.N + TN - 1) / TN, tm, tn);
    const int m0 = tm * TM, n0 = tn * TN;
    const int total = (a.K + kStep - 1) / kStep;
    const int k0 = blockIdx.y * a.steps;
    const int steps = min(total - k0, a.steps);
    const size_t K = (size_t)a.K;

    const int mrows = min(TM, a.M - m0), nrows = min(TN, a.N - n0);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (size_t)m0 * K, (size_t)mrows * K);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (size_t)n0 * K, (size_t)nrows * K);

    // A load instruction fills 8 rows: lane l writes chunk l & 7 of row l >> 3
    const int lr = lane >> 3, kc = (lane & 7) ^ chunk_swizzle(lr);
    uint32_t xoff[XI], woff[WI];
#pragma unroll
    for (int i = 0; i < XI; ++i)
        xoff[i] = (uint32_t)min(8 * (wave * XI + i) + lr, mrows - 1) * (uint32_t)a.K + 16u * kc;
#pragma unroll
    for (int i = 0; i < WI; ++i)
        woff[i] = (uint32_t)min(8 * (wave * WI + i) + lr, nrows - 1) * (uint32_t)a.K + 16u * kc;
    auto issue = [&](int step, int slot) {
        const uint32_t at = (uint32_t)(k0 + step) * kStep;
        // chunks past K, and all of the steps past the last one, load zeros
        const bool ok = step < steps && (int)at + 16 * kc < a.K;
        unsigned char* xb = smem + slot * BUF;
#pragma unroll
        for (int i = 0; i < XI; ++i)
            load16_lds(rx, xb + (wave * XI + i) * 1024, ok ? xoff[i] : kOutOfRange, at);
#pragma unroll
        for (int i = 0; i < WI; ++i)
            load16_lds(rw, xb + XB + (wave * WI + i) * 1024, ok ? woff[i] : kOutOfRange, at);
    };
    int fat[2];                                    // this lane's chunks of a fragment: k 0..63 and 64..127
#pragma unroll
    for (int q = 0; q < 2; ++q) fat[q] = j * kStep + (((4 * q + h) ^ chunk_swizzle(j)) << 4);
    const unsigned char* xf = smem + wm * FM * 2048;
    const unsigned char* wf = smem + XB + wn * FN * 2048;

    int4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int c = 0; c < FN; ++c) acc[i][c] = (int4_t){0, 0, 0, 0};
    int4_t xv[2][FM][2], wv[2][FN][2];
    auto fragments = [&](int slot, int f) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int c = 0; c < FN; ++c) wv[f][c][q] = *reinterpret_cast<const int4_t*>(wf + slot * BUF + c * 2048 + fat[q]);
#pragma unroll
            for (int i = 0; i < FM; ++i) xv[f][i][q] = *reinterpret_cast<const int4_t*>(xf + slot * BUF + i * 2048 + fat[q]);
        }
    };

#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(s, s);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(LPS * (S - 2)));
    asm volatile("s_barrier" ::: "memory");
    fragments(0, 0);
    static_assert(S % 2 == 0, "fragment sets alternate with the steps");
    for (int step0 = 0;; step0 += S) {
        bool more = true;
#pragma unroll
        for (int st = 0; st < S; ++st) {
            const int step = step0 + st;
            if (step >= steps) { more = false; break; }
            // this wave's part of step + 1 has landed and its fragments of step
            // have been read; then everybody's (a bare barrier: a fence would
            // drain the loads of the steps after)
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(LPS * (S - 3)));
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            issue(step + S - 1, (st + S - 1) % S);
            fragments((st + 1) % S, (st + 1) & 1);
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int c = 0; c < FN; ++c)
                        acc[i][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[st & 1][c][q], xv[st & 1][i][q],
                                                                          acc[i][c], 0, 0, 0);
            // the MFMAs' operands are in registers: the next loads and fragment
            // reads are issued between them
#pragma unroll
            for (int q = 0; q < LPS; ++q) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            }
#pragma unroll
            for (int q = 0; q < 2 * FM * FN - LPS; ++q) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!more) break;
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));

    const int mb = m0 + wm * FM * 16, nb = n0 + wn * FN * 16;
    if (a.part) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int c = 0; c < FN; ++c) {
                const int m = mb + 16 * i + j, n = nb + 16 * c + 4 * h;
                if (m < a.M && n < a.N) store4<E>(a, m, n, acc[i][c], 0.0f, (float4_t){}, (float4_t){});
            }
        return;
    }
    float4_t sw[FN], bias[FN];
    float sx[FM];
#pragma unroll
    for (int c = 0; c < FN; ++c) {
        sw[c] = load4(a.sw, nb + 16 * c + 4 * h, a.N);
        bias[c] = a.bias ? load4(a.bias, nb + 16 * c + 4 * h, a.N) : (float4_t){0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) sx[i] = a.sx[min(mb + 16 * i + j, a.M - 1)];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");    // every fragment is read
    unsigned char* stage = smem + wave * (FM * 16 * FN * 32);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int c = 0; c < FN; ++c) stage4<E, FN * 16>(stage, 16 * i + j, 16 * c + 4 * h, acc[i][c], sx[i], sw[c], bias[c]);
    store_rows<FM * 16, FN * 16>(a, stage, mb, nb);
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles of the largest products, 8 waves, one workgroup per compute
// unit that takes tile after tile.  8192 x 14336 x 4096: 367 to 398 us (2420 to
// 2620 TOP/s), MFMAs running 68 % of the time at a clock of 1.9 GHz; up to 484 us in
// a first burst of launches, while the clock is lower still (24 launches, in order:
// 373 three times, 386 rising to 484 in the ninth, 441 to 446, 407 in the last).
//
// Steps of 128 k (whole 128-byte lines of every row), two of them in LDS, each
// as four half tiles of 128 rows: X0, X1, W0, W1.  A wave computes 64 rows of
// X0 and of X1 against 32 columns of W0 and of W1, in four phases of 16 MFMAs:
//   phase   reads (LDS)   multiplies   loads (to LDS)
//     0     X0 (t)        X0 W0        W0 (t + 2)
//     1     W1 (t)        X0 W1        X0 (t + 2)
//     2     X1 (t)        X1 W1        W1 (t + 2)
//     3     W0 (t + 1)    X1 W0        X1 (t + 2)
// Each half tile is read once and its buffer is loaded again in the next phase;
// a phase waits for the one half tile that the next phase reads, with the six
// after it (12 loads a wave) still in flight.
//
// A phase is a memory part and a multiply part with a barrier after each.  The
// waves 4..7 run one barrier behind 0..3 (a SIMD holds one of each): while one
// multiplies, the other reads, loads and waits.
//
// A tile's results leave while the next tile's first half tiles are loading:
// each wave turns them in 4 KB of LDS of its own (32 rows of 64 columns) and
// stores whole 128-byte lines.  For that the 64 columns of a wave are adjacent:
// row r of half W_p is column 64 (r / 32) + 32 p + r % 32 of the tile.
// ---------------------------------------------------------------------------
namespace wide {
constexpr int T = 256;                             // tile rows and columns
constexpr int HALF = 128 * kStep;                  // bytes of a half tile
constexpr int BUF = 4 * HALF;                      // X0 X1 W0 W1 of one step
constexpr int IN_FLIGHT = 12;                      // loads behind the half tile a phase waits for
constexpr int STAGE = 32 * 128;                    // a wave's output rows
constexpr size_t LDS = 2 * BUF + 8 * STAGE;
}  // namespace wide

template <class E>
__global__ __launch_bounds__(512, 2) void k_w8a8_wide(Args a, int tiles) {
    using namespace wide;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, h = lane >> 4;
    const int wm = wave >> 2, wn = wave & 3;
    const int steps = (a.K + kStep - 1) / kStep;
    const size_t K = (size_t)a.K;

    // a load fills 8 rows: lane l writes chunk l & 7 of row l >> 3
    const int lr = lane >> 3, kc = (lane & 7) ^ chunk_swizzle(lr);
    const int at0 = ((h ^ chunk_swizzle(j)) << 4) + j * kStep;        // this lane's chunk, k 0..63 of the step
    const int at1 = (((4 + h) ^ chunk_swizzle(j)) << 4) + j * kStep;  // k 64..127

    int4_t x[4][2], w0[2][2][2], w1[2][2], acc[2][2][4][2];
    auto read_x = [&](const unsigned char* half) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i][0] = *reinterpret_cast<const int4_t*>(half + (wm * 4 + i) * 2048 + at0);
            x[i][1] = *reinterpret_cast<const int4_t*>(half + (wm * 4 + i) * 2048 + at1);
        }
    };
    auto read_w = [&](const unsigned char* half, int4_t (*w)[2]) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            w[c][0] = *reinterpret_cast<const int4_t*>(half + (wn * 2 + c) * 2048 + at0);
            w[c][1] = *reinterpret_cast<const int4_t*>(half + (wn * 2 + c) * 2048 + at1);
        }
    };
    auto multiply = [&](int4_t (*out)[2], const int4_t (*w)[2]) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    out[i][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[c][s], x[i][s], out[i][c], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
    };
    // end of a memory part: its fragments are in registers (their LDS may be
    // loaded again) and the half tile of the next part has landed (stores of the
    // tile before only make the wait stricter)
    auto ready = [&]() {
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(IN_FLIGHT));
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto next = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    constexpr int X0 = 0, X1 = 1, W0 = 2, W1 = 3;
    struct Source { __amdgpu_buffer_rsrc_t rx, rw; uint32_t off[4][2]; };
    Source src;
    auto aim = [&](int id) {                       // the loads of a tile
        int tm, tn;
        tile_of(id, (a.M + T - 1) / T, (a.N + T - 1) / T, tm, tn);
        const int mrows = min(T, a.M - tm * T), nrows = min(T, a.N - tn * T);
        src.rx = make_rsrc(a.x + (size_t)tm * T * K, (size_t)mrows * K);
        src.rw = make_rsrc(a.w + (size_t)tn * T * K, (size_t)nrows * K);
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = (wave * 2 + i) * 8 + lr;       // of the half tile
                const int row = p < 2 ? (p & 1) * 128 + r : r / 32 * 64 + (p & 1) * 32 + r % 32;
                src.off[p][i] = (uint32_t)min(row, (p < 2 ? mrows : nrows) - 1) * (uint32_t)a.K + 16u * kc;
            }
    };
    auto issue = [&](int part, int step) {
        const uint32_t at = (uint32_t)step * kStep;
        // chunks past K, and all of the steps past the last one, load zeros
        const bool ok = (int)at + 16 * kc < a.K;
        unsigned char* lds = smem + (step & 1) * BUF + part * HALF + wave * 2048;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            load16_lds(part < 2 ? src.rx : src.rw, lds + i * 1024, ok ? src.off[part][i] : kOutOfRange, at);
    };
    auto begin = [&]() {
        issue(W0, 0); issue(X0, 0); issue(W1, 0); issue(X1, 0);
        issue(W0, 1); issue(X0, 1); issue(W1, 1); issue(X1, 1);
    };
    auto step = [&](int t, int odd) {
        const unsigned char* b = smem + odd * BUF;
        read_x(b + X0 * HALF);
        issue(W0, t + 2);
        ready();
        multiply(acc[0][0], w0[odd]);
        next();
        read_w(b + W1 * HALF, w1);
        issue(X0, t + 2);
        ready();
        multiply(acc[0][1], w1);
        next();
        read_x(b + X1 * HALF);
        issue(W1, t + 2);
        ready();
        multiply(acc[1][1], w1);
        next();
        read_w(smem + (odd ^ 1) * BUF + W0 * HALF, w0[odd ^ 1]);
        issue(X1, t + 2);
        ready();
        multiply(acc[1][0], w0[odd]);
        next();
    };

    aim(blockIdx.x);
    begin();
    for (int id = blockIdx.x; id < tiles; id += gridDim.x) {
        int tm, tn;
        tile_of(id, (a.M + T - 1) / T, (a.N + T - 1) / T, tm, tn);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) acc[q][p][i][c] = (int4_t){0, 0, 0, 0};
        // W0 (0), then X0 (0), have landed for everybody
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(IN_FLIGHT));
        asm volatile("s_barrier" ::: "memory");
        read_w(smem + W0 * HALF, w0[0]);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (wave >= 4) next();                     // one barrier behind
        for (int t = 0; t < steps; t += 2) {
            step(t, 0);
            if (t + 1 < steps) step(t + 1, 1);
        }
        if (wave < 4) next();                      // the same number of barriers for all
        const int nb = tn * T + wn * 64, mb = tm * T + wm * 64;
        float4_t sw[2][2], bias[2][2];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int n = nb + 32 * p + 16 * c + 4 * h;
                sw[p][c] = load4(a.sw, n, a.N);
                bias[p][c] = a.bias ? load4(a.bias, n, a.N) : (float4_t){0.f, 0.f, 0.f, 0.f};
            }
        float sx[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) sx[q][i] = a.sx[min(mb + 128 * q + 16 * i + j, a.M - 1)];
        // The loads past the last step write zeros to LDS: they are done before
        // the next tile's.  So are the scales': a register load still pending
        // on entry would be waited for, with all loads behind it, in every step.
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        asm volatile("s_barrier" ::: "memory");
        if (id + (int)gridDim.x < tiles) {
            aim(id + gridDim.x);
            begin();
        }
        unsigned char* stage = smem + 2 * BUF + wave * STAGE;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i0 = 0; i0 < 4; i0 += 2) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            stage4<E, 64>(stage, 16 * i + j, 32 * p + 16 * c + 4 * h, acc[q][p][i0 + i][c], sx[q][i0 + i],
                                          sw[p][c], bias[p][c]);
                store_rows<32, 64>(a, stage, mb + 128 * q + 16 * i0, nb);
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

// how a product is cut: the kernel, its tile and the K splits
enum Kernel { ROW, FEW, BATCH, TILE, WIDE };
struct Plan {
    Kernel kernel;
    int waves;                                     // BATCH
    int blocks, splits, steps;                     // workgroups per split, splits, K steps of each
};

// k_w8a8_row: its rows (1, 2 or 4) and the LDS of a split's codes
int row_rows(int M) { return M > 2 ? 4 : M; }
int row_lds(int M, int steps) { return row_rows(M) * ((steps * kStep + kRowStep - 1) / kRowStep * kRowStep); }
int row_steps(int M) { return kRowLds / row_rows(M) / kStep; }       // K steps whose codes fit

// K cut into `splits` at least, or more of at least 16 steps where there are
// fewer workgroups than compute units, in units of `unit` steps.  At 8 / 16 / 32
// steps at least (M x N x K): 16 x 1024 x 8192 8.6 / 8.0 / 9.1 us, 64 x 4096 x 11008
// 17.1 / 17.1 / 21.6, 128 x 4096 x 4096 15.0 / 15.3 / 16.0, 512 x 1024 x 8192 17.5 /
// 15.8 / 20.2; 8 gains for 128 x 2048 x 8192 (12.3 / 13.7 / 19.0) and 65 x 4096 x 4096
// (12.2 / 13.5 / 15.5), and one row of 1024 x 4096 is better whole (5.0 / 5.0 / 3.0).
void split(Plan& p, int total, int splits, int unit, int cus) {
    p.splits = 1;
    p.steps = (total + unit - 1) / unit * unit;
    const int s = max(splits, min(cus / p.blocks, total / 16));
    if (s <= 1) return;
    p.steps = ((total + s - 1) / s + unit - 1) / unit * unit;
    p.splits = (total + p.steps - 1) / p.steps;
}

Plan plan(int M, int N, int K) {
    Plan p{};
    int cus = device_cu_count();
    const int total = (K + kStep - 1) / kStep;
    const int small = (N + 63) / 64;               // 4-wave workgroups of a decode batch
    int unit = 1;
    if (M <= 4) {
        const int cols = kWaves * kRowColumns;
        p.kernel = ROW;
        p.blocks = (N + cols - 1) / cols;
        split(p, total, (total + row_steps(M) - 1) / row_steps(M), 1, cus);
        return p;
    }
    // a narrow product of a short K, which a decode batch would split (4096 x 4096 at
    // M = 16: 7.5 against 9.1 us; 6144 x 4096: 11.7 and 10.3)
    if (M <= 16 && 4 * small <= cus && total <= 48) {
        p.kernel = FEW;
        p.blocks = (N + 15) / 16;
    } else if (M <= 64) {
        p.kernel = BATCH;
        p.waves = (N + 127) / 128 >= cus * 5 / 8 ? 8 : 4;
        p.blocks = p.waves == 8 ? (N + 127) / 128 : small;
        unit = kBatchSteps;
    } else {
        // The tile whose rounds over the compute units take less: a 128-k step of
        // a 256 x 256 tile takes 1.5 us and a tile 4 us besides, 0.62 and 3 us at
        // 128 x 128 (342 x 6528 x 23735: 76 against 100 us, 4684 x 4160 x 1292: 54
        // against 46)
        const long long wide = (long long)((M + 255) / 256) * ((N + 255) / 256);
        const long long tiles = (long long)((M + 127) / 128) * ((N + 127) / 128);
        const bool w = (wide + cus - 1) / cus * (5 * total + 13) <= (tiles + cus - 1) / cus * (2 * total + 10);
        p.kernel = w ? WIDE : TILE;
        p.blocks = (int)(w ? wide : tiles);
        if (w) cus = 0;                            // no splits
    }
    split(p, total, 1, unit, cus);
    return p;
}

template <class E, int MR>
int launch_row(const Args& a, const Plan& p, hipStream_t st) {
    auto kern = k_w8a8_row<E, MR, false>;
    if constexpr (MR <= kFusedRows)
        if (a.rows) kern = k_w8a8_row<E, MR, true>;
    const int lds = row_lds(MR, p.steps);
    if (lds > 48 * 1024)
        if (int e = (int)hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds))
            return e;
    hipLaunchKernelGGL(kern, dim3(p.blocks, p.splits), dim3(64 * kWaves), lds, st, a);
    return (int)hipGetLastError();
}

template <class E>
int launch_few(const Args& a, const Plan& p, hipStream_t st) {
    hipLaunchKernelGGL((k_w8a8_few<E, 4>), dim3(p.blocks, p.splits), dim3(64 * kWaves), 0, st, a);
    return (int)hipGetLastError();
}

template <class E, int TM, int TN, int WM, int WN, int S>
int launch_tile(const Args& a, const Plan& p, hipStream_t st) {
    constexpr size_t lds = S * (TM + TN) * kStep;
    auto kern = k_w8a8_tile<E, TM, TN, WM, WN, S>;
    if (int e = (int)hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                         hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds))
        return e;
    hipLaunchKernelGGL(kern, dim3(p.blocks, p.splits), dim3(64 * WM * WN), lds, st, a);
    return (int)hipGetLastError();
}

template <class E>
int launch_wide(const Args& a, const Plan& p, hipStream_t st) {
    auto kern = k_w8a8_wide<E>;
    if (int e = (int)hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                         hipFuncAttributeMaxDynamicSharedMemorySize, (int)wide::LDS))
        return e;
    hipLaunchKernelGGL(kern, dim3(min(p.blocks, device_cu_count())), dim3(512), wide::LDS, st, a, p.blocks);
    return (int)hipGetLastError();
}

template <class E, int MT, int WV>
int launch_batch_t(const Args& a, const Plan& p, hipStream_t st) {
    using T = BatchShape<MT, WV>;
    auto kern = k_w8a8_batch<E, MT, WV>;
    if (T::LDS > 48 * 1024)
        if (int e = (int)hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)T::LDS))
            return e;
    hipLaunchKernelGGL(kern, dim3(p.blocks, p.splits), dim3(64 * WV), T::LDS, st, a);
    return (int)hipGetLastError();
}

template <class E, int MT>
int launch_batch(const Args& a, const Plan& p, hipStream_t st) {
    return p.waves == 8 ? launch_batch_t<E, MT, 8>(a, p, st) : launch_batch_t<E, MT, 4>(a, p, st);
}

template <class E>
int launch_t(const Args& a, const Plan& p, hipStream_t st) {
    int e;
    if (p.kernel == ROW) e = a.M == 1 ? launch_row<E, 1>(a, p, st) : a.M == 2 ? launch_row<E, 2>(a, p, st)
                                                                              : launch_row<E, 4>(a, p, st);
    else if (p.kernel == FEW) e = launch_few<E>(a, p, st);
    else if (p.kernel == WIDE) e = launch_wide<E>(a, p, st);
    else if (p.kernel == TILE) e = launch_tile<E, 128, 128, 2, 4, 4>(a, p, st);
    else if (a.M <= 16) e = launch_batch<E, 1>(a, p, st);
    else if (a.M <= 32) e = launch_batch<E, 2>(a, p, st);
    else e = launch_batch<E, 4>(a, p, st);
    if (e || !a.part) return e;
    const size_t total = (size_t)a.M * a.N;
    hipLaunchKernelGGL((k_w8a8_join<E>), dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, a, p.splits);
    return (int)hipGetLastError();
}

// the decode product quantizes its rows itself
bool fused_rows(const Plan& p, int M, int K) {
        return p.kernel == ROW && p.splits == 1 && M <= kFusedRows && M * (K / 8) <= kFusedChunks * 64 * kWaves;
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
