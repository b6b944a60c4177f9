// Norms before and after a block fused with its gate and the scaled residual,
// and the row quantizer of the 8-bit product.
//
//   t  = post(b)                     (or b without a norm after the block)
//   r' = alpha * r + g * t
//   h  = pre(r')                     from the fp32 r', before it is rounded
//   RMS:   norm(v) = v / sqrt(mean(v^2) + eps) * w (+ bias)
//   layer: the same of v - mean(v)
//
// HBM-bound: b and r are read once and r' and h written once (8 bytes an
// element; 7 with h as 8-bit codes).  A row lives in the registers of one
// workgroup from its load to its last store: NT threads hold C 16-byte chunks
// each, the means and mean squares are fp32 reductions over the workgroup (a
// layer norm takes its mean first and sums squares of differences, so nothing
// cancels), and r' is rounded once on its way out while h goes on from the
// fp32 value.  Chunks past the row's end hold zeros and take no part.
//
// Both norms, cold rows: 8192 x 8192 94 us (5.7 TB/s), 86 us with h as codes (5.5
// TB/s); 2048 x 4096 14.4 us (4.7 TB/s), 17.2 us with codes (3.4 TB/s).  One norm,
// 2048 x 4096: 14.4 and 15.9 us; 14.9 in a build whose codes never divide, and 16.0
// where the third reduction is left out as well.  64 x 8192 3.8 us and 1 x 4096 3.1
// us: a launch and the latency of a load, two reductions and a store.
#include "rows.h"

namespace awq {
namespace {

struct NormArgs {
    const uint4 *block, *residual;                 // [T][H / 8] chunks
    const uint4 *post_weight, *post_bias, *gate, *pre_weight, *pre_bias;
    uint4* residual_out;
    void* h;                                       // 16-bit elements, or int8 codes with h_scales
    float* h_scales;
    int H, rows_per_gate;
    float alpha, eps;
    int layer;
    int row0;                                      // of this launch
};

template <class E, int NT, int C>
__global__ __launch_bounds__(NT) void k_norm(NormArgs a) {
    constexpr int W = NT / 64;
    __shared__ uint32_t slots[5][W];               // one row of slots per reduction
    const int tid = threadIdx.x;
    const int chunks = a.H / 8;
    const size_t row = (size_t)a.row0 + blockIdx.x;
    const size_t at = row * (size_t)chunks;
    const size_t gat = a.gate ? row / (size_t)a.rows_per_gate * (size_t)chunks : 0;
    const float inv_h = 1.0f / (float)a.H;

    auto fetch = [&](const uint4* p, size_t base, int c) -> uint4 {
        const int i = tid + NT * c;
        return p && i < chunks ? p[base + i] : make_uint4(0, 0, 0, 0);
    };
    uint4 br[C], rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) br[c] = fetch(a.block, at, c);
#pragma unroll
    for (int c = 0; c < C; ++c) rr[c] = fetch(a.residual, at, c);

    float v[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) unpack8<E>(br[c], v[c]);

    // v -> norm(v) * weight (+ bias); slots s0 (layer norms only) and s0 + 1
    auto normalize = [&](const uint4* weight, const uint4* bias, int s0) {
        uint4 w[C], b[C];
#pragma unroll
        for (int c = 0; c < C; ++c) w[c] = fetch(weight, 0, c);
#pragma unroll
        for (int c = 0; c < C; ++c) b[c] = fetch(bias, 0, c);
        if (a.layer) {
            float sum = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += v[c][e];
            const float mean = __builtin_bit_cast(float, group_reduce<W>(__builtin_bit_cast(uint32_t, sum),
                                                                         slots[s0], SumF32())) * inv_h;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (tid + NT * c < chunks)
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[c][e] -= mean;
        }
        float sq = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) sq = __builtin_fmaf(v[c][e], v[c][e], sq);
        const float ms = __builtin_bit_cast(float, group_reduce<W>(__builtin_bit_cast(uint32_t, sq),
                                                                   slots[s0 + 1], SumF32())) * inv_h;
        const float inv = rsqrtf(ms + a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float wf[8], bf[8];
            unpack8<E>(w[c], wf);
            unpack8<E>(b[c], bf);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = __builtin_fmaf(v[c][e] * inv, wf[e], bf[e]);
        }
    };

    if (a.post_weight) normalize(a.post_weight, a.post_bias, 0);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float r[8];
        unpack8<E>(rr[c], r);
        if (a.gate) {
            float g[8];
            unpack8<E>(fetch(a.gate, gat, c), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = __builtin_fmaf(a.alpha, r[e], g[e] * v[c][e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = __builtin_fmaf(a.alpha, r[e], v[c][e]);
        }
        const int i = tid + NT * c;
        if (i < chunks) a.residual_out[at + i] = pack8<E>(v[c]);
    }
    normalize(a.pre_weight, a.pre_bias, 2);

    if (a.h_scales) {
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[c][e]));
        const RowScale s(group_reduce<W>(top, slots[4], MaxU32()));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = tid + NT * c;
            const uint2 q = pack_codes8(v[c], s);
            if (i < chunks) reinterpret_cast<uint2*>(a.h)[at + i] = q;
        }
        if (tid == 0) a.h_scales[row] = s.scale();
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = tid + NT * c;
            if (i < chunks) reinterpret_cast<uint4*>(a.h)[at + i] = pack8<E>(v[c]);
        }
    }
}

// Row quantizer: scale = max|x| / 127, q = rint(127 x / max|x|).  The row is
// held in registers between the maximum and the codes, or (LONG: past the
// widest instance) read a second time.  509 x 4096: 3.8 us, mostly the launch; 2048
// x 4096 7.7 us (3.3 TB/s), 11008 x 4096 26.7 us (5.1 TB/s), 28672 x 8192 118 us (6.0
// TB/s).
struct QuantArgs {
    const uint4* x;
    uint2* q;
    float* scales;
    int K;
    int row0;                                      // of this launch
};

template <class E, int NT, int C, bool LONG>
__global__ __launch_bounds__(NT) void k_quantize_rows(QuantArgs a) {
    constexpr int W = NT / 64;
    __shared__ uint32_t slots[W];
    const int tid = threadIdx.x;
    const int chunks = a.K / 8;
    const size_t row = (size_t)a.row0 + blockIdx.x;
    const size_t at = row * (size_t)chunks;
    uint32_t top = 0;
    float v[C][8];
    if constexpr (LONG) {
        for (int i = tid; i < chunks; i += NT) {
            unpack8<E>(a.x[at + i], v[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[0][e]));
        }
    } else {
        uint4 r[C];
#pragma unroll
        for (int c = 0; c < C; ++c) r[c] = tid + NT * c < chunks ? a.x[at + tid + NT * c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            unpack8<E>(r[c], v[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[c][e]));
        }
    }
    const RowScale s(group_reduce<W>(top, slots, MaxU32()));
    if constexpr (LONG) {
        for (int i = tid; i < chunks; i += NT) {
            unpack8<E>(a.x[at + i], v[0]);
            a.q[at + i] = pack_codes8(v[0], s);
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint2 q = pack_codes8(v[c], s);
            if (tid + NT * c < chunks) a.q[at + tid + NT * c] = q;
        }
    }
    if (tid == 0) a.scales[row] = s.scale();
}

// Threads and chunks per thread of a row of `chunks` 16-byte chunks: one wave
// for the narrow rows, which needs no barrier (the norm of 8192 rows of 512: 7.3 us,
// 9.1 with 256 threads; of 1024 12.7 with one wave of 2, 14.8 with 256 threads or 128,
// one row 2.5 against 2.1; of 2048 26.0 with 256 of 1, 27.7 with 64 of 4, 25.2 with 128
// of 2, one row 2.2, 3.7 and 2.4); 1024 threads where there are fewer rows than compute
// units (a row's latency is the cost); else few enough threads that several
// rows share a compute unit.  2048 x 16384: 54.7 us with 512 threads of 4
// chunks, 61.7 with 1024 of 2; 8193 x 8192: 97.5 with 512 of 2, 98.8 with 256
// of 4, 102.5 with 1024 of 1; 2048 x 4096: 14.0 with 256 of 2, 16.7 with 512 of 1.
template <int NT, int C>
struct Shape {
    static constexpr int threads = NT, chunks = C;
};

template <class F>
void pick_row(int chunks, int rows, int cus, F&& f) {
    if (chunks <= 64) return f(Shape<64, 1>());
    if (chunks <= 128) return f(Shape<64, 2>());
    if (chunks <= 256) return f(Shape<256, 1>());
    if (rows < cus) {
        if (chunks <= 1024) return f(Shape<1024, 1>());
        if (chunks <= 2048) return f(Shape<1024, 2>());
    }
    if (chunks <= 512) return f(Shape<256, 2>());
    if (chunks <= 1024) return f(Shape<512, 2>());
    if (chunks <= 2048) return f(Shape<512, 4>());
    return f(Shape<1024, 4>());
}

// A launch counts its threads in 32 bits: 2^21 rows of up to 1024 threads at a time
constexpr int kLaunchRows = 1 << 21;

template <class E>
int launch_norm_t(NormArgs a, int T, hipStream_t st) {
    for (a.row0 = 0;; a.row0 += kLaunchRows) {
        const int rows = min(T - a.row0, kLaunchRows);
        pick_row(a.H / 8, T, device_cu_count(), [&](auto shape) {
            using S = decltype(shape);
            hipLaunchKernelGGL((k_norm<E, S::threads, S::chunks>), dim3(rows), dim3(S::threads), 0, st, a);
        });
        if (int e = (int)hipGetLastError()) return e;
        if (T - a.row0 <= kLaunchRows) return 0;
    }
}

template <class E>
int launch_quantize_rows_t(QuantArgs a, int M, hipStream_t st) {
    for (a.row0 = 0;; a.row0 += kLaunchRows) {
        const int rows = min(M - a.row0, kLaunchRows);
        if (a.K / 8 > 4096) {
            hipLaunchKernelGGL((k_quantize_rows<E, 1024, 1, true>), dim3(rows), dim3(1024), 0, st, a);
        } else {
            pick_row(a.K / 8, M, device_cu_count(), [&](auto shape) {
                using S = decltype(shape);
                hipLaunchKernelGGL((k_quantize_rows<E, S::threads, S::chunks, false>), dim3(rows), dim3(S::threads), 0, st, a);
            });
        }
        if (int e = (int)hipGetLastError()) return e;
        if (M - a.row0 <= kLaunchRows) return 0;
    }
}

}  // namespace

int launch_norm(const NormProblem& p, hipStream_t st) {
    NormArgs a{};
    a.block = (const uint4*)p.block;
    a.residual = (const uint4*)p.residual;
    a.post_weight = (const uint4*)p.post_weight;
    a.post_bias = (const uint4*)p.post_bias;
    a.gate = (const uint4*)p.gate;
    a.pre_weight = (const uint4*)p.pre_weight;
    a.pre_bias = (const uint4*)p.pre_bias;
    a.residual_out = (uint4*)p.residual_out;
    a.h = p.h;
    a.h_scales = p.h_scales;
    a.H = p.H;
    a.rows_per_gate = p.gate ? p.T / p.gate_rows : 1;
    a.alpha = p.residual_scale;
    a.eps = p.eps;
    a.layer = p.kind == AWQ_NORM_LAYER;
    return p.dtype == AWQ_BF16 ? launch_norm_t<BF16>(a, p.T, st) : launch_norm_t<F16>(a, p.T, st);
}

int launch_quantize_rows(const void* x, int M, int K, int dtype, void* q, float* scales, hipStream_t st) {
    const QuantArgs a{(const uint4*)x, (uint2*)q, scales, K, 0};
    return dtype == AWQ_BF16 ? launch_quantize_rows_t<BF16>(a, M, st) : launch_quantize_rows_t<F16>(a, M, st);
}

}  // namespace awq
