// Attention over the 8-bit cache for many rows: prompts and chunks of them.
//
// The formulas and the treatment of scales are those of attend.hip.  Here a
// workgroup holds a tile of rows (a query's rows of all heads that share a kv
// head count as rows of their own, so keys and values are read once for the group)
// and goes over the keys 64 at a time:
//
//   codes -> registers -> fp16 operands in LDS, two tiles of keys by turns
//   scores  S^T = K Q^T          32 x 32 x 16 products, 32 rows (or 64) a wave
//   weights exp2(S - M)          stay in the lane that the next product wants them in
//   output  O^T += V^T W         32 x 32 x 16 products
//
// Keys of a score tile are permuted so that a lane's registers hold 8 consecutive
// keys of one row for each chunk of 16: the B operand of the second product.  Values
// are transposed on their way into LDS (four keys by four channels a thread).  Both
// images are swizzled by 16 bytes so that the eight lanes that read together meet
// eight different banks' quarters.
#include "attend.h"

namespace awq {
namespace {

constexpr int kKeys = 64;                // keys of a tile

template <int D>
struct Image {
    static constexpr int KS = D == 96 ? 128 : D;            // halves of a key row (swizzled in blocks of 64)
    static constexpr int keys = kKeys * KS * 2, values = D * kKeys * 2;
    static constexpr int bytes = keys + values;
};

// rows of A (32 of them, r) to keys and channels, so that a lane's 16 results are
// 2 x 8 consecutive keys, or 16 consecutive channels
__device__ __forceinline__ int key_of(int r) { return 16 * (r >> 4) + 8 * (r >> 2 & 1) + 4 * (r >> 3 & 1) + (r & 3); }
__device__ __forceinline__ int channel_of(int r) { return 16 * (r >> 2 & 1) + 4 * (r >> 3) + (r & 3); }
__device__ __forceinline__ int key_swizzle(int key) { return (key & 3) | (key >> 3 & 1) << 2; }
__device__ __forceinline__ int channel_swizzle(int d) { return ((d ^ d >> 2) & 3) | (d >> 4 & 1) << 2; }

template <int D, int CT, int NW>
__global__ __launch_bounds__(64 * NW, D <= 128 ? 2 : 1) void k_attend_tile(AttendArgs a, int parts) {
    constexpr int NT = 64 * NW, R = 32 * CT * NW, NC = D / 16, ND = D / 32;
    constexpr int KP = kKeys * D / 16, VP = kKeys / 4 * D / 4;       // pieces of a tile: 16 codes; 4 x 4 codes
    constexpr int KN = (KP + NT - 1) / NT, VN = (VP + NT - 1) / NT;
    using I = Image<D>;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, hf = lane >> 5;
    const Sequences& s = a.seqs;
    const int kv = a.cache.kv, page_log2 = a.cache.page_log2;

    // the tile: heads first (neighbouring workgroups, on different XCDs, read different
    // heads), long rows of keys before short ones
    const LineWalk walk(a, R, true);
    if (parts > 1 && blockIdx.x == 0)              // the join wants to know the line
        walk([&](int b, long long, long long before) {
            if (b < s.B) a.line[b] = before;
            return false;
        });
    const long long unit = blockIdx.x / parts;
    const auto mine = walk([&](int, long long u, long long before) { return unit < before + u; });
    const int b = mine.b;
    if (b < 0) return;
    const Line& l = mine.line;
    const int at = (int)(blockIdx.x - mine.before * parts);
    const int head = at % kv;
    const int part = at / kv % parts;
    const int tile = l.tiles - 1 - at / kv / parts;
    const int pos0 = l.len - l.n;                                    // position of the sequence's first row
    const int pos_lo = pos0 + tile * R / a.group;
    const int pos_hi = pos0 + min(tile * R + R - 1, l.rows - 1) / a.group;
    // tiles of keys [t0, t1) that some row sees, and this part's share
    const int span = s.span(l.len, page_log2);
    const int first = a.window > 0 ? max((int)max((long long)pos_lo + 1 - a.window, 0LL), 0) : 0;
    const int last = min(pos_hi, span - 1);                          // -1: nothing
    int t0 = first / kKeys, t1 = last >= first ? last / kKeys + 1 : t0;
    {
        const int n = t1 - t0;
        t1 = t0 + (int)((long long)n * (part + 1) / parts);
        t0 = t0 + (int)((long long)n * part / parts);
    }

    // rows of the wave: column col of column tile ct is row 32 (CT wave + ct) + col
    int pos[CT];
    half8_t q[CT][NC];
    float qf[CT], bias[CT];
    const int row0 = tile * R + 32 * CT * wave;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int row = min(row0 + 32 * ct + col, l.rows - 1);
        const int j = row / a.group, h = head * a.group + (row - j * a.group);
        pos[ct] = pos0 + j;
        const uint16_t* from = a.q + (size_t)(l.start + j) * a.q_stride + (size_t)h * D + 8 * hf;
        uint4 raw[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) raw[c] = *(const uint4*)(from + 16 * c);
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float f[8];
            if (a.bf16) unpack8<BF16>(raw[c], f); else unpack8<F16>(raw[c], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
        }
        top = fmaxf(top, __shfl_xor(top, 32));
        const int e2 = query_exponent(top);
        const float up = power_of_two(e2) * a.sign;
        qf[ct] = power_of_two(-e2);
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float f[8];
            if (a.bf16) unpack8<BF16>(raw[c], f); else unpack8<F16>(raw[c], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                q[ct][c][e] = (_Float16)(f[e] * up);
                sum += (float)q[ct][c][e];
            }
        }
        sum += __shfl_xor(sum, 32);
        bias[ct] = sum * -0x1p-17f;
    }
    // positions of the wave's rows; a wave without rows only helps to stage
    const bool idle = row0 >= l.rows;
    const int wave_lo = pos0 + min(row0, l.rows - 1) / a.group;
    const int wave_hi = idle ? -1 : pos0 + min(row0 + 32 * CT - 1, l.rows - 1) / a.group;

    float M[CT], sum[CT];
    float16_t o[CT][ND];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        M[ct] = kLow;
        sum[ct] = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[ct][d][i] = 0.0f;
    }

    // pages and scales of the next 64 chunks of 16 keys (16 tiles), one a lane
    int page_l = -1;
    float c_l = -1.0f, lv_l = 0.0f, iv_l = 1.0f;
    auto fetch_pages = [&](int t) {
        const long long key = (long long)t * kKeys + 16 * lane;
        const int p = key < span ? s.page(b, (int)(key >> page_log2), a.cache.pages) : -1;
        const size_t i = (size_t)max(p, 0) * kv + head;
        page_l = p;
        c_l = p >= 0 ? a.cache.scales[0][i] * a.scale : -1.0f;
        const float vs = p >= 0 ? fmaxf(a.cache.scales[1][i], 0x1p-100f) : 1.0f;
        lv_l = __builtin_amdgcn_logf(vs);
        iv_l = 1.0f / vs;
    };
    // a tile's codes on their way, and its chunks' scales
    uint4 kr[KN];
    uint32_t vr[VN][4];
    float cs[4], lvs[4], ivs[4];
    auto load = [&](int t) {
        const int i = (t - t0) & 15;
        if (i == 0) fetch_pages(t);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            cs[c] = lane_value(c_l, 4 * i + c);
            lvs[c] = lane_value(lv_l, 4 * i + c);
            ivs[c] = lane_value(iv_l, 4 * i + c);
        }
        const int mask = (1 << page_log2) - 1;
#pragma unroll
        for (int x = 0; x < KN; ++x) {
            const int p = tid + NT * x, key = p / NC, c = p - key * NC;
            const int page = max(__shfl(page_l, 4 * i + (key >> 4 & 3)), 0);
            if (KP % NT == 0 || p < KP)
                kr[x] = *(const uint4*)(a.cache.codes[0] + a.cache.block(page, head) +
                                        (uint32_t)(((t * kKeys + key) & mask) * D + 16 * c));
        }
#pragma unroll
        for (int x = 0; x < VN; ++x) {
            const int p = tid + NT * x, kg = p / (D / 4), dg = p - kg * (D / 4);
            const int page = max(__shfl(page_l, 4 * i + (kg >> 2 & 3)), 0);
            if (VP % NT == 0 || p < VP) {
                const int8_t* from = a.cache.codes[1] + a.cache.block(page, head) +
                                     (uint32_t)(((t * kKeys + 4 * kg) & mask) * D + 4 * dg);
#pragma unroll
                for (int y = 0; y < 4; ++y) vr[x][y] = *(const uint32_t*)(from + y * D);
            }
        }
    };
    auto store = [&](unsigned char* image) {
#pragma unroll
        for (int x = 0; x < KN; ++x) {
            const int p = tid + NT * x, key = p / NC, c = p - key * NC;
            if (KP % NT == 0 || p < KP) {
                const uint32_t w[4] = {kr[x].x ^ 0x80808080u, kr[x].y ^ 0x80808080u, kr[x].z ^ 0x80808080u, kr[x].w ^ 0x80808080u};
                unsigned char* row = image + key * (2 * I::KS);
                const int sw = key_swizzle(key);
                *(uint4*)(row + ((2 * c ^ sw) << 4)) = make_uint4(key_pair(w[0], 0), key_pair(w[0], 1), key_pair(w[1], 0), key_pair(w[1], 1));
                *(uint4*)(row + (((2 * c + 1) ^ sw) << 4)) = make_uint4(key_pair(w[2], 0), key_pair(w[2], 1), key_pair(w[3], 0), key_pair(w[3], 1));
            }
        }
#pragma unroll
        for (int x = 0; x < VN; ++x) {
            const int p = tid + NT * x, kg = p / (D / 4), dg = p - kg * (D / 4);
            if (VP % NT == 0 || p < VP) {
                uint32_t w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) w[y] = vr[x][y] ^ 0x80808080u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // 1024 + (code + 128) for two keys, less 1152
                    const uint32_t sel = 0x0C000C00u | (uint32_t)(4 + j) << 16 | (uint32_t)j;
                    const half2_t m = {(_Float16)-1152.0f, (_Float16)-1152.0f};
                    const half2_t lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(w[1], w[0], sel) | 0x64006400u) + m;
                    const half2_t hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(w[3], w[2], sel) | 0x64006400u) + m;
                    const int d = 4 * dg + j;
                    *(uint2*)(image + I::keys + d * (2 * kKeys) + (((kg >> 1) ^ channel_swizzle(d)) << 4) + (kg & 1) * 8) =
                        make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
                }
            }
        }
    };

    const int key_row = key_of(col) * (2 * I::KS), key_x = hf ^ key_swizzle(key_of(col));
    const int channel_row = I::keys + channel_of(col) * (2 * kKeys), channel_x = hf ^ channel_swizzle(channel_of(col));

    auto compute = [&](const unsigned char* image, int t, const float* c4, const float* lv4, const float* iv4) {
        const int key0 = t * kKeys;
        if (key0 > wave_hi) return;
        float16_t sc[CT][2];
#pragma unroll
        for (int st = 0; st < 2; ++st) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int i = 0; i < 16; ++i) sc[ct][st][i] = bias[ct];
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const half8_t k = *(const half8_t*)(image + st * (32 * 2 * I::KS) + key_row + ((2 * c ^ key_x) << 4));
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    sc[ct][st] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[ct][c], sc[ct][st], 0, 0, 0);
            }
        }
        const bool pages = c4[0] >= 0.0f && c4[1] >= 0.0f && c4[2] >= 0.0f && c4[3] >= 0.0f;
        const bool open = pages && key0 + kKeys - 1 <= wave_lo && (a.window <= 0 || key0 > wave_hi - a.window);
        half8_t w[CT][4];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            // a chunk's scores are f * product; the product of no product is left at 0
            float f[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) f[c] = fmaxf(c4[c] * qf[ct] * kLog2e, 0x1p-126f);
            if (a.softcap > 0.0f) {
                // cap tanh(x / cap) = cap (1 - 2 / (exp(2 x / cap) + 1))
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float e = 2.0f / a.softcap * f[c];
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const float x = sc[ct][c >> 1][8 * (c & 1) + y] * e;
                        sc[ct][c >> 1][8 * (c & 1) + y] = 1.0f - 2.0f * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(x) + 1.0f);
                    }
                    f[c] = kLog2e * a.softcap;
                }
            }
            if (!open) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int key = key0 + 16 * c + 8 * hf;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const bool seen = c4[c] >= 0.0f && key + y <= pos[ct] && (a.window <= 0 || key + y > pos[ct] - a.window);
                        if (!seen) sc[ct][c >> 1][8 * (c & 1) + y] = -INFINITY;
                    }
                }
            }
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float m = sc[ct][c >> 1][8 * (c & 1)];
#pragma unroll
                for (int y = 1; y < 8; ++y) m = fmaxf(m, sc[ct][c >> 1][8 * (c & 1) + y]);
                top = fmaxf(top, __builtin_fmaf(m, f[c], lv4[c]));
            }
            if (__builtin_amdgcn_ballot_w64(top > M[ct] + kSlack)) {
                top = fmaxf(top, __shfl_xor(top, 32));
                const float m = fmaxf(M[ct], top);
                const float down = __builtin_amdgcn_exp2f(M[ct] - m);
                M[ct] = m;
                sum[ct] *= down;
#pragma unroll
                for (int d = 0; d < ND; ++d) o[ct][d] *= down;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float less = lv4[c] - M[ct];
                float p8 = 0.0f;
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[ct][c >> 1][8 * (c & 1) + y], f[c], less));
                    p8 += p;
                    w[ct][c][y] = (_Float16)p;
                }
                sum[ct] = __builtin_fmaf(p8, iv4[c], sum[ct]);
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const half8_t v = *(const half8_t*)(image + channel_row + d * (32 * 2 * kKeys) + ((2 * c ^ channel_x) << 4));
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    o[ct][d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, w[ct][c], o[ct][d], 0, 0, 0);
            }
    };

    if (t0 < t1) {
        load(t0);
        for (int t = t0; t < t1; ++t) {
            unsigned char* image = smem + ((t - t0) & 1) * I::bytes;
            float c4[4], lv4[4], iv4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) c4[c] = cs[c], lv4[c] = lvs[c], iv4[c] = ivs[c];
            store(image);                // the other image is still being read by slower waves
            if (t + 1 < t1) load(t + 1);
            __syncthreads();
            compute(image, t, c4, lv4, iv4);
        }
    }

    float* slot = parts > 1 ? a.parts + (size_t)blockIdx.x * (size_t)(R * (D + 2)) : nullptr;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const float all = sum[ct] + __shfl_xor(sum[ct], 32);
        const int in = 32 * (CT * wave + ct) + col, row = tile * R + in;
        if (row >= l.rows) continue;
        if (parts > 1) {
            if (hf == 0) {
                slot[in] = M[ct];
                slot[R + in] = all;
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                float4* to = (float4*)(slot + 2 * R + in * D + 32 * d + 16 * hf);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    to[i] = make_float4(o[ct][d][4 * i], o[ct][d][4 * i + 1], o[ct][d][4 * i + 2], o[ct][d][4 * i + 3]);
            }
            continue;
        }
        const int j = row / a.group, h = head * a.group + (row - j * a.group);
        const size_t out = (size_t)(l.start + j) * a.heads + h;
        const float inv = all > 0.0f ? 1.0f / all : 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            float f[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = o[ct][d][i] * inv;
            uint4* to = (uint4*)(a.out + out * D + 32 * d + 16 * hf);
            to[0] = a.bf16 ? pack8<BF16>(f) : pack8<F16>(f);
            to[1] = a.bf16 ? pack8<BF16>(f + 8) : pack8<F16>(f + 8);
        }
        if (hf == 0 && a.lse) a.lse[out] = all > 0.0f ? (M[ct] + __builtin_amdgcn_logf(all)) * kLn2 : -INFINITY;
    }
}

template <int D, int CT, int NW>
int launch_t(const AttendArgs& a, int parts, hipStream_t st) {
    constexpr int bytes = 2 * Image<D>::bytes;
    auto kern = k_attend_tile<D, CT, NW>;
    if (bytes > 65536)
        if (int e = (int)hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes))
            return e;
    hipLaunchKernelGGL(kern, dim3(a.groups), dim3(64 * NW), bytes, st, a, parts);
    return (int)hipGetLastError();
}

template <int D>
int launch_d(const AttendArgs& a, const TilePlan& p, hipStream_t st) {
    if constexpr (D <= 128)
        if (p.rows == 256) return launch_t<D, 1, 8>(a, p.parts, st);
    return launch_t<D, 1, 4>(a, p.parts, st);
}

}  // namespace

TilePlan tile_plan(int T, int B, int group, int kv, int dim, int max_new, int max_len, int cus) {
    TilePlan p;
    const long long rows = (long long)T * group;
    p.rows = dim <= 128 && (rows / 256 + B) * kv >= cus && (long long)max_new * group > 128 ? 256 : 128;
    const long long tiles = (rows / p.rows + B) * kv;
    const long long most = max_len / (8 * kKeys);
    long long parts = cus / tiles;
    if (parts > most) parts = most;
    p.parts = parts > 8 ? 8 : parts < 1 ? 1 : (int)parts;
    return p;
}

int launch_attend_tile(const AttendArgs& a, const TilePlan& p, hipStream_t st) {
    switch (a.cache.dim) {
        case 64: return launch_d<64>(a, p, st);
        case 96: return launch_d<96>(a, p, st);
        case 128: return launch_d<128>(a, p, st);
        case 192: return launch_d<192>(a, p, st);
        default: return launch_d<256>(a, p, st);
    }
}

}  // namespace awq
