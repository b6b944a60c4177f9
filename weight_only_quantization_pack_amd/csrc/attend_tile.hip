// Attention over the 8-bit cache for many rows: prompts and chunks of them.
//
// The formulas and the treatment of scales are those of attend.hip.  Here a
// workgroup holds a tile of rows (a query's rows of all heads that share a kv
// head count as rows of their own, so keys and values are read once for the group)
// and goes over the keys 64 at a time:
//
//   codes -> registers -> fp16 operands in LDS, two tiles of keys by turns
//   scores  S^T = K Q^T          16 x 16 x 32 products, one or two columns of 16 rows a wave
//   weights exp2(S - M)          stay in the lane that the next product wants them in
//   output  O^T += V^T W         16 x 16 x 32 products
//
// Keys of a score tile are permuted so that a lane's registers hold 8 consecutive
// keys of one row for each chunk of 32: the B operand of the second product.  Values
// are transposed on their way into LDS (four keys by four channels a thread).  Both
// images are swizzled by 16 bytes so that lanes that read together meet different
// banks.
//
// What bounds it: the instructions that a SIMD can issue.  A tile of 64 keys costs a
// wave, with two columns and heads of 128, 64 products of 16 cycles and 280 other vector
// instructions of 4 (weights, running maximum, conversion of the codes): 1024 and 1120
// cycles, which overlap only across the two waves of a SIMD.  Counted on a prompt of
// 8192 tokens, 32 heads over 8, heads of 128: products in 40 % of the SIMDs' cycles, vector
// instructions in 44 %.  It takes 578 us, 950 TFLOP/s (572 where all rows of a wave raise their
// maximum together, which made a row's bits depend on its neighbours).  Tried and slower there:
// 32 x 32 x 16 products 613, 64 rows a wave 944, tiles of 128 rows 662, waves in two
// groups that take products and weights by turns 800, exponentials of half of the keys between
// the products of the other half 592.
//
// Eight waves: 256 rows in two columns a wave where the registers hold them, for heads to
// 128.  Wider heads, and calls of fewer rows, take one column: heads of 256, 2048 tokens,
// 114 us, and 190 with four waves of two columns (one wave a SIMD); 64 sequences of 500
// tokens, 64 rows each, heads of 128, 37 us and 40.
#include "attend.h"

namespace awq {
namespace {

constexpr int kKeys = kTileKeys, NW = 8;        // keys of a tile, waves of a workgroup

template <int D>
struct Image {
    static constexpr int KS = D == 96 ? 128 : D;            // halves of a key row (swizzled in blocks of 64)
    static constexpr int keys = kKeys * KS * 2, values = D * kKeys * 2;
};

// Row r of the A operand with the keys of score tile t (of two that make 32 keys), and
// with the channels of output tile t (of two that make 32): a lane's results are then 8
// consecutive keys of each 32, which is what it holds as B of the next product, and 8
// consecutive channels.
__device__ __forceinline__ int row_of(int t, int r) { return 8 * (r >> 2) + 4 * t + (r & 3); }

// Position of 16-byte chunk c of a row of an image, for rows of ROW bytes: the 16 lanes
// that read a chunk of 16 rows together (they differ in bits 0, 1, 3 and 4 of the row)
// meet 16 different quarters of the 64 banks; the other bits spread the writes.
template <int ROW>
__device__ __forceinline__ int swizzle(int row) {
    if constexpr (ROW % 256 == 0) return ((row & 3) | (row >> 3 & 3) << 2) ^ (row >> 2 & 1);
    return ((row >> 1 & 1) | (row >> 3 & 3) << 1) ^ (row >> 2 & 1);
}

// CT: columns of 16 rows a wave
template <int D, int CT>
__global__ __launch_bounds__(64 * NW, D <= 128 && CT == 1 ? 4 : 2) void k_attend_tile(AttendArgs a, int parts) {
    constexpr int NT = 64 * NW, R = 16 * CT * NW, NC = D / 32, ND = D / 16;
    constexpr int KP = kKeys * D / 16, VP = kKeys / 4 * D / 4;       // pieces of a tile: 16 codes; 4 x 4 codes
    constexpr int KN = (KP + NT - 1) / NT, VN = (VP + NT - 1) / NT;
    using I = Image<D>;
    constexpr int kRow = 2 * I::KS, vRow = 2 * kKeys;                // bytes of the images' rows
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    const Sequences& s = a.seqs;
    const int kv = a.cache.kv, page_log2 = a.cache.page_log2;

    // the tile: heads first (neighbouring workgroups, on different XCDs, read different
    // heads), long rows of keys before short ones
    const int head = blockIdx.x % kv, part = blockIdx.x / kv % parts;
    const TilePlace found = find_tile(a, R, blockIdx.x / kv / parts);
    const int b = found.b;
    if (b < 0) return;
    const Line& l = found.line;
    const int tile = l.tiles - 1 - found.tile;
    const TileSpan keys(a, l, R, tile, parts);
    if (part >= keys.parts) return;
    const int pos0 = l.len - l.n;                                    // position of the sequence's first row
    const int t0 = keys.t0 + (int)((long long)(keys.t1 - keys.t0) * part / keys.parts);
    const int t1 = keys.t0 + (int)((long long)(keys.t1 - keys.t0) * (part + 1) / keys.parts);
    const int span = s.span(l.len, page_log2);

    // rows of the wave: column col of column tile ct is row 16 (CT wave + ct) + col
    int pos[CT];
    half8_t q[CT][NC];
    float qf[CT];
    float4_t bias[CT];
    float reach = 0.0f;
    const int row0 = tile * R + 16 * CT * wave;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int row = min(row0 + 16 * ct + col, l.rows - 1);
        const int j = row / a.group, h = head * a.group + (row - j * a.group);
        pos[ct] = pos0 + j;
        const uint16_t* from = a.q + (size_t)(l.start + j) * a.q_stride + (size_t)h * D + 8 * g;
        uint4 raw[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) raw[c] = *(const uint4*)(from + 32 * c);
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float f[8];
            if (a.bf16) unpack8<BF16>(raw[c], f); else unpack8<F16>(raw[c], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const int e2 = query_exponent(top);
        const float up = power_of_two(e2) * a.sign;
        qf[ct] = power_of_two(-e2) * kLog2e;
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
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        reach = fmaxf(reach, qf[ct]);
        bias[ct] = float4_t{1, 1, 1, 1} * (sum * -0x1p-17f);
    }
    // What no product of the wave's rows passes, qf taken in: D channels below 2^14, codes of up to 255 and the bias's
    // 128 in units of 2^-24.
    reach = __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(uint32_t, reach), MaxU32())) * (0.5f * D);
    // positions of the wave's rows; a wave without rows goes along with the last one
    const int wave_lo = pos0 + min(row0, l.rows - 1) / a.group;
    const int wave_hi = pos0 + min(row0 + 16 * CT - 1, l.rows - 1) / a.group;

    float M[CT], sum[CT];
    float4_t o[CT][ND];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        M[ct] = kLow;
        sum[ct] = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[ct][d] = float4_t{0, 0, 0, 0};
    }

    // Pages of 64 chunks of 16 keys (16 tiles), one a lane, asked for a block of chunks
    // ahead; their scales are asked for with the block's first codes and taken over when
    // its first scores need them.
    auto page_ids = [&](int t) {
        const long long key = (long long)t * kKeys + 16 * lane;
        return key < span ? s.page(b, (int)(key >> page_log2), a.cache.pages) : -1;
    };
    int page_l = -1, page_next = page_ids(t0);
    float ks_next = 0.0f, vs_next = 0.0f;
    bool none = true;
    float c_l = -1.0f, lv_l = 0.0f, iv_l = 1.0f;
    // a tile's codes on their way
    const int mask = (1 << page_log2) - 1;
    const uint32_t page_bytes = (uint32_t)kv * (uint32_t)D << page_log2, head_bytes = (uint32_t)head * (uint32_t)D << page_log2;
    uint4 kr[KN];
    uint32_t vr[VN][4];
    auto load = [&](int t) {
        const int i = (t - t0) & 15;
        if (i == 0) {
            page_l = page_next;
            page_next = page_ids(t + 16);
            const size_t at = (size_t)max(page_l, 0) * kv + head;
            ks_next = a.cache.scales[0][at];
            vs_next = a.cache.scales[1][at];
            none = page_l < 0;
        }
        // tiles start at a page or in the middle of one: a key's slot is the tile's plus its own
        const uint32_t slot = (uint32_t)((t * kKeys) & mask) * D + head_bytes;
#pragma unroll
        for (int x = 0; x < KN; ++x) {
            const int p = tid + NT * x, key = p / (D / 16), c = p - key * (D / 16);
            const uint32_t page = (uint32_t)max(__shfl(page_l, 4 * i + (key >> 4 & 3)), 0);
            if (KP % NT == 0 || p < KP)
                kr[x] = *(const uint4*)(a.cache.codes[0] + ((uint64_t)page * page_bytes + slot) + (uint32_t)((key & mask) * D + 16 * c));
        }
#pragma unroll
        for (int x = 0; x < VN; ++x) {
            const int p = tid + NT * x, kg = p / (D / 4), dg = p - kg * (D / 4);
            const uint32_t page = (uint32_t)max(__shfl(page_l, 4 * i + (kg >> 2 & 3)), 0);
            if (VP % NT == 0 || p < VP) {
                const int8_t* from = a.cache.codes[1] + ((uint64_t)page * page_bytes + slot) + (uint32_t)((4 * kg & mask) * D + 4 * dg);
#pragma unroll
                for (int y = 0; y < 4; ++y) vr[x][y] = *(const uint32_t*)(from + y * D);
            }
        }
    };
    auto store = [&](unsigned char* keys, unsigned char* values) {
#pragma unroll
        for (int x = 0; x < KN; ++x) {
            const int p = tid + NT * x, key = p / (D / 16), c = p - key * (D / 16);
            if (KP % NT == 0 || p < KP) {
                const uint32_t w[4] = {kr[x].x ^ 0x80808080u, kr[x].y ^ 0x80808080u, kr[x].z ^ 0x80808080u, kr[x].w ^ 0x80808080u};
                unsigned char* row = keys + key * kRow;
                const int sw = swizzle<kRow>(key);
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
                    *(uint2*)(values + d * vRow + (((kg >> 1) ^ swizzle<vRow>(d)) << 4) + (kg & 1) * 8) =
                        make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
                }
            }
        }
    };

    // A operands: row_of(0 or 1, col) + 32 n, chunk 4 c + g; rows 32 apart swizzle alike, and
    // the two tiles of 32 rows differ in bit 2 of the row, which flips bit 0
    const int key_row = row_of(0, col) * kRow, key_x = g ^ swizzle<kRow>(row_of(0, col));
    const int channel_row = row_of(0, col) * vRow, channel_x = g ^ swizzle<vRow>(row_of(0, col));
    auto key_operand = [&](const unsigned char* keys, int kt, int c) {
        return *(const half8_t*)(keys + (32 * (kt >> 1) + 4 * (kt & 1)) * kRow + key_row + ((4 * c ^ key_x ^ (kt & 1)) << 4));
    };
    auto value_operand = [&](const unsigned char* values, int d, int kc) {
        return *(const half8_t*)(values + (32 * (d >> 1) + 4 * (d & 1)) * vRow + channel_row + ((4 * kc ^ channel_x ^ (d & 1)) << 4));
    };

    float4_t sc[CT][4];
    half8_t w[CT][2];
    bool large = false;                            // some score of the 16 tiles may pass 2^20
    auto scores = [&](const unsigned char* keys) {
#pragma unroll
        for (int kt = 0; kt < 4; ++kt)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const half8_t k = key_operand(keys, kt, c);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    sc[ct][kt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[ct][c], c == 0 ? bias[ct] : sc[ct][kt], 0, 0, 0);
            }
        // eight operands under way before the first product needs one
        constexpr int kAhead = 8;
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int i = 0; i < 4 * NC - kAhead; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, CT, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, CT * kAhead, 0);
    };
    auto weights = [&](int t) {
        const int i = (t - t0) & 15, key0 = t * kKeys;
        if (i == 0) {
            c_l = none ? -1.0f : key_factor(ks_next, vs_next, a.scale);
            const float vs = none ? 1.0f : value_scale(vs_next);
            lv_l = __builtin_amdgcn_logf(vs);
            iv_l = 1.0f / vs;
            large = a.softcap <= 0.0f && __builtin_amdgcn_ballot_w64(c_l * reach > 0x1p20f) != 0;
        }
        // scales of this lane's halves of the two 32 keys
        float ks[2], lv[2], iv[2];
#pragma unroll
        for (int kc = 0; kc < 2; ++kc) {
            const int from = 4 * i + 2 * kc + (g >> 1);
            ks[kc] = __shfl(c_l, from);
            lv[kc] = __shfl(lv_l, from);
            iv[kc] = __shfl(iv_l, from);
        }
        const bool closed = __builtin_amdgcn_ballot_w64(!(ks[0] >= 0.0f && ks[1] >= 0.0f)) || key0 + kKeys - 1 > wave_lo ||
                            (a.window > 0 && key0 <= wave_hi - a.window) || large;
        float f[CT][2];                            // log2 weights are f * product + lv
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
            for (int kc = 0; kc < 2; ++kc) f[ct][kc] = fmaxf(ks[kc] * qf[ct], 0x1p-126f);
            if (a.softcap > 0.0f) {
                // cap tanh(x / cap) = cap - 2 cap / (exp(2 x / cap) + 1): the product becomes
                // -1 / (exp(2 x / cap) + 1), its factor 2 cap, and cap is added with lv
#pragma unroll
                for (int kc = 0; kc < 2; ++kc) {
                    const float e = 2.0f / a.softcap * f[ct][kc];
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const float x = sc[ct][2 * kc + (y >> 2)][y & 3] * e;
                        sc[ct][2 * kc + (y >> 2)][y & 3] = __builtin_amdgcn_rcpf(-1.0f - __builtin_amdgcn_exp2f(x));
                    }
                    f[ct][kc] = 2.0f * kLog2e * a.softcap;
                    if (ct == 0) lv[kc] = __builtin_fmaf(kLog2e, a.softcap, lv[kc]);
                }
            }
            if (closed) {
                // The maximum is a rounded score, and f * product + lv - M below is not: beyond 2^20 they differ by more than
                // the room that fp16 leaves, from 2^24 on by whole units.  Such scores are rounded here, as the
                // maximum will be, and their difference is exact.
                if (large) {
#pragma unroll
                    for (int kc = 0; kc < 2; ++kc) {
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            sc[ct][2 * kc + (y >> 2)][y & 3] = __builtin_fmaf(sc[ct][2 * kc + (y >> 2)][y & 3], f[ct][kc], lv[kc]);
                        f[ct][kc] = 1.0f;
                        if (ct == CT - 1) lv[kc] = 0.0f;
                    }
                }
                // the product of a key that the row does not see is -infinity (f > 0)
#pragma unroll
                for (int kc = 0; kc < 2; ++kc) {
                    const int key = key0 + 32 * kc + 8 * g;
                    const int hi = ks[kc] < 0.0f ? -1 : pos[ct] - key;                   // keys y <= hi, > lo are seen
                    const int lo = a.window > 0 ? pos[ct] - a.window - key : -1;
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        sc[ct][2 * kc + (y >> 2)][y & 3] = y <= hi && y > lo ? sc[ct][2 * kc + (y >> 2)][y & 3] : -INFINITY;
                    if (ks[kc] != ks[kc] && hi >= 0 && lo < 7) sum[ct] = ks[kc];         // NaN for rows that see the block
                }
            }
        }
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            float top = -INFINITY;
#pragma unroll
            for (int kc = 0; kc < 2; ++kc) {
                float m = sc[ct][2 * kc][0];
#pragma unroll
                for (int y = 1; y < 8; ++y) m = fmaxf(m, sc[ct][2 * kc + (y >> 2)][y & 3]);
                top = fmaxf(top, __builtin_fmaf(m, f[ct][kc], lv[kc]));
            }
            // (rare, and laid out of the way: the prompt of 8192 tokens 578 us, 582 where it is not)
            if (__builtin_expect(__builtin_amdgcn_ballot_w64(top - M[ct] > kRoom + kSlack) != 0, 0)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                // a row by its own scores only: its bits do not depend on the rows beside it
                const float m = top - M[ct] > kRoom + kSlack ? top - kRoom : M[ct];
                const float down = __builtin_amdgcn_exp2f(M[ct] - m);
                M[ct] = m;
                sum[ct] *= down;
#pragma unroll
                for (int d = 0; d < ND; ++d) o[ct][d] *= down;
            }
        }
#pragma unroll
        for (int kc = 0; kc < 2; ++kc)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                // summed in fp32: a block whose values are small (or zeros) has weights that fp16
                // loses, but not its share of the softmax
                const float less = lv[kc] - M[ct];
                float all = 0.0f;
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[ct][2 * kc + (y >> 2)][y & 3], f[ct][kc], less));
                    all += p;
                    w[ct][kc][y] = (_Float16)p;
                }
                sum[ct] = __builtin_fmaf(all, iv[kc], sum[ct]);
            }
    };
    auto values = [&](const unsigned char* values) {
#pragma unroll
        for (int kc = 0; kc < 2; ++kc)
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const half8_t v = value_operand(values, d, kc);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    o[ct][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w[ct][kc], o[ct][d], 0, 0, 0);
            }
    };

    unsigned char* const value_images = smem + 2 * I::keys;
    if (t0 < t1) {
        load(t0);
        for (int t = t0; t < t1; ++t) {
            const int at = (t - t0) & 1;
            store(smem + at * I::keys, value_images + at * I::values);      // slower waves still read the other place
            if (t + 1 < t1) load(t + 1);
            __syncthreads();
            scores(smem + at * I::keys);
            weights(t);
            values(value_images + at * I::values);
        }
    }

    float* slot = keys.parts > 1 ? a.parts + (size_t)blockIdx.x * (size_t)(R * (D + 2)) : nullptr;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        float all = sum[ct];
        all += __shfl_xor(all, 16);
        all += __shfl_xor(all, 32);
        const int in = 16 * (CT * wave + ct) + col, row = tile * R + in;
        if (row >= l.rows) continue;
        if (keys.parts > 1) {
            if (g == 0) {
                slot[in] = M[ct];
                slot[R + in] = all;
            }
#pragma unroll
            for (int d = 0; d < ND; d += 2) {
                float4* to = (float4*)(slot + 2 * R + in * D + 16 * d + 8 * g);
                to[0] = make_float4(o[ct][d][0], o[ct][d][1], o[ct][d][2], o[ct][d][3]);
                to[1] = make_float4(o[ct][d + 1][0], o[ct][d + 1][1], o[ct][d + 1][2], o[ct][d + 1][3]);
            }
            continue;
        }
        const int j = row / a.group, h = head * a.group + (row - j * a.group);
        const size_t out = (size_t)(l.start + j) * a.heads + h;
        const float inv = all == 0.0f ? 0.0f : 1.0f / all;
#pragma unroll
        for (int d = 0; d < ND; d += 2) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = o[ct][d + (i >> 2)][i & 3] * inv;
            *(uint4*)(a.out + out * D + 16 * d + 8 * g) = a.bf16 ? pack8<BF16>(f) : pack8<F16>(f);
        }
        if (g == 0 && a.lse) a.lse[out] = all == 0.0f ? -INFINITY : (M[ct] + __builtin_amdgcn_logf(all)) * kLn2;
    }
}

template <int D, int CT>
int launch_t(const AttendArgs& a, int parts, hipStream_t st) {
    constexpr int bytes = 2 * (Image<D>::keys + Image<D>::values);
    auto kern = k_attend_tile<D, CT>;
    if (bytes > 65536)
        if (int e = (int)hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes))
            return e;
    hipLaunchKernelGGL(kern, dim3(a.groups), dim3(64 * NW), bytes, st, a, parts);
    return (int)hipGetLastError();
}

template <int D>
int launch_d(const AttendArgs& a, const TilePlan& p, hipStream_t st) {
    if constexpr (D <= 128)
        if (p.rows == 256) return launch_t<D, 2>(a, p.parts, st);
    return launch_t<D, 1>(a, p.parts, st);
}

}  // namespace

TilePlan tile_plan(int T, int B, int group, int kv, int dim, int max_new, int max_len, int cus) {
    TilePlan p;
    const long long rows = (long long)max_new * group;
    p.rows = dim <= 128 && rows > 128 ? 256 : 128;
    // tiles there will be, if the bounds hold
    const long long most_tiles = ((long long)T * group / p.rows + B) * kv;
    const long long tiles = min(most_tiles, B * ((rows + p.rows - 1) / p.rows) * kv);
    // As many parts as workgroups run at a time, if they pay.  A tile of keys takes 2.4 us, however
    // few workgroups there are; the join about as much as 2.5 of them, and one more for each 4 MB that
    // the parts leave to it.  1000 rows of 4 heads each behind 9000 tokens, 8 kv heads: 213 us in 2 parts
    // and 329 in one; 300 behind 2000, 43 in 6, 48 in 3, 82 in one; a prompt of 1024, 58 in 2 and 48 in
    // one; 32 rows of 8 heads over 30000 tokens, one kv head, 36 in 64 and 77 in 16.
    const long long slots = (p.rows == 128 && dim <= 128 ? 2 : 1) * cus, steps = (max_len + kKeys - 1LL) / kKeys;
    long long most = min(slots / tiles, 64LL);
    most = min(most, 2 * slots / most_tiles);      // the workspace holds for every T rows, whatever max_new says
    const double join = (double)T * group * kv * (dim + 2) * sizeof(float) / 4e6;
    double best = (double)steps;
    p.parts = 1;
    for (int n = 2; n <= most; ++n) {
        const double cost = (double)((steps + n - 1) / n) + 2.5 + n * join;
        if (cost < best) {
            best = cost;
            p.parts = n;
        }
    }
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
