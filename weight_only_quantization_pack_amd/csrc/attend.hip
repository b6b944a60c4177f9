// Attention of a sequence's last tokens over its cached keys and values.
//
//   s_j = scale * q.k_j            (or cap * tanh(that / cap))
//   p = softmax(s) over the keys j at or before the query's position (and within
//   the window);  o = sum_j p_j v_j
//
// Keys and values are int8 codes with one scale for each page and kv head, so a
// step of 32 keys has one key scale ks and one value scale vs (two with 16-token
// pages).  The running maximum M is taken over t = log2(e) s + log2(vs): the weight
// w = exp2(t - M) is then what multiplies a value's code, and the softmax's sum is
// the sum of w / vs.  (M stays a little below, so that fp16 holds more of the small
// weights: attend.h.)  One fused multiply-add a score brings ks, scale and vs in.
//
// Queries are the columns and keys the rows of a 16 x 16 x 32 product, so that a
// lane ends with 8 consecutive keys of one query: exactly the operand that the
// product with the values wants, with no exchange between lanes.  Codes become
// fp16 operands by one byte permutation for two of them: code + 128 is put into
// the low bits of an fp16 number, where it stands for (code + 128) 2^-24, exactly.
// The bias leaves the scores through the product's initial value (-128 2^-24 times
// the sum of q) and the output through one more product, of a constant with the
// weights.  The keys' and values' bytes are read once, straight into registers.
//
// Work is cut evenly: all (sequence, head, tile of rows) with their steps of 32
// keys form one line, and every workgroup takes an equal stretch of it.  Stretches
// that end inside a tile leave (M, sum, o) in the workspace and a second launch
// joins them in order.  Every wave of a call whose sequences are split reads all starts
// and lengths, 64 at a time, twice: 4096 sequences of 300 to 500 tokens, 8 heads over
// one of 64, 112 us, and 51 where the bound on the lengths says not to split.
//
// What bounds it is the read of the cache.  64 sequences of 200 to 8000 tokens, 64 heads
// over 8 of 128 channels: 70 us, 4.1 TB/s, 6 us of it the join; one of 131072 tokens, 32
// heads over 8: 61 us, 4.4 TB/s.  The vector instructions that turn codes into operands and
// scores into weights take 25 % of the SIMDs' cycles, the products 8 %; waves wait
// for 26 % of their time.  One token over 131 keys is latency: 8.5 us.
#include "attend.h"

namespace awq {
namespace {

constexpr int kW = 4;                    // waves of a workgroup

// units a workgroup takes: an even share, but at least two steps for every wave
__device__ __forceinline__ long long stretch(long long total, int groups) {
    return max(quotient(total + groups - 1, groups), (long long)(2 * kW));
}

// one step's codes of a wave: keys as 16 x 32 operands, values as 8 rows of D / 16
template <int D>
struct Codes {
    static constexpr int VD = D == 96 ? 128 : D;   // 96 channels: 12 of 16 lanes hold 8 values each
    static constexpr int NK = D / 32, VB = VD / 16, VW = VB / 4;
    uint32_t k[2][NK][2];                          // [key tile][chunk]: 8 codes
    uint32_t v[8][VW];                             // [key]: VB codes
    float c[2], lv[2], iv[2];                      // per half of the step: ks scale 2^24 (< 0: no page), log2(vs), 1 / vs
};

// byte j of two rows' words
__device__ __forceinline__ uint32_t value_pair(uint32_t lo, uint32_t hi, int j) {
    return __builtin_amdgcn_perm(hi, lo, 0x0C000C00u | (uint32_t)(4 + j) << 16 | (uint32_t)j);
}

template <int D, int C, bool SMALL>
__global__ __launch_bounds__(64 * kW, D * C > 256 ? 1 : 2) void k_attend(AttendArgs a) {
    using K = Codes<D>;
    // The next step's codes beside this one's, where the registers hold both: 16 sequences of
    // 1000 to 4000 tokens, heads of 256, 38 us one step at a time and 62 with two (spilled).
    constexpr bool kDeep = K::VD * C <= 192;
    constexpr int R = 16 * C, NK = K::NK, VB = K::VB, VW = K::VW;
    constexpr int JB = VB > 8 ? VB / 2 : VB;       // channels of a lane that one pass of the join takes
    __shared__ float join[kW][4][64][JB + 1];      // [wave][i][lane][j]; padded against bank conflicts
    __shared__ float stat[kW][2][R];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const Sequences& s = a.seqs;
    const int kv = a.cache.kv, page_log2 = a.cache.page_log2;

    // this workgroup's stretch [u, u_end) of the line of units, relative to sequence b: an even
    // share of it, or just one tile's
    long long u, u_end;
    int b;
    Line l(a, 0, 0, 0, R);
    const LineWalk walk(a, R);
    if (a.split) {
        const bool note = blockIdx.x == 0;         // the join wants to know the line
        const long long total = walk([&](int b, long long, long long before) {
            if (note && b < s.B) a.line[b] = before;
            return false;
        }).before;
        const long long share = stretch(total, a.groups);
        if (note && threadIdx.x == 0) a.line[s.B] = share;
        u = blockIdx.x * share;
        u_end = min(u + share, total);
        if (u >= u_end) return;
        const auto p = walk([&](int, long long n, long long before) { return u < before + n; });
        if (p.b < 0) return;
        b = p.b;
        l = p.line;
        u -= p.before;
        u_end -= p.before;
    } else {
        const TilePlace p = find_tile(a, R, blockIdx.x / kv);
        if (p.b < 0) return;
        b = p.b;
        l = p.line;
        u = ((long long)(blockIdx.x % kv) * l.tiles + p.tile) * l.tile_units();
        u_end = u + l.tile_units();
    }

    while (true) {
        const long long units = l.units(kv);
        if (u >= units) {                          // on to the next sequence
            u -= units;
            u_end -= units;
            if (++b >= s.B || u >= u_end) return;
            l = walk.line(b);
            continue;
        }
        // of the tile's units the stretch has [from, to); its steps are those behind kFixed
        const int tile_at = __builtin_amdgcn_readfirstlane((int)quotient(u, l.tile_units()));
        const int head = tile_at / l.tiles, tile = tile_at - head * l.tiles;
        const int from = __builtin_amdgcn_readfirstlane((int)(u - (long long)tile_at * l.tile_units()));
        const int to = (int)min((long long)l.tile_units(), from + (u_end - u));
        u += to - from;
        const int s0 = max(from - kFixed, 0), s1 = to - kFixed;
        if (s0 >= s1) {
            if (u >= u_end) return;
            continue;
        }
        const bool whole = s0 == 0 && s1 == l.steps;

        // rows of the tile: column r of column tile ct is row 16 ct + r.  Their loads are on
        // their way while the first step's pages and codes are asked for
        int pos[C];
        uint4 raw[C][NK];
#pragma unroll
        for (int ct = 0; ct < C; ++ct) {
            const int row = min(tile * R + 16 * ct + r, l.rows - 1);
            const int j = row / a.group, h = head * a.group + (row - j * a.group);
            pos[ct] = l.len - l.n + j;
            const uint16_t* row_q = a.q + (size_t)(l.start + j) * a.q_stride + (size_t)h * D;
#pragma unroll
            for (int c = 0; c < NK; ++c)
                raw[ct][c] = *(const uint4*)(row_q + (NK % 2 == 1 && c == NK - 1 ? 32 * c + 8 * g : 64 * (c / 2) + 16 * g + 8 * (c & 1)));
        }
        // pages and scales of the wave's next 64 steps, one a lane
        int page_l[2];
        float c_l[2], lv_l[2], iv_l[2];
        auto fetch_pages = [&](int i0) {           // the wave's steps i0 ..
            const int step = s0 + wave + kW * (i0 + lane);
#pragma unroll
            for (int x = 0; x < (SMALL ? 2 : 1); ++x) {
                const long long key = (long long)(l.step0 + step) * kStep + 16 * x;
                const int p = step < s1 ? s.page(b, (int)(key >> page_log2), a.cache.pages) : -1;
                page_l[x] = p;
                const size_t at = (size_t)max(p, 0) * kv + head;
                const float ks = a.cache.scales[0][at], raw = a.cache.scales[1][at];
                c_l[x] = p >= 0 ? key_factor(ks, raw, a.scale) : -1.0f;
                const float vs = p >= 0 ? value_scale(raw) : 1.0f;
                lv_l[x] = __builtin_amdgcn_logf(vs);
                iv_l[x] = 1.0f / vs;
            }
        };
        auto load = [&](K& d, int i) {             // the wave's step i
            if ((i & 63) == 0) fetch_pages(i);
            const int at = i & 63;
            const int step = s0 + wave + kW * i;
            const int slot = ((l.step0 + step) * kStep) & ((1 << page_log2) - 1);
            const int8_t *kb[2], *vb[2];
#pragma unroll
            for (int x = 0; x < (SMALL ? 2 : 1); ++x) {
                const int p = __builtin_amdgcn_readlane(page_l[x], at);
                const size_t off = a.cache.block(max(p, 0), head) + (SMALL ? (size_t)0 : (size_t)slot * D);
                kb[x] = a.cache.codes[0] + off;
                vb[x] = a.cache.codes[1] + off;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int key = 8 * (r >> 2) + 4 * t + (r & 3);
                const int8_t* row = SMALL ? (r < 8 ? kb[0] : kb[1]) + (uint32_t)((key & 15) * D) : kb[0] + (uint32_t)(key * D);
#pragma unroll
                for (int c = 0; c + 1 < NK; c += 2) {
                    const uint4 w = *(const uint4*)(row + 32 * c + 16 * g);
                    d.k[t][c][0] = w.x;
                    d.k[t][c][1] = w.y;
                    d.k[t][c + 1][0] = w.z;
                    d.k[t][c + 1][1] = w.w;
                }
                if constexpr (NK % 2 == 1) {
                    const uint2 w = *(const uint2*)(row + 32 * (NK - 1) + 8 * g);
                    d.k[t][NK - 1][0] = w.x;
                    d.k[t][NK - 1][1] = w.y;
                }
            }
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const int key = 8 * g + y;
                const int8_t* row = SMALL ? (g < 2 ? vb[0] : vb[1]) + (uint32_t)((key & 15) * D) : vb[0] + (uint32_t)(key * D);
                const int lr = D == 96 ? min(r, 11) : r;      // lanes 12.. repeat the last channels
                const uint32_t* from = (const uint32_t*)(row + VB * lr);
#pragma unroll
                for (int x = 0; x < VW; ++x) d.v[y][x] = from[x];
            }
#pragma unroll
            for (int x = 0; x < (SMALL ? 2 : 1); ++x) {
                d.c[x] = lane_value(c_l[x], at);
                d.lv[x] = lane_value(lv_l[x], at);
                d.iv[x] = lane_value(iv_l[x], at);
            }
        };
        const int mine = s1 - s0 > wave ? (s1 - s0 - wave + kW - 1) / kW : 0;      // steps of this wave
        K da;
        if (mine > 0) load(da, 0);

        half8_t q[C][NK];
        float qf[C];                               // what brings a column's products back to q.k
        float4_t bias[C];
#pragma unroll
        for (int ct = 0; ct < C; ++ct) {
            float f[NK][8], top = 0.0f;
#pragma unroll
            for (int c = 0; c < NK; ++c) {
                if (a.bf16) unpack8<BF16>(raw[ct][c], f[c]); else unpack8<F16>(raw[ct][c], f[c]);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[c][e]));
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const int e2 = query_exponent(top);
            const float up = power_of_two(e2) * a.sign;
            qf[ct] = power_of_two(-e2);
            float sum = 0.0f;
#pragma unroll
            for (int c = 0; c < NK; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    q[ct][c][e] = (_Float16)(f[c][e] * up);
                    sum += (float)q[ct][c][e];
                }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            bias[ct] = float4_t{1, 1, 1, 1} * (sum * -0x1p-17f);
        }
        // positions of the tile's first and last row: what no key of a step needs a mask for
        const int pos_lo = l.len - l.n + min(tile * R, l.rows - 1) / a.group;
        const int pos_hi = l.len - l.n + min(tile * R + R - 1, l.rows - 1) / a.group;

        float M[C], sum[C];
        float4_t o[C][VB], obias[C];
#pragma unroll
        for (int ct = 0; ct < C; ++ct) {
            M[ct] = kLow;
            sum[ct] = 0.0f;
            obias[ct] = float4_t{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < VB; ++j) o[ct][j] = float4_t{0, 0, 0, 0};
        }

        auto compute = [&](K& d, int i) {
            const int key0 = (l.step0 + s0 + wave + kW * i) * kStep;
            // scores
            float4_t sc[C][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int ct = 0; ct < C; ++ct) sc[ct][t] = bias[ct];
#pragma unroll
                for (int c = 0; c < NK; ++c) {
                    Half8 x;
                    const uint32_t w0 = d.k[t][c][0] ^ 0x80808080u, w1 = d.k[t][c][1] ^ 0x80808080u;
                    x.w[0] = key_pair(w0, 0);
                    x.w[1] = key_pair(w0, 1);
                    x.w[2] = key_pair(w1, 0);
                    x.w[3] = key_pair(w1, 1);
#pragma unroll
                    for (int ct = 0; ct < C; ++ct)
                        sc[ct][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x.h, q[ct][c], sc[ct][t], 0, 0, 0);
                }
            }
            const int half = SMALL ? g >> 1 : 0;   // keys 8 g .. lie in one half
            const float ks = SMALL && half ? d.c[1] : d.c[0];
            const float lv = SMALL && half ? d.lv[1] : d.lv[0];
            const float iv = SMALL && half ? d.iv[1] : d.iv[0];
            const bool pages = SMALL ? !(d.c[0] < 0.0f) && !(d.c[1] < 0.0f) : !(d.c[0] < 0.0f);
            const bool open = pages && key0 + kStep - 1 <= pos_lo && (a.window <= 0 || key0 > pos_hi - a.window);
            half8_t w[C];
#pragma unroll
            for (int ct = 0; ct < C; ++ct) {
                float t[8];
                const float f = ks * qf[ct];
                if (a.softcap > 0.0f) {
                    // cap tanh(x / cap) = cap - 2 cap / (exp(2 x / cap) + 1)
                    const float e = 2.0f * kLog2e / a.softcap * f, cap = kLog2e * a.softcap;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const float z = __builtin_amdgcn_exp2f(sc[ct][y >> 2][y & 3] * e);
                        t[y] = __builtin_fmaf(2.0f * cap, __builtin_amdgcn_rcpf(-1.0f - z), lv + cap);
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < 8; ++y) t[y] = __builtin_fmaf(sc[ct][y >> 2][y & 3], f * kLog2e, lv);
                }
                if (!open) {
                    const int key = key0 + 8 * g;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const bool seen = !(ks < 0.0f) && key + y <= pos[ct] && (a.window <= 0 || key + y > pos[ct] - a.window);
                        t[y] = seen ? t[y] : -INFINITY;
                    }
                }
                float top = t[0];
#pragma unroll
                for (int y = 1; y < 8; ++y) top = fmaxf(top, t[y]);
                if (__builtin_amdgcn_ballot_w64(top - M[ct] > kRoom + kSlack)) {
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    // a row by its own scores only: its bits do not depend on the rows beside it
                    const float m = top - M[ct] > kRoom + kSlack ? top - kRoom : M[ct];
                    const float down = __builtin_amdgcn_exp2f(M[ct] - m);
                    M[ct] = m;
                    sum[ct] *= down;
                    obias[ct] *= down;
#pragma unroll
                    for (int j = 0; j < VB; ++j) o[ct][j] *= down;
                }
                float part = 0.0f;
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const float p = __builtin_amdgcn_exp2f(t[y] - M[ct]);
                    part += p;
                    w[ct][y] = (_Float16)p;
                }
                sum[ct] = __builtin_fmaf(part, iv, sum[ct]);
            }
            // values
            const Half8 one{{0x00800080u, 0x00800080u, 0x00800080u, 0x00800080u}};      // 128 2^-24
#pragma unroll
            for (int ct = 0; ct < C; ++ct) obias[ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(one.h, w[ct], obias[ct], 0, 0, 0);
#pragma unroll
            for (int x = 0; x < VW; ++x) {
                uint32_t v[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) v[y] = d.v[y][x] ^ 0x80808080u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    Half8 e;
#pragma unroll
                    for (int y = 0; y < 4; ++y) e.w[y] = value_pair(v[2 * y], v[2 * y + 1], j);
#pragma unroll
                    for (int ct = 0; ct < C; ++ct)
                        o[ct][4 * x + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(e.h, w[ct], o[ct][4 * x + j], 0, 0, 0);
                }
            }
        };

        if constexpr (kDeep) {
            // loads under no condition, so that a wait counts only those before it: behind the
            // last step they repeat it
            K db;
            for (int i = 0; i < mine; i += 2) {
                load(db, min(i + 1, mine - 1));
                compute(da, i);
                load(da, min(i + 2, mine - 1));
                if (i + 1 < mine) compute(db, i + 1);
            }
        } else {
            for (int i = 0; i < mine; ++i) {
                compute(da, i);
                if (i + 1 < mine) load(da, i + 1);
            }
        }

        // the four waves' results: one maximum, sums and outputs added in order
#pragma unroll
        for (int ct = 0; ct < C; ++ct) {
            sum[ct] += __shfl_xor(sum[ct], 16);
            sum[ct] += __shfl_xor(sum[ct], 32);
            if (g == 0) {
                stat[wave][0][16 * ct + r] = M[ct];
                stat[wave][1][16 * ct + r] = sum[ct];
            }
        }
        __syncthreads();
        float* part = nullptr;
        // a tile that began before the stretch leaves its part in the first place, one that goes on in the second
        if (!whole) part = a.parts + ((size_t)blockIdx.x * 2 + (from > 0 ? 0 : 1)) * (size_t)(R * (D + 2));
#pragma unroll
        for (int ct = 0; ct < C; ++ct) {
            float m = stat[0][0][16 * ct + r];
#pragma unroll
            for (int x = 1; x < kW; ++x) m = fmaxf(m, stat[x][0][16 * ct + r]);
            float all = 0.0f;
#pragma unroll
            for (int x = 0; x < kW; ++x)
                all += stat[x][1][16 * ct + r] * __builtin_amdgcn_exp2f(stat[x][0][16 * ct + r] - m);
            const float down = __builtin_amdgcn_exp2f(M[ct] - m) * 0x1p24f;
            const int row = tile * R + 16 * ct + r;
            const bool live = row < l.rows;
            const int j = row / a.group, h = head * a.group + (row - j * a.group);
            const float inv = all == 0.0f ? 0.0f : 1.0f / all;
            const size_t at = (size_t)(l.start + j) * a.heads + h;
            for (int jb = 0; jb < VB; jb += JB) {
#pragma unroll
                for (int x = 0; x < VB; ++x)
                    if (x >= jb && x < jb + JB)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            join[wave][y][lane][x - jb] = (o[ct][x][y] - obias[ct][y]) * down;
                __syncthreads();
                float v[JB];
#pragma unroll
                for (int x = 0; x < JB; ++x) {
                    v[x] = join[0][wave][lane][x];
#pragma unroll
                    for (int z = 1; z < kW; ++z) v[x] += join[z][wave][lane][x];
                }
                // channels VB (4 g + wave) + jb ..
                const int d0 = VB * (4 * g + wave) + jb;
                if (d0 < D) {
                    if (whole) {
                        if (live) {
                            uint32_t* to = (uint32_t*)(a.out + at * D + d0);
#pragma unroll
                            for (int x = 0; x < JB; x += 2)
                                to[x / 2] = a.bf16 ? pack2<BF16>(v[x] * inv, v[x + 1] * inv) : pack2<F16>(v[x] * inv, v[x + 1] * inv);
                        }
                    } else if (live) {
                        float* to = part + 2 * R + (16 * ct + r) * D + d0;
#pragma unroll
                        for (int x = 0; x < JB; ++x) to[x] = v[x];
                    }
                }
                __syncthreads();
            }
            if (wave == 0 && g == 0) {
                if (!whole) {
                    part[16 * ct + r] = m;
                    part[R + 16 * ct + r] = all;
                } else if (live && a.lse) {
                    a.lse[at] = all == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(all)) * kLn2;
                }
            }
        }
        if (u >= u_end) return;
    }
}

// Joins the parts of a row (one of the call's, one head).  WAVES waves share a row:
// its parts in turns, four at a time in flight; one wave each where there are rows
// enough.
struct JoinArgs {
    AttendArgs a;
    int rows, dim;                       // of a tile
    int tile_parts;                      // 0: stretches; else the parts of a tile (attend_tile.hip)
};

template <int WAVES>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void k_attend_join(JoinArgs ja) {
    const AttendArgs& a = ja.a;
    const int R = ja.rows, D = ja.dim;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int id = __builtin_amdgcn_readfirstlane(WAVES == 1 ? blockIdx.x * 4 + wave : blockIdx.x);
    const Sequences& s = a.seqs;
    const int t = id / a.heads, h = id - t * a.heads;
    if (t >= s.T) return;
    const int b = s.of_row_by_wave(t);
    if (b < 0) return;
    const long long before = ja.tile_parts ? 0 : a.line[b], share = ja.tile_parts ? 1 : a.line[s.B];
    const Line l(a, b, R);
    const int head = h / a.group;
    const int row = (t - l.start) * a.group + (h - head * a.group);
    const int tile = row / R, in = row - tile * R;
    const size_t size = (size_t)(R * (D + 2));
    const float* base;
    int w0 = 0, w1;
    size_t second = 0, step;                       // what part w0's place is past base, and the others' distance
    if (ja.tile_parts) {
        w1 = TileSpan(a, l, R, tile, ja.tile_parts).parts - 1;
        if (w1 == 0) return;                       // written by its workgroup
        step = (size_t)a.cache.kv * size;
        base = a.parts + ((size_t)(first_place(a, R, b, l.start) + l.tiles - 1 - tile) * ja.tile_parts * a.cache.kv + head) * size;
    } else {
        const long long u0 = before + ((long long)head * l.tiles + tile) * l.tile_units();
        w0 = (int)quotient(u0 + kFixed, share);
        w1 = (int)quotient(u0 + l.tile_units() - 1, share);
        if (w0 == w1) return;                      // written by its workgroup
        // stretches that begin inside the tile leave their parts in the first place
        base = a.parts;
        step = 2 * size;
        second = u0 < w0 * share ? 0 : size;
    }
    auto part = [&](int w) { return base + (size_t)w * step + (w == w0 ? second : 0); };
    constexpr int kMost = 4, kDeep = 4;            // 64 channels at a time; parts in flight
    float m = kLow, all = 0.0f, v[kMost] = {0, 0, 0, 0};
    for (int w = w0 + (WAVES == 1 ? 0 : wave); w <= w1; w += WAVES * kDeep) {
        float pm[kDeep], ps[kDeep], pv[kDeep][kMost];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const float* p = part(min(w + WAVES * i, w1));
            pm[i] = p[in];
            ps[i] = p[R + in];
#pragma unroll
            for (int x = 0; x < kMost; ++x) pv[i][x] = lane + 64 * x < D ? p[2 * R + (size_t)in * D + lane + 64 * x] : 0.0f;
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            if (w + WAVES * i > w1) pm[i] = -INFINITY;       // a part twice
            top = fmaxf(top, pm[i]);
        }
        const float down = __builtin_amdgcn_exp2f(m - top);
        m = top;
        all *= down;
#pragma unroll
        for (int x = 0; x < kMost; ++x) v[x] *= down;
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const float f = __builtin_amdgcn_exp2f(pm[i] - m);
            all = __builtin_fmaf(ps[i], f, all);
#pragma unroll
            for (int x = 0; x < kMost; ++x) v[x] = __builtin_fmaf(pv[i][x], f, v[x]);
        }
    }
    if constexpr (WAVES > 1) {
        __shared__ float acc[WAVES][kMost][64], stat[WAVES][2];
#pragma unroll
        for (int x = 0; x < kMost; ++x) acc[wave][x][lane] = v[x];
        if (lane == 0) stat[wave][0] = m, stat[wave][1] = all;
        __syncthreads();
        if (wave > 0) return;
        float top = stat[0][0];
#pragma unroll
        for (int z = 1; z < WAVES; ++z) top = fmaxf(top, stat[z][0]);
        m = top;
        all = 0.0f;
#pragma unroll
        for (int x = 0; x < kMost; ++x) v[x] = 0.0f;
#pragma unroll
        for (int z = 0; z < WAVES; ++z) {
            const float f = __builtin_amdgcn_exp2f(stat[z][0] - m);
            all = __builtin_fmaf(stat[z][1], f, all);
#pragma unroll
            for (int x = 0; x < kMost; ++x) v[x] = __builtin_fmaf(acc[z][x][lane], f, v[x]);
        }
    }
    const float inv = all == 0.0f ? 0.0f : 1.0f / all;
    const size_t at = (size_t)t * a.heads + h;
#pragma unroll
    for (int x = 0; x < kMost; ++x)
        if (lane + 64 * x < D) a.out[at * D + lane + 64 * x] = a.bf16 ? BF16::store(v[x] * inv) : F16::store(v[x] * inv);
    if (lane == 0 && a.lse) a.lse[at] = all == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(all)) * kLn2;
}

// columns of 16 rows (0: attend_tile.hip's tiles), the workgroups and whether tiles
// are split over them
struct Plan {
    int columns, split, groups;
    TilePlan tile;
    long long keys;                                // of tiles: keys that one's rows see at most
    int rows() const { return columns ? 16 * columns : tile.rows; }
    int places() const { return columns ? 2 : 1; }           // parts that a workgroup may leave
};

size_t line_bytes(int B) { return ((size_t)B + 1) * sizeof(long long) / 16 * 16 + 16; }

// Up to 32 rows a kv head (a query's rows of all its heads): this file's kernel.  Up to 64
// as well while tiles of 128 rows would not fill the card: its stretches are even
// whatever the lengths, tiles are converted once for all their rows.  48 rows, 36
// sequences of 400 to 7800 tokens, 3 kv heads: 55 us here, 89 in tiles; 64 rows, 64
// sequences of 250 to 1000, 8 kv heads: 70 here, 49 in tiles; 128 rows, 16 of 500 to 2000:
// 53 here, 44 in tiles.
Plan plan(int T, int B, int heads, int kv, int dim, int max_new, int max_len, int window) {
    Plan p;
    p.keys = max_len;
    const int group = heads / kv, cus = device_cu_count();
    const long long rows = (long long)max_new * group;
    p.tile = TilePlan{0, 1};
    if (rows > 64 || (rows > 32 && (long long)B * kv >= 2 * cus)) {
        p.columns = 0;
        p.tile = tile_plan(T, B, group, kv, dim, max_new, max_len, cus);
        // With a window a tile has few keys however long the sequence is: parts by these, and by the length where it
        // is shorter (the workspace's size knows no window).  512 rows of 32 heads over 8 behind 100000 tokens, window 128:
        // 20 us, and 37 in the 4 parts that the length would give; window 4096: 72, in parts either way.
        if (window > 0 && window + (long long)p.tile.rows / group + kTileKeys < max_len) {
            p.keys = window + (long long)p.tile.rows / group + kTileKeys;
            p.tile.parts = min(p.tile.parts, tile_plan(T, B, group, kv, dim, max_new, (int)p.keys, cus).parts);
        }
        p.split = p.tile.parts > 1;
        p.groups = (int)(((long long)T * group / p.tile.rows + B) * kv * p.tile.parts);
        return p;
    }
    p.columns = rows <= 16 ? 1 : 2;
    // two steps a wave at least: shorter sequences go unsplit, a workgroup for each tile
    p.split = max_len > 2 * kW * kStep;
    p.groups = p.split ? cus * 2 : (int)(((long long)T * group / (16 * p.columns) + B) * kv);
    return p;
}

template <int D, int C>
void launch_c(const AttendArgs& a, hipStream_t st) {
    if (a.cache.page_log2 == 4)
        hipLaunchKernelGGL((k_attend<D, C, true>), dim3(a.groups), dim3(64 * kW), 0, st, a);
    else
        hipLaunchKernelGGL((k_attend<D, C, false>), dim3(a.groups), dim3(64 * kW), 0, st, a);
}

template <int D>
void launch_d(const AttendArgs& a, int columns, hipStream_t st) {
    if (columns == 1) return launch_c<D, 1>(a, st);
    return launch_c<D, 2>(a, st);
}

}  // namespace

size_t attend_workspace_bytes(int T, int B, int heads, int kv, int dim, int max_new, int max_len) {
    const Plan p = plan(T, B, heads, kv, dim, max_new, max_len, 0);
    if (!p.split) return 0;
    return line_bytes(B) + (size_t)p.groups * p.places() * p.rows() * (dim + 2) * sizeof(float);
}

int launch_cache_attention(const AttendProblem& p, void* workspace, hipStream_t st) {
    const Plan pl = plan(p.seqs.T, p.seqs.B, p.heads, p.cache.kv, p.cache.dim, p.max_new, p.max_len,
                         p.window);
    AttendArgs a{};
    a.q = (const uint16_t*)p.q;
    a.q_stride = p.q_stride;
    a.out = (uint16_t*)p.out;
    a.lse = p.lse;
    a.cache = p.cache;
    a.seqs = p.seqs;
    a.scale = fabsf(p.scale) * 0x1p24f;
    a.sign = p.scale < 0.0f ? -1.0f : 1.0f;
    a.softcap = p.softcap;
    a.heads = p.heads;
    a.group = p.heads / p.cache.kv;
    a.window = p.window;
    a.bf16 = p.dtype == AWQ_BF16;
    a.split = pl.split;
    // tiles of keys that a part takes: a tile's largest number of them, over the parts
    a.piece = (int)((pl.keys + kTileKeys - 1) / kTileKeys + pl.tile.parts - 1) / pl.tile.parts;
    a.groups = pl.groups;
    a.line = (long long*)workspace;
    a.parts = (float*)((char*)workspace + (pl.split ? line_bytes(p.seqs.B) : 0));
    int e = 0;
    if (!pl.columns) e = launch_attend_tile(a, pl.tile, st);
    else switch (p.cache.dim) {
        case 64: launch_d<64>(a, pl.columns, st); break;
        case 96: launch_d<96>(a, pl.columns, st); break;
        case 128: launch_d<128>(a, pl.columns, st); break;
        case 192: launch_d<192>(a, pl.columns, st); break;
        default: launch_d<256>(a, pl.columns, st); break;
    }
    if (e || (e = (int)hipGetLastError())) return e;
    if (!pl.split) return 0;
    const JoinArgs ja{a, pl.rows(), p.cache.dim, pl.columns ? 0 : pl.tile.parts};
    const unsigned rows = (unsigned)p.seqs.T * p.heads;
    if (rows < (unsigned)device_cu_count() * 4)
        hipLaunchKernelGGL((k_attend_join<16>), dim3(rows), dim3(1024), 0, st, ja);
    else
        hipLaunchKernelGGL((k_attend_join<1>), dim3((rows + 3) / 4), dim3(256), 0, st, ja);
    return (int)hipGetLastError();
}

}  // namespace awq
