// Rotary positions, and rows into and out of the paged 8-bit cache.
//
//   a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t),  t = position * inv_freq[i]
//
// for the pairs (a, b) of a head's first 2 * pairs channels: (i, i + pairs) or
// (2i, 2i + 1).  Angles of far positions need more than fp32 has: position and
// frequency are multiplied in 64 bits as turns (t / 2 pi), whole turns are taken
// off there, and only the rest goes to fp32's sine and cosine.
//
// Into the cache: the tokens x of a call that fall into one page make up a block
// of every kv head, with the scale s' = max(s, max|x| / 127), where s is the scale
// that the block had (0 if it held no tokens).  Codes that it held become
// rint(code * s / s'), the new ones are rint(x / s').  A workgroup (or a wave) owns a
// block, so nothing is exchanged.
//
// All of it is one pass over the rows and bound by memory: 4099 rows of 64 heads of 128,
// half of each turned, 29 us (4.6 TB/s); 16384 rows of 64 + 8 + 8 heads into the
// cache 154 us, half of them for the queries (4.2 TB/s with the read back, 19 us).  One row
// is a launch: 2.4 us for the kernel.  64 single tokens into pages that hold some: 7.4 us,
// three dependent loads (place, old scale and codes) behind the launch, and 9.3 where all
// held codes go to a new scale.
#include "cache.h"

namespace awq {
namespace {

constexpr int kNT = 256;

// cos and sin of a pair's angle, times the magnitude; inverse turns the other way
__device__ __forceinline__ float2 angle(const Rotation& r, int position, int i) {
    const double turns = (double)position * ((double)r.inv_freq[i] * 0.15915494309189533577);
    const float rest = (float)(turns - __builtin_rint(turns));
    float s, c;
    sincospif(2.0f * rest, &s, &c);
    return make_float2(r.magnitude * c, r.inverse ? -r.magnitude * s : r.magnitude * s);
}

// A head's channels go in units of 16 as two chunks of 8: unit j of the rotated
// part holds 8 pairs (two neighbouring chunks where pairs are interleaved, chunks j
// and j + pairs / 8 else), later units two neighbouring chunks.
struct Unit {
    int c0, c1;                          // channels of the chunks
    int pair;                            // its first pair, or -1: not rotated
    __device__ __forceinline__ Unit(const Rotation& r, int j) {
        const bool turned = r.inv_freq && j < r.pairs / 8;
        pair = turned ? 8 * j : -1;
        c0 = turned && !r.interleaved ? 8 * j : 16 * j;
        c1 = turned && !r.interleaved ? 8 * j + r.pairs : 16 * j + 8;
    }
};

// the rows of a and b (channels c0.. and c1..) rotated; cs: cos and sin of the unit's 8 pairs
__device__ __forceinline__ void rotate(float* v, const float2* cs, bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = v[2 * e], b = v[2 * e + 1];
            v[2 * e] = __builtin_fmaf(a, cs[e].x, -(b * cs[e].y));
            v[2 * e + 1] = __builtin_fmaf(b, cs[e].x, a * cs[e].y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = v[e], b = v[8 + e];
            v[e] = __builtin_fmaf(a, cs[e].x, -(b * cs[e].y));
            v[8 + e] = __builtin_fmaf(b, cs[e].x, a * cs[e].y);
        }
    }
}

// Rows [t0, t0 + n) of x, all heads, by one workgroup: positions in LDS (a row whose
// live is 0 is left alone), their angles once for all heads.
struct RowsArgs {
    const uint16_t* x;
    long long x_stride;
    uint16_t* out;
    long long out_stride;
    Rotation rot;
    int heads, dim;
};

constexpr int kRows = 4;                 // rows of a workgroup
constexpr int kMaxPairs = 256;

template <class E>
__device__ __forceinline__ void rotate_rows(const RowsArgs& a, int t0, int n, const int* positions, const int* live,
                                            float2* table) {
    if (a.rot.inv_freq) {
        for (int i = threadIdx.x; i < n * a.rot.pairs; i += kNT) {
            const int t = i / a.rot.pairs;
            table[i] = angle(a.rot, positions[t], i - t * a.rot.pairs);
        }
    }
    __syncthreads();
    const int per = a.dim / 16, units = a.heads * per;
    for (int i = threadIdx.x; i < n * units; i += kNT) {
        const int t = i / units;
        const int rest = i - t * units;
        const int h = rest / per;
        const Unit u(a.rot, rest - h * per);
        if (!live[t]) continue;
        const uint16_t* from = a.x + (size_t)(t0 + t) * a.x_stride + (size_t)h * a.dim;
        uint16_t* to = a.out + (size_t)(t0 + t) * a.out_stride + (size_t)h * a.dim;
        uint4 w0 = *(const uint4*)(from + u.c0), w1 = *(const uint4*)(from + u.c1);
        if (u.pair >= 0) {
            float v[16];
            unpack8<E>(w0, v);
            unpack8<E>(w1, v + 8);
            rotate(v, table + t * a.rot.pairs + u.pair, a.rot.interleaved);
            w0 = pack8<E>(v);
            w1 = pack8<E>(v + 8);
        }
        *(uint4*)(to + u.c0) = w0;
        *(uint4*)(to + u.c1) = w1;
    }
}

template <class E>
__global__ __launch_bounds__(kNT) void k_rope(RowsArgs a, const int* positions, int T) {
    __shared__ float2 table[kRows * kMaxPairs];
    __shared__ int pos[kRows], live[kRows];
    const int t0 = blockIdx.x * kRows, n = min(T - t0, kRows);
    if ((int)threadIdx.x < n) {
        pos[threadIdx.x] = positions[t0 + threadIdx.x];
        live[threadIdx.x] = 1;
    }
    __syncthreads();
    rotate_rows<E>(a, t0, n, pos, live, table);
}

struct AppendArgs {
    RowsArgs q;                          // q.x null: no queries
    const uint16_t* in[2];               // keys, values
    long long stride[2];
    Rotation rot;
    Cache cache;
    Sequences seqs;
    int items, by_rows;                  // of find_item
    int row_groups;                      // workgroups that rotate queries
};

// Item i of the call as (sequence, page of its table row), or sequence -1: by a wave.  With
// by_rows an item is a row, and the first one of a sequence in a page stands for the page;
// else sequence b has the items from start(b) / page + 2 b on, enough for its pages (n
// rows reach at most n / page + 2), and finding it takes the starts alone.
__device__ __forceinline__ int2 find_item(const Sequences& s, int page_log2, bool by_rows, int i) {
    int b;
    if (by_rows) {
        b = s.of_row_by_wave(i);
    } else {
        b = first_by_wave(s.B, [&](int k) { return (s.start(k + 1) >> page_log2) + 2 * (k + 1) > i; });
        if (b >= 0 && (s.start(b) >> page_log2) + 2 * b > i) b = -1;
    }
    if (b < 0) return make_int2(-1, 0);
    const int len = s.len(b), rows = s.rows(b), start = s.start(b);
    if (by_rows) {
        const int pos = len - rows + (i - start);              // below 0: not cached
        if (pos < 0 || ((pos & ((1 << page_log2) - 1)) != 0 && pos != max(len - rows, 0))) return make_int2(-1, 0);
        return make_int2(b, pos >> page_log2);
    }
    const int first = max(len - rows, 0);
    const int w = (first >> page_log2) + i - ((start >> page_log2) + 2 * b);
    return len > first && w <= (len - 1) >> page_log2 ? make_int2(b, w) : make_int2(-1, 0);
}

// the codes of a unit's 16 values, rint(v / s), by multiplication where it decides
// (|v| <= 127 s): v * inv is within 127 * 2^-22 of the quotient.  0 with a scale of 0 or
// one that is not finite, which then stands for the whole block.
__device__ __forceinline__ void unit_codes(const float* v, float s, float inv, uint2* c0, uint2* c1) {
    int k[16];
    float far = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float t = v[e] * inv, r = __builtin_rintf(t);
        k[e] = (int)r;
        far = fmaxf(far, fabsf(t - r));
    }
    const bool slow = !(far <= 0.5f - 0x1p-14f) || !(s >= 0x1p-100f && s < INFINITY);
    if (__builtin_amdgcn_ballot_w64(slow)) {
        if (slow) {
#pragma unroll
            for (int e = 0; e < 16; ++e) k[e] = s > 0.0f && s < INFINITY ? (int)__builtin_rintf(v[e] / s) : 0;
        }
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i] |= (uint32_t)(min(max(k[4 * i + e], -127), 127) & 255) << (8 * e);
    }
    *c0 = make_uint2(w[0], w[1]);
    *c1 = make_uint2(w[2], w[3]);
}

// A block (a page's tokens of one head) by W waves, all four of a workgroup or one: then
// four heads share the search for their page and the angles of its positions.  U: units of
// 16 channels that a thread holds, 64 W U >= page * dim / 16.
template <class E, int U, int W>
__global__ __launch_bounds__(kNT) void k_append(AppendArgs a) {
    constexpr int BT = 64 * W;                     // threads of a block
    __shared__ float2 table[kNT * 8];              // angles: of kRows rows of queries; of BT units (W = 4); of the page (W = 1)
    __shared__ int pos[kRows], live[kRows];
    __shared__ int2 item;
    __shared__ uint32_t slots[4];
    static_assert(kNT * 8 >= kRows * kMaxPairs / 2, "angles of a group's rows (dim at most 256)");
    const Sequences& s = a.seqs;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), bt = W == 4 ? tid : tid & 63;
    if ((int)blockIdx.x < a.row_groups) {          // queries
        const int t0 = blockIdx.x * kRows, n = min(s.T - t0, kRows);
        static_assert(kRows == kNT / 64, "a wave finds a row's sequence");
        if (wave < n) {
            const int b = s.of_row_by_wave(t0 + wave);
            if ((tid & 63) == 0) {
                live[wave] = b >= 0;
                pos[wave] = b >= 0 ? s.len(b) - s.rows(b) + (t0 + wave - s.start(b)) : 0;
            }
        }
        __syncthreads();
        rotate_rows<E>(a.q, t0, n, pos, live, table);
        return;
    }
    const int kv = a.cache.kv, dim = a.cache.dim, page_log2 = a.cache.page_log2;
    const int groups = W == 4 ? kv : (kv + 3) / 4;                   // of heads
    const int at = blockIdx.x - a.row_groups;
    const int which = at & 1;                      // keys, values
    const int head = W == 4 ? (at >> 1) % groups : (at >> 1) % groups * 4 + wave;
    if (wave == 0) {
        const int2 f = find_item(s, page_log2, a.by_rows, (at >> 1) / groups);
        if (tid == 0) item = f;
    }
    __syncthreads();
    const int b = item.x, w = item.y;
    if (b < 0 || w < 0) return;
    const int page_id = s.page(b, w, a.cache.pages);
    if (page_id < 0) return;
    const int len = s.len(b), first = max(len - s.rows(b), 0);
    const int lo = max(first, w << page_log2);                       // positions [lo, hi) are written
    const int hi = (int)min((long long)len, (long long)(w + 1) << page_log2);
    const int slot0 = lo - (w << page_log2), n = hi - lo;
    // rows of the call: the last one of the sequence is position len - 1
    const int row0 = s.start(b) + s.rows(b) - (len - lo);
    const uint16_t* x = a.in[which] + (size_t)row0 * a.stride[which] + (size_t)head * dim;
    Rotation rot = a.rot;
    if (which == 1) rot.inv_freq = nullptr;
    const int per = dim / 16;
    const int units = W == 4 || head < kv ? n * per : 0;             // a wave without a head only helps with the angles

    float v[U][16];
    uint32_t top = 0;
    {
        uint4 raw[U][2];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = bt + BT * i;
            raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
            if (BT * i < units && u < units) {
                const int t = u / per;
                const Unit unit(rot, u - t * per);
                const uint16_t* r = x + (size_t)t * a.stride[which];
                raw[i][0] = *(const uint4*)(r + unit.c0);
                raw[i][1] = *(const uint4*)(r + unit.c1);
            }
        }
        if (W == 1 && rot.inv_freq) {              // while the rows are on their way
            for (int k = tid; k < n * rot.pairs; k += kNT) {
                const int t = k / rot.pairs;
                table[k] = angle(rot, lo + t, k - t * rot.pairs);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            unpack8<E>(raw[i][0], v[i]);
            unpack8<E>(raw[i][1], v[i] + 8);
        }
    }
    if (rot.inv_freq) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u0 = BT * i, count = min(units - u0, BT);
            if (count <= 0) break;
            if constexpr (W == 4) {
                // the angles of this step's units, 8 pairs each, by all threads
                if (i) __syncthreads();
                for (int k = tid; k < 8 * count; k += kNT) {
                    const int u = u0 + k / 8, t = u / per;
                    const Unit unit(rot, u - t * per);
                    if (unit.pair >= 0) table[k] = angle(rot, lo + t, unit.pair + (k & 7));
                }
                __syncthreads();
            }
            const int u = u0 + bt, t = u / per;
            const Unit unit(rot, u - t * per);
            if (u < units && unit.pair >= 0)
                rotate(v[i], table + (W == 4 ? 8 * tid : t * rot.pairs + unit.pair), rot.interleaved);
        }
    }
    if (units == 0) return;                        // W = 1: no barrier from here on
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = max(top, abs_bits(v[i][e]));
    const float amax = __builtin_bit_cast(float, group_reduce<W>(top, slots, MaxU32()));

    float* scale = a.cache.scales[which] + (size_t)page_id * kv + head;
    int8_t* block = a.cache.codes[which] + a.cache.block(page_id, head);
    const float before = slot0 > 0 ? *scale : 0.0f;
    // the larger one, and NaN if either is
    const float top127 = amax / 127.0f;
    const float after = before >= top127 || before != before ? before : top127;
    if (W == 4) __syncthreads();                   // everyone has read the old scale
    if (bt == 0) *scale = after;
    if (after > before && slot0 > 0) {             // the codes that the block held, on the new scale
        const float shrink = before / after;
        uint4* held = (uint4*)block;
        for (int i = bt; i < slot0 * per; i += BT) {
            uint4 c = held[i];
            uint32_t* words = (uint32_t*)&c;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t r = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    r |= (uint32_t)((int)__builtin_rintf((float)(int8_t)(words[k] >> (8 * e)) * shrink) & 255) << (8 * e);
                words[k] = r;
            }
            held[i] = c;
        }
    }
    const float inv = after > 0.0f ? 1.0f / after : 0.0f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = bt + BT * i;
        if (BT * i >= units) break;
        uint2 c0, c1;
        unit_codes(v[i], after, inv, &c0, &c1);
        if (u < units) {
            const int t = u / per;
            const Unit unit(rot, u - t * per);
            int8_t* r = block + (size_t)(slot0 + t) * dim;
            *(uint2*)(r + unit.c0) = c0;
            *(uint2*)(r + unit.c1) = c1;
        }
    }
}

struct ReadArgs {
    Cache cache;
    Sequences seqs;
    uint16_t* out[2];
};

// The sequences' last rows as the values that their codes stand for: 4 rows a
// workgroup, 16 codes a thread at a time.
template <class E>
__global__ __launch_bounds__(kNT) void k_read(ReadArgs a) {
    __shared__ int where[kRows][2];                // page (-1: no token, -2: no row), slot
    const Sequences& s = a.seqs;
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * kRows, n = min(s.T - t0, kRows);
    const int page_log2 = a.cache.page_log2, kv = a.cache.kv, dim = a.cache.dim;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);           // a row each
    if (wave < n) {
        const int b = s.of_row_by_wave(t0 + wave);
        int page = -2, pos = 0;
        if (b >= 0) {
            pos = s.len(b) - s.rows(b) + (t0 + wave - s.start(b));
            page = pos >= 0 ? s.page(b, pos >> page_log2, a.cache.pages) : -1;
        }
        if ((tid & 63) == 0) {
            where[wave][0] = page;
            where[wave][1] = pos & (a.cache.page() - 1);
        }
    }
    __syncthreads();
    const int per = dim / 16, units = 2 * kv * per;
    for (int i = tid; i < n * units; i += kNT) {
        const int t = i / units;
        int rest = i - t * units;
        const int which = rest >= kv * per;
        rest -= which * kv * per;
        const int h = rest / per, c = (rest - h * per) * 16;
        const int page = where[t][0];
        if (page == -2) continue;
        float v[16];
        if (page >= 0) {
            const int8_t* from = a.cache.codes[which] + a.cache.block(page, h) + (size_t)where[t][1] * dim + c;
            const uint4 q = *(const uint4*)from;
            const float scale = a.cache.scales[which][(size_t)page * kv + h];
            const uint32_t words[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = (float)(int8_t)(words[e / 4] >> (8 * (e % 4))) * scale;
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.0f;
        }
        uint4* to = (uint4*)(a.out[which] + ((size_t)(t0 + t) * kv + h) * dim + c);
        to[0] = pack8<E>(v);
        to[1] = pack8<E>(v + 8);
    }
}

template <class E, int U, int W>
int launch_append_t(const AppendArgs& a, hipStream_t st) {
    const unsigned groups = a.row_groups + 2u * a.items * (W == 4 ? a.cache.kv : (a.cache.kv + 3) / 4);
    hipLaunchKernelGGL((k_append<E, U, W>), dim3(groups), dim3(kNT), 0, st, a);
    return (int)hipGetLastError();
}

// A wave a block where a wave can hold it: four heads then share a page's search and its
// angles (3374 rows of 3 sequences, 16-token pages of 8 heads of 128: 23 us with a
// workgroup a block, 19 with a wave).  One row a sequence is one token a block.
template <class E>
int pick_append(const AppendArgs& a, hipStream_t st) {
    if (!a.seqs.starts) return launch_append_t<E, 1, 1>(a, st);
    const int units = a.cache.page() * a.cache.dim / 16;
    if (units <= 128) return launch_append_t<E, 2, 1>(a, st);
    if (units <= 256) return launch_append_t<E, 4, 1>(a, st);
    if (units <= 512) return launch_append_t<E, 2, 4>(a, st);
    if (units <= 1024) return launch_append_t<E, 4, 4>(a, st);
    return launch_append_t<E, 8, 4>(a, st);
}

}  // namespace

int launch_rope(const RopeProblem& p, hipStream_t st) {
    const RowsArgs a{(const uint16_t*)p.x, p.x_stride, (uint16_t*)p.out, p.out_stride, p.rot, p.heads, p.dim};
    const dim3 grid((p.T + kRows - 1) / kRows);
    if (p.dtype == AWQ_BF16)
        hipLaunchKernelGGL((k_rope<BF16>), grid, dim3(kNT), 0, st, a, p.positions, p.T);
    else
        hipLaunchKernelGGL((k_rope<F16>), grid, dim3(kNT), 0, st, a, p.positions, p.T);
    return (int)hipGetLastError();
}

int launch_cache_append(const AppendProblem& p, hipStream_t st) {
    AppendArgs a{};
    a.q = RowsArgs{(const uint16_t*)p.q, p.q_stride, (uint16_t*)p.q_out, (long long)p.heads * p.cache.dim, p.rot,
                   p.heads, p.cache.dim};
    a.in[0] = (const uint16_t*)p.k;
    a.in[1] = (const uint16_t*)p.v;
    a.stride[0] = p.k_stride;
    a.stride[1] = p.v_stride;
    a.rot = p.rot;
    a.cache = p.cache;
    a.seqs = p.seqs;
    const long long most = (p.seqs.T >> p.cache.page_log2) + 2LL * p.seqs.B;
    a.by_rows = !p.seqs.starts || p.seqs.T <= most;
    a.items = a.by_rows ? p.seqs.T : (int)most;
    a.row_groups = p.q ? (p.seqs.T + kRows - 1) / kRows : 0;
    return p.dtype == AWQ_BF16 ? pick_append<BF16>(a, st) : pick_append<F16>(a, st);
}

int launch_cache_read(const ReadProblem& p, hipStream_t st) {
    const ReadArgs a{p.cache, p.seqs, {(uint16_t*)p.k_out, (uint16_t*)p.v_out}};
    const dim3 grid((p.seqs.T + kRows - 1) / kRows);
    if (p.dtype == AWQ_BF16)
        hipLaunchKernelGGL((k_read<BF16>), grid, dim3(kNT), 0, st, a);
    else
        hipLaunchKernelGGL((k_read<F16>), grid, dim3(kNT), 0, st, a);
    return (int)hipGetLastError();
}

}  // namespace awq
