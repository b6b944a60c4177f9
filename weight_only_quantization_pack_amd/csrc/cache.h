// Declarations shared by the operators of the paged 8-bit key and value cache
// (rope.hip, pages.hip, attend.hip and the C ABI layer).
#pragma once

#include "rows.h"

namespace awq {

// One layer's cache: codes int8 [pages][kv][page][dim] and a scale for each
// (page, kv head), keys and values apart.
struct Cache {
    int8_t* codes[2];                    // keys, values
    float* scales[2];
    int pages, kv, page_log2, dim;
    __host__ __device__ int page() const { return 1 << page_log2; }
    // first code of a page's block of one head: page * kv passes 2^31 bytes early
    __host__ __device__ size_t block(int page_id, int head) const {
        return (((size_t)page_id * (size_t)kv + (size_t)head) << page_log2) * (size_t)dim;
    }
};

// The first i in 0..n-1 with above(i), for an `above` that stays true once it is; -1 without
// one.  By a whole wave, 64 places a load.  (Whatever `above` says, i is in 0..n-1.)
template <class F>
__device__ __forceinline__ int first_by_wave(int n, F above) {
    const int lane = threadIdx.x & 63;
    int lo = 0;
    while (n > 64) {
        const int step = (n + 63) / 64;            // lane i looks at the end of its stretch of `step` places
        const uint64_t hit = __builtin_amdgcn_ballot_w64(above(lo + min((lane + 1) * step, n) - 1));
        if (!hit) return -1;
        const int i = __builtin_ctzll(hit);
        lo += i * step;
        n = min(step, n - i * step);
    }
    const uint64_t hit = __builtin_amdgcn_ballot_w64(lane < n && above(lo + min(lane, n - 1)));
    return hit ? lo + __builtin_ctzll(hit) : -1;
}

// The sequences of a call.  Sequence b holds lens[b] tokens, the last starts[b + 1]
// - starts[b] of which are rows starts[b].. of the call's T rows (starts null: one
// row each).  All of it is device data that the host has not seen: an accessor
// brings every row number into 0..T and every page lookup into the table, and a
// page outside the cache reads as -1, the page that holds no tokens.
struct Sequences {
    const int *tables, *lens, *starts;
    int T, B, W;
    __device__ __forceinline__ int start(int b) const { return starts ? min(max(starts[b], 0), T) : b; }
    __device__ __forceinline__ int rows(int b) const { return starts ? max(start(b + 1) - start(b), 0) : 1; }
    __device__ __forceinline__ int len(int b) const { return max(lens[b], 0); }
    // of `len` tokens those that a table row has room for
    __device__ __forceinline__ int span(int len, int page_log2) const {
        return (int)min((long long)len, (long long)W << page_log2);
    }
    __device__ __forceinline__ int page(int b, int w, int pages) const {
        const int p = (unsigned)w < (unsigned)W ? tables[(size_t)b * W + w] : -1;
        return (unsigned)p < (unsigned)pages ? p : -1;
    }
    // the sequence of row t, or -1 behind the last one; by a whole wave, t the same in all lanes
    __device__ __forceinline__ int of_row_by_wave(int t) const {
        if (!starts) return t < B ? t : -1;
        const int b = first_by_wave(B, [&](int i) { return starts[i + 1] > t; });
        return b >= 0 && starts[b] <= t ? b : -1;
    }
};

// inclusive prefix of v over the lanes (DPP: no LDS round trip)
__device__ __forceinline__ uint32_t lane_prefix(uint32_t v) {
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true);   // row_shr:1
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, true);   // row_shr:2
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, true);   // row_shr:4
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, true);   // row_shr:8
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);  // row_bcast:15
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);  // row_bcast:31
    return v;
}

struct Rotation {
    const float* inv_freq;               // [pairs], or null: no rotation
    float magnitude;
    int pairs;                           // rotated channels / 2, a multiple of 8
    int interleaved;
    int inverse;
};

struct RopeProblem {
    const void* x;
    long long x_stride;                  // elements from a row to the next
    const int* positions;
    void* out;
    long long out_stride;
    Rotation rot;
    int T, heads, dim, dtype;
};
int launch_rope(const RopeProblem& p, hipStream_t st);

struct AppendProblem {
    const void *q, *k, *v;               // q may be null
    long long q_stride, k_stride, v_stride;
    void* q_out;
    Rotation rot;
    Cache cache;
    Sequences seqs;
    int heads, dtype;
};
int launch_cache_append(const AppendProblem& p, hipStream_t st);

struct ReadProblem {
    Cache cache;
    Sequences seqs;
    void *k_out, *v_out;
    int dtype;
};
int launch_cache_read(const ReadProblem& p, hipStream_t st);

// scores: cap * tanh(scale * q.k / cap) with softcap > 0, scale * q.k without
struct AttendProblem {
    const void* q;
    long long q_stride;
    void* out;
    float* lse;                          // or null
    Cache cache;
    Sequences seqs;
    float scale, softcap;
    int heads, window, max_new, max_len, dtype;
};
size_t attend_workspace_bytes(int T, int B, int heads, int kv, int dim, int max_new, int max_len);
int launch_cache_attention(const AttendProblem& p, void* workspace, hipStream_t st);

constexpr int kMaxReserveRows = 4096;    // a call's rows are kept in LDS
int launch_cache_fork(const int* tables, const int* lens, int* refs, const int* parents, int* out_tables,
                      int* out_lens, int B, int B_out, int W, int pages, int page_log2, hipStream_t st);
int launch_cache_reserve(int* tables, int* lens, int* refs, const int* counts, int* pairs, int* status, int B,
                         int W, int pages, int page_log2, hipStream_t st);
int launch_cache_compact(int* tables, const int* lens, int* refs, int* moves, int* count, int B, int W, int pages,
                         int page_log2, hipStream_t st);

constexpr int kMaxCopyTensors = 8;
struct CopyProblem {
    char* tensors[kMaxCopyTensors];
    size_t page_bytes[kMaxCopyTensors];  // multiples of 4
    int n, layers, max_pairs, pages;
    const int *pairs, *count;            // count may be null
};
int launch_cache_copy_pages(const CopyProblem& p, hipStream_t st);

}  // namespace awq
