// The bookkeeping of a cache whose pages sequences share, on the device.
//
// tables[b][0 .. ceil(lens[b] / page)) are the pages of sequence b; refs[p] counts
// the table rows that hold page p (0: free).  Four calls: a batch of rows from its
// parents (forked, reordered, dropped), room for new tokens (lowest free pages
// first; a last page that others hold too is replaced by a copy before it is
// written), used pages moved to the front of the cache, and the copies of whole
// pages that the last two ask for.
//
// All but the copies are integers by the thousand: a launch and a few dependent
// loads are their cost (64 rows of up to 32 pages: fork 4 us, reserve 11; compact over
// 5300 pages 19 and its table cells 5).  The copies run at the rate of memory: 2.3 GB
// moved in 487 us, 4.8 TB/s.  Their results do not depend on any order: counts change
// by integer atomics, and whatever is ranked is ranked by a scan.
#include "cache.h"

namespace awq {
namespace {

__device__ __forceinline__ int pages_of(int len, int page_log2) {
    return len > 0 ? ((len - 1) >> page_log2) + 1 : 0;
}

// rows [b_out] from rows [parents[b_out]]; one thread for each table cell.  Old
// rows give their references back, new ones take theirs; a row that stays where
// it is does neither.
__global__ __launch_bounds__(256) void k_fork(const int* tables, const int* lens, int* refs, const int* parents,
                                              int* out_tables, int* out_lens, int B, int B_out, int W, int pages,
                                              int page_log2) {
    const int w = blockIdx.x * 256 + threadIdx.x;
    const int b = blockIdx.y;
    if (w >= W) return;
    if (b < B_out) {
        const int parent = parents[b];
        const bool alive = (unsigned)parent < (unsigned)B;
        const int len = alive ? max(lens[parent], 0) : 0;
        const int p = w < pages_of(len, page_log2) ? tables[(size_t)parent * W + w] : -1;
        out_tables[(size_t)b * W + w] = p;
        if (w == 0) out_lens[b] = len;
        if (parent != b && (unsigned)p < (unsigned)pages) atomicAdd(refs + p, 1);
    }
    if (b < B && (b >= B_out || parents[b] != b) && w < pages_of(lens[b], page_log2)) {
        const int p = tables[(size_t)b * W + w];
        if ((unsigned)p < (unsigned)pages) atomicAdd(refs + p, -1);
    }
}

constexpr int kT = 1024, kWaves = kT / 64;     // one workgroup that sees the whole book

// Exclusive prefix of v >= 0 over the workgroup's threads, and the total.  `slots` holds
// kWaves words; two barriers.
__device__ __forceinline__ int group_scan(int v, int* slots, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int s = (int)lane_prefix((uint32_t)v);
    if (lane == 63) slots[wave] = s;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const int c = slots[w];
        if (w < wave) before += c;
        total += c;
    }
    __syncthreads();
    return before + s - v;
}

// A look over refs[0 .. pages) in chunks of kWaves * 1024 pages (each wave 16 lines of 64
// in order, so that ranks follow page numbers) for the pages with pick(page, ref).
constexpr int kLines = 16, kChunk = kT * kLines;
template <class Pick>
struct Ranked {
    const int* refs;
    int pages;
    int* slots;
    Pick pick;
    uint64_t hit[kLines];                // of the chunk looked at last
    int before;                          // its pages that were picked in waves before this one
    // looks at a chunk, says how many it holds; two barriers
    __device__ __forceinline__ int chunk(int base) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int first = base + wave * (64 * kLines) + lane;
        int r[kLines];
#pragma unroll
        for (int i = 0; i < kLines; ++i) r[i] = first + 64 * i < pages ? refs[first + 64 * i] : 0;
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kLines; ++i) {
            const int p = first + 64 * i;
            hit[i] = __builtin_amdgcn_ballot_w64(p < pages && pick(p, r[i]));
            mine += __builtin_popcountll(hit[i]);
        }
        if (lane == 0) slots[wave] = mine;
        __syncthreads();
        int total = 0;
        before = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int c = slots[w];
            if (w < wave) before += c;
            total += c;
        }
        __syncthreads();
        return total;
    }
    // f(page, rank) for the chunk's picked pages, `met` of which came in chunks before
    template <class F>
    __device__ __forceinline__ void each(int base, int met, F f) const {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        int rank = met + before;
#pragma unroll
        for (int i = 0; i < kLines; ++i) {
            if (hit[i] >> lane & 1)
                f(base + wave * (64 * kLines) + 64 * i + lane, rank + __builtin_popcountll(hit[i] & ((1ull << lane) - 1)));
            rank += __builtin_popcountll(hit[i]);
        }
    }
    // the bases of the chunks: base + kChunk may pass 2^31
    __device__ __forceinline__ bool next(int& base) const {
        if (base > pages - kChunk) return false;
        base += kChunk;
        return base < pages;
    }
    // counts until `most` are met (or all)
    __device__ __forceinline__ int count(int most) {
        int met = 0, base = 0;
        do met += chunk(base); while (met < most && next(base));
        return met;
    }
    template <class F>
    __device__ __forceinline__ int all(int most, F f) {
        int met = 0, base = 0;
        do {
            const int n = chunk(base);
            each(base, met, f);
            met += n;
        } while (met < most && next(base));
        return met;
    }
};
template <class Pick>
__device__ __forceinline__ Ranked<Pick> ranked(const int* refs, int pages, int* slots, Pick pick) {
    return {refs, pages, slots, pick, {}, 0};
}

__global__ __launch_bounds__(kT) void k_reserve(int* tables, int* lens, int* refs, const int* counts, int* pairs,
                                                int* status, int B, int W, int pages, int page_log2) {
    constexpr int R = kMaxReserveRows / kT;
    __shared__ int writer[kMaxReserveRows];        // the shared page that a row writes to, or -1
    __shared__ int offset[kMaxReserveRows + 1];    // fresh pages before a row
    __shared__ int slots[kWaves];
    const int tid = threadIdx.x;
    const int per = (B + kT - 1) / kT;             // rows of a thread, in order
    int len[R], fresh[R], cow[R], last[R];
    int over = 0, any = 0;
    bool full = false;                             // a length that passes 31 bits
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int b = tid * per + i;
        fresh[i] = cow[i] = len[i] = 0;
        last[i] = -1;
        if (i >= per || b >= B) continue;
        len[i] = max(lens[b], 0);
        const int n = max(counts[b], 0);
        const int have = pages_of(len[i], page_log2);
        const long long total = (long long)len[i] + n;
        const long long want = (total + (1 << page_log2) - 1) >> page_log2;
        full = total > 0x7FFFFFFFLL || want > W;
        over += full;
        fresh[i] = full ? 0 : (int)want - have;
        int w = -1;
        if (!full && n > 0 && (len[i] & ((1 << page_log2) - 1)) != 0) {
            last[i] = tables[(size_t)b * W + have - 1];
            if ((unsigned)last[i] < (unsigned)pages && refs[last[i]] > 1) w = last[i];
        }
        writer[b] = w;
        any |= w >= 0;
        pairs[2 * b] = pairs[2 * b + 1] = -1;
    }
    // a barrier for `writer` as well
    if (__syncthreads_or(any)) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int b = tid * per + i;
            if (i >= per || b >= B || writer[b] < 0) continue;
            int same = 0, lower = 0;
            for (int o = 0; o < B; ++o) {
                const int hit = writer[o] == writer[b];
                same += hit;
                lower += hit & (o < b);
            }
            // the first of a page's writers keeps it where no one else holds it
            cow[i] = !(lower == 0 && same == refs[writer[b]]);
            fresh[i] += cow[i];
        }
    }
    int mine = 0, need = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) mine += fresh[i];
    int at = group_scan(mine, slots, need);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int b = tid * per + i;
        if (i >= per || b >= B) continue;
        offset[b] = at;
        at += fresh[i];
        writer[b] = cow[i] ? last[i] : -1;         // from here on: the page that a row copies
    }
    if (tid == 0) offset[B] = need;
    __syncthreads();
    auto free_pages = ranked(refs, pages, slots, [](int, int r) { return r == 0; });
    const int met = need > 0 ? free_pages.count(need) : 0;
    int overs = 0;
    group_scan(over, slots, overs);
    if (tid == 0) {
        status[0] = max(need - met, 0);
        status[1] = overs;
    }
    if (met < need || overs > 0) return;           // nothing changes
    // the page of rank r goes to the row whose fresh pages hold r
    auto take = [&](int p, int r) {
        if (r >= need) return;
        int lo = 0, hi = B;                        // the last row with offset <= r; rows without fresh pages
        while (hi - lo > 1) {                      // share their offset with the next one and are passed over
            const int mid = (lo + hi) >> 1;
            if (offset[mid] <= r) lo = mid; else hi = mid;
        }
        const int have = pages_of(max(lens[lo], 0), page_log2);
        const int src = writer[lo];
        const int i = r - offset[lo] - (src >= 0);
        refs[p] = 1;
        tables[(size_t)lo * W + have + i] = p;     // i = -1: the copy in place of the last page
        if (i < 0) {
            pairs[2 * lo] = src;
            pairs[2 * lo + 1] = p;
        }
    };
    if (need > 0) {
        if (pages <= kChunk) free_pages.each(0, 0, take); else free_pages.all(need, take);
    }
    __syncthreads();                               // every lens read, every free page ranked
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int b = tid * per + i;
        if (i >= per || b >= B) continue;
        if (cow[i]) atomicAdd(refs + last[i], -1);
        lens[b] = len[i] + max(counts[b], 0);
    }
}

// Moves: the k-th used page behind the first `used` goes to the k-th free one
// among them.  refs follow here, table rows in the launch after.
__global__ __launch_bounds__(kT) void k_compact(int* refs, int* moves, int* count, int pages) {
    __shared__ int slots[kWaves];
    const int tid = threadIdx.x;
    const int all = 0x7FFFFFFF;
    auto is_used = ranked(refs, pages, slots, [](int, int r) { return r > 0; });
    const int used = is_used.count(all);
    const int holes = ranked(refs, used, slots, [](int, int r) { return r <= 0; }).all(all, [&](int p, int k) {
        moves[2 * (size_t)k + 1] = p;
    });
    ranked(refs + used, pages - used, slots, [](int, int r) { return r > 0; }).all(all, [&](int p, int k) {
        moves[2 * (size_t)k] = used + p;
    });
    if (tid == 0) *count = holes;
    for (int k = holes + tid; k < pages; k += kT) moves[2 * (size_t)k] = moves[2 * (size_t)k + 1] = -1;
    __threadfence();
    __syncthreads();
    for (int k = tid; k < holes; k += kT) {
        const int src = moves[2 * (size_t)k], dst = moves[2 * (size_t)k + 1];
        refs[dst] = refs[src];
        refs[src] = 0;
    }
}

// page ids of the rows by the moves, whose sources ascend
__global__ __launch_bounds__(256) void k_remap(int* tables, const int* lens, const int* moves, const int* count, int B,
                                               int W, int page_log2) {
    const int w = blockIdx.x * 256 + threadIdx.x, b = blockIdx.y;
    if (w >= W || w >= pages_of(lens[b], page_log2)) return;
    int& cell = tables[(size_t)b * W + w];
    const int p = cell;
    int lo = 0, hi = *count;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (moves[2 * (size_t)mid] < p) lo = mid + 1; else hi = mid;
    }
    if (lo < *count && moves[2 * (size_t)lo] == p) cell = moves[2 * (size_t)lo + 1];
}

// Copies of pages.  A unit is up to kSpan bytes of one page of one tensor and layer;
// workgroups take units in turns.  A short list that comes without a count is mostly
// empty (a pair for each row of a batch): its valid pairs are gathered first.
constexpr int kSpan = 8192, kGather = 4096;
struct CopyArgs {
    CopyProblem p;
    int first[kMaxCopyTensors + 1];      // units of a page before each tensor's
};

__global__ __launch_bounds__(256) void k_copy_pages(CopyArgs a) {
    __shared__ int gathered[kGather], counts[4];
    const CopyProblem& p = a.p;
    const int per = a.first[kMaxCopyTensors];
    auto valid = [&](int src, int dst) { return (unsigned)src < (unsigned)p.pages && (unsigned)dst < (unsigned)p.pages; };
    int n = p.count ? min(max(*p.count, 0), p.max_pairs) : p.max_pairs;
    const bool gather = !p.count && n <= kGather;
    if (gather) {
        // in the list's order, the same in every workgroup: a quarter of the list a wave,
        // counted and then placed
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int quarter = (n + 255) / 256 * 64, end = min(n, (wave + 1) * quarter);
        auto hits = [&](int i) {
            return __builtin_amdgcn_ballot_w64(i + lane < end && valid(p.pairs[2 * (i + lane)], p.pairs[2 * (i + lane) + 1]));
        };
        int mine = 0;
        for (int i = wave * quarter; i < end; i += 64) mine += __builtin_popcountll(hits(i));
        if (lane == 0) counts[wave] = mine;
        __syncthreads();
        int at = 0;
        n = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) at += counts[w];
            n += counts[w];
        }
        for (int i = wave * quarter; i < end; i += 64) {
            const uint64_t hit = hits(i);
            if (hit >> lane & 1) gathered[at + __builtin_popcountll(hit & ((1ull << lane) - 1))] = i + lane;
            at += __builtin_popcountll(hit);
        }
        __syncthreads();
    }
    const size_t units = (size_t)n * p.layers * per;
    for (size_t u = blockIdx.x; u < units; u += gridDim.x) {
        size_t pair, layer;
        int part;
        if (units >> 32 == 0) {
            const uint32_t rest = (uint32_t)u / (uint32_t)per;
            part = (int)((uint32_t)u - rest * (uint32_t)per);
            pair = rest / (uint32_t)p.layers;
            layer = rest - (uint32_t)pair * (uint32_t)p.layers;
        } else {
            part = (int)(u % per);
            pair = u / per / p.layers;
            layer = u / per % p.layers;
        }
        if (gather) pair = gathered[pair];
        const int src = p.pairs[2 * pair], dst = p.pairs[2 * pair + 1];
        if (!valid(src, dst)) continue;
        char* tensor = p.tensors[0];
        size_t bytes = p.page_bytes[0];
        int first = 0;
#pragma unroll
        for (int t = 1; t < kMaxCopyTensors; ++t)
            if (part >= a.first[t]) {
                tensor = p.tensors[t];
                bytes = p.page_bytes[t];
                first = a.first[t];
            }
        const size_t at = (size_t)(part - first) * kSpan;
        const size_t left = bytes - at < kSpan ? bytes - at : (size_t)kSpan;
        char* base = tensor + layer * (size_t)p.pages * bytes + at;
        const char* from = base + (size_t)src * bytes;
        char* to = base + (size_t)dst * bytes;
        if (bytes % 16 == 0) {
            const uint4* f = (const uint4*)from;
            uint4* d = (uint4*)to;
            const int words = (int)(left / 16);
            if (words == kSpan / 16) {
                uint4 v[kSpan / 4096];
#pragma unroll
                for (int i = 0; i < kSpan / 4096; ++i) v[i] = f[threadIdx.x + 256 * i];
#pragma unroll
                for (int i = 0; i < kSpan / 4096; ++i) d[threadIdx.x + 256 * i] = v[i];
            } else {
                for (int i = threadIdx.x; i < words; i += 256) d[i] = f[i];
            }
        } else {
            for (int i = threadIdx.x; i < (int)(left / 4); i += 256) ((uint32_t*)to)[i] = ((const uint32_t*)from)[i];
        }
    }
}

}  // namespace

int launch_cache_fork(const int* tables, const int* lens, int* refs, const int* parents, int* out_tables,
                      int* out_lens, int B, int B_out, int W, int pages, int page_log2, hipStream_t st) {
    hipLaunchKernelGGL(k_fork, dim3((W + 255) / 256, max(B, B_out)), dim3(256), 0, st, tables, lens, refs, parents,
                       out_tables, out_lens, B, B_out, W, pages, page_log2);
    return (int)hipGetLastError();
}

int launch_cache_reserve(int* tables, int* lens, int* refs, const int* counts, int* pairs, int* status, int B,
                         int W, int pages, int page_log2, hipStream_t st) {
    hipLaunchKernelGGL(k_reserve, dim3(1), dim3(kT), 0, st, tables, lens, refs, counts, pairs, status, B, W, pages,
                       page_log2);
    return (int)hipGetLastError();
}

int launch_cache_compact(int* tables, const int* lens, int* refs, int* moves, int* count, int B, int W, int pages,
                         int page_log2, hipStream_t st) {
    hipLaunchKernelGGL(k_compact, dim3(1), dim3(kT), 0, st, refs, moves, count, pages);
    if (int e = (int)hipGetLastError()) return e;
    if (B == 0 || W == 0) return 0;
    hipLaunchKernelGGL(k_remap, dim3((W + 255) / 256, B), dim3(256), 0, st, tables, lens, moves, count, B, W, page_log2);
    return (int)hipGetLastError();
}

int launch_cache_copy_pages(const CopyProblem& p, hipStream_t st) {
    CopyArgs a{p, {0}};
    // tensors that are not there begin behind the last unit
    for (int t = 0; t < kMaxCopyTensors; ++t)
        a.first[t + 1] = a.first[t] + (t < p.n ? (int)((p.page_bytes[t] + kSpan - 1) / kSpan) : 0);
    for (int t = p.n; t < kMaxCopyTensors; ++t) a.first[t] = 0x7FFFFFFF;
    const size_t units = (size_t)p.max_pairs * p.layers * a.first[kMaxCopyTensors];
    // compact and 2.3 GB of copies in 8 KB: 521 us with 64 workgroups for each compute unit, 537 with 16
    const size_t most = (size_t)device_cu_count() * 64;
    hipLaunchKernelGGL(k_copy_pages, dim3((unsigned)(units < most ? units : most)), dim3(256), 0, st, a);
    return (int)hipGetLastError();
}

}  // namespace awq
