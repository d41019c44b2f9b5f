// Eviction from paged caches (include/lla.h): paged_evict keeps every (sequence, key head)'s positions of largest score,
// paged_trim cuts the lengths and gives the pages behind them back.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/lla.h"
#include "lla_internal.h"
#include "lla_paged.h"

namespace lla {
namespace cache {
namespace {

namespace cg = cooperative_groups;

int failf(int status, const char* fmt, ...) {
    char msg[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return set_error(status, msg);
}
int cuda_failf(cudaError_t e, const char* what) {
    return failf(LLA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}
bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int page_shift_of(int page) {
    for (int s = 3; s <= 8; ++s)
        if (page == 1 << s) return s;
    return -1;
}
int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

// ------------------------------------------------------------------------------------------ evict
//
// The kept positions of a (sequence, key head) are the b = min(L, keep) largest of its L scores.  Slots below b that are
// not kept are holes, kept slots from b on are movers: as many, and they are matched in ascending order.  What is read
// lies at or behind slot b and what is written before it, so rows move in place without an order among them, and only
// what changes is touched: after a step of 64 new positions 64 rows move, where closing the gaps in order would move
// half the cache.
//
// Scores become integers of the same order, held in shared memory (those behind kHeld are read again).  The threshold is
// found by histograms of 2048 equal ranges between the lowest and the highest of them, each pass within the range that holds the
// threshold: two passes for most scores, three at most.  (Two bits a pass took sixteen, and most of 177 us on 64 x 16 heads
// of 4145 positions.)  Then windows of kWindow slots are marked, with one scan for all of a window's ballots.
constexpr int kEvictThreads = 512, kEvictWarps = kEvictThreads / 32;
constexpr int kHeld = 10240;             // scores of a sequence that shared memory holds
constexpr int kBins = 4 * kEvictThreads;
constexpr int kChunks = 8, kWindow = kChunks * kEvictThreads;

struct EvictArgs {
    const float* scores;
    float* scores_out;
    const int* positions;                // or null
    int* positions_out;
    char* k;
    char* v;
    const int* table;
    const int* kv_lens;
    const int* keep;
    const int* dropped;                  // or null
    long long page_bytes;                // from page to page of a cache
    int S, Hkv, width, page_shift, num_pages, vec_shift, sinks, recent;   // vec_shift: log2 of 16-byte pieces of a row
    unsigned* err;
};

// Floats as integers of the same order, -inf (and NaN, which counts as it) at 0x007fffff; both zeros alike.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = x != x ? 0xff800000u : __float_as_uint(x + 0.f);             // -0 becomes 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct Pair {
    const int* row;                      // the sequence's table row
    int s, h, L, b;
    int newest;                          // position behind the last, where positions are known
};

// Page of slot j, checked; -1 where the table holds none.
__device__ __forceinline__ int page_of(const EvictArgs& a, const Pair& p, int j) {
    const int page = p.row[j >> a.page_shift];
    return page >= 0 && page < a.num_pages ? page : -1;
}
// Element of scores and positions that slot j has; its page must be there.
__device__ __forceinline__ long long element_of(const EvictArgs& a, const Pair& p, int page, int j) {
    return (((long long)page * a.Hkv + p.h) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
}
// Rank of slot j: mandatory positions above all scores, slots without a page below all.
__device__ __forceinline__ uint32_t rank_of(const EvictArgs& a, const Pair& p, int j) {
    const int page = page_of(a, p, j);
    if (page < 0) {
        atomicOr(a.err, (unsigned)kDevErrPagedArg);
        return 0u;
    }
    const long long e = element_of(a, p, page, j);
    if (a.positions) {
        const int x = a.positions[e];
        if (x < a.sinks || x >= p.newest - a.recent) return 0xffffffffu;
    }
    return order_of(a.scores[e]);
}

// Inclusive sum of x over the block's threads, and the block's total.
__device__ __forceinline__ int2 scan_block(int x, int* sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += t;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kEvictWarps; ++i) {
        const int t = sh[i];
        if (i < warp) before += t;
        all += t;
    }
    __syncthreads();
    return make_int2(x + before, all);
}

struct EvictShared {
    int red[kEvictWarps];
    uint32_t low[kEvictWarps], high[kEvictWarps];
    int count[kChunks * kEvictWarps];        // of a window's ballots, then the sums before them
    union {
        unsigned bins[kBins];
        uint16_t list[2][kWindow];           // holes and movers, from their windows' first slots on
    };
    int found[3];                            // bin, what it has, what is still needed of it
};

// Marks of a window's slots: flag(slot), asked of every slot in [first, end), and for those that have it put(slot, rank), the rank counted
// from `base` on.  Returns how many there are.
template <typename Flag, typename Put>
__device__ __forceinline__ int mark_window(EvictShared& sh, int first, int end, int base, Flag flag, Put put) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned mine = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int j = first + c * kEvictThreads + tid;
        const bool yes = j < end && flag(j);
        const unsigned some = __ballot_sync(0xffffffffu, yes);
        if (lane == 0) sh.count[c * kEvictWarps + warp] = __popc(some);
        mine |= (unsigned)yes << c;
    }
    __syncthreads();
    constexpr int kEntries = kChunks * kEvictWarps;
    static_assert(kEntries <= kEvictThreads, "an entry to a thread");
    const int n = tid < kEntries ? sh.count[tid] : 0;
    const int2 t = scan_block(n, sh.red);
    if (tid < kEntries) sh.count[tid] = base + t.x - n;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const bool yes = mine >> c & 1;
        const unsigned some = __ballot_sync(0xffffffffu, yes);
        if (yes) put(first + c * kEvictThreads + tid, sh.count[c * kEvictWarps + warp] + __popc(some & ((1u << lane) - 1)));
    }
    __syncthreads();
    return t.y;
}

__global__ void __launch_bounds__(kEvictThreads, 3) paged_evict_kernel(EvictArgs a) {
    extern __shared__ uint32_t held[];               // kHeld ranks
    __shared__ EvictShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pair = blockIdx.x / ranks;
    cudaGridDependencySynchronize();
    Pair p;
    p.s = pair / a.Hkv;
    p.h = pair % a.Hkv;
    p.row = a.table + (size_t)p.s * a.width;
    const int kv = a.kv_lens[p.s], room = a.width << a.page_shift;
    p.L = min(max(kv, 0), room);
    if (p.L != kv && tid == 0) atomicOr(a.err, (unsigned)kDevErrPagedArg);
    p.b = min(p.L, max(a.keep[p.s], 0));
    p.newest = p.L + (a.dropped ? a.dropped[p.s] : 0);
    const bool out = a.scores_out != a.scores, pos_out = a.positions && a.positions_out != a.positions;
    auto carry = [&](int j) {                        // a kept slot that stays, where the results go elsewhere
        if ((!out && !pos_out) || j % ranks != me) return;
        const int page = page_of(a, p, j);
        if (page < 0) return;
        const long long e = element_of(a, p, page, j);
        if (out) a.scores_out[e] = a.scores[e];
        if (pos_out) a.positions_out[e] = a.positions[e];
    };
    if (p.b == p.L) {
        for (int j = tid; j < p.L; j += kEvictThreads) carry(j);
        return;
    }
    if (p.b == 0) return;

    // ranks, the lowest and highest of those that are not mandatory, and how many are
    constexpr uint32_t kMust = 0xffffffffu;          // above every score's rank
    uint32_t lo = kMust, hi = 0;
    int need = 0;
#pragma unroll 4
    for (int j = tid; j < p.L; j += kEvictThreads) {
        const uint32_t x = rank_of(a, p, j);
        if (j < kHeld) held[j] = x;
        if (x == kMust) ++need;
        else {
            lo = min(lo, x);
            hi = max(hi, x);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    need = __reduce_add_sync(0xffffffffu, need);
    if (lane == 0) {
        sh.low[warp] = lo;
        sh.high[warp] = hi;
        sh.red[warp] = need;
    }
    __syncthreads();
    need = p.b;
#pragma unroll
    for (int i = 0; i < kEvictWarps; ++i) {
        lo = min(lo, sh.low[i]);
        hi = max(hi, sh.high[i]);
        need -= sh.red[i];
    }
    auto rank = [&](int j) { return j < kHeld ? held[j] : rank_of(a, p, j); };
    // kept: every rank above `threshold`, and of those at it the first `ties`
    uint32_t threshold = kMust;
    int ties = p.b;                                  // more mandatory ones than are kept
    if (need == 0) {
        threshold = kMust - 1;                       // (no score has it)
        ties = 0;
    }
    while (need > 0) {
        if (lo == hi) {
            threshold = lo;
            ties = need;
            break;
        }
        const int shift = max(32 - __clz(hi - lo) - 11, 0);      // (hi - lo) >> shift < 2048
#pragma unroll
        for (int i = 0; i < kBins / kEvictThreads; ++i) sh.bins[i * kEvictThreads + tid] = 0;
        __syncthreads();
#pragma unroll 4
        for (int j = tid; j < p.L; j += kEvictThreads) {
            const uint32_t x = rank(j);
            if (x >= lo && x <= hi) atomicAdd(&sh.bins[(x - lo) >> shift], 1u);
        }
        __syncthreads();
        // bins from the highest down, four to a thread
        constexpr int kOf = kBins / kEvictThreads;
        int n[kOf], sum = 0;
#pragma unroll
        for (int i = 0; i < kOf; ++i) {
            n[i] = (int)sh.bins[kBins - 1 - (tid * kOf + i)];
            sum += n[i];
        }
        const int2 t = scan_block(sum, sh.red);
        int before = t.x - sum;
        if (before < need && need <= t.x) {
#pragma unroll
            for (int i = 0; i < kOf; ++i) {
                if (before < need && need <= before + n[i]) {
                    sh.found[0] = kBins - 1 - (tid * kOf + i);
                    sh.found[1] = n[i];
                    sh.found[2] = need - before;
                }
                before += n[i];
            }
        }
        __syncthreads();
        lo += (uint32_t)sh.found[0] << shift;
        hi = min(hi, lo + ((1u << shift) - 1));
        const bool all = sh.found[1] == sh.found[2];
        need = sh.found[2];
        __syncthreads();
        if (all) {                                   // all of the bin are kept: what lies in it need not be told apart
            threshold = lo - 1;                      // (lo > 0: with it the lowest would be kept, and with that all)
            ties = 0;
            break;
        }
    }

    auto page_element = [&](int page, int j, int c) {          // byte offset of piece c of slot j in a cache
        const int in = (1 << a.page_shift) - 1;
        return page * a.page_bytes + ((((long long)((p.h << a.page_shift) + (j & in))) << a.vec_shift) + c) * 16;
    };
    // windows of holes from slot 0 on, of movers from b on; as many as both have are moved, then the empty one's next window is marked
    int next[2] = {0, p.b}, base[2] = {0, 0}, have[2] = {0, 0}, used[2] = {0, 0}, tied = 0, tied_behind = 0;
    const int end[2] = {p.b, p.L};
    if (ties > 0) {                                  // ties below b come before those behind it
        int mine = 0;
        for (int j = tid; j < p.b; j += kEvictThreads) mine += rank(j) == threshold;
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) sh.red[warp] = mine;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kEvictWarps; ++i) tied_behind += sh.red[i];
        __syncthreads();
    }
    for (;;) {
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            while (used[side] == have[side] && next[side] < end[side]) {
                const int first = next[side], last = min(first + kWindow, end[side]);
                int& before = side == 0 ? tied : tied_behind;
                // ties are kept while they last: those that are not leave their mark in the list's place
                if (ties > 0 && before < ties) {
                    const int n = mark_window(sh, first, last, before, [&](int j) { return rank(j) == threshold; },
                                              [&](int j, int k) { sh.list[side][j - first] = k < ties; });
                    have[side] = 0;
                    unsigned keep = 0;               // bit c: the thread's slot of chunk c is a tie that is kept
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        const int j = first + c * kEvictThreads + tid;
                        if (j < last && rank(j) == threshold && sh.list[side][j - first]) keep |= 1u << c;
                    }
                    __syncthreads();
                    have[side] = mark_window(sh, first, last, 0, [&](int j) {
                        const bool kept = rank(j) > threshold || (keep >> ((j - first) / kEvictThreads) & 1);
                        if (side == 0 && kept) carry(j);
                        return kept == (side == 1);
                    }, [&](int j, int k) { sh.list[side][k] = (uint16_t)(j - first); });
                    before += n;
                } else {
                    have[side] = mark_window(sh, first, last, 0, [&](int j) {
                        const bool kept = rank(j) > threshold;
                        if (side == 0 && kept) carry(j);
                        return kept == (side == 1);
                    }, [&](int j, int k) { sh.list[side][k] = (uint16_t)(j - first); });
                }
                base[side] = first;
                next[side] = last;
                used[side] = 0;
            }
        }
        // every CTA has looked at the slots before next[0] and next[1] (all look at the same ones): they may be written
        if (ranks > 1) cluster.sync();
        else __syncthreads();
        const int n = min(have[0] - used[0], have[1] - used[1]);
        if (n == 0) break;                           // (holes and movers end together)
        const int vecs = 1 << a.vec_shift, mine = ((n - me + ranks - 1) / ranks) << a.vec_shift;
        for (int e0 = tid; e0 < mine; e0 += 4 * kEvictThreads) {
            uint4 x[4], y[4];
            long long to[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int e = e0 + u * kEvictThreads;
                to[u] = -1;
                if (e >= mine) continue;
                const int i = (e >> a.vec_shift) * ranks + me, c = e & (vecs - 1);
                const int from_j = base[1] + sh.list[1][used[1] + i], to_j = base[0] + sh.list[0][used[0] + i];
                const int sp = page_of(a, p, from_j), dp = page_of(a, p, to_j);
                if (sp < 0 || dp < 0) continue;
                const long long from = page_element(sp, from_j, c);
                x[u] = *reinterpret_cast<const uint4*>(a.k + from);
                y[u] = *reinterpret_cast<const uint4*>(a.v + from);
                to[u] = page_element(dp, to_j, c);
                if (c == 0) {
                    const long long se = element_of(a, p, sp, from_j), de = element_of(a, p, dp, to_j);
                    a.scores_out[de] = a.scores[se];
                    if (a.positions) a.positions_out[de] = a.positions[se];
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (to[u] >= 0) {
                    *reinterpret_cast<uint4*>(a.k + to[u]) = x[u];
                    *reinterpret_cast<uint4*>(a.v + to[u]) = y[u];
                }
        }
        used[0] += n;
        used[1] += n;
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------------- trim
//
// Every CTA of one cluster counts the pages that its sequences give back, the counts are summed over the cluster, and
// each writes its own: the free stack gets them sequence after sequence.  Latency bounds it (three dependent reads).
constexpr int kTrimThreads = 1024, kTrimMaxSeqs = 8192, kTrimCtas = 8;

struct TrimArgs {
    const int* kv_lens;
    const int* keep;
    const int* table;
    int* free_pages;
    const int* free_count;
    const int* dropped;          // or null
    int* new_lens;
    int* new_dropped;            // or null
    int* free_left;
    int S, width, page_shift, capacity;
    unsigned* err;
};

struct Cut {
    int L, b, c0, c1;            // lengths, and the columns of the table that are given back
};
__device__ __forceinline__ Cut cut_of(const TrimArgs& a, int s) {
    Cut c;
    const int kv = a.kv_lens[s], page = 1 << a.page_shift;
    c.L = min(max(kv, 0), a.width << a.page_shift);
    if (c.L != kv) atomicOr(a.err, (unsigned)kDevErrPagedArg);
    c.b = min(c.L, max(a.keep[s], 0));
    c.c0 = (c.b + page - 1) >> a.page_shift;
    c.c1 = (c.L + page - 1) >> a.page_shift;
    return c;
}

__global__ void __launch_bounds__(kTrimThreads) paged_trim_kernel(TrimArgs a) {
    extern __shared__ int at[];          // [per]: pages that this CTA's earlier sequences give back
    __shared__ int total, warps[32], carry;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.S + ranks - 1) / ranks, s0 = min(me * per, a.S), s1 = min(s0 + per, a.S);
    cudaGridDependencySynchronize();
    const int have = min(max(*a.free_count, 0), a.capacity);
    // a warp to a sequence: columns that hold a page
    for (int s = s0 + warp; s < s1; s += 32) {
        const Cut c = cut_of(a, s);
        int n = 0;
        for (int x = c.c0 + lane; x < c.c1; x += 32) n += a.table[(size_t)s * a.width + x] >= 0;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) at[s - s0] = n;
    }
    if (tid == 0) carry = 0;
    __syncthreads();
    for (int x0 = 0; x0 < s1 - s0; x0 += kTrimThreads) {         // exclusive sums, a chunk at a time
        const int n = x0 + tid < s1 - s0 ? at[x0 + tid] : 0;
        int v = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
        }
        if (lane == 31) warps[warp] = v;
        __syncthreads();
        int before = carry, all = 0;
        for (int i = 0; i < 32; ++i) {
            if (i < warp) before += warps[i];
            all += warps[i];
        }
        if (x0 + tid < s1 - s0) at[x0 + tid] = before + v - n;
        __syncthreads();
        if (tid == 0) carry += all;
        __syncthreads();
    }
    if (tid == 0) total = carry;
    cluster.sync();
    int base = 0, all = 0;
    for (int r = 0; r < ranks; ++r) {
        const int t = *cluster.map_shared_rank(&total, r);
        if (r < me) base += t;
        all += t;
    }
    cluster.sync();                      // every CTA has read the counts, the lengths and the free count
    for (int s = s0 + warp; s < s1; s += 32) {
        const Cut c = cut_of(a, s);
        int to = have + base + at[s - s0];
        for (int x0 = c.c0; x0 < c.c1; x0 += 32) {
            const int id = x0 + lane < c.c1 ? a.table[(size_t)s * a.width + x0 + lane] : -1;
            const unsigned some = __ballot_sync(0xffffffffu, id >= 0);
            const int mine = to + __popc(some & ((1u << lane) - 1));
            if (id >= 0) {
                if (mine < a.capacity) a.free_pages[mine] = id;
                else atomicOr(a.err, (unsigned)kDevErrPagedArg);
            }
            to += __popc(some);
        }
        __syncwarp();
        if (lane == 0) {
            if (a.new_dropped) a.new_dropped[s] = c.L - c.b + (a.dropped ? a.dropped[s] : 0);
            a.new_lens[s] = c.b;
        }
    }
    if (me == 0 && tid == 0) *a.free_left = min(have + all, a.capacity);
}

}  // namespace
}  // namespace cache
}  // namespace lla

namespace lc = lla::cache;

extern "C" {

int lla_paged_evict(int dtype, const float* scores, float* scores_out, const int* positions, int* positions_out, void* k_cache,
                    void* v_cache, const int* block_table, const int* kv_lens, const int* keep, const int* dropped, int S,
                    int Hkv, int d, int page_size, int num_pages, int table_width, long long page_stride, int sinks, int recent,
                    void* stream_) {
    lla::set_error(LLA_OK, "");
    if (!scores || !scores_out || !k_cache || !v_cache || !block_table || !kv_lens || !keep)
        return lc::failf(LLA_ERR_INVALID_ARG, "null tensor pointer");
    if ((positions != nullptr) != (positions_out != nullptr))
        return lc::failf(LLA_ERR_INVALID_ARG, "positions and positions_out go together");
    if (!positions && (sinks > 0 || recent > 0)) return lc::failf(LLA_ERR_INVALID_ARG, "sinks and recent need the slots' positions");
    const void* words[] = {scores, scores_out, positions, positions_out, block_table, kv_lens, keep, dropped};
    for (const void* x : words)
        if (!lc::aligned(x, 4)) return lc::failf(LLA_ERR_INVALID_ARG, "int32 and fp32 pointers must be 4-byte aligned");
    if (!lc::aligned(k_cache, 16) || !lc::aligned(v_cache, 16)) return lc::failf(LLA_ERR_INVALID_ARG, "caches must be 16-byte aligned");
    if (dtype != LLA_DTYPE_BF16 && dtype != LLA_DTYPE_FP32) return lc::failf(LLA_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (d != 16 && d != 32 && d != 64 && d != 128)
        return lc::failf(LLA_ERR_INVALID_ARG, "head dim d must be 16, 32, 64 or 128 (got %d)", d);
    const int shift = lc::page_shift_of(page_size);
    if (shift < 0) return lc::failf(LLA_ERR_INVALID_ARG, "page_size must be a power of two in 8 .. 256 (got %d)", page_size);
    if (S < 1 || Hkv < 1 || num_pages < 1 || table_width < 1 || sinks < 0 || recent < 0)
        return lc::failf(LLA_ERR_INVALID_ARG, "S, Hkv, num_pages and table_width must be >= 1, sinks and recent >= 0");
    if (S > (1 << 20) || Hkv > 65535 || (long long)S * Hkv > (1LL << 27) || (long long)table_width * page_size > (1LL << 28))
        return lc::failf(LLA_ERR_INVALID_ARG, "problem too large (S <= 2^20, S*Hkv <= 2^27, table_width*page_size <= 2^28)");
    if (page_stride < (long long)Hkv * page_size * d || page_stride % ((long long)page_size * d))
        return lc::failf(LLA_ERR_INVALID_ARG, "page_stride must be >= Hkv*page_size*d and a multiple of page_size*d");
    const int es = dtype == LLA_DTYPE_BF16 ? 2 : 4;
    const int sms = lc::sm_count();
    if (sms < 1) return lc::failf(LLA_ERR_CUDA, "lla_paged_evict: no device");
    unsigned* err = lla::device_error_word();
    if (!err) return lc::failf(LLA_ERR_CUDA, "lla_paged_evict: device error word not found");
    lc::EvictArgs a{scores, scores_out, positions, positions_out, static_cast<char*>(k_cache), static_cast<char*>(v_cache),
                    block_table, kv_lens, keep, dropped, page_stride * es, S, Hkv, table_width, shift, num_pages, lla::paged::log2_up(d * es / 16), sinks,
                    recent, err};
    constexpr size_t smem = lc::kHeld * sizeof(uint32_t);
    cudaError_t e = cudaFuncSetAttribute(lc::paged_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return lc::cuda_failf(e, "lla_paged_evict");
    const long long pairs = (long long)S * Hkv;
    int ranks = 1;
    while (ranks < 8 && pairs * ranks * 2 <= 2LL * sms) ranks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs * ranks));
    cfg.blockDim = dim3(lc::kEvictThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream_);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ranks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ranks > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, lc::paged_evict_kernel, a);
    if (e != cudaSuccess) return lc::cuda_failf(e, "lla_paged_evict launch");
    return LLA_OK;
}

int lla_paged_trim(const int* kv_lens, const int* keep, int S, int page_size, const int* block_table, int table_width,
                   int* free_pages, int free_capacity, const int* free_count, const int* dropped, int* new_lens, int* new_dropped,
                   int* free_left, void* stream_) {
    lla::set_error(LLA_OK, "");
    if (!kv_lens || !keep || !block_table || !free_pages || !free_count || !new_lens || !free_left)
        return lc::failf(LLA_ERR_INVALID_ARG, "null pointer");
    if (dropped && !new_dropped) return lc::failf(LLA_ERR_INVALID_ARG, "dropped goes with new_dropped");
    if (S < 1 || S > lc::kTrimMaxSeqs) return lc::failf(LLA_ERR_INVALID_ARG, "S must be in [1, %d] (got %d)", lc::kTrimMaxSeqs, S);
    const int shift = lc::page_shift_of(page_size);
    if (shift < 0) return lc::failf(LLA_ERR_INVALID_ARG, "page_size must be a power of two in 8 .. 256 (got %d)", page_size);
    if (table_width < 1 || (long long)table_width * page_size > (1LL << 28))
        return lc::failf(LLA_ERR_INVALID_ARG, "table_width must be >= 1 and table_width*page_size <= 2^28");
    if (free_capacity < 1) return lc::failf(LLA_ERR_INVALID_ARG, "free_capacity must be >= 1");
    const void* ints[] = {kv_lens, keep, block_table, free_pages, free_count, dropped, new_lens, new_dropped, free_left};
    for (const void* x : ints)
        if (!lc::aligned(x, 4)) return lc::failf(LLA_ERR_INVALID_ARG, "int32 pointers must be 4-byte aligned");
    unsigned* err = lla::device_error_word();
    if (!err) return lc::failf(LLA_ERR_CUDA, "lla_paged_trim: device error word not found");
    lc::TrimArgs a{kv_lens, keep, block_table, free_pages, free_count, dropped, new_lens, new_dropped, free_left, S, table_width,
                   shift, free_capacity, err};
    const int ctas = S > 64 ? lc::kTrimCtas : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(lc::kTrimThreads);
    cfg.dynamicSmemBytes = (size_t)((S + ctas - 1) / ctas) * sizeof(int);
    cfg.stream = static_cast<cudaStream_t>(stream_);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, lc::paged_trim_kernel, a);
    if (e != cudaSuccess) return lc::cuda_failf(e, "lla_paged_trim launch");
    return LLA_OK;
}

}  // extern "C"
