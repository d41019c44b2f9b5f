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
// Scores become integers of the same order, held in shared memory (those behind kHeld are read again), four neighbouring
// slots to a thread: they lie on one page.  The threshold is found by histograms of 2048 equal ranges between the lowest and
// the highest of them, each pass within the range that holds the threshold: two passes for most scores, three at most.  (Two
// bits a pass took sixteen, and most of 177 us on 64 x 16 heads of 4145 positions.)  Then windows of slots are
// marked with one scan each.
//
// Lengths are known on the device only, so the table's width says how much shared memory a block gets: 64 x 16 heads of 4145 positions
// take 40 us with a table of 4288 (four blocks to an SM), and 53 with one of 16,384 or more (three, so a third wave of blocks).
// In place or elsewhere makes no difference (39 and 40).
constexpr int kHeld = 16384;             // scores of a sequence that shared memory holds at most
constexpr int kBins = 2048;

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
    int S, Hkv, width, page_shift, num_pages, vec_shift, sinks, recent, held;   // vec_shift: log2 of 16-byte pieces of a row; held: scores in shared memory
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
// Ranks of slots 4 q .. 4 q + 3: mandatory positions (kMust) above all scores, a slot without a page (1) below all, and behind the
// last slot 0, which no range begins with.  A slot below b without a page counts as mandatory: it stays, so no row is moved to where
// it would be lost, and one position less of the lowest rank is kept.  (Of more mandatory ones than b the first b slots' stay, and these
// are below b: it is always among them.)
constexpr uint32_t kMust = 0xffffffffu;
// Where `copy`, and the results go elsewhere, the scores and positions of slots below b go there on the way: holes' too,
// which their movers' replace later.
__device__ __forceinline__ uint4 ranks_of(const EvictArgs& a, const Pair& p, int q, bool copy = false) {
    uint32_t r[4] = {0, 0, 0, 0};
    const int j = 4 * q, page = page_of(a, p, j);
    if (page < 0) atomicOr(a.err, (unsigned)kDevErrPagedArg);
    const long long e = element_of(a, p, max(page, 0), j);
    const float4 x = *reinterpret_cast<const float4*>(a.scores + e);
    const float s[4] = {x.x, x.y, x.z, x.w};
    int4 at = make_int4(0, 0, 0, 0);
    if (a.positions) at = *reinterpret_cast<const int4*>(a.positions + e);
    const int w[4] = {at.x, at.y, at.z, at.w};
    if (copy && page >= 0 && j < p.b) {
        const bool out = a.scores_out != a.scores, pos_out = a.positions && a.positions_out != a.positions;
        if (j + 4 <= p.b) {
            if (out) *reinterpret_cast<float4*>(a.scores_out + e) = x;
            if (pos_out) *reinterpret_cast<int4*>(a.positions_out + e) = at;
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (j + i < p.b) {
                    if (out) a.scores_out[e + i] = s[i];
                    if (pos_out) a.positions_out[e + i] = w[i];
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (j + i < p.L) r[i] = page < 0 ? (j + i < p.b ? kMust : 1u) : a.positions && (w[i] < a.sinks || w[i] >= p.newest - a.recent) ? kMust : order_of(s[i]);
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Sums of x[0 .. N-1] over the block, in the order x[0] of all its threads, x[1] of all, ...: what lies before each of the thread's
// own goes to x, the sum of all is returned.  sh: N integers a warp.
template <int T, int N>
__device__ __forceinline__ int scan_block(int (&x)[N], int* sh) {
    constexpr int W = T / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int own[N];
#pragma unroll
    for (int i = 0; i < N; ++i) own[i] = x[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = __shfl_up_sync(0xffffffffu, x[i], o);
            if (lane >= o) x[i] += t;
        }
    if (lane == 31) {
#pragma unroll
        for (int i = 0; i < N; ++i) sh[i * W + warp] = x[i];
    }
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] -= own[i];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            if (k == warp) x[i] += all;
            all += sh[i * W + k];
        }
    }
    __syncthreads();
    return all;
}

template <int WINDOW>
struct EvictShared {
    int red[16];
    uint32_t low[16], high[16];
    union {
        unsigned bins[kBins];
        uint16_t list[2][WINDOW];           // holes and movers, from their windows' first slots on
    };
    int red2[4 * 16];
    int found[3];                            // bin, what it has, what is still needed of it
};

// T threads: 512, or 256 where there are pairs enough to fill the device with such blocks: each step waits for the one before,
// and more blocks side by side hide that (us; 96 x 8 heads of 4145 positions 47 and 36, of 1000 to 4000 cut to 1000, where rows
// that move count most, 114 and 123; 128 threads 40 and 152; 16 x 8 heads of 4145 14 and 18).
template <int T>
__global__ void __launch_bounds__(T, 1024 / T) paged_evict_kernel(EvictArgs a) {
    constexpr int kWindow = T == 512 ? 8192 : 2048;
    constexpr int W = T / 32, N = kWindow / 4 / T;             // warps; quads of a window that a thread has
    extern __shared__ uint4 held[];                  // a.held / 4 of ranks_of
    __shared__ EvictShared<kWindow> sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), me = (int)cluster.block_rank();         // a power of two of CTAs
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pair = blockIdx.x / ranks;
    cudaGridDependencySynchronize();
    Pair p;
    p.s = pair / a.Hkv;
    p.h = pair - p.s * a.Hkv;
    p.row = a.table + (size_t)p.s * a.width;
    const int kv = a.kv_lens[p.s], room = a.width << a.page_shift;
    p.L = min(max(kv, 0), room);
    if (p.L != kv && tid == 0) atomicOr(a.err, (unsigned)kDevErrPagedArg);
    p.b = min(p.L, max(a.keep[p.s], 0));
    p.newest = p.L + (a.dropped ? a.dropped[p.s] : 0);
    const int quads = (p.L + 3) >> 2, held4 = a.held >> 2;
    if (p.b == p.L) {                                // nothing leaves
        if (a.scores_out != a.scores || a.positions_out != a.positions)
            for (int q = tid; q < quads; q += T) ranks_of(a, p, q, (q & (ranks - 1)) == me);
        return;
    }
    if (p.b == 0) return;

    // ranks, the lowest and highest of those that are not mandatory, and how many are
    uint32_t lo = kMust, hi = 0;
    int need = 0;
#pragma unroll 4
    for (int q = tid; q < quads; q += T) {
        const uint4 r = ranks_of(a, p, q, (q & (ranks - 1)) == me);
        if (q < held4) held[q] = r;
        const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            need += x[i] == kMust;
            hi = max(hi, x[i] == kMust ? 0u : x[i]);
            lo = min(lo, x[i] == 0u ? kMust : x[i]);
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
    for (int i = 0; i < W; ++i) {
        lo = min(lo, sh.low[i]);
        hi = max(hi, sh.high[i]);
        need -= sh.red[i];
    }
    auto rank = [&](int q) { return q < held4 ? held[q] : ranks_of(a, p, q); };
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
        for (int i = 0; i < kBins / T; ++i) sh.bins[i * T + tid] = 0;
        __syncthreads();
#pragma unroll 2
        for (int q = tid; q < quads; q += T) {
            const uint4 r = rank(q);
            if (r.x >= lo && r.x <= hi) atomicAdd(&sh.bins[(r.x - lo) >> shift], 1u);
            if (r.y >= lo && r.y <= hi) atomicAdd(&sh.bins[(r.y - lo) >> shift], 1u);
            if (r.z >= lo && r.z <= hi) atomicAdd(&sh.bins[(r.z - lo) >> shift], 1u);
            if (r.w >= lo && r.w <= hi) atomicAdd(&sh.bins[(r.w - lo) >> shift], 1u);
        }
        __syncthreads();
        // bins from the highest down, a run of them to a thread
        constexpr int R = kBins / T;
        int sum[1] = {0};
#pragma unroll
        for (int i = 0; i < R; ++i) sum[0] += (int)sh.bins[kBins - 1 - (tid * R + i)];
        const int mine = sum[0];
        scan_block<T>(sum, sh.red);
        int before = sum[0];
        if (before < need && need <= before + mine) {
            for (int i = 0; i < R; ++i) {
                const int n = (int)sh.bins[kBins - 1 - (tid * R + i)];
                if (before < need && need <= before + n) {
                    sh.found[0] = kBins - 1 - (tid * R + i);
                    sh.found[1] = n;
                    sh.found[2] = need - before;
                }
                before += n;
            }
        }
        __syncthreads();
        lo += (uint32_t)sh.found[0] << shift;
        hi = min(hi, lo + ((1u << shift) - 1));
        need = sh.found[2];
        const bool all = sh.found[1] == need;
        __syncthreads();
        if (all) {                                   // all of the bin are kept: what lies in it need not be told apart
            threshold = lo - 1;
            ties = 0;
            break;
        }
    }

    // slots of quad q whose rank is above the threshold, and at it
    auto above = [&](const uint4& r) {
        return (unsigned)(r.x > threshold) | (unsigned)(r.y > threshold) << 1 | (unsigned)(r.z > threshold) << 2 | (unsigned)(r.w > threshold) << 3;
    };
    auto equal = [&](const uint4& r) {
        return (unsigned)(r.x == threshold) | (unsigned)(r.y == threshold) << 1 | (unsigned)(r.z == threshold) << 2 |
               (unsigned)(r.w == threshold) << 3;
    };
    // bits of quad q that lie in [from, to)
    auto within = [&](int q, int from, int to) {
        const int f = from - 4 * q, t = to - 4 * q;
        return (f <= 0 ? 15u : f >= 4 ? 0u : 15u << f & 15u) & (t >= 4 ? 15u : t <= 0 ? 0u : (1u << t) - 1);
    };
    // windows of holes from slot 0 on, of movers from b on; as many as both have are moved, then the empty one's next window is marked
    struct Side {
        int next, base, have, used, tied;            // next window; the present one's first slot, its marks, those used; ties before `next`
    } hole = {0, 0, 0, 0, 0}, mover = {p.b & ~3, 0, 0, 0, 0};
    if (ties > 0) {                                  // ties below b come before those behind it
        int mine = 0;
        for (int q = tid; 4 * q < p.b; q += T) mine += __popc(equal(rank(q)) & within(q, 0, p.b));
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) sh.red2[warp] = mine;         // (not to sh.red: without a histogram another warp may still read its counts)
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) mover.tied += sh.red2[i];
        __syncthreads();
    }
    auto refill = [&](Side& d, bool holes, int begin, int end) {
        while (d.used == d.have && d.next < end) {
            const int q0 = d.next >> 2;
            unsigned in = 0, kept = 0, tie = 0;      // four bits to a quad of the thread's N
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int q = q0 + i * T + tid;
                const unsigned here = within(q, begin, end);
                if (here) {
                    const uint4 r = rank(q);
                    in |= here << 4 * i;
                    kept |= (above(r) & here) << 4 * i;
                    tie |= (equal(r) & here) << 4 * i;
                }
            }
            int n[N];
            if (ties > d.tied) {                     // ties are kept while they last, the lowest slots first
#pragma unroll
                for (int i = 0; i < N; ++i) n[i] = __popc(tie >> 4 * i & 15u);
                const int all = scan_block<T>(n, sh.red2);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    int before = d.tied + n[i];
#pragma unroll
                    for (int k = 4 * i; k < 4 * i + 4; ++k)
                        if (tie >> k & 1) kept |= (unsigned)(before++ < ties) << k;
                }
                d.tied += all;
            }
            const unsigned mark = holes ? in & ~kept : kept;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                n[i] = __popc(mark >> 4 * i & 15u);
            }
            d.have = scan_block<T>(n, sh.red2);
#pragma unroll
            for (int i = 0; i < N; ++i)
                for (unsigned m = mark >> 4 * i & 15u, k = n[i]; m; m &= m - 1, ++k)
                    sh.list[!holes][k] = (uint16_t)(4 * (i * T + tid) + __ffs((int)m) - 1);
            d.base = d.next;
            d.used = 0;
            d.next += kWindow;
        }
    };
    for (;;) {
        refill(hole, true, 0, p.b);
        refill(mover, false, p.b, p.L);
        // every CTA has looked at the slots before the next windows (all look at the same ones): they may be written
        if (ranks > 1) cluster.sync();
        else __syncthreads();
        const int n = min(hole.have - hole.used, mover.have - mover.used);
        if (n == 0) break;                           // (holes and movers end together)
        const int in = (1 << a.page_shift) - 1, vecs = 1 << a.vec_shift, mine = ((n - me + ranks - 1) / ranks) << a.vec_shift;
        constexpr int U = 4;
        for (int e0 = tid; e0 < mine; e0 += U * T) {
            uint4 x[U], y[U];
            long long to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = e0 + u * T;
                to[u] = -1;
                if (e >= mine) continue;
                const int i = (e >> a.vec_shift) * ranks + me, c = e & (vecs - 1);
                const int from_j = mover.base + sh.list[1][mover.used + i], to_j = hole.base + sh.list[0][hole.used + i];
                const int sp = page_of(a, p, from_j), dp = page_of(a, p, to_j);
                if (sp < 0 || dp < 0) continue;
                const long long from = sp * a.page_bytes + (((p.h << a.page_shift) + (from_j & in)) * (long long)vecs + c) * 16;
                x[u] = *reinterpret_cast<const uint4*>(a.k + from);
                y[u] = *reinterpret_cast<const uint4*>(a.v + from);
                to[u] = dp * a.page_bytes + (((p.h << a.page_shift) + (to_j & in)) * (long long)vecs + c) * 16;
                if (c == 0) {
                    const long long se = element_of(a, p, sp, from_j), de = element_of(a, p, dp, to_j);
                    a.scores_out[de] = a.scores[se];
                    if (a.positions) a.positions_out[de] = a.positions[se];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (to[u] >= 0) {
                    *reinterpret_cast<uint4*>(a.k + to[u]) = x[u];
                    *reinterpret_cast<uint4*>(a.v + to[u]) = y[u];
                }
        }
        hole.used += n;
        mover.used += n;
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------------- trim
//
// Every CTA of one cluster counts the pages that its sequences give back, the counts are summed over the cluster, and
// each writes its own: the free stack gets them sequence after sequence.  Latency bounds it: a warp takes its sequences one after
// another, each in two passes of lengths and then 32 columns of the table at a time, and in the second pass a step's loads stand behind the
// stores of the step before (512 sequences of up to 8000 positions in pages of 16: 14 us).
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
    const void* words[] = {block_table, kv_lens, keep, dropped}, *wide[] = {scores, scores_out, positions, positions_out, k_cache, v_cache};
    for (const void* x : words)
        if (!lc::aligned(x, 4)) return lc::failf(LLA_ERR_INVALID_ARG, "lengths and tables must be 4-byte aligned");
    for (const void* x : wide)
        if (!lc::aligned(x, 16)) return lc::failf(LLA_ERR_INVALID_ARG, "caches, scores and positions must be 16-byte aligned");
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
    const long long room = (long long)table_width * page_size;
    const int held = room < lc::kHeld ? (int)room : lc::kHeld;
    lc::EvictArgs a{scores, scores_out, positions, positions_out, static_cast<char*>(k_cache), static_cast<char*>(v_cache),
                    block_table, kv_lens, keep, dropped, page_stride * es, S, Hkv, table_width, shift, num_pages, lla::paged::log2_up(d * es / 16), sinks,
                    recent, held, err};
    const size_t smem = (size_t)held * sizeof(uint32_t);
    const long long pairs = (long long)S * Hkv;
    const bool small = pairs >= 4LL * sms;
    auto* kern = small ? lc::paged_evict_kernel<256> : lc::paged_evict_kernel<512>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(lc::kHeld * sizeof(uint32_t)));
    if (e != cudaSuccess) return lc::cuda_failf(e, "lla_paged_evict");
    int ranks = 1;
    while (ranks < 8 && pairs * ranks * 2 <= 2LL * sms) ranks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs * ranks));
    cfg.blockDim = dim3(small ? 256 : 512);
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
    e = cudaLaunchKernelEx(&cfg, kern, a);
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
