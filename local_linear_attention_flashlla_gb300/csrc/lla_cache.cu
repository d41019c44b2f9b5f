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
// The threshold is found bit by bit from the top, two bits a pass over the scores (in shared memory as integers of the
// same order), the counts of the four digits in one 64-bit word a thread.
constexpr int kEvictThreads = 512, kEvictWarps = kEvictThreads / 32;
constexpr int kHeld = 12288;             // scores of a sequence that shared memory holds; those behind are read again
constexpr int kBuffer = 2 * kEvictThreads;

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
    int S, Hkv, width, page_shift, num_pages, row_bytes, sinks, recent;
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

// Inclusive prefix over the block of two 16-bit counts a thread (in one word), and the block's total.
__device__ __forceinline__ uint2 scan_pairs(uint32_t x, uint32_t* sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += t;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kEvictWarps; ++i) {
        const uint32_t t = sh[i];
        if (i < warp) before += t;
        all += t;
    }
    __syncthreads();
    return make_uint2(x + before, all);
}

__global__ void __launch_bounds__(kEvictThreads) paged_evict_kernel(EvictArgs a) {
    extern __shared__ uint32_t held[];               // kHeld ranks
    __shared__ unsigned long long counts[kEvictWarps][2];
    __shared__ uint32_t red[kEvictWarps];
    __shared__ int holes[kBuffer], movers[kBuffer];
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

    uint32_t threshold = 0;
    int ties = INT_MAX;                              // slots at the threshold that are kept, the lowest ones
    const bool cut = p.b < p.L;
    auto rank = [&](int j) { return j < kHeld ? held[j] : rank_of(a, p, j); };
    if (cut && p.b > 0) {
        for (int j = tid; j < min(p.L, kHeld); j += kEvictThreads) held[j] = rank_of(a, p, j);
        __syncthreads();
        int need = p.b;                              // of those that agree with the threshold so far
        uint32_t mask = 0;
        for (int shift = 30; shift >= 0; shift -= 2) {
            uint32_t c01 = 0, c23 = 0;               // counts of digits 0, 1 and 2, 3: 16 bits each
            unsigned long long w01 = 0, w23 = 0;
            int n = 0;
            for (int j = tid; j < p.L; j += kEvictThreads) {
                const uint32_t x = rank(j);
                if ((x & mask) == threshold) {
                    const uint32_t digit = (x >> shift) & 3u, one = 1u << ((digit & 1u) * 16);
                    if (digit & 2u) c23 += one;
                    else c01 += one;
                }
                if (++n == 65535) {                  // before a 16-bit count can overflow
                    w01 += (c01 & 0xffffu) | ((unsigned long long)(c01 >> 16) << 32);
                    w23 += (c23 & 0xffffu) | ((unsigned long long)(c23 >> 16) << 32);
                    c01 = c23 = 0;
                    n = 0;
                }
            }
            w01 += (c01 & 0xffffu) | ((unsigned long long)(c01 >> 16) << 32);
            w23 += (c23 & 0xffffu) | ((unsigned long long)(c23 >> 16) << 32);
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                w01 += __shfl_xor_sync(0xffffffffu, w01, o);
                w23 += __shfl_xor_sync(0xffffffffu, w23, o);
            }
            if (lane == 0) {
                counts[warp][0] = w01;
                counts[warp][1] = w23;
            }
            __syncthreads();
            w01 = w23 = 0;
#pragma unroll
            for (int i = 0; i < kEvictWarps; ++i) {
                w01 += counts[i][0];
                w23 += counts[i][1];
            }
            __syncthreads();
            const int c[4] = {(int)(uint32_t)w01, (int)(w01 >> 32), (int)(uint32_t)w23, (int)(w23 >> 32)};
            int digit = 3;
            while (digit > 0 && need > c[digit]) need -= c[digit--];
            threshold |= (uint32_t)digit << shift;
            mask |= 3u << shift;
            if (need == c[digit]) {                  // all that agree are kept: the bits below need not be known
                ties = INT_MAX;
                break;
            }
            ties = need;
        }
    }
    // kept: rank above the threshold, or at it (its unknown bits are zeros) while ties last

    const int vecs = a.row_bytes / 16;
    auto move_rows = [&](int n) {                    // rows movers[i] -> holes[i], i < n, those of this CTA
        for (int e = tid; e < ((n + ranks - 1 - me) / ranks) * vecs; e += kEvictThreads) {
            const int i = e / vecs * ranks + me, c = e % vecs;
            const int sp = page_of(a, p, movers[i]), dp = page_of(a, p, holes[i]);
            if (sp < 0 || dp < 0) continue;
            const int in = (1 << a.page_shift) - 1;
            const long long from = sp * a.page_bytes + ((long long)((p.h << a.page_shift) + (movers[i] & in)) * vecs + c) * 16;
            const long long to = dp * a.page_bytes + ((long long)((p.h << a.page_shift) + (holes[i] & in)) * vecs + c) * 16;
            const uint4 x = *reinterpret_cast<const uint4*>(a.k + from), y = *reinterpret_cast<const uint4*>(a.v + from);
            *reinterpret_cast<uint4*>(a.k + to) = x;
            *reinterpret_cast<uint4*>(a.v + to) = y;
            if (c == 0) {
                const long long se = element_of(a, p, sp, movers[i]), de = element_of(a, p, dp, holes[i]);
                a.scores_out[de] = a.scores[se];
                if (a.positions) a.positions_out[de] = a.positions[se];
            }
        }
    };
    auto carry = [&](int j) {                        // a kept slot that stays, where the results go elsewhere
        if ((!out && !pos_out) || j % ranks != me) return;
        const int page = page_of(a, p, j);
        if (page < 0) return;
        const long long e = element_of(a, p, page, j);
        if (out) a.scores_out[e] = a.scores[e];
        if (pos_out) a.positions_out[e] = a.positions[e];
    };
    if (!cut) {
        for (int j = tid; j < p.L; j += kEvictThreads) carry(j);
        return;
    }
    if (p.b == 0) return;
    // Slots in order, holes and movers into two buffers; as many as both have are moved whenever one is full.
    int hole_at = 0, mover_at = p.b;                 // next slots to look at
    int nh = 0, nm = 0;                              // in the buffers
    int tied = 0;                                    // slots at the threshold before hole_at and before mover_at
    int tied_m = 0;
    // ties below b come before those behind it
    if (ties != INT_MAX) {
        int mine = 0;
        for (int j = tid; j < p.b; j += kEvictThreads) mine += rank(j) == threshold;
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) red[warp] = (uint32_t)mine;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kEvictWarps; ++i) tied_m += (int)red[i];
        __syncthreads();
    }
    auto keeps = [&](uint32_t x, int before) { return x > threshold || (x == threshold && (ties == INT_MAX || before < ties)); };
    for (;;) {
        while (nh + kEvictThreads <= kBuffer && hole_at < p.b) {
            const int j = hole_at + tid;
            const bool in = j < p.b;
            const uint32_t x = in ? rank(j) : 0u;
            const uint32_t tie = in && x == threshold && ties != INT_MAX ? 1u : 0u;
            uint2 t = scan_pairs(tie, red);
            const bool kept = in && keeps(x, tied + (int)(t.x - tie));
            tied += (int)t.y;
            if (kept) carry(j);
            const uint32_t hole = in && !kept ? 1u : 0u;
            t = scan_pairs(hole, red);
            if (hole) holes[nh + t.x - 1] = j;
            nh += (int)t.y;
            hole_at += kEvictThreads;
        }
        while (nm + kEvictThreads <= kBuffer && mover_at < p.L) {
            const int j = mover_at + tid;
            const bool in = j < p.L;
            const uint32_t x = in ? rank(j) : 0u;
            const uint32_t tie = in && x == threshold && ties != INT_MAX ? 1u : 0u;
            uint2 t = scan_pairs(tie, red);
            const uint32_t move = in && keeps(x, tied_m + (int)(t.x - tie)) ? 1u : 0u;
            tied_m += (int)t.y;
            t = scan_pairs(move, red);
            if (move) movers[nm + t.x - 1] = j;
            nm += (int)t.y;
            mover_at += kEvictThreads;
        }
        // every CTA has looked at the slots before hole_at and mover_at (all look at the same ones): they may be written
        if (ranks > 1) cluster.sync();
        else __syncthreads();
        const int n = min(nh, nm);
        move_rows(n);
        __syncthreads();
        if (hole_at >= p.b && mover_at >= p.L) break;
        // the rest to the front
        const int left_h = nh - n, left_m = nm - n;
        int keep_h[2], keep_m[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = tid + i * kEvictThreads;
            keep_h[i] = at < left_h ? holes[n + at] : 0;
            keep_m[i] = at < left_m ? movers[n + at] : 0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = tid + i * kEvictThreads;
            if (at < left_h) holes[at] = keep_h[i];
            if (at < left_m) movers[at] = keep_m[i];
        }
        nh = left_h;
        nm = left_m;
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
                    block_table, kv_lens, keep, dropped, page_stride * es, S, Hkv, table_width, shift, num_pages, d * es, sinks,
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
