// Paged-cache entry points of the C ABI (include/lla.h): page planning, cache append and the Parallax
// attention over pages; argument checks, path choice, scratch, and the kernels of the first two.
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
namespace {

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

// log2 of a page size the kernels take (8, 16, ... 256), or -1.
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

// ------------------------------------------------------------------------------------------- plan
//
// Three running sums over the sequences (token rows, pages asked for, and from them who is served)
// are taken by every CTA for itself, in shared memory; the token rows and new pages are then dealt to
// the CTAs of one cluster, each finding its sequence by bisection of the sums.  What it moves is a few
// bytes a sequence and 12 a row: latency bounds it (two dependent reads and the scans), so it is one
// launch (on the device 3.6 us for 64 decoding sequences, where 256 threads do: 1024 took 5.5; 10.4 us for 512 sequences
// with 64,000 new rows, where a thread has one sequence: 11.8 with room for eight, more in one CTA).  The cluster barrier
// lets kv_lens take ctx_lens' place and free_left free_count's: they are written after every CTA has read.
constexpr int kPlanMaxSeqs = 8192;

struct PlanArgs {
    const int* ctx;
    const int* fresh;        // new_lens
    int* table;
    const int* free_pages;
    const int* free_count;
    int* kv_lens;
    int* cu_q;
    long long* slots;
    int* positions;
    int* granted;
    int* free_left;
    int S, width, page_shift, free_cap, T;
};

// Inclusive sum over the block's TH threads in thread order.
template <int TH>
__device__ long long scan_block(long long v, long long* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) red[warp] = v;
    __syncthreads();
    if (warp == 0) {
        long long x = lane < TH / 32 ? red[lane] : 0;
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += t;
        }
        red[lane] = x;
    }
    __syncthreads();
    const long long r = v + (warp ? red[warp - 1] : 0);
    __syncthreads();
    return r;
}

// Largest s with a[s] <= x (a ascending, a[0] <= x), s < n.
__device__ __forceinline__ int bisect(const int* a, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int TH, int PER>           // at most TH PER sequences
__global__ void __launch_bounds__(TH) paged_plan_kernel(PlanArgs a) {
    namespace cg = cooperative_groups;
    extern __shared__ int psm[];
    __shared__ long long red[32];
    __shared__ int taken_sh;
    int* cu = psm;                     // [S] first token row (cut to T)
    int* base = cu + a.S;              // [S] pages given to earlier sequences
    int* ctx = base + a.S;             // [S]
    int* okay = ctx + a.S;             // [S] granted
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, page = 1 << a.page_shift;
    const int per = (a.S + TH - 1) / TH, s0 = tid * per;
    const int have = min(max(*a.free_count, 0), a.free_cap);

    if (tid == 0) taken_sh = 0;
    int c[PER], n[PER];
    long long rows = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        c[i] = n[i] = 0;
        if (i < per && s0 + i < a.S) {
            c[i] = max(a.ctx[s0 + i], 0);
            n[i] = max(a.fresh[s0 + i], 0);
            rows += n[i];
        }
    }
    const long long rows_end = scan_block<TH>(rows, red);
    long long row = rows_end - rows, asks = 0;
    const long long room = (long long)a.width << a.page_shift;
    int need[PER];
    bool fits[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        need[i] = 0;
        fits[i] = false;
        if (i < per && s0 + i < a.S) {
            cu[s0 + i] = (int)(row < a.T ? row : a.T);
            ctx[s0 + i] = c[i];
            row += n[i];
            const long long total = (long long)c[i] + n[i];
            fits[i] = total <= room && row <= a.T;
            if (fits[i]) need[i] = (int)((total + page - 1) >> a.page_shift) - (int)(((long long)c[i] + page - 1) >> a.page_shift);
            asks += need[i];
        }
    }
    const long long asks_end = scan_block<TH>(asks, red);
    long long ask = asks_end - asks;
    int taken = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (i < per && s0 + i < a.S) {
            base[s0 + i] = (int)(ask < have ? ask : have);
            ask += need[i];
            const bool ok = fits[i] && (need[i] == 0 || ask <= have);
            okay[s0 + i] = ok;
            if (ok && need[i]) taken = (int)ask;
        }
    if (taken) atomicMax(&taken_sh, taken);
    // rows_end of the last thread is the number of token rows
    if (tid == TH - 1) red[0] = rows_end;
    __syncthreads();
    const int total_rows = (int)(red[0] < a.T ? red[0] : a.T);
    taken = taken_sh;

    // a warp takes runs of 32 kRun rows, a lane every 32nd of them: a bisection where the sequence changes, the table
    // reads side by side
    constexpr int kRun = 4;
    const int lane = tid & 31, warps = ranks * (TH / 32);
    for (int t0 = (rank * (TH / 32) + (tid >> 5)) * 32 * kRun; t0 < a.T; t0 += warps * 32 * kRun) {
        int pos[kRun], id[kRun], s = bisect(cu, a.S, min(t0 + lane, max(total_rows - 1, 0)));
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int t = t0 + lane + 32 * i;
            pos[i] = 0;
            id[i] = -1;
            if (t < total_rows) {
                if (s + 1 < a.S && cu[s + 1] <= t) s += 1 + bisect(cu + s + 1, a.S - s - 1, t);   // another sequence
                pos[i] = ctx[s] + (t - cu[s]);
                if (okay[s]) {
                    const int lp = pos[i] >> a.page_shift, held = (ctx[s] + page - 1) >> a.page_shift;
                    id[i] = lp < held ? a.table[(size_t)s * a.width + lp]
                                      : a.free_pages[have - 1 - (base[s] + lp - held)];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int t = t0 + lane + 32 * i;
            if (t < a.T) {
                a.slots[t] = id[i] >= 0 ? ((long long)id[i] << a.page_shift) + (pos[i] & (page - 1)) : -1;
                if (a.positions) a.positions[t] = pos[i];
            }
        }
    }
    for (int k = rank * TH + tid; k < taken; k += ranks * TH) {
        const int s = bisect(base, a.S, k);
        const int held = (ctx[s] + page - 1) >> a.page_shift;
        a.table[(size_t)s * a.width + held + (k - base[s])] = a.free_pages[have - 1 - k];
    }
    cluster.sync();
    if (rank == 0) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i < per && s0 + i < a.S) {
                a.kv_lens[s0 + i] = c[i] + (okay[s0 + i] ? n[i] : 0);
                a.granted[s0 + i] = okay[s0 + i];
                a.cu_q[s0 + i] = cu[s0 + i];
            }
        if (tid == 0) {
            a.cu_q[a.S] = total_rows;
            *a.free_left = have - taken;
        }
    }
}

// ----------------------------------------------------------------------------------------- append
//
// A thread moves 16 bytes of a key row and the 16 bytes of the value row at the same place: both
// directions are whole rows of d elements, so every warp reads and writes full lines.  Bound by the
// copied bytes: 145 MB of prompt rows (8 heads, d = 128) in 26.6 us, 5.4 TB/s (24.7 replayed from a graph).
struct AppendArgs {
    const char* k_new;
    const char* v_new;
    const long long* slots;
    char* k_cache;
    char* v_cache;
    long long k_stride, v_stride, page_stride;   // bytes
    int T, Hkv, vecs, page_shift, num_pages;     // vecs: 16-byte pieces of a row
    unsigned* err;
};

__global__ void __launch_bounds__(256) paged_append_kernel(AppendArgs a) {
    const int per = a.Hkv * a.vecs;
    const long long n = (long long)a.T * per;
    for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (long long)gridDim.x * blockDim.x) {
        const int t = (int)(e / per), x = (int)(e % per), h = x / a.vecs, c = x % a.vecs;
        const long long slot = a.slots[t];
        if (slot < 0) continue;                     // a padding row, or a token that got no page
        const long long page = slot >> a.page_shift;
        if (page >= a.num_pages) {
            atomicOr(a.err, (unsigned)kDevErrPagedArg);
            continue;
        }
        const long long off = slot & ((1 << a.page_shift) - 1);
        const long long to = page * a.page_stride + ((((long long)h << a.page_shift) + off) * a.vecs + c) * 16;
        const uint4 k = *reinterpret_cast<const uint4*>(a.k_new + t * a.k_stride + (long long)x * 16);
        const uint4 v = *reinterpret_cast<const uint4*>(a.v_new + t * a.v_stride + (long long)x * 16);
        *reinterpret_cast<uint4*>(a.k_cache + to) = k;
        *reinterpret_cast<uint4*>(a.v_cache + to) = v;
    }
}

// ------------------------------------------------------------------------------- attention: checks
int check_paged_sizes(int dtype, int path, int T, int S, int Hq, int Hkv, int d, int page_size, int num_pages,
                      int table_width, int max_new, int* rpath) {
    if (T < 1 || S < 1 || Hq < 1 || Hkv < 1 || num_pages < 1 || table_width < 1 || max_new < 1)
        return failf(LLA_ERR_INVALID_ARG, "T, S, Hq, Hkv, num_pages, table_width and max_new must be >= 1");
    if (Hq % Hkv != 0) return failf(LLA_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
    if (d != 16 && d != 32 && d != 64 && d != 128)
        return failf(LLA_ERR_INVALID_ARG, "head dim d must be 16, 32, 64 or 128 (got %d)", d);
    if (page_shift_of(page_size) < 0)
        return failf(LLA_ERR_INVALID_ARG, "page_size must be a power of two in 8 .. 256 (got %d)", page_size);
    if (dtype != LLA_DTYPE_BF16 && dtype != LLA_DTYPE_FP32) return failf(LLA_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (path < LLA_PATH_AUTO || path > LLA_PATH_FP32) return failf(LLA_ERR_INVALID_ARG, "unknown path %d", path);
    if (S > (1 << 20) || (long long)T * Hq > (1LL << 30) || (long long)table_width * page_size > (1LL << 28) ||
        (long long)table_width * page_size * (Hq / Hkv) > (1LL << 30) || Hkv > 65535 || Hq / Hkv > 1024)
        return failf(LLA_ERR_INVALID_ARG, "problem too large (S <= 2^20, T*Hq <= 2^30, table_width*page_size <= 2^28 and "
                                          "<= 2^30 Hkv/Hq, Hq/Hkv <= 1024)");
    *rpath = lla_resolve_path(dtype, path, d);
    if (*rpath == LLA_PATH_TENSOR && (dtype != LLA_DTYPE_BF16 || (d != 64 && d != 128)))
        return failf(LLA_ERR_UNSUPPORTED, "tensor path needs bf16 inputs and d in {64, 128}");
    return LLA_OK;
}

PagedSplit split_of(const PagedProblem& p, int rpath, int sms) {
    if (paged_decode_fits(p, rpath)) return paged_decode_split(p, sms);
    return rpath == LLA_PATH_TENSOR ? paged_tc_split(p, sms) : paged_simt_split(p, sms);
}

}  // namespace
}  // namespace lla

using lla::aligned;
using lla::cuda_failf;
using lla::failf;

extern "C" {

int lla_paged_plan(const int* ctx_lens, const int* new_lens, int S, int page_size, int* block_table, int table_width,
                   const int* free_pages, int free_capacity, const int* free_count, int T, int* kv_lens, int* cu_q,
                   long long* slots, int* positions, int* granted, int* free_left, void* stream_) {
    lla::set_error(LLA_OK, "");
    if (!ctx_lens || !new_lens || !block_table || !free_pages || !free_count || !kv_lens || !cu_q || !slots || !granted ||
        !free_left)
        return failf(LLA_ERR_INVALID_ARG, "null pointer");
    if (S < 1 || S > lla::kPlanMaxSeqs) return failf(LLA_ERR_INVALID_ARG, "S must be in [1, %d] (got %d)", lla::kPlanMaxSeqs, S);
    const int shift = lla::page_shift_of(page_size);
    if (shift < 0) return failf(LLA_ERR_INVALID_ARG, "page_size must be a power of two in 8 .. 256 (got %d)", page_size);
    if (table_width < 1 || (long long)table_width * page_size > (1LL << 28))
        return failf(LLA_ERR_INVALID_ARG, "table_width must be >= 1 and table_width*page_size <= 2^28");
    if (free_capacity < 1 || T < 1 || T > (1 << 30))
        return failf(LLA_ERR_INVALID_ARG, "free_capacity must be >= 1 and T in [1, 2^30]");
    const void* ints[] = {ctx_lens, new_lens, block_table, free_pages, free_count, kv_lens, cu_q, positions, granted, free_left};
    for (const void* x : ints)
        if (!aligned(x, 4)) return failf(LLA_ERR_INVALID_ARG, "int32 pointers must be 4-byte aligned");
    if (!aligned(slots, 8)) return failf(LLA_ERR_INVALID_ARG, "slots must be 8-byte aligned");

    lla::PlanArgs a{ctx_lens, new_lens, block_table, free_pages, free_count, kv_lens, cu_q, slots, positions,
                    granted, free_left, S, table_width, shift, free_capacity, T};
    const size_t smem = (size_t)S * 4 * sizeof(int);
    cudaError_t e = cudaSuccess;
    auto* kern = S <= 256 && T <= 1024 ? lla::paged_plan_kernel<256, 1>
                 : S <= 1024           ? lla::paged_plan_kernel<1024, 1>
                                       : lla::paged_plan_kernel<1024, lla::kPlanMaxSeqs / 1024>;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return cuda_failf(e, "lla_paged_plan");
    const int ctas = T > 4096 ? 8 : T > 1024 ? 4 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(S <= 256 && T <= 1024 ? 256 : 1024);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream_);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ctas > 1;                   // a CTA alone is a cluster of one
    e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess) return cuda_failf(e, "lla_paged_plan launch");
    return LLA_OK;
}

int lla_paged_append(int dtype, const void* k_new, const void* v_new, const long long* slots, void* k_cache,
                     void* v_cache, int T, int Hkv, int d, int page_size, int num_pages, long long k_stride,
                     long long v_stride, long long page_stride, void* stream_) {
    lla::set_error(LLA_OK, "");
    if (!k_new || !v_new || !slots || !k_cache || !v_cache) return failf(LLA_ERR_INVALID_ARG, "null tensor pointer");
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slots, 8))
        return failf(LLA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned (slots: 8)");
    if (dtype != LLA_DTYPE_BF16 && dtype != LLA_DTYPE_FP32) return failf(LLA_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (d != 16 && d != 32 && d != 64 && d != 128)
        return failf(LLA_ERR_INVALID_ARG, "head dim d must be 16, 32, 64 or 128 (got %d)", d);
    const int shift = lla::page_shift_of(page_size);
    if (shift < 0) return failf(LLA_ERR_INVALID_ARG, "page_size must be a power of two in 8 .. 256 (got %d)", page_size);
    if (T < 1 || Hkv < 1 || num_pages < 1 || Hkv > 65535 || T > (1 << 30))
        return failf(LLA_ERR_INVALID_ARG, "T, Hkv and num_pages must be >= 1 (T <= 2^30, Hkv <= 65535)");
    const int es = dtype == LLA_DTYPE_BF16 ? 2 : 4, ve = 16 / es;
    if (k_stride < (long long)Hkv * d || v_stride < (long long)Hkv * d || k_stride % ve || v_stride % ve)
        return failf(LLA_ERR_INVALID_ARG, "token strides must be >= Hkv*d and multiples of 16 bytes");
    if (page_stride < (long long)Hkv * page_size * d || page_stride % ((long long)page_size * d))
        return failf(LLA_ERR_INVALID_ARG, "page_stride must be >= Hkv*page_size*d and a multiple of page_size*d");
    if (page_stride / ((long long)page_size * d) * num_pages > INT_MAX)
        return failf(LLA_ERR_INVALID_ARG, "problem too large (head slices of the cache must number < 2^31)");
    unsigned* err = lla::device_error_word();
    if (!err) return failf(LLA_ERR_CUDA, "lla_paged_append: device error word not found");
    lla::AppendArgs a{static_cast<const char*>(k_new), static_cast<const char*>(v_new), slots,
                      static_cast<char*>(k_cache), static_cast<char*>(v_cache), k_stride * es, v_stride * es,
                      page_stride * es, T, Hkv, d * es / 16, shift, num_pages, err};
    const long long n = (long long)T * Hkv * a.vecs;
    const int blocks = (int)((n + 255) / 256 < 65536 ? (n + 255) / 256 : 65536);
    lla::paged_append_kernel<<<blocks, 256, 0, static_cast<cudaStream_t>(stream_)>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_failf(e, "lla_paged_append launch");
    return LLA_OK;
}

size_t lla_paged_parallax_workspace_size(int dtype, int path, int T, int S, int Hq, int Hkv, int d, int page_size,
                                         int table_width, int max_new) {
    int rpath = 0;
    if (lla::check_paged_sizes(dtype, path, T, S, Hq, Hkv, d, page_size, 1, table_width, max_new, &rpath) != LLA_OK) return 0;
    lla::PagedProblem p{};
    p.T = T; p.S = S; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.d = d; p.max_new = max_new; p.dtype = dtype;
    p.page_shift = lla::page_shift_of(page_size); p.width = table_width;
    const int sms = lla::sm_count();
    const lla::PagedSplit sp = lla::split_of(p, rpath, sms > 0 ? sms : 152);
    return lla::paged_workspace_bytes(sp.ctas, sp.rows, d);
}

int lla_paged_parallax(int dtype, int path, const void* q, const void* probe, const void* k_cache, const void* v_cache,
                       const int* block_table, const int* cu_q, const int* kv_lens, void* out, int T, int S, int Hq,
                       int Hkv, int d, int page_size, int num_pages, int table_width, int max_new, long long q_stride,
                       long long probe_stride, long long page_stride, float tau, int causal, void* workspace,
                       size_t workspace_bytes, void* stream_) {
    lla::set_error(LLA_OK, "");
    if (!q || !probe || !k_cache || !v_cache || !block_table || !cu_q || !kv_lens || !out)
        return failf(LLA_ERR_INVALID_ARG, "null tensor pointer");
    if (!aligned(q, 16) || !aligned(probe, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return failf(LLA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    if (!aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4))
        return failf(LLA_ERR_INVALID_ARG, "int32 pointers must be 4-byte aligned");
    int rpath = 0;
    const int st = lla::check_paged_sizes(dtype, path, T, S, Hq, Hkv, d, page_size, num_pages, table_width, max_new, &rpath);
    if (st != LLA_OK) return st;
    if (!(tau > 0.f) || !(tau < 1e30f)) return failf(LLA_ERR_INVALID_ARG, "tau must be finite and > 0");
    const int es = dtype == LLA_DTYPE_BF16 ? 2 : 4, ve = 16 / es;
    if (q_stride < (long long)Hq * d || probe_stride < (long long)Hq * d || q_stride % ve || probe_stride % ve)
        return failf(LLA_ERR_INVALID_ARG, "token strides must be >= Hq*d and multiples of 16 bytes");
    if (page_stride < (long long)Hkv * page_size * d || page_stride % ((long long)page_size * d))
        return failf(LLA_ERR_INVALID_ARG, "page_stride must be >= Hkv*page_size*d and a multiple of page_size*d");
    if (page_stride / ((long long)page_size * d) * num_pages > INT_MAX)
        return failf(LLA_ERR_INVALID_ARG, "problem too large (head slices of the cache must number < 2^31)");

    lla::PagedProblem p{};
    p.q = q; p.probe = probe; p.k = k_cache; p.v = v_cache; p.table = block_table; p.cu_q = cu_q; p.kv_lens = kv_lens;
    p.out = out; p.T = T; p.S = S; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.d = d;
    p.page_shift = lla::page_shift_of(page_size); p.num_pages = num_pages; p.width = table_width; p.max_new = max_new;
    p.q_stride = q_stride; p.r_stride = probe_stride; p.page_stride = page_stride;
    p.tau = tau; p.causal = causal != 0; p.dtype = dtype;
    const int sms = lla::sm_count();
    if (sms < 1) return failf(LLA_ERR_CUDA, "lla_paged_parallax: no device");
    const lla::PagedSplit sp = lla::split_of(p, rpath, sms);
    if (sp.ctas > lla::kPagedMaxCtas) return failf(LLA_ERR_UNSUPPORTED, "device has too many SMs (%d)", sms);
    const size_t need = lla::paged_workspace_bytes(sp.ctas, sp.rows, d);
    if (workspace) {
        if (workspace_bytes < need)
            return failf(LLA_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
        if (!aligned(workspace, 256)) return failf(LLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    }
    p.err = lla::device_error_word();
    if (!p.err) return failf(LLA_ERR_CUDA, "lla_paged_parallax: device error word not found");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    p.ws = workspace;
    cudaError_t e = cudaSuccess;
    if (!workspace && (e = cudaMallocAsync(&p.ws, need, stream)) != cudaSuccess)
        return cuda_failf(e, "cudaMallocAsync(workspace)");
    const char* why = nullptr;
    if (lla::paged_decode_fits(p, rpath)) e = lla::launch_paged_decode(p, sp, stream, &why);
    else if (rpath == LLA_PATH_TENSOR) e = lla::launch_paged_tc(p, sp, stream, &why);
    else e = lla::launch_paged_simt(p, sp, stream);
    if (e == cudaSuccess) e = lla::launch_paged_merge(p, sp, stream);
    if (!workspace) {
        const cudaError_t e2 = cudaFreeAsync(p.ws, stream);
        if (e == cudaSuccess && e2 != cudaSuccess) return cuda_failf(e2, "cudaFreeAsync(workspace)");
    }
    if (e != cudaSuccess) return cuda_failf(e, why ? why : "paged attention launch");
    return LLA_OK;
}

}  // extern "C"
