// Attention weights summed over a step's rows, key by key, into the scores of a paged cache (include/lla.h, paged_weigh):
//
//   score_j <- decay score_j (0 for the step's own tokens) + sum_rows exp(tau q.k_j - lse_row).
//
// The attention wrote each row's logsumexp, so that one pass over the keys is enough and no row needs what another CTA
// has.  Keys are the rows of the mma operand (16 to a tile) and query rows its columns, so the sum over query rows is a sum
// over a thread's own values and the four lanes of a quad, and a key belongs to one warp: no atomics.
//
// Every warp has its own keys, 16 of a 64-key tile, and copies them with cp.async through stages of its own: no block
// barrier.  A decode step is bound by reading the keys once.  fp32 keys and queries are multiplied as three tf32 products
// of their upper and lower 11 bits, as in lla_paged_decode.cu.
#include <cuda_bf16.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "../../include/lla.h"
#include "lla_internal.h"
#include "lla_weigh.h"
#include "tc_ptx.cuh"

namespace lla {
namespace weigh {
namespace {

constexpr int kTile = 64, kBlock = 32;       // keys of a tile, rows of a block
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kKeys = kTile / kWarps;        // a warp's

template <typename T, int D>
struct Shape {
    static constexpr int kRow = D * (int)sizeof(T);              // bytes of a key
    static constexpr int kPieces = kRow / 16;                    // 16-byte pieces of it
    static constexpr int kStage = kKeys * kRow;                  // a warp's 16 keys
    static constexpr int kStages = kRow >= 512 ? 3 : kRow >= 256 ? 4 : 6;
    static constexpr int kSteps = kRow / 32;                     // mma steps over d: 32 bytes of a row each
    static constexpr int kSets = kRow >= 512 ? 1 : 2;            // sets of eight rows at a time
    static constexpr size_t smem = (size_t)kWarps * kStages * kStage;
};

struct Args {
    Work w;
    const void* q;
    const float* lse;
    const char* k;
    int Hq;
    long long q_stride, page_bytes;          // q_stride in elements
    float scale;                             // tau log2(e)
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo, 11 bits each (but for 2^-23 of x); a NaN stays one in lo.
__device__ __forceinline__ void split(uint32_t x, uint32_t& hi, uint32_t& lo) {
    hi = (x + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) weigh_mma_kernel(Args a) {
    using Sh = Shape<T, D>;
    constexpr int NS = Sh::kStages, SETS = Sh::kSets, STEPS = Sh::kSteps, P = Sh::kPieces;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ long long scratch[40];
    const Work& w = a.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const uint32_t base = tc::smem_u32(ring) + warp * NS * Sh::kStage;
    cudaGridDependencySynchronize();
    Walk ahead = begin_walk(w, scratch), wk = ahead;

    // copies of this warp's keys of a piece into a stage
    auto fetch = [&](int stage, bool& more) {
        Piece p;
        more = more && next_piece(w, ahead, p);
        if (more) {
            const int key0 = (p.t << w.keys_shift) + warp * kKeys;
            const int* row = w.table + (size_t)p.s * w.width;
#pragma unroll
            for (int i = 0; i < (kKeys * P + 31) / 32; ++i) {
                const int e = i * 32 + lane, r = e / P, x = e % P, key = key0 + r;
                if (e >= kKeys * P || key >= p.q.L) continue;        // keys behind the last are never weighed
                const int page = row[key >> w.page_shift];
                if (page < 0 || page >= w.num_pages) continue;       // (reported where its score would be written)
                const int in = key & ((1 << w.page_shift) - 1);
                copy16(base + stage * Sh::kStage + r * Sh::kRow + ((x ^ (r & (P < 8 ? P - 1 : 7))) << 4),
                       a.k + page * a.page_bytes + ((long long)((p.h << w.page_shift) + in) * P + x) * 16);
            }
        }
        copies_end();
    };
    bool more = true;
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) fetch(i, more);

    const uint32_t* q32 = static_cast<const uint32_t*>(a.q);
    int stage = 0;
    Piece p;
    p.parts = p.s = p.h = p.t = 0;
    p.slot = -1;
    int at_s = -1, at_h = -1;                // whose rows the operand holds, where they are all of them
    uint32_t b[SETS][STEPS][2];
    float lse[SETS][2];
    int limit[SETS][2];
    while (next_piece(w, wk, p)) {
        copies_wait<NS - 2>();
        __syncwarp();
        const int key0 = (p.t << w.keys_shift) + warp * kKeys, rows = rows_of(w, p.q);
        const bool all = rows <= SETS * 8;   // the operand can stay from tile to tile
        float sum[2] = {0.f, 0.f};           // of keys g and g + 8
        const uint32_t at = base + stage * Sh::kStage;
        if (key0 < p.q.L) {
#pragma unroll 1
            for (int r0 = p.b0 * kBlock; r0 < min(p.b1 * kBlock, rows); r0 += SETS * 8) {
                if (!all || at_s != p.s || at_h != p.h) {
                    at_s = all ? p.s : -1;
                    at_h = p.h;
#pragma unroll
                    for (int n = 0; n < SETS; ++n) {
                        const int r = r0 + n * 8 + g;               // the lane's row of the operand
                        const int i = over_g(w, min(r, rows - 1)), head = p.h * w.G + min(r, rows - 1) - i * w.G;
                        const uint32_t* src = q32 + ((p.q.token0 + p.q.first + i) * a.q_stride + (long long)head * D) * (int)sizeof(T) / 4;
#pragma unroll
                        for (int k = 0; k < STEPS; ++k) {
                            b[n][k][0] = r < rows ? src[k * 8 + c] : 0u;
                            b[n][k][1] = r < rows ? src[k * 8 + c + 4] : 0u;
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {               // the lane's columns of the products
                            const int x = r0 + n * 8 + 2 * c + e;
                            limit[n][e] = 0;
                            lse[n][e] = 0.f;
                            if (x < rows) {
                                const int ix = over_g(w, x);
                                const float y = a.lse[(long long)(p.q.token0 + p.q.first + ix) * a.Hq + p.h * w.G + x - ix * w.G];
                                lse[n][e] = y * 1.4426950408889634f;
                                limit[n][e] = y == -INFINITY ? 0 : keys_seen(w, p.q, ix);     // -inf: a row without weights
                            }
                        }
                    }
                }
                float s[SETS][4], small[sizeof(T) == 4 ? SETS : 1][4];
#pragma unroll
                for (int n = 0; n < SETS; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[n][i] = 0.f;
                        if (sizeof(T) == 4) small[sizeof(T) == 4 ? n : 0][i] = 0.f;
                    }
#pragma unroll
                for (int k = 0; k < STEPS; ++k) {
                    uint32_t f[4];
                    const int r = lane & 15, x = k * 2 + (lane >> 4);
                    ldsm4(at + r * Sh::kRow + ((x ^ (r & (P < 8 ? P - 1 : 7))) << 4), f);
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int n = 0; n < SETS; ++n) mma(s[n], f, b[n][k][0], b[n][k][1]);
                    } else {
                        uint32_t fh[4], fl[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) split(f[i], fh[i], fl[i]);
#pragma unroll
                        for (int n = 0; n < SETS; ++n) {
                            uint32_t h0, l0, h1, l1;
                            split(b[n][k][0], h0, l0);
                            split(b[n][k][1], h1, l1);
                            mma_tf32(small[n], fl, h0, h1);
                            mma_tf32(small[n], fh, l0, l1);
                            mma_tf32(s[n], fh, h0, h1);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < SETS; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key0 + g + (i >> 1) * 8;
                        float x = s[n][i];
                        if constexpr (sizeof(T) == 4) x += small[n][i];
                        if (key < limit[n][i & 1]) sum[i >> 1] += tc::ex2(fmaf(x, a.scale, -lse[n][i & 1]));
                    }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
            }
            const float mine = c == 0 ? sum[0] : sum[1];
            const int k = warp * kKeys + g + c * 8;
            if (c < 2) {
                if (p.slot < 0) put_score(w, p.q, p.s, p.h, (p.t << w.keys_shift) + k, mine);
                else part_of(w, blockIdx.x, p.slot)[k] = mine;
            }
        } else if (p.slot >= 0 && c < 2) {
            part_of(w, blockIdx.x, p.slot)[warp * kKeys + g + c * 8] = 0.f;
        }
        __syncwarp();                        // the stage before this one is read: it may be filled again
        fetch((stage + NS - 1) % NS, more);
        if (++stage == NS) stage = 0;
    }
    copies_wait<0>();
    if (tid == 0) w.hdr[blockIdx.x] = WeighHeader{p.slot == 1 ? p.parts : 0, p.s, p.h, p.t};
}

// Adds the parts of the tile that CTA blockIdx.x starts and others finish: its slot 1, then slots 0 of those behind it.
__global__ void __launch_bounds__(256) weigh_join_kernel(Work w) {
    cudaGridDependencySynchronize();
    const WeighHeader h = w.hdr[blockIdx.x];
    if (h.parts == 0) return;
    const Seq q = load_seq(w, h.s);
    for (int k = threadIdx.x; k < 1 << w.keys_shift; k += 256) {
        float x = part_of(w, blockIdx.x, 1)[k];
        for (int i = 1; i < h.parts; ++i) x += part_of(w, blockIdx.x + i, 0)[k];
        put_score(w, q, h.s, h.h, (h.tile << w.keys_shift) + k, x);
    }
}

template <typename T, int D>
cudaError_t launch_one(const Args& a, cudaStream_t stream) {
    constexpr size_t smem = Shape<T, D>::smem;
    cudaError_t e = cudaFuncSetAttribute(weigh_mma_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return paged::launch_after(weigh_mma_kernel<T, D>, dim3(a.w.ctas), kThreads, smem, stream, a);
}
template <typename T>
cudaError_t launch_typed(const Args& a, int d, cudaStream_t stream) {
    switch (d) {
        case 16: return launch_one<T, 16>(a, stream);
        case 32: return launch_one<T, 32>(a, stream);
        case 64: return launch_one<T, 64>(a, stream);
        default: return launch_one<T, 128>(a, stream);
    }
}

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

int check_sizes(int dtype, int T, int S, int Hq, int Hkv, int d, int page_size, int num_pages, int table_width, int max_new) {
    if (T < 1 || S < 1 || Hq < 1 || Hkv < 1 || num_pages < 1 || table_width < 1 || max_new < 1)
        return failf(LLA_ERR_INVALID_ARG, "T, S, Hq, Hkv, num_pages, table_width and max_new must be >= 1");
    if (Hq % Hkv != 0) return failf(LLA_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
    if (d != 16 && d != 32 && d != 64 && d != 128)
        return failf(LLA_ERR_INVALID_ARG, "head dim d must be 16, 32, 64 or 128 (got %d)", d);
    if (page_shift_of(page_size) < 0)
        return failf(LLA_ERR_INVALID_ARG, "page_size must be a power of two in 8 .. 256 (got %d)", page_size);
    if (dtype != LLA_DTYPE_BF16 && dtype != LLA_DTYPE_FP32) return failf(LLA_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (S > (1 << 20) || (long long)T * Hq > (1LL << 30) || (long long)table_width * page_size > (1LL << 28) ||
        (long long)table_width * page_size * (Hq / Hkv) > (1LL << 30) || Hkv > 65535 || Hq / Hkv > 1024)
        return failf(LLA_ERR_INVALID_ARG, "problem too large (S <= 2^20, T*Hq <= 2^30, table_width*page_size <= 2^28 and "
                                          "<= 2^30 Hkv/Hq, Hq/Hkv <= 1024)");
    return LLA_OK;
}

WeighSplit split_of(const WeighProblem& p, int sms) { return weigh_mma_split(p, sms); }

}  // namespace
}  // namespace weigh

WeighSplit weigh_mma_split(const WeighProblem& p, int sms) {
    const int row = p.d * (p.dtype == LLA_DTYPE_BF16 ? 2 : 4);
    return WeighSplit{weigh::kTile, weigh::kBlock, (row >= 512 ? 2 : 3) * sms, 0};
}

cudaError_t launch_weigh_mma(const WeighProblem& p, const WeighSplit& sp, cudaStream_t stream) {
    const int es = p.dtype == LLA_DTYPE_BF16 ? 2 : 4;
    weigh::Args a{weigh::make_work(p, sp), p.q, p.lse, static_cast<const char*>(p.k), p.Hq, p.q_stride, p.page_stride * es,
                  p.tau * 1.4426950408889634f};
    return p.dtype == LLA_DTYPE_BF16 ? weigh::launch_typed<__nv_bfloat16>(a, p.d, stream) : weigh::launch_typed<float>(a, p.d, stream);
}

cudaError_t launch_weigh_join(const WeighProblem& p, const WeighSplit& sp, cudaStream_t stream) {
    return paged::launch_after(weigh::weigh_join_kernel, dim3(sp.ctas), 256, 0, stream, weigh::make_work(p, sp));
}

}  // namespace lla

namespace lw = lla::weigh;

extern "C" {

size_t lla_paged_weigh_workspace_size(int dtype, int T, int S, int Hq, int Hkv, int d, int page_size, int table_width, int max_new) {
    if (lw::check_sizes(dtype, T, S, Hq, Hkv, d, page_size, 1, table_width, max_new) != LLA_OK) return 0;
    lla::WeighProblem p{};
    p.T = T; p.S = S; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.d = d; p.max_new = max_new; p.dtype = dtype;
    const int sms = lw::sm_count();
    return lla::weigh_workspace_bytes(lw::split_of(p, sms > 0 ? sms : 152));
}

int lla_paged_weigh(int dtype, const void* q, const float* lse, const void* k_cache, const float* scores, float* scores_out,
                    int* positions, const int* dropped, const int* block_table, const int* cu_q, const int* kv_lens, int T, int S,
                    int Hq, int Hkv, int d, int page_size, int num_pages, int table_width, int max_new, long long q_stride,
                    long long page_stride, float tau, float decay, int last, int causal, void* workspace, size_t workspace_bytes,
                    void* stream_) {
    lla::set_error(LLA_OK, "");
    if (!q || !lse || !k_cache || !scores || !scores_out || !block_table || !cu_q || !kv_lens)
        return lw::failf(LLA_ERR_INVALID_ARG, "null tensor pointer");
    if (!lw::aligned(q, 16) || !lw::aligned(k_cache, 16)) return lw::failf(LLA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    const void* words[] = {lse, scores, scores_out, positions, dropped, block_table, cu_q, kv_lens};
    for (const void* x : words)
        if (!lw::aligned(x, 4)) return lw::failf(LLA_ERR_INVALID_ARG, "int32 and fp32 pointers must be 4-byte aligned");
    const int st = lw::check_sizes(dtype, T, S, Hq, Hkv, d, page_size, num_pages, table_width, max_new);
    if (st != LLA_OK) return st;
    if (!(tau > 0.f) || !(tau < 1e30f)) return lw::failf(LLA_ERR_INVALID_ARG, "tau must be finite and > 0");
    if (!(decay >= 0.f) || !(decay < INFINITY)) return lw::failf(LLA_ERR_INVALID_ARG, "decay must be finite and >= 0");
    if (last < 0) return lw::failf(LLA_ERR_INVALID_ARG, "last must be >= 0 (0: every row)");
    const int es = dtype == LLA_DTYPE_BF16 ? 2 : 4, ve = 16 / es;
    if (q_stride < (long long)Hq * d || q_stride % ve)
        return lw::failf(LLA_ERR_INVALID_ARG, "the token stride must be >= Hq*d and a multiple of 16 bytes");
    if (page_stride < (long long)Hkv * page_size * d || page_stride % ((long long)page_size * d))
        return lw::failf(LLA_ERR_INVALID_ARG, "page_stride must be >= Hkv*page_size*d and a multiple of page_size*d");
    if (page_stride / ((long long)page_size * d) * num_pages > 0x7fffffffLL)
        return lw::failf(LLA_ERR_INVALID_ARG, "problem too large (head slices of the cache must number < 2^31)");

    lla::WeighProblem p{};
    p.q = q; p.lse = lse; p.k = k_cache; p.scores = scores; p.out = scores_out; p.positions = positions; p.dropped = dropped;
    p.table = block_table; p.cu_q = cu_q; p.kv_lens = kv_lens; p.T = T; p.S = S; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.d = d;
    p.page_shift = lw::page_shift_of(page_size); p.num_pages = num_pages; p.width = table_width; p.max_new = max_new;
    p.last = last; p.causal = causal != 0; p.dtype = dtype; p.q_stride = q_stride; p.page_stride = page_stride; p.tau = tau;
    p.decay = decay;
    const int sms = lw::sm_count();
    if (sms < 1) return lw::failf(LLA_ERR_CUDA, "lla_paged_weigh: no device");
    const lla::WeighSplit sp = lw::split_of(p, sms);
    if (sp.ctas > lla::kPagedMaxCtas) return lw::failf(LLA_ERR_UNSUPPORTED, "device has too many SMs (%d)", sms);
    const size_t need = lla::weigh_workspace_bytes(sp);
    if (workspace) {
        if (workspace_bytes < need) return lw::failf(LLA_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
        if (!lw::aligned(workspace, 256)) return lw::failf(LLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    }
    p.err = lla::device_error_word();
    if (!p.err) return lw::failf(LLA_ERR_CUDA, "lla_paged_weigh: device error word not found");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    p.ws = workspace;
    cudaError_t e = cudaSuccess;
    if (!workspace && (e = cudaMallocAsync(&p.ws, need, stream)) != cudaSuccess) return lw::cuda_failf(e, "cudaMallocAsync(workspace)");
    e = lla::launch_weigh_mma(p, sp, stream);
    // a tile of one block is never cut
    const long long most = (long long)(last > 0 && last < max_new ? last : max_new) * p.G;
    if (e == cudaSuccess && most > sp.rows) e = lla::launch_weigh_join(p, sp, stream);
    if (!workspace) {
        const cudaError_t e2 = cudaFreeAsync(p.ws, stream);
        if (e == cudaSuccess && e2 != cudaSuccess) return lw::cuda_failf(e2, "cudaFreeAsync(workspace)");
    }
    if (e != cudaSuccess) return lw::cuda_failf(e, "lla_paged_weigh launch");
    return LLA_OK;
}

}  // extern "C"
