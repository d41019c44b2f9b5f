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

// RS sets of eight query rows at a time.
template <typename T, int D>
struct Shape {
    static constexpr int kRow = D * (int)sizeof(T);              // bytes of a key
    static constexpr int kPieces = kRow / 16;                    // 16-byte pieces of it
    static constexpr int kStage = kKeys * (kRow + 8);            // a warp's 16 keys, their pages and old scores
    static constexpr int kStages = kRow >= 512 ? 3 : kRow >= 256 ? 4 : 6;
    static constexpr int kSteps = kRow / 32;                     // mma steps over d: 32 bytes of a row each
    static constexpr size_t smem = (size_t)kWarps * kStages * kStage;
    // on an SM; named to the compiler, which else kept to 128 registers or took too many for three (64 x 16 heads at 4096: 171 us for 168)
    static constexpr int kCtas = kRow >= 512 ? 2 : 3;
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

// Where a tile is one unit (rows of one block, no extra units), the next piece is the next tile: no divisions.
__device__ __forceinline__ bool next_tile(const Work& w, Walk& k, Piece& p, int& tiles) {
    if (k.u >= k.end) return false;
    p.s = k.s; p.h = k.h; p.t = k.t; p.q = k.q;
    p.b0 = 0; p.b1 = 1;
    p.slot = -1; p.parts = 0;
    ++k.u;
    if (++k.t == tiles) {
        k.t = 0;
        if (++k.h == w.Hkv) {
            k.h = 0;
            if (k.u < k.end) {
                do {
                    if (++k.s >= w.S) {                  // lengths that changed during the call
                        k.end = k.u;
                        break;
                    }
                    k.q = load_seq(w, k.s);
                } while (tiles_of(w, k.q) == 0);
                tiles = tiles_of(w, k.q);
            }
        }
    }
    return true;
}

// ONE: no sequence has more than 8 RS rows to a key head, so a tile is one unit and its rows stay in registers from tile to
// tile.  Else blocks of kBlock rows, RS sets of them at a time.
template <typename T, int D, int RS, bool ONE>
__global__ void __launch_bounds__(kThreads, (Shape<T, D>::kCtas)) weigh_mma_kernel(Args a) {
    using Sh = Shape<T, D>;
    constexpr int NS = Sh::kStages, STEPS = Sh::kSteps, P = Sh::kPieces, SW = P < 8 ? P - 1 : 7;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ long long scratch[40];
    const Work& w = a.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    unsigned char* mine = ring + warp * NS * Sh::kStage;         // stages: keys, pages [16], old scores [16]
    const uint32_t base = tc::smem_u32(mine);
    cudaGridDependencySynchronize();
    Walk ahead = begin_walk(w, scratch), wk = ahead;
    int tiles_a = tiles_of(w, ahead.q), tiles_w = tiles_a;
    auto next = [&](Walk& k, Piece& p, int& tiles) { return ONE ? next_tile(w, k, p, tiles) : next_piece(w, k, p); };

    // The piece to be copied next, and the page of its key `lane & 15` (loaded a piece ahead of its use).
    Piece n;
    int page = -1;
    bool more;
    auto look = [&] {
        more = next(ahead, n, tiles_a);
        page = -1;
        const int key = (n.t << w.keys_shift) + warp * kKeys + (lane & 15);
        if (more && key < n.q.L) page = w.table[(size_t)n.s * w.width + (key >> w.page_shift)];
    };
    look();
    auto fetch = [&](int stage) {
        if (more) {
            const int key0 = (n.t << w.keys_shift) + warp * kKeys, in = (1 << w.page_shift) - 1;
            const int id = page >= 0 && page < w.num_pages ? page : -1;      // (reported where its score would be written)
#pragma unroll
            for (int i = 0; i < (kKeys * P + 31) / 32; ++i) {
                const int e = i * 32 + lane, r = e / P, x = e % P;
                const int pg = __shfl_sync(0xffffffffu, id, r & 15);         // keys behind the last have none: never weighed
                if (pg >= 0 && e < kKeys * P)
                    copy16(base + stage * Sh::kStage + r * Sh::kRow + ((x ^ (r & SW)) << 4),
                           a.k + pg * a.page_bytes + ((long long)((n.h << w.page_shift) + ((key0 + r) & in)) * P + x) * 16);
            }
            if (lane < kKeys) {
                const int key = key0 + lane;
                reinterpret_cast<int*>(mine + stage * Sh::kStage + kKeys * Sh::kRow)[lane] = page;
                if (id >= 0 && n.slot < 0 && w.decay != 0.f && !(w.causal && key >= n.q.L - n.q.n))
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                                 ::"r"(base + stage * Sh::kStage + kKeys * (Sh::kRow + 4) + lane * 4),
                                 "l"(w.scores + ((((long long)id * w.Hkv + n.h) << w.page_shift) + (key & in)) ) : "memory");
            }
            look();
        }
        copies_end();
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) fetch(i);

    const uint32_t* q32 = static_cast<const uint32_t*>(a.q);
    int stage = 0;
    Piece p;
    p.parts = p.s = p.h = p.t = 0;
    p.slot = -1;
    int at_s = -1, at_h = -1;                // whose rows the operand holds, where they are all of them
    uint32_t b[RS][STEPS][2];
    float lse[RS][2];
    int limit[RS][2];
    while (next(wk, p, tiles_w)) {
        copies_wait<NS - 2>();
        __syncwarp();
        const int key0 = (p.t << w.keys_shift) + warp * kKeys, rows = rows_of(w, p.q);
        float sum[2] = {0.f, 0.f};           // of keys g and g + 8
        const uint32_t at = base + stage * Sh::kStage;
        if (key0 < p.q.L) {
            const int r1 = ONE ? 1 : min(p.b1 * kBlock, rows);
#pragma unroll 1
            for (int r0 = ONE ? 0 : p.b0 * kBlock; r0 < r1; r0 += RS * 8) {
                if (!ONE || at_s != p.s || at_h != p.h) {
                    at_s = p.s;
                    at_h = p.h;
#pragma unroll
                    for (int m = 0; m < RS; ++m) {
                        const int r = r0 + m * 8 + g;               // the lane's row of the operand
                        const int i = over_g(w, min(r, rows - 1)), head = p.h * w.G + min(r, rows - 1) - i * w.G;
                        const uint32_t* src = q32 + ((p.q.token0 + p.q.first + i) * a.q_stride + (long long)head * D) * (int)sizeof(T) / 4;
#pragma unroll
                        for (int k = 0; k < STEPS; ++k) {
                            b[m][k][0] = r < rows ? src[k * 8 + c] : 0u;
                            b[m][k][1] = r < rows ? src[k * 8 + c + 4] : 0u;
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {               // the lane's columns of the products
                            const int x = r0 + m * 8 + 2 * c + e;
                            limit[m][e] = 0;
                            lse[m][e] = 0.f;
                            if (x < rows) {
                                const int ix = over_g(w, x);
                                const float y = a.lse[(long long)(p.q.token0 + p.q.first + ix) * a.Hq + p.h * w.G + x - ix * w.G];
                                lse[m][e] = y * 1.4426950408889634f;
                                limit[m][e] = y == -INFINITY ? 0 : keys_seen(w, p.q, ix);     // -inf: a row without weights
                            }
                        }
                    }
                }
                // even and odd steps of bf16, large and small products of fp32, have sums of their own
                float s[RS][4], other[RS][4];
#pragma unroll
                for (int m = 0; m < RS; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[m][i] = other[m][i] = 0.f;
#pragma unroll
                for (int k = 0; k < STEPS; ++k) {
                    uint32_t f[4];
                    const int r = lane & 15, x = k * 2 + (lane >> 4);
                    ldsm4(at + r * Sh::kRow + ((x ^ (r & SW)) << 4), f);
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int m = 0; m < RS; ++m) mma(k & 1 ? other[m] : s[m], f, b[m][k][0], b[m][k][1]);
                    } else {
                        uint32_t fh[4], fl[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) split(f[i], fh[i], fl[i]);
#pragma unroll
                        for (int m = 0; m < RS; ++m) {
                            uint32_t h0, l0, h1, l1;
                            split(b[m][k][0], h0, l0);
                            split(b[m][k][1], h1, l1);
                            mma_tf32(other[m], fl, h0, h1);
                            mma_tf32(other[m], fh, l0, l1);
                            mma_tf32(s[m], fh, h0, h1);
                        }
                    }
                }
#pragma unroll
                for (int m = 0; m < RS; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (key0 + g + (i >> 1) * 8 < limit[m][i & 1])
                            sum[i >> 1] += tc::ex2(fmaf(s[m][i] + other[m][i], a.scale, -lse[m][i & 1]));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
            }
        }
        if (c < 2) {
            const int k = g + c * 8, key = key0 + k;
            float x = c == 0 ? sum[0] : sum[1];
            if (p.slot >= 0) {
                part_of(w, blockIdx.x, p.slot)[warp * kKeys + k] = x;
            } else if (key < p.q.L) {
                const unsigned char* st = mine + stage * Sh::kStage + kKeys * Sh::kRow;
                const int pg = reinterpret_cast<const int*>(st)[k];
                if (pg < 0 || pg >= w.num_pages) {
                    atomicOr(w.err, (unsigned)kDevErrPagedArg);
                } else {
                    const long long e = (((long long)pg * w.Hkv + p.h) << w.page_shift) + (key & ((1 << w.page_shift) - 1));
                    const bool fresh = w.causal && key >= p.q.L - p.q.n;
                    if (!fresh && w.decay != 0.f) x = fmaf(w.decay, reinterpret_cast<const float*>(st)[kKeys + k], x);
                    w.out[e] = x;
                    if (fresh && w.positions) w.positions[e] = key + (w.dropped ? w.dropped[p.s] : 0);
                }
            }
        }
        __syncwarp();                        // the stage before this one is read: it may be filled again
        fetch((stage + NS - 1) % NS);
        if (++stage == NS) stage = 0;
    }
    copies_wait<0>();
    if (!ONE && tid == 0) w.hdr[blockIdx.x] = WeighHeader{p.slot == 1 ? p.parts : 0, p.s, p.h, p.t};
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

template <typename T, int D, int RS, bool ONE>
cudaError_t launch_rows(const Args& a, cudaStream_t stream) {
    constexpr size_t smem = Shape<T, D>::smem;
    auto* kern = weigh_mma_kernel<T, D, RS, ONE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return paged::launch_after(kern, dim3(a.w.ctas), kThreads, smem, stream, a);
}
// rows: the most that a sequence has to a key head.  Sets that stay in registers, as many as there is room for.  bf16 with d = 128
// comes here with 16 rows at most, with d = 64 32 (weigh_tc_fits).
template <typename T, int D>
cudaError_t launch_one(const Args& a, long long rows, cudaStream_t stream) {
    constexpr bool kTc = sizeof(T) == 2 && D >= 64;
    if (rows <= 8) return launch_rows<T, D, 1, true>(a, stream);
    if (rows <= 16 || (kTc && D == 128)) return launch_rows<T, D, 2, true>(a, stream);
    if constexpr (D * sizeof(T) <= 256 && !(kTc && D == 128)) {
        if (rows <= 32 || kTc) return launch_rows<T, D, 4, true>(a, stream);
    }
    if constexpr (!kTc) return launch_rows<T, D, 2, false>(a, stream);
    return cudaErrorInvalidValue;
}
template <typename T>
cudaError_t launch_typed(const Args& a, int d, long long rows, cudaStream_t stream) {
    switch (d) {
        case 16: return launch_one<T, 16>(a, rows, stream);
        case 32: return launch_one<T, 32>(a, rows, stream);
        case 64: return launch_one<T, 64>(a, rows, stream);
        default: return launch_one<T, 128>(a, rows, stream);
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

WeighSplit split_of(const WeighProblem& p, int sms) { return weigh_tc_fits(p) ? weigh_tc_split(p, sms) : weigh_mma_split(p, sms); }

}  // namespace
}  // namespace weigh

WeighSplit weigh_mma_split(const WeighProblem& p, int sms) {
    const int row = p.d * (p.dtype == LLA_DTYPE_BF16 ? 2 : 4);
    return WeighSplit{weigh::kTile, weigh::kBlock, (row >= 512 ? 2 : 3) * sms, 0};      // Shape::kCtas
}

cudaError_t launch_weigh_mma(const WeighProblem& p, const WeighSplit& sp, cudaStream_t stream) {
    const int es = p.dtype == LLA_DTYPE_BF16 ? 2 : 4;
    weigh::Args a{weigh::make_work(p, sp), p.q, p.lse, static_cast<const char*>(p.k), p.Hq, p.q_stride, p.page_stride * es,
                  p.tau * 1.4426950408889634f};
    const long long rows = most_rows(p);
    return p.dtype == LLA_DTYPE_BF16 ? weigh::launch_typed<__nv_bfloat16>(a, p.d, rows, stream)
                                     : weigh::launch_typed<float>(a, p.d, rows, stream);
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
                    int* positions, const int* dropped, const int* block_table, const int* cu_q, const int* kv_lens,
                    const int* granted, int T, int S, int Hq, int Hkv, int d, int page_size, int num_pages, int table_width, int max_new, long long q_stride,
                    long long page_stride, float tau, float decay, int last, int causal, void* workspace, size_t workspace_bytes,
                    void* stream_) {
    lla::set_error(LLA_OK, "");
    if (!q || !lse || !k_cache || !scores || !scores_out || !block_table || !cu_q || !kv_lens)
        return lw::failf(LLA_ERR_INVALID_ARG, "null tensor pointer");
    if (!lw::aligned(q, 16) || !lw::aligned(k_cache, 16)) return lw::failf(LLA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    const void* words[] = {lse, scores, scores_out, positions, dropped, block_table, cu_q, kv_lens, granted};
    for (const void* x : words)
        if (!lw::aligned(x, 4)) return lw::failf(LLA_ERR_INVALID_ARG, "int32 and fp32 pointers must be 4-byte aligned");
    const int st = lw::check_sizes(dtype, T, S, Hq, Hkv, d, page_size, num_pages, table_width, max_new);
    if (st != LLA_OK) return st;
    // (the tensor cores' logsumexp is -lse / tau: it stays finite)
    if (!(tau >= 1e-30f) || !(tau < 1e30f)) return lw::failf(LLA_ERR_INVALID_ARG, "tau must be in [1e-30, 1e30)");
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
    p.table = block_table; p.cu_q = cu_q; p.kv_lens = kv_lens; p.granted = granted; p.T = T; p.S = S; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.d = d;
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
    const char* why = "lla_paged_weigh launch";
    e = lla::weigh_tc_fits(p) ? lla::launch_weigh_tc(p, sp, stream, &why) : lla::launch_weigh_mma(p, sp, stream);
    // a tile of one block is never cut
    if (e == cudaSuccess && lla::most_rows(p) > sp.rows) e = lla::launch_weigh_join(p, sp, stream);
    if (!workspace) {
        const cudaError_t e2 = cudaFreeAsync(p.ws, stream);
        if (e == cudaSuccess && e2 != cudaSuccess) return lw::cuda_failf(e2, "cudaFreeAsync(workspace)");
    }
    if (e != cudaSuccess) return lw::cuda_failf(e, why);
    return LLA_OK;
}

}  // extern "C"
