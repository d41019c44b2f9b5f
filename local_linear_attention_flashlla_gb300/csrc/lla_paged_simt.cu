// Parallax attention over a paged cache on CUDA cores (every product in fp32: bf16 of any head dim, fp32 with
// d = 16 or 128), and the merge of row tiles that several CTAs share (all paths).
//
// Per query row, over its keys in blocks, one pass (base-2 logits l = tau log2(e) q.k, t = probe.k):
//   m <- max(m, max l),  p = 2^(l - m),  w += p,  A += p (t - s0),  O1 += p v,  O2 += p (t - s0) v,
//   out = ((1 + A/w) O1 - O2) / w.
// The centre s0 is the softmax mean of t over the row's first block: the formula holds for any value,
// and one near the mean keeps O2 from holding a large multiple of O1 that the end would cancel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/lla.h"
#include "lla_internal.h"
#include "lla_paged.h"
#include "tc_ptx.cuh"

namespace lla {
namespace paged {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Four values side by side (16- or 8-byte aligned).
__device__ __forceinline__ void put4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void put4(__nv_bfloat16* p, float4 x) {
    __nv_bfloat162 y[2] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w)};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(y);
}

constexpr int kThreads = 256;

// Few rows (a decode step): eight rows of a tile, a warp to a row, a lane two of the 64 keys of a block; warps without
// a row only help to load.  fp32, 32 sequences x 16 heads at 4096 keys, d = 128: 496, 506 or 520 us from process to process
// (the same program and inputs), 4.1 to 4.3 TB/s, bound by the shared-memory reads of K beside the loads.  bf16, 64
// sequences, d = 32 and 16: 274 and 428 us.
template <int D>
struct FewShape {
    static constexpr int R = 8, BN = 64, TX = 32;
    static constexpr int KPT = BN / TX;                 // keys of a thread
    static constexpr int CPT = (D + TX - 1) / TX;       // output columns of a thread,
    static constexpr int VW = CPT < 4 ? CPT : 4;        // this many side by side
    static constexpr int KS = D + 4;                    // row strides of K and of the weights: the float4 reads of
    static constexpr int PS = BN + 4;                   // a warp's rows do not collide
    static constexpr size_t smem = sizeof(float) * (2 * R * D + BN * KS + BN * D + 2 * R * PS);
};

struct SimtArgs {
    Work w;
    const void* q;
    const void* probe;
    const void* k;
    const void* v;
    void* out;
    int Hq;
    long long q_stride, r_stride, page_stride;
    float scale;     // tau log2(e)
};

// 16 bytes of T as floats.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& raw, float* dst) {
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(T)); i += 4)
        *reinterpret_cast<float4*>(dst + i) = make_float4(to_f(e[i]), to_f(e[i + 1]), to_f(e[i + 2]), to_f(e[i + 3]));
}

// The e-th 16-byte piece of K and of V of the block of `keys` keys from key0 on; zeros behind the last key that the
// tile sees, whatever the page holds there.
template <typename T, int D>
__device__ __forceinline__ void fetch_piece(const SimtArgs& a, const Piece& p, int key0, int keys, int e, uint4& k, uint4& v) {
    constexpr int VE = 16 / sizeof(T);
    const Work& w = a.w;
    const int kk = e / (D / VE), c = (e % (D / VE)) * VE, key = key0 + kk;
    k = v = make_uint4(0, 0, 0, 0);
    if (kk < keys && key < p.keys) {
        const int page = w.table[(size_t)p.s * w.width + (key >> w.page_shift)];
        if (page < 0 || page >= w.num_pages) {
            atomicOr(w.err, (unsigned)kDevErrPagedArg);
        } else {
            const long long off = page * a.page_stride +
                (((long long)p.h << w.page_shift) + (key & ((1 << w.page_shift) - 1))) * D + c;
            k = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + off);
            v = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + off);
        }
    }
}

// A tile's queries and probes, in fp32; rows behind its last are zeros.
template <typename T, int D>
__device__ __forceinline__ void load_tile_rows(const SimtArgs& a, const Piece& p, int rows, int threads, float* Qs, float* Rs) {
    constexpr int VE = 16 / sizeof(T);
    const Work& w = a.w;
    for (int e = threadIdx.x; e < rows * (D / VE); e += threads) {
        const int r = e / (D / VE), c = (e % (D / VE)) * VE;
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (r < p.rows) {
            const int fr = p.row0 + r, tk = over_g(w, fr);
            const long long token = p.q.token0 + tk, hc = (long long)(p.h * w.G + fr - tk * w.G) * D + c;
            x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + token * a.q_stride + hc);
            y = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.probe) + token * a.r_stride + hc);
        }
        unpack<T>(x, Qs + r * D + c);
        unpack<T>(y, Rs + r * D + c);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) paged_simt_few_kernel(SimtArgs a) {
    using Sh = FewShape<D>;
    constexpr int R = Sh::R, TX = Sh::TX, BN = Sh::BN, KPT = Sh::KPT, CPT = Sh::CPT, VW = Sh::VW, KS = Sh::KS, PS = Sh::PS;
    constexpr int VE = 16 / sizeof(T);                  // elements of a 16-byte piece
    constexpr int PPT = (BN * D / VE + kThreads - 1) / kThreads;   // pieces of K (and of V) that a thread loads
    extern __shared__ __align__(16) float sm[];
    __shared__ long long scratch[40];
    float* Qs = sm;
    float* Rs = Qs + R * D;
    float* Ks = Rs + R * D;
    float* Vs = Ks + BN * KS;
    float* P1 = Vs + BN * D;
    float* P2 = P1 + R * PS;
    const Work& w = a.w;
    const int tid = threadIdx.x, row = tid / TX, tx = tid % TX;

    cudaGridDependencySynchronize();           // the lengths may be the previous kernel's
    Walk wk = begin_walk(w, blockIdx.x, scratch);
    cudaTriggerProgrammaticLaunchCompletion();   // the merge waits for this grid's end all the same
    Piece p;
    p.parts = 0; p.row0 = p.rows = p.h = 0; p.q.token0 = 0;
    bool shared = false;
    // a block of K and V on its way: loaded into registers while the block before is computed
    uint4 kraw[PPT], vraw[PPT];
    auto fetch = [&](int j) {
#pragma unroll
        for (int i = 0; i < PPT; ++i) fetch_piece<T, D>(a, p, j * BN, BN, tid + i * kThreads, kraw[i], vraw[i]);
    };

    while (next_piece(w, wk, p)) {
        shared = p.slot == 1;
        if (p.j0 < p.j1) fetch(p.j0);
        load_tile_rows<T, D>(a, p, R, kThreads, Qs, Rs);
        int limit = 0;                                   // keys this row sees
        if (row < p.rows) limit = w.causal ? min(max(p.q.L - p.q.nq + over_g(w, p.row0 + row) + 1, 0), p.q.L) : p.q.L;
        const bool busy = __any_sync(0xffffffffu, row < p.rows);   // a warp without rows only helps to load
        float m = -INFINITY, om = 0.f, A = 0.f, s0 = 0.f;
        float o1[CPT], o2[CPT];
#pragma unroll
        for (int i = 0; i < CPT; ++i) o1[i] = o2[i] = 0.f;

        for (int j = p.j0; j < p.j1; ++j) {
            const int key0 = j * BN;
#pragma unroll
            for (int i = 0; i < PPT; ++i) {
                const int e = tid + i * kThreads, kk = e / (D / VE), c = (e % (D / VE)) * VE;
                if (e < BN * (D / VE)) {
                    unpack<T>(kraw[i], Ks + kk * KS + c);
                    unpack<T>(vraw[i], Vs + kk * D + c);
                }
            }
            __syncthreads();
            if (j + 1 < p.j1) fetch(j + 1);
            if (busy) {
                float s[KPT], t[KPT];
#pragma unroll
                for (int u = 0; u < KPT; ++u) s[u] = t[u] = 0.f;
#pragma unroll 4
                for (int c = 0; c < D; c += 4) {
                    const float4 q4 = *reinterpret_cast<const float4*>(Qs + row * D + c);
                    const float4 r4 = *reinterpret_cast<const float4*>(Rs + row * D + c);
#pragma unroll
                    for (int u = 0; u < KPT; ++u) {
                        const float4 k4 = *reinterpret_cast<const float4*>(Ks + (tx + TX * u) * KS + c);
                        s[u] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[u]))));
                        t[u] = fmaf(r4.x, k4.x, fmaf(r4.y, k4.y, fmaf(r4.z, k4.z, fmaf(r4.w, k4.w, t[u]))));
                    }
                }
                float bm = -INFINITY;
#pragma unroll
                for (int u = 0; u < KPT; ++u) {
                    s[u] = key0 + tx + TX * u < limit ? s[u] * a.scale : -INFINITY;
                    bm = fmaxf(bm, s[u]);
                }
#pragma unroll
                for (int o = TX / 2; o; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
                const float mn = fmaxf(m, bm);
                const float base = mn == -INFINITY ? 0.f : mn;
                const float corr = exp2f(m - base);      // m = -inf: 0
                float ps = 0.f, pt = 0.f;
#pragma unroll
                for (int u = 0; u < KPT; ++u) {
                    s[u] = exp2f(s[u] - base);
                    ps += s[u];
                    pt = fmaf(s[u], t[u], pt);
                }
#pragma unroll
                for (int o = TX / 2; o; o >>= 1) {
                    ps += __shfl_xor_sync(0xffffffffu, ps, o);
                    pt += __shfl_xor_sync(0xffffffffu, pt, o);
                }
                if (om == 0.f && ps > 0.f) s0 = pt / ps; // the row's first block with keys
                m = mn;
                om = om * corr + ps;
                A = A * corr + (pt - s0 * ps);
#pragma unroll
                for (int u = 0; u < KPT; ++u) {
                    P1[row * PS + tx + TX * u] = s[u];
                    P2[row * PS + tx + TX * u] = s[u] * (t[u] - s0);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < CPT; ++i) {
                    o1[i] *= corr;
                    o2[i] *= corr;
                }
#pragma unroll 2
                for (int kk = 0; kk < BN; kk += 4) {
                    const float4 w1 = *reinterpret_cast<const float4*>(P1 + row * PS + kk);
                    const float4 w2 = *reinterpret_cast<const float4*>(P2 + row * PS + kk);
                    const float a1[4] = {w1.x, w1.y, w1.z, w1.w}, a2[4] = {w2.x, w2.y, w2.z, w2.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int g = 0; g < CPT / VW; ++g) {
                            const int c = (tx + TX * g) * VW;
                            float v[VW];
                            if (D % TX == 0 || c < D) {
                                if constexpr (VW == 4) {
                                    const float4 y = *reinterpret_cast<const float4*>(Vs + (kk + x) * D + c);
                                    v[0] = y.x; v[1] = y.y; v[2] = y.z; v[3] = y.w;
                                } else if constexpr (VW == 2) {
                                    const float2 y = *reinterpret_cast<const float2*>(Vs + (kk + x) * D + c);
                                    v[0] = y.x; v[1] = y.y;
                                } else {
                                    v[0] = Vs[(kk + x) * D + c];
                                }
#pragma unroll
                                for (int i = 0; i < VW; ++i) {
                                    o1[g * VW + i] = fmaf(a1[x], v[i], o1[g * VW + i]);
                                    o2[g * VW + i] = fmaf(a2[x], v[i], o2[g * VW + i]);
                                }
                            }
                        }
                }
            }
            __syncthreads();
        }

        if (row < p.rows) {
            if (p.slot < 0) {
                const int fr = p.row0 + row, token = p.q.token0 + over_g(w, fr), head = p.h * w.G + (fr - over_g(w, fr) * w.G);
                T* o = static_cast<T*>(a.out) + ((long long)token * a.Hq + head) * D;
                const float inv = om != 0.f ? 1.f / om : 0.f, c1 = 1.f + A * inv;
#pragma unroll
                for (int i = 0; i < CPT; ++i) {
                    const int c = (tx + TX * (i / VW)) * VW + i % VW;
                    if (D % TX == 0 || c < D) put(o + c, (c1 * o1[i] - o2[i]) * inv);
                }
            } else {
                if (tx == 0) part_stats(w, blockIdx.x, p.slot, D)[row] = make_float4(m, om, A, s0);
                float4* ps = part_sums(w, blockIdx.x, p.slot, D);
#pragma unroll
                for (int i = 0; i < CPT; ++i) {
                    const int c = (tx + TX * (i / VW)) * VW + i % VW;
                    if (D % TX == 0 || c < D) {
                        *part_element(ps, R, D, 0, row, c) = o1[i];
                        *part_element(ps, R, D, 1, row, c) = o2[i];
                    }
                }
            }
        }
        __syncthreads();
    }
    if (tid == 0) write_header(w, blockIdx.x, p, shared);
}

// ------------------------------------------------------------------------------------------ many rows
//
// 32 rows to a tile, a warp to eight of them.  Its lanes are four pairs of rows by eight key columns: in the first
// product a lane has two rows and an eighth of the keys, in the second the same rows and an eighth of the output
// columns.  So a 16-byte read of K or V serves two rows and one of q, the probe or the weights eight keys or columns:
// eight reads to 64 products (a row a thread and four keys: six to 32), and shared-memory reads bound this kernel:
// 64 sequences of 1 to 97 new tokens over 200 to 1024 keys, 4 heads, fp32, d = 128: 369 us, 24 TFLOP/s (d = 32, which
// the tensor cores have now, 16 sequences: 35 us, 44 with a row a thread).
// Products and sums are pairs of fp32 (fma.rn.f32x2: each rounded as the scalar instruction).
constexpr int kManyThreads = 128;

template <int D>
struct ManyShape {
    static constexpr int R = 32, BN = 32;
    static constexpr int kCtas = D == 128 ? 2 : D == 64 ? 3 : 4;   // to an SM (registers)
    static constexpr int KPT = BN / 8;                  // keys of a lane
    static constexpr int CPT = D / 8;                   // output columns of a lane, in runs of VW
    static constexpr int VW = CPT < 4 ? CPT : 4;
    static constexpr int KS = D + 4, PS = BN + 4;       // row strides of K and of the weights
    static constexpr size_t smem = sizeof(float) * (2 * R * D + BN * KS + BN * D + 2 * R * PS);
};

template <typename T, int D>
__global__ void __launch_bounds__(kManyThreads, ManyShape<D>::kCtas) paged_simt_many_kernel(SimtArgs a) {
    using Sh = ManyShape<D>;
    constexpr int R = Sh::R, BN = Sh::BN, KPT = Sh::KPT, CPT = Sh::CPT, VW = Sh::VW, KS = Sh::KS, PS = Sh::PS;
    constexpr int VE = 16 / sizeof(T);
    constexpr int PPT = (BN * D / VE + kManyThreads - 1) / kManyThreads;
    extern __shared__ __align__(16) float sm[];
    __shared__ long long scratch[40];
    float* Qs = sm;
    float* Rs = Qs + R * D;
    float* Ks = Rs + R * D;
    float* Vs = Ks + BN * KS;
    float* P1 = Vs + BN * D;
    float* P2 = P1 + R * PS;
    const Work& w = a.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = warp * 8 + (lane >> 3) * 2, g8 = lane & 7;   // the lane's first row; its key and column group

    cudaGridDependencySynchronize();           // the lengths may be the previous kernel's
    Walk wk = begin_walk(w, blockIdx.x, scratch);
    cudaTriggerProgrammaticLaunchCompletion();   // the merge waits for this grid's end all the same
    Piece p;
    p.parts = 0; p.row0 = p.rows = p.h = 0; p.q.token0 = 0;
    bool shared = false;
    uint4 kraw[PPT], vraw[PPT];                // a block of K and V on its way, while the one before is computed
    auto fetch = [&](int j) {
#pragma unroll
        for (int i = 0; i < PPT; ++i) fetch_piece<T, D>(a, p, j * BN, BN, tid + i * kManyThreads, kraw[i], vraw[i]);
    };

    while (next_piece(w, wk, p)) {
        shared = p.slot == 1;
        if (p.j0 < p.j1) fetch(p.j0);
        load_tile_rows<T, D>(a, p, R, kManyThreads, Qs, Rs);
        const bool busy = warp * 8 < p.rows;             // a warp without rows only helps to load
        int limit[2], all = INT_MAX;                     // keys a row sees, keys that all of the warp's rows see
        float m[2], om[2], A[2], s0[2];                  // om, A: this lane's keys
        uint64_t o1[2][CPT / 2], o2[2][CPT / 2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            limit[i] = 0;
            if (row + i < p.rows)
                limit[i] = w.causal ? min(max(p.q.L - p.q.nq + over_g(w, p.row0 + row + i) + 1, 0), p.q.L) : p.q.L;
            all = min(all, row + i < p.rows ? limit[i] : INT_MAX);
            m[i] = -INFINITY;
            om[i] = A[i] = s0[i] = 0.f;
#pragma unroll
            for (int c = 0; c < CPT / 2; ++c) o1[i][c] = o2[i][c] = tc::f2_pack(0.f, 0.f);
        }

        all = __reduce_min_sync(0xffffffffu, all);

        for (int j = p.j0; j < p.j1; ++j) {
            const int key0 = j * BN;
#pragma unroll
            for (int i = 0; i < PPT; ++i) {
                const int e = tid + i * kManyThreads, kk = e / (D / VE), c = (e % (D / VE)) * VE;
                if (e < BN * (D / VE)) {
                    unpack<T>(kraw[i], Ks + kk * KS + c);
                    unpack<T>(vraw[i], Vs + kk * D + c);
                }
            }
            __syncthreads();
            if (j + 1 < p.j1) fetch(j + 1);
            if (busy) {
                float s[2][KPT], t[2][KPT];
                {
                    uint64_t s2[2][KPT], t2[2][KPT];     // even and odd columns apart
#pragma unroll
                    for (int u = 0; u < KPT; ++u) s2[0][u] = s2[1][u] = t2[0][u] = t2[1][u] = tc::f2_pack(0.f, 0.f);
#pragma unroll 2
                    for (int c = 0; c < D; c += 4) {
                        ulonglong2 q4[2], r4[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            q4[i] = *reinterpret_cast<const ulonglong2*>(Qs + (row + i) * D + c);
                            r4[i] = *reinterpret_cast<const ulonglong2*>(Rs + (row + i) * D + c);
                        }
#pragma unroll
                        for (int u = 0; u < KPT; ++u) {
                            const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(Ks + (g8 + 8 * u) * KS + c);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                s2[i][u] = tc::f2_fma(q4[i].y, k4.y, tc::f2_fma(q4[i].x, k4.x, s2[i][u]));
                                t2[i][u] = tc::f2_fma(r4[i].y, k4.y, tc::f2_fma(r4[i].x, k4.x, t2[i][u]));
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int u = 0; u < KPT; ++u) {
                            float x, y;
                            tc::f2_unpack(s2[i][u], x, y);
                            s[i][u] = x + y;
                            tc::f2_unpack(t2[i][u], x, y);
                            t[i][u] = x + y;
                        }
                }
                if (key0 + BN > all) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int u = 0; u < KPT; ++u)
                            if (key0 + g8 + 8 * u >= limit[i]) s[i][u] = -INFINITY;
                }
                float mn[2];
                bool grown = false, first[2];                // first: the row's first block with keys
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float bm = s[i][0];
#pragma unroll
                    for (int u = 1; u < KPT; ++u) bm = fmaxf(bm, s[i][u]);
#pragma unroll
                    for (int o = 4; o; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
                    mn[i] = fmaxf(m[i], bm * a.scale);
                    grown |= mn[i] > m[i];
                    first[i] = m[i] == -INFINITY && mn[i] != -INFINITY;
                }
                grown = __any_sync(0xffffffffu, grown);
                if (grown) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float corr = tc::ex2(m[i] - (mn[i] == -INFINITY ? 0.f : mn[i]));   // m = -inf: 0
                        const uint64_t c2 = tc::f2_pack(corr, corr);
                        om[i] *= corr;
                        A[i] *= corr;
#pragma unroll
                        for (int c = 0; c < CPT / 2; ++c) {
                            o1[i][c] = tc::f2_mul(o1[i][c], c2);
                            o2[i][c] = tc::f2_mul(o2[i][c], c2);
                        }
                        m[i] = mn[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float base = m[i] == -INFINITY ? 0.f : m[i];
                    float ps = 0.f;
#pragma unroll
                    for (int u = 0; u < KPT; ++u) {
                        s[i][u] = tc::ex2(fmaf(s[i][u], a.scale, -base));
                        ps += s[i][u];
                    }
                    if (grown) {                             // so it is in a row's first block with keys
                        float x = ps, y = 0.f;
#pragma unroll
                        for (int u = 0; u < KPT; ++u) y = fmaf(s[i][u], t[i][u], y);
#pragma unroll
                        for (int o = 4; o; o >>= 1) {
                            x += __shfl_xor_sync(0xffffffffu, x, o);
                            y += __shfl_xor_sync(0xffffffffu, y, o);
                        }
                        if (first[i]) s0[i] = x > 0.f ? y / x : 0.f;
                    }
                    om[i] += ps;
#pragma unroll
                    for (int u = 0; u < KPT; ++u) {
                        const float z = s[i][u] * (t[i][u] - s0[i]);
                        A[i] += z;
                        P1[(row + i) * PS + g8 + 8 * u] = s[i][u];
                        P2[(row + i) * PS + g8 + 8 * u] = z;
                    }
                }
                __syncwarp();
#pragma unroll 2
                for (int kk = 0; kk < BN; kk += 4) {
                    float w1[2][4], w2[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        *reinterpret_cast<float4*>(w1[i]) = *reinterpret_cast<const float4*>(P1 + (row + i) * PS + kk);
                        *reinterpret_cast<float4*>(w2[i]) = *reinterpret_cast<const float4*>(P2 + (row + i) * PS + kk);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
#pragma unroll
                        for (int g = 0; g < CPT / VW; ++g) {
                            const float* src = Vs + (kk + x) * D + (g8 + 8 * g) * VW;
                            uint64_t v[VW / 2];
                            if constexpr (VW == 4) {
                                const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(src);
                                v[0] = y.x;
                                v[VW / 2 - 1] = y.y;
                            } else {
                                v[0] = *reinterpret_cast<const uint64_t*>(src);
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int c = 0; c < VW / 2; ++c) {
                                    const int n = g * (VW / 2) + c;
                                    o1[i][n] = tc::f2_fma(tc::f2_pack(w1[i][x], w1[i][x]), v[c], o1[i][n]);
                                    o2[i][n] = tc::f2_fma(tc::f2_pack(w2[i][x], w2[i][x]), v[c], o2[i][n]);
                                }
                        }
                    }
                }
            }
            __syncthreads();
        }

        if (busy) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int o = 4; o; o >>= 1) {
                    om[i] += __shfl_xor_sync(0xffffffffu, om[i], o);
                    A[i] += __shfl_xor_sync(0xffffffffu, A[i], o);
                }
                const int r = row + i;
                if (r >= p.rows) continue;
                const int fr = p.row0 + r, tk = over_g(w, fr);
                T* o = static_cast<T*>(a.out) + ((long long)(p.q.token0 + tk) * a.Hq + p.h * w.G + fr - tk * w.G) * D;
                float4* ps = p.slot >= 0 ? part_sums(w, blockIdx.x, p.slot, D) : nullptr;
                if (p.slot >= 0 && g8 == 0) part_stats(w, blockIdx.x, p.slot, D)[r] = make_float4(m[i], om[i], A[i], s0[i]);
                const float inv = om[i] != 0.f ? 1.f / om[i] : 0.f, c1 = 1.f + A[i] * inv;
#pragma unroll
                for (int n = 0; n < CPT / 2; ++n) {
                    const int c = (g8 + 8 * (2 * n / VW)) * VW + 2 * n % VW;
                    float x1, y1, x2, y2;
                    tc::f2_unpack(o1[i][n], x1, y1);
                    tc::f2_unpack(o2[i][n], x2, y2);
                    if (p.slot < 0) {
                        put(o + c, (c1 * x1 - x2) * inv);
                        put(o + c + 1, (c1 * y1 - y2) * inv);
                    } else {
                        *reinterpret_cast<float2*>(part_element(ps, R, D, 0, r, c)) = make_float2(x1, y1);
                        *reinterpret_cast<float2*>(part_element(ps, R, D, 1, r, c)) = make_float2(x2, y2);
                    }
                }
            }
        }
        __syncthreads();
    }
    if (tid == 0) write_header(w, blockIdx.x, p, shared);
}

// Joins the parts of the tile that CTA blockIdx.x starts and others finish: part 0 is its slot 1, part
// i > 0 slot 0 of CTA blockIdx.x + i.  With the common maximum and one centre,
//   out = sum_i f_i ((1 + A/w - (s0_i - s0)) O1_i - O2_i) / w,   f_i = 2^(m_i - m).
// The order of the sum is fixed by the parts: results do not depend on which CTA was first.  A block has
// eight rows and kC groups of four columns: a warp turns a row's statistics into two factors per part in
// shared memory, after which the loads of the sums are independent of one another.  Eight rows side by side
// are a full line of a part, and the four columns of four neighbouring threads a full sector of the output.
// Where parts are many and rows few, kLanes threads share a (row, columns) and take the parts in turn.
// A lane loads the statistics of three parts (two of a large tile) at once: the 152 parts of 32,768 keys of one sequence
// 1.5 us sooner than one after another, and as soon as eight at once where parts are few: more registers let
// fewer of the blocks that have nothing to join pass at a time.
// 128-row tiles of 152 CTAs: 12 us (36 MB of parts); blocks that looped over several joins took longer than idle ones.
constexpr int kMergeRows = 8;

template <int D, int R>
struct MergeShape {
    static constexpr int kC = R <= 16 ? 4 : D / 4;                     // groups of four columns of a block
    static constexpr int kItems = kMergeRows * kC, kLanes = 256 / kItems;
    static constexpr int kBlocks = R / kMergeRows * (D / 4 / kC);      // of a tile
    static constexpr int kHeld = R <= 16 ? 3 : 2;                      // parts whose statistics a lane loads at once
    static constexpr int kChunk = 32 * kHeld;                          // parts whose factors are held at a time
};

template <typename T, int D, int R>
__global__ void __launch_bounds__(256, 5) paged_merge_kernel(Work w, T* __restrict__ out, int Hq) {
    using Sh = MergeShape<D, R>;
    constexpr int kItems = Sh::kItems, kLanes = Sh::kLanes, kHeld = Sh::kHeld, kChunk = Sh::kChunk;
    __shared__ float2 fac[kChunk][kMergeRows];
    __shared__ float4 red[kLanes > 1 ? 256 : 1];
    const int tid = threadIdx.x, warp = tid >> 5, ln = tid & 31;
    cudaGridDependencySynchronize();
    const PartHeader h = w.hdr[blockIdx.x];
    const int row0 = blockIdx.y % (R / kMergeRows) * kMergeRows, c0 = blockIdx.y / (R / kMergeRows) * Sh::kC;
    if (h.parts == 0 || row0 >= h.rows) return;

    // this warp's row: statistics of its parts, a lane's first ones in registers
    const int row = row0 + warp;
    const bool live = row < h.rows;
    auto stats = [&](int i) { return part_stats(w, blockIdx.x + i, i == 0, D)[row]; };
    float4 held[kHeld];
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
        held[u] = live && ln + 32 * u < h.parts ? stats(ln + 32 * u) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    float m = held[0].x;
#pragma unroll
    for (int u = 1; u < kHeld; ++u) m = fmaxf(m, held[u].x);
    if (live)
        for (int i = ln + kChunk; i < h.parts; i += 32) m = fmaxf(m, stats(i).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m, s0 = __shfl_sync(0xffffffffu, held[0].w, 0);
    float om = 0.f, A = 0.f;
    auto add = [&](const float4& st) {
        const float f = exp2f(st.x - base);
        om = fmaf(f, st.y, om);
        A = fmaf(f, fmaf(st.w - s0, st.y, st.z), A);
    };
#pragma unroll
    for (int u = 0; u < kHeld; ++u) add(held[u]);
    if (live)
        for (int i = ln + kChunk; i < h.parts; i += 32) add(stats(i));
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        om += __shfl_xor_sync(0xffffffffu, om, o);
        A += __shfl_xor_sync(0xffffffffu, A, o);
    }
    const float inv = om != 0.f ? 1.f / om : 0.f, c1 = 1.f + A * inv;   // om 0: no key in any part; NaN stays NaN

    const int r = tid % kMergeRows, c4 = c0 + tid / kMergeRows % Sh::kC, lane = tid / kItems;
    const bool mine = row0 + r < h.rows;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < h.parts; i0 += kChunk) {
        const int n = min(kChunk, h.parts - i0);
        if (live) {
#pragma unroll
            for (int u = 0; u < kHeld; ++u) {
                const int i = ln + 32 * u;
                if (i < n) {
                    const float4 st = i0 == 0 ? held[u] : stats(i0 + i);
                    const float g = exp2f(st.x - base) * inv;
                    fac[i][warp] = make_float2(g * (c1 - (st.w - s0)), g);
                }
            }
        }
        __syncthreads();
        if (mine) {
#pragma unroll 4
            for (int i = lane; i < n; i += kLanes) {
                const float2 g = fac[i][r];
                const float4* o = part_sums(w, blockIdx.x + i0 + i, i0 + i == 0, D) + (size_t)c4 * R + row0 + r;
                const float4 x = o[0], y = o[(size_t)(D / 4) * R];
                acc.x = fmaf(g.x, x.x, fmaf(-g.y, y.x, acc.x));
                acc.y = fmaf(g.x, x.y, fmaf(-g.y, y.y, acc.y));
                acc.z = fmaf(g.x, x.z, fmaf(-g.y, y.z, acc.z));
                acc.w = fmaf(g.x, x.w, fmaf(-g.y, y.w, acc.w));
            }
        }
        __syncthreads();
    }
    if (kLanes > 1) {
        red[tid] = acc;
        __syncthreads();
        if (lane == 0)
#pragma unroll
            for (int i = 1; i < kLanes; ++i) {
                const float4 x = red[i * kItems + tid];
                acc.x += x.x;
                acc.y += x.y;
                acc.z += x.z;
                acc.w += x.w;
            }
    }
    if (lane == 0 && mine) {
        const int fr = h.row0 + row0 + r, tk = over_g(w, fr);
        put4(out + ((long long)(h.token0 + tk) * Hq + h.head * w.G + fr - tk * w.G) * D + c4 * 4, acc);
    }
}

template <typename T, int D>
cudaError_t launch_one(const SimtArgs& a, cudaStream_t stream) {
    const bool few = a.w.rows == 8;
    auto* kern = few ? paged_simt_few_kernel<T, D> : paged_simt_many_kernel<T, D>;
    const size_t smem = few ? FewShape<D>::smem : ManyShape<D>::smem;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(a.w.ctas), few ? kThreads : kManyThreads, smem, stream, a);
}

cudaError_t launch_fp32(const SimtArgs& a, int d, cudaStream_t stream) {
    return d == 16 ? launch_one<float, 16>(a, stream) : launch_one<float, 128>(a, stream);
}

cudaError_t launch_bf16(const SimtArgs& a, int d, cudaStream_t stream) {
    using T = __nv_bfloat16;
    switch (d) {
        case 16: return launch_one<T, 16>(a, stream);
        case 32: return launch_one<T, 32>(a, stream);
        case 64: return launch_one<T, 64>(a, stream);
        default: return launch_one<T, 128>(a, stream);
    }
}

template <typename T, int D, int R>
cudaError_t merge_one(const Work& w, void* out, int Hq, cudaStream_t stream) {
    return launch_after(paged_merge_kernel<T, D, R>, dim3(w.ctas, MergeShape<D, R>::kBlocks), 256, 0, stream, w,
                        static_cast<T*>(out), Hq);
}

template <typename T, int D>
cudaError_t merge_rows(const Work& w, void* out, int Hq, cudaStream_t stream) {
    switch (w.rows) {
        case 8: return merge_one<T, D, 8>(w, out, Hq, stream);
        case 16: return merge_one<T, D, 16>(w, out, Hq, stream);
        case 32: return merge_one<T, D, 32>(w, out, Hq, stream);
        case 128: return merge_one<T, D, 128>(w, out, Hq, stream);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t merge_typed(const Work& w, void* out, int Hq, int d, cudaStream_t stream) {
    switch (d) {
        case 16: return merge_rows<T, 16>(w, out, Hq, stream);
        case 32: return merge_rows<T, 32>(w, out, Hq, stream);
        case 64: return merge_rows<T, 64>(w, out, Hq, stream);
        default: return merge_rows<T, 128>(w, out, Hq, stream);
    }
}

}  // namespace
}  // namespace paged

PagedSplit paged_simt_split(const PagedProblem& p, int sms) {
    // rows: 8 where no sequence has more than eight query rows to a key head (a decode step), else 32
    const bool few = (long long)p.max_new * p.G <= 8;
    if (few) return PagedSplit{8, 64, 2 * sms, 0};
    return PagedSplit{32, paged::ManyShape<128>::BN, (p.d == 128 ? paged::ManyShape<128>::kCtas : p.d == 64 ? paged::ManyShape<64>::kCtas : paged::ManyShape<32>::kCtas) * sms, 0};
}

cudaError_t launch_paged_simt(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream) {
    paged::SimtArgs a{paged::make_work(p, sp), p.q, p.probe, p.k, p.v, p.out, p.Hq, p.q_stride, p.r_stride,
                      p.page_stride, p.tau * 1.4426950408889634f};
    return p.dtype == LLA_DTYPE_BF16 ? paged::launch_bf16(a, p.d, stream) : paged::launch_fp32(a, p.d, stream);
}

cudaError_t launch_paged_merge(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream) {
    const paged::Work w = paged::make_work(p, sp);
    return p.dtype == LLA_DTYPE_BF16 ? paged::merge_typed<__nv_bfloat16>(w, p.out, p.Hq, p.d, stream)
                                     : paged::merge_typed<float>(w, p.out, p.Hq, p.d, stream);
}

}  // namespace lla
