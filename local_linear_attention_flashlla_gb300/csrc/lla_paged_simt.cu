// Parallax attention over a paged cache on CUDA cores (every product in fp32; any head dim, bf16 or
// fp32), and the merge of row tiles that several CTAs share (all paths).
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

// R rows of a tile, TX threads to a row (they lie in one warp), BN keys of a block.
template <int D, int R>
struct Shape {
    static constexpr int TX = kThreads / R;
    static constexpr int BN = R == 32 ? 32 : 64;
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

template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads, 2) paged_simt_kernel(SimtArgs a) {
    using Sh = Shape<D, R>;
    constexpr int TX = Sh::TX, BN = Sh::BN, KPT = Sh::KPT, CPT = Sh::CPT, VW = Sh::VW, KS = Sh::KS, PS = Sh::PS;
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
    const T* gq = static_cast<const T*>(a.q);
    const T* gr = static_cast<const T*>(a.probe);
    const T* gk = static_cast<const T*>(a.k);
    const T* gv = static_cast<const T*>(a.v);

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
        for (int i = 0; i < PPT; ++i) {
            const int e = tid + i * kThreads, kk = e / (D / VE), c = (e % (D / VE)) * VE, key = j * BN + kk;
            kraw[i] = vraw[i] = make_uint4(0, 0, 0, 0);  // keys that no row sees: zeros, whatever the page holds
            if (e < BN * (D / VE) && key < p.keys) {
                const int page = w.table[(size_t)p.s * w.width + (key >> w.page_shift)];
                if (page < 0 || page >= w.num_pages) {
                    atomicOr(w.err, (unsigned)kDevErrPagedArg);
                } else {
                    const long long off = page * a.page_stride +
                        (((long long)p.h << w.page_shift) + (key & ((1 << w.page_shift) - 1))) * D + c;
                    kraw[i] = *reinterpret_cast<const uint4*>(gk + off);
                    vraw[i] = *reinterpret_cast<const uint4*>(gv + off);
                }
            }
        }
    };
    auto unpack = [&](const uint4& raw, float* dst) {
        const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int i = 0; i < VE; i += 4)
            *reinterpret_cast<float4*>(dst + i) = make_float4(to_f(e[i]), to_f(e[i + 1]), to_f(e[i + 2]), to_f(e[i + 3]));
    };

    while (next_piece(w, wk, p)) {
        shared = p.slot == 1;
        if (p.j0 < p.j1) fetch(p.j0);
        for (int e = tid; e < R * (D / VE); e += kThreads) {
            const int r = e / (D / VE), c = (e % (D / VE)) * VE;
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (r < p.rows) {
                const int fr = p.row0 + r, tk = over_g(w, fr);
                const long long token = p.q.token0 + tk, hc = (long long)(p.h * w.G + fr - tk * w.G) * D + c;
                x = *reinterpret_cast<const uint4*>(gq + token * a.q_stride + hc);
                y = *reinterpret_cast<const uint4*>(gr + token * a.r_stride + hc);
            }
            unpack(x, Qs + r * D + c);
            unpack(y, Rs + r * D + c);
        }
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
                    unpack(kraw[i], Ks + kk * KS + c);
                    unpack(vraw[i], Vs + kk * D + c);
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

// Joins the parts of the tile that CTA blockIdx.x starts and others finish: part 0 is its slot 1, part
// i > 0 slot 0 of CTA blockIdx.x + i.  With the common maximum and one centre,
//   out = sum_i f_i ((1 + A/w - (s0_i - s0)) O1_i - O2_i) / w,   f_i = 2^(m_i - m).
// The order of the sum is fixed by the parts: results do not depend on which CTA was first.  A block has
// eight rows and kC groups of four columns: a warp turns a row's statistics into two factors per part in
// shared memory, after which the loads of the sums are independent of one another.  Eight rows side by side
// are a full line of a part, and the four columns of four neighbouring threads a full sector of the output.
// Where parts are many and rows few, kLanes threads share a (row, columns) and take the parts in turn.
constexpr int kMergeRows = 8;
constexpr int kChunk = 128;                    // parts whose factors are held at a time

template <int D, int R>
struct MergeShape {
    static constexpr int kC = R <= 16 ? 4 : D / 4;                     // groups of four columns of a block
    static constexpr int kItems = kMergeRows * kC, kLanes = 256 / kItems;
    static constexpr int kBlocks = R / kMergeRows * (D / 4 / kC);      // of a tile
};

template <typename T, int D, int R>
__global__ void __launch_bounds__(256) paged_merge_kernel(Work w, T* __restrict__ out, int Hq) {
    using Sh = MergeShape<D, R>;
    constexpr int kItems = Sh::kItems, kLanes = Sh::kLanes;
    __shared__ float2 fac[kChunk][kMergeRows];
    __shared__ float4 red[kLanes > 1 ? 256 : 1];
    const int tid = threadIdx.x, warp = tid >> 5, ln = tid & 31;
    cudaGridDependencySynchronize();
    const PartHeader h = w.hdr[blockIdx.x];
    const int row0 = blockIdx.y % (R / kMergeRows) * kMergeRows, c0 = blockIdx.y / (R / kMergeRows) * Sh::kC;
    if (h.parts == 0 || row0 >= h.rows) return;

    // this warp's row: statistics of its parts (a lane's first in a register)
    const int row = row0 + warp;
    const bool live = row < h.rows;
    auto stats = [&](int i) { return part_stats(w, blockIdx.x + i, i == 0, D)[row]; };
    float4 first = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    if (live && ln < h.parts) first = stats(ln);
    float m = first.x;
    if (live)
        for (int i = ln + 32; i < h.parts; i += 32) m = fmaxf(m, stats(i).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m, s0 = __shfl_sync(0xffffffffu, first.w, 0);
    float f = exp2f(first.x - base), om = f * first.y, A = f * fmaf(first.w - s0, first.y, first.z);
    if (live)
        for (int i = ln + 32; i < h.parts; i += 32) {
            const float4 st = stats(i);
            f = exp2f(st.x - base);
            om = fmaf(f, st.y, om);
            A = fmaf(f, fmaf(st.w - s0, st.y, st.z), A);
        }
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
        if (live)
            for (int i = ln; i < n; i += 32) {
                const float4 st = i0 + i < 32 ? first : stats(i0 + i);
                const float g = exp2f(st.x - base) * inv;
                fac[i][warp] = make_float2(g * (c1 - (st.w - s0)), g);
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

template <typename T, int D, int R>
cudaError_t launch_one(const SimtArgs& a, cudaStream_t stream) {
    constexpr size_t smem = Shape<D, R>::smem;
    auto* kern = paged_simt_kernel<T, D, R>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(a.w.ctas), kThreads, smem, stream, a);
}

template <typename T>
cudaError_t launch_typed(const SimtArgs& a, int d, cudaStream_t stream) {
    const bool few = a.w.rows == 8;
    switch (d) {
        case 16: return few ? launch_one<T, 16, 8>(a, stream) : launch_one<T, 16, 32>(a, stream);
        case 32: return few ? launch_one<T, 32, 8>(a, stream) : launch_one<T, 32, 32>(a, stream);
        case 64: return few ? launch_one<T, 64, 8>(a, stream) : launch_one<T, 64, 32>(a, stream);
        default: return few ? launch_one<T, 128, 8>(a, stream) : launch_one<T, 128, 32>(a, stream);
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
    return PagedSplit{few ? 8 : 32, few ? 64 : 32, 2 * sms, 2, 0};
}

cudaError_t launch_paged_simt(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream) {
    paged::SimtArgs a{paged::make_work(p, sp), p.q, p.probe, p.k, p.v, p.out, p.Hq, p.q_stride, p.r_stride,
                      p.page_stride, p.tau * 1.4426950408889634f};
    return p.dtype == LLA_DTYPE_BF16 ? paged::launch_typed<__nv_bfloat16>(a, p.d, stream)
                                     : paged::launch_typed<float>(a, p.d, stream);
}

cudaError_t launch_paged_merge(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream) {
    const paged::Work w = paged::make_work(p, sp);
    return p.dtype == LLA_DTYPE_BF16 ? paged::merge_typed<__nv_bfloat16>(w, p.out, p.Hq, p.d, stream)
                                     : paged::merge_typed<float>(w, p.out, p.Hq, p.d, stream);
}

}  // namespace lla
