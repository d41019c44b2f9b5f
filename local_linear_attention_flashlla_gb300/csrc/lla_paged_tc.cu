// Parallax attention over a paged bf16 cache for many query rows to a key head (prompts, chunks of
// prompts, cross attention, drafts over many shared heads): tcgen05 with 128-row tiles.
//
// Per block of 128 keys four products of 128 x 128 x d: S = Q K^T, T = R K^T, O1 += P V and O2 += P' V
// with P = 2^(l - m) and P' = P (T - s0) (the formulas of lla_paged_simt.cu).  S, T, O1 and O2 fill the
// 512 TMEM columns, so S and T have one buffer each, and P and P' (bf16) overwrite the halves of S and T
// that they came from.  The products are issued as
//     S(j+1)  O2(j)  T(j+1)  O1(j+1)  S(j+2)  O2(j+1) ...
// : the softmax of S(j+1) runs under O2(j) and T(j+1), the weighting of T(j+1) under O1(j+1) and S(j+2).
//
// Two groups of four warps hold the rows, a thread a row, and take the blocks in turn, so that one
// group's weighting runs beside the other's softmax: a row's maximum needs no exchange, and each
// scheduler has a warp that waits for exponentials and one that does not need them.  Two more warps
// feed K and V through TMA rings (a box per page) and issue the products.
#include <math.h>

#include "../../include/lla.h"
#include "lla_internal.h"
#include "lla_paged.h"
#include "paged_tc.cuh"

namespace lla {
namespace paged {
namespace {

using namespace tc;

constexpr int kRows = 128;
constexpr int kKeys = 128;
constexpr int kSoft = 256;                     // threads that hold rows
constexpr int kThreads = kSoft + 64;

template <int D>
struct TcShape {
    static constexpr int kStages = D == 128 ? 2 : 4;       // of K and of V
    static constexpr int kTile = kKeys * D * 2;            // bytes of a K or V block, and of Q or R: [D / 64][128 rows][128 B]
    static constexpr size_t smem = (size_t)(2 + 2 * kStages) * kTile + 1024;
};

struct TcArgs {
    Work w;
    const __nv_bfloat16* q;
    const __nv_bfloat16* probe;
    __nv_bfloat16* out;
    int Hq;
    long long q_stride, r_stride;
    float scale;                               // tau log2(e)
};

template <int D>
struct TcBars {
    uint64_t kfull[TcShape<D>::kStages], kempty[TcShape<D>::kStages];
    uint64_t vfull[TcShape<D>::kStages], vempty[TcShape<D>::kStages];
    uint64_t sfull[2], tfull[2], p1[2], p2[2];  // by block parity
    uint64_t qfull, done, fin;
    uint32_t tmem;
    int err;
    float m[kRows], s0[kRows];                 // the groups' common reference point and centre of a row
    float2 tot[2][kRows];                      // group: omega and A of a tile
};

__device__ __forceinline__ uint32_t piece_off(int r, int c) {
    return (uint32_t)((c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// One box to a lane; K and V of a block go to rings of their own (K is given back a product earlier).
template <int D>
__device__ void feed_kv(const Work& w, Walk wk, const CUtensorMap* mk, const CUtensorMap* mv, uint32_t kring,
                        uint32_t vring, TcBars<D>& b) {
    constexpr int NS = TcShape<D>::kStages, kTile = TcShape<D>::kTile;
    const int lane = threadIdx.x & 31;
    const int box = min(1 << w.page_shift, kBoxRows), boxes = kKeys / box;     // <= 16
    int n = 0;                                 // blocks issued
    bool ok = true;
    Piece p;
    while (ok && next_piece(w, wk, p)) {
        const int* row = w.table + (size_t)p.s * w.width;
        for (int j = p.j0; j < p.j1; ++j, ++n) {
            const int key = j * kKeys + lane * box;
            const bool mine = lane < boxes && key < p.keys;
            const int page = mine ? checked_page(w, row, key) : 0;
            const int y = key & ((1 << w.page_shift) - 1);
            const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, mine)) * box * D * 2);
            const int st = n % NS;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                uint64_t* full = kv ? &b.vfull[st] : &b.kfull[st];
                uint64_t* empty = kv ? &b.vempty[st] : &b.kempty[st];
                ok = __all_sync(0xffffffffu, mbar_wait(empty, ((n / NS) & 1) ^ 1, &b.err));
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
                if (mine) {
                    const uint32_t dst = (kv ? vring : kring) + (uint32_t)(st * kTile + lane * box * 128);
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_4d(dst + x * (kKeys * 128), kv ? mv : mk, full, x * 64, y, p.h, page);
                }
                __syncwarp();
            }
            if (!ok) break;
        }
    }
    if (!ok || *(volatile int*)&b.err)         // copies in flight land before the CTA gives its memory back
        for (int t = max(n - NS, 0); t < n; ++t) {
            drain(&b.kfull[t % NS], (t / NS) & 1);
            drain(&b.vfull[t % NS], (t / NS) & 1);
        }
}

// D[tmem] = A B^T, 128 x 128 x D, both operands K-major in shared memory.
template <int D>
__device__ __forceinline__ void gemm_ss(uint32_t d, uint32_t a_addr, uint32_t b_addr) {
    constexpr uint32_t ID = idesc_bf16(kRows, kKeys, false, false);
    const uint64_t a0 = sdesc_sw128(a_addr, 16, 1024), b0 = sdesc_sw128(b_addr, 16, 1024);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const uint64_t off = (uint64_t)(((ks >> 2) * (kRows * 128) + (ks & 3) * 32) >> 4);
        if (ks == 0) umma_ss_c<false>(d, a0 + off, b0 + off, ID);
        else umma_ss_c<true>(d, a0 + off, b0 + off, ID);
    }
}
// D[tmem] (+)= P V, 128 x D x 128: P bf16 pairs in TMEM (keys 0-63 at column 0, 64-127 at column 64), V
// [128 keys x D] read MN-major.
template <int D>
__device__ __forceinline__ void gemm_ts(uint32_t d, uint32_t p, uint32_t v_addr, bool acc) {
    constexpr uint32_t ID = idesc_bf16(kRows, D, false, true);
    const uint64_t b0 = sdesc_sw128(v_addr, kKeys * 128, 1024);
    if (acc) umma_ts_c<true>(d, p, b0, ID);
    else umma_ts_c<false>(d, p, b0, ID);
#pragma unroll
    for (int ks = 1; ks < kKeys / 16; ++ks)
        umma_ts_c<true>(d, p + (ks >> 2) * 64 + (ks & 3) * 8, b0 + (uint64_t)((ks * 2048) >> 4), ID);
}

// The issuing warp.  All lanes run the loop and one elected lane issues: with everything that the products'
// descriptors are made of uniform across the warp the descriptors stay in uniform registers, which
// tcgen05.mma takes (issued from a branch of lane 0 each product's eight instructions took 570 to 830
// cycles to issue, more than the 512 it takes to run).
template <int D>
__device__ void issue(const Work& w, Walk wk, uint32_t tm, uint32_t qa, uint32_t ra, uint32_t kring, uint32_t vring,
                      TcBars<D>& b) {
    constexpr int NS = TcShape<D>::kStages, kTile = TcShape<D>::kTile;
    const uint32_t tS = tm, tT = tm + 128, tO1 = tm + 256, tO2 = tm + 256 + D;
    int n = 0, pieces = 0;
    bool ok = true;
    Piece p;
    while (ok && next_piece(w, wk, p)) {
        const int nb = __shfl_sync(0xffffffffu, p.j1 - p.j0, 0);
        if (nb == 0) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(&b.qfull, pieces & 1, &b.err) &&
                                         mbar_wait(&b.kfull[n % NS], (n / NS) & 1, &b.err));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
            gemm_ss<D>(tS, qa, kring + (n % NS) * kTile);
            umma_commit(&b.sfull[n & 1]);
            gemm_ss<D>(tT, ra, kring + (n % NS) * kTile);
            umma_commit(&b.tfull[n & 1]);
            umma_commit(&b.kempty[n % NS]);
        }
        __syncwarp();
        for (int j = 0; j < nb; ++j, ++n) {
            const int st = n % NS, sk = (n + 1) % NS;
            const bool more = j + 1 < nb;
            ok = __all_sync(0xffffffffu, mbar_wait(&b.vfull[st], (n / NS) & 1, &b.err) &&
                                             (!more || mbar_wait(&b.kfull[sk], ((n + 1) / NS) & 1, &b.err)) &&
                                             mbar_wait(&b.p1[n & 1], (n >> 1) & 1, &b.err));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                gemm_ts<D>(tO1, tS, vring + st * kTile, j > 0);
                if (more) {
                    gemm_ss<D>(tS, qa, kring + sk * kTile);
                    umma_commit(&b.sfull[(n + 1) & 1]);
                }
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, mbar_wait(&b.p2[n & 1], (n >> 1) & 1, &b.err));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                gemm_ts<D>(tO2, tT, vring + st * kTile, j > 0);
                umma_commit(&b.vempty[st]);
                if (more) {
                    gemm_ss<D>(tT, ra, kring + sk * kTile);
                    umma_commit(&b.tfull[(n + 1) & 1]);
                    umma_commit(&b.kempty[sk]);
                } else {
                    umma_commit(&b.done);
                }
            }
            __syncwarp();
        }
        ++pieces;
    }
    __syncwarp();
    if (elect_one()) umma_commit(&b.fin);
    drain(&b.fin, 0);                          // no product runs when TMEM is given back
}

// 32 columns of this thread's row x f.
__device__ __forceinline__ void scale32(uint32_t t, float f) {
    float x[32];
    tmem_ld32(t, x);
    tmem_ld_wait();
    uint32_t y[16], z[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        y[i] = __float_as_uint(x[i] * f);
        z[i] = __float_as_uint(x[16 + i] * f);
    }
    tmem_st16(t, y);
    tmem_st16(t + 16, z);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(TcArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using Sh = TcShape<D>;
    constexpr int NS = Sh::kStages, kTile = Sh::kTile, HD = D / 2;
    extern __shared__ unsigned char raw[];
    __shared__ long long scratch[40];
    __shared__ TcBars<D> b;
    unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    unsigned char* qs = base;
    unsigned char* rs = base + kTile;
    unsigned char* vs = base + (size_t)(2 + NS) * kTile;
    const uint32_t kring = smem_u32(base) + 2 * kTile, vring = kring + NS * kTile;
    const Work& w = a.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&b.kfull[i], 1);
            mbar_init(&b.kempty[i], 1);
            mbar_init(&b.vfull[i], 1);
            mbar_init(&b.vempty[i], 1);
        }
        mbar_init(&b.qfull, kSoft / 32);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.p1[i], kSoft / 64);
            mbar_init(&b.p2[i], kSoft / 64);
            mbar_init(&b.sfull[i], 1);
            mbar_init(&b.tfull[i], 1);
        }
        mbar_init(&b.done, 1);
        mbar_init(&b.fin, 1);
        b.err = 0;
        mbar_fence_init();
    }
    if (warp == kSoft / 32) {
        tmem_alloc(&b.tmem, 512);
        tmem_relinquish();
    }
    Walk wk = begin_walk(w, scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = b.tmem;

    if (warp == kSoft / 32) {
        feed_kv<D>(w, wk, &mk, &mv, kring, vring, b);
    } else if (warp == kSoft / 32 + 1) {
        issue<D>(w, wk, __shfl_sync(0xffffffffu, tm, 0), __shfl_sync(0xffffffffu, smem_u32(qs), 0),
                 __shfl_sync(0xffffffffu, smem_u32(rs), 0), __shfl_sync(0xffffffffu, kring, 0),
                 __shfl_sync(0xffffffffu, vring, 0), b);
    } else {
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;      // group, row
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lanes, tT = lanes + 128, tO = lanes + 256;
        const uint32_t tO1 = tO + half * HD, tO2 = tO1 + D;   // the output columns this group writes
        int n = 0, pieces = 0;
        bool shared = false;
        Piece p;
        p.parts = 0; p.row0 = p.rows = p.h = 0; p.q.token0 = 0;
        // after a wait that gave up, the others give up at once (they see the flag) and every barrier is still
        // passed: the CTA ends, with results that the error word disowns
        while (next_piece(w, wk, p)) {
            shared = p.slot == 1;
            const int nb = p.j1 - p.j0;
            const int fr = p.row0 + r;
            const long long token = p.q.token0 + fr / w.G;
            const int head = p.h * w.G + fr % w.G;
            float m = -INFINITY, om = 0.f, A = 0.f, s0 = 0.f;
            // rows behind the tile's last compute on zeros and are not written
            int limit = p.keys;
            if (r < p.rows && w.causal) limit = min(max(p.q.L - p.q.nq + fr / w.G + 1, 0), p.q.L);
            if (nb > 0) {
                for (int e = tid; e < kRows * (D / 8); e += kSoft) {
                    const int rr = e / (D / 8), c = e % (D / 8), f2 = p.row0 + rr;
                    uint4 x = make_uint4(0, 0, 0, 0), y = x;
                    if (rr < p.rows) {
                        const long long tk = p.q.token0 + f2 / w.G;
                        const long long hc = (long long)(p.h * w.G + f2 % w.G) * D + c * 8;
                        x = *reinterpret_cast<const uint4*>(a.q + tk * a.q_stride + hc);
                        y = *reinterpret_cast<const uint4*>(a.probe + tk * a.r_stride + hc);
                    }
                    *reinterpret_cast<uint4*>(qs + piece_off(rr, c)) = x;
                    *reinterpret_cast<uint4*>(rs + piece_off(rr, c)) = y;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.qfull);
            }
            bool centred = false;
            for (int j = 0; j < nb; ++j, ++n) {
                if ((n & 1) != half) continue;
                const int key0 = (p.j0 + j) * kKeys, ph = (n >> 1) & 1;
                const bool masked = !__all_sync(0xffffffffu, limit >= key0 + kKeys);
                const bool tail = p.keys < key0 + kKeys;
                // ---------------------------------------------------------------- S: the weights p
                float mo = -INFINITY;              // the reference point before this block
                if (j > 0) {
                    mbar_wait(&b.p1[half ^ 1], ((n - 1) >> 1) & 1, &b.err);
                    mo = b.m[r];
                }
                mbar_wait(&b.sfull[half], ph, &b.err);
                tc_fence_after();
                float mn = mo;
                if (j == 0 || masked) {            // the maximum first; keys that the row does not see out of the way
                    float bm = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < kKeys; c += 32) {
                        float x[32];
                        tmem_ld32(tS + c, x);
                        tmem_ld_wait();
                        const int in = limit - key0 - c;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (i >= in) x[i] = -INFINITY;
                            bm = fmaxf(bm, x[i]);
                        }
                        if (masked) {
                            uint32_t y[16], z[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                y[i] = __float_as_uint(x[i]);
                                z[i] = __float_as_uint(x[16 + i]);
                            }
                            tmem_st16(tS + c, y);
                            tmem_st16(tS + c + 16, z);
                        }
                    }
                    tmem_st_wait();
                    bm *= a.scale;
                    if (__any_sync(0xffffffffu, bm > mo + 8.f)) mn = fmaxf(mo, bm);
                }
                if (tail) {
                    // value rows behind the last key hold a page's rest or an earlier block; a zero weight does
                    // not remove a NaN, so they are cleared before the products read them
                    const int st = n % NS;
                    mbar_wait(&b.vfull[st], (n / NS) & 1, &b.err);
                    for (int e = tid & 127; e < kKeys * (D / 8); e += 128) {
                        const int rr = e / (D / 8), c = e % (D / 8);
                        if (key0 + rr >= p.keys)
                            *reinterpret_cast<uint4*>(vs + (size_t)st * kTile + piece_off(rr, c)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                uint32_t pk[64];
                float ps;
                // One pass with the reference point of the blocks before: it follows the maximum only when that
                // has grown by more than 8 (weights to 2^8), and then the pass is repeated (S is still there).
                for (;;) {
                    const float mb = mn == -INFINITY ? 0.f : mn;
                    const uint64_t sc2 = f2_pack(a.scale, a.scale), nm2 = f2_pack(-mb, -mb);
                    uint64_t sum2 = f2_pack(0.f, 0.f);
                    float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
                    for (int c = 0; c < kKeys; c += 32) {
                        float x[32];
                        tmem_ld32(tS + c, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            b0 = fmaxf(b0, x[2 * i]);
                            b1 = fmaxf(b1, x[2 * i + 1]);
                            float u, v;
                            f2_unpack(f2_fma(f2_pack(x[2 * i], x[2 * i + 1]), sc2, nm2), u, v);
                            u = ex2(u);
                            v = ex2(v);
                            sum2 = f2_add(sum2, f2_pack(u, v));
                            // the value products take the weights in bf16 (half a step is 2^-8 of each), the same
                            // rounded weight in both; their sums and the normaliser are fp32
                            pk[c / 2 + i] = pack_bf16(u, v);
                        }
                    }
                    float u;
                    f2_unpack(sum2, ps, u);
                    ps += u;
                    const float bm = a.scale * fmaxf(b0, b1);
                    if (!__any_sync(0xffffffffu, bm > mn + 8.f)) break;
                    mn = fmaxf(mn, bm);
                }
                float f = 1.f;                     // from the reference before to this block's
                const bool grow = __any_sync(0xffffffffu, mn > mo);
                if (grow) {
                    f = mn == -INFINITY ? 1.f : ex2(mo - mn);
                    if (j > 0) {                   // O1 of the blocks before (complete: S of this one came after it)
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) scale32(tO + c, f);
                    }
                }
                if (grow || j == 0) b.m[r] = mn;
                tmem_st16(tS, *reinterpret_cast<uint32_t (*)[16]>(&pk[0]));
                tmem_st16(tS + 16, *reinterpret_cast<uint32_t (*)[16]>(&pk[16]));
                tmem_st16(tS + 64, *reinterpret_cast<uint32_t (*)[16]>(&pk[32]));
                tmem_st16(tS + 80, *reinterpret_cast<uint32_t (*)[16]>(&pk[48]));
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p1[half]);
                // this group's sums to the new reference (m: the reference of its last block)
                const float fs = mn == -INFINITY || m == -INFINITY ? 1.f : ex2(m - mn);
                om = om * fs + ps;
                A *= fs;
                m = mn;

                // ------------------------------------------------------------- T: the weights p (t - s0)
                if (j > 0 && !centred) {
                    mbar_wait(&b.p2[half ^ 1], ((n - 1) >> 1) & 1, &b.err);
                    s0 = b.s0[r];
                }
                mbar_wait(&b.tfull[half], ph, &b.err);
                tc_fence_after();
                if (j == 0) {                  // centre: the softmax mean of t over the first keys
                    float x = 0.f, y = 0.f, t[32];
                    tmem_ld32(tT, t);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float q = __uint_as_float(i & 1 ? pk[i / 2] & 0xffff0000u : pk[i / 2] << 16);
                        if (key0 + i < limit) {
                            x += q;
                            y = fmaf(q, t[i], y);
                        }
                    }
                    s0 = x > 0.f ? y / x : t[0];
                    b.s0[r] = s0;
                } else if (grow) {             // O2 of the blocks before (complete: T of this one came after it)
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) scale32(tO + D + c, f);
                }
                centred = true;
                if (tail) {                    // t of keys behind the last may be anything, a NaN too
#pragma unroll 1
                    for (int c = 0; c < kKeys; c += 32) {
                        float x[32];
                        tmem_ld32(tT + c, x);
                        tmem_ld_wait();
                        const int in = p.keys - key0 - c;
                        uint32_t y[16], z[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            y[i] = __float_as_uint(i < in ? x[i] : s0);
                            z[i] = __float_as_uint(16 + i < in ? x[16 + i] : s0);
                        }
                        tmem_st16(tT + c, y);
                        tmem_st16(tT + c + 16, z);
                    }
                    tmem_st_wait();
                }
                const uint64_t ns2 = f2_pack(-s0, -s0);
                uint64_t sum2 = f2_pack(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) {
                    float t[32];
                    tmem_ld32(tT + c, t);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t q = pk[c / 2 + i];
                        const uint64_t x2 = f2_mul(f2_pack(__uint_as_float(q << 16), __uint_as_float(q & 0xffff0000u)),
                                                   f2_add(f2_pack(t[2 * i], t[2 * i + 1]), ns2));
                        sum2 = f2_add(sum2, x2);
                        float u, v;
                        f2_unpack(x2, u, v);
                        pk[c / 2 + i] = pack_bf16(u, v);
                    }
                }
                tmem_st16(tT, *reinterpret_cast<uint32_t (*)[16]>(&pk[0]));
                tmem_st16(tT + 16, *reinterpret_cast<uint32_t (*)[16]>(&pk[16]));
                tmem_st16(tT + 64, *reinterpret_cast<uint32_t (*)[16]>(&pk[32]));
                tmem_st16(tT + 80, *reinterpret_cast<uint32_t (*)[16]>(&pk[48]));
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p2[half]);
                float x, y;
                f2_unpack(sum2, x, y);
                A += x + y;
            }

            if (nb > 0) {
                mbar_wait(&b.done, pieces & 1, &b.err);
                tc_fence_after();
                ++pieces;
                // the last reference and the centre: written before the arrivals that `done` came after
                const int last = (n - 1) & 1;
                if (last != half) {
                    mbar_wait(&b.p1[last], ((n - 1) >> 1) & 1, &b.err);
                    mbar_wait(&b.p2[last], ((n - 1) >> 1) & 1, &b.err);
                    const float mn = b.m[r], fs = m == -INFINITY ? 0.f : ex2(m - mn);
                    om *= fs;
                    A *= fs;
                    m = mn;
                    s0 = b.s0[r];
                }
                b.tot[half][r] = make_float2(om, A);
                named_bar_sync(1, kSoft);
                om = b.tot[0][r].x + b.tot[1][r].x;
                A = b.tot[0][r].y + b.tot[1][r].y;
            }
            const float inv = om != 0.f ? 1.f / om : 0.f, c1 = (1.f + A * inv) * inv;
#pragma unroll
            for (int c = 0; c < HD; c += 32) {
                float o1[32], o2[32];
                if (nb > 0) {
                    tmem_ld32(tO1 + c, o1);
                    tmem_ld32(tO2 + c, o2);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o1[i] = o2[i] = 0.f;
                }
                if (r < p.rows) {
                    const int col = half * HD + c;
                    if (p.slot < 0) {
                        uint4* o = reinterpret_cast<uint4*>(a.out + (token * a.Hq + head) * D + col);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int k = i * 8 + e * 2;
                                y[e] = pack_bf16(c1 * o1[k] - inv * o2[k], c1 * o1[k + 1] - inv * o2[k + 1]);
                            }
                            o[i] = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    } else {
                        float4* d1 = reinterpret_cast<float4*>(part_sums(w, blockIdx.x, p.slot, D) + (size_t)r * 2 * D + col);
                        float4* d2 = d1 + D / 4;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            d1[i] = make_float4(o1[4 * i], o1[4 * i + 1], o1[4 * i + 2], o1[4 * i + 3]);
                            d2[i] = make_float4(o2[4 * i], o2[4 * i + 1], o2[4 * i + 2], o2[4 * i + 3]);
                        }
                    }
                }
            }
            if (r < p.rows && half == 0 && p.slot >= 0)
                *reinterpret_cast<float4*>(part_stats(w, blockIdx.x, p.slot, D) + r * 4) = make_float4(m, om, A, s0);
            tc_fence_before();                 // O is read: the next tile's products may write it
            named_bar_sync(1, kSoft);          // and tot is free
        }
        if (tid == 0) write_header(w, p, shared);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoft / 32) {
        __syncwarp();
        tmem_dealloc(tm, 512);
    }
    if (tid == 0 && b.err) atomicOr(w.err, (unsigned)kDevErrMbarTimeout);
}

template <int D>
cudaError_t launch_tc(const TcArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
    constexpr size_t smem = TcShape<D>::smem;
    cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    paged_tc_kernel<D><<<a.w.ctas, kThreads, smem, stream>>>(a, mk, mv);
    return cudaGetLastError();
}

}  // namespace
}  // namespace paged

PagedSplit paged_tc_split(const PagedProblem& p, int sms) {
    (void)p;
    return PagedSplit{paged::kRows, paged::kKeys, sms, 2};
}

cudaError_t launch_paged_tc(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream, const char** why) {
    CUtensorMap mk, mv;
    if (!paged::make_cache_map(&mk, p.k, p) || !paged::make_cache_map(&mv, p.v, p)) {
        *why = "tensor map of a paged cache";
        return cudaErrorInvalidValue;
    }
    paged::TcArgs a{paged::make_work(p, sp), static_cast<const __nv_bfloat16*>(p.q), static_cast<const __nv_bfloat16*>(p.probe),
                    static_cast<__nv_bfloat16*>(p.out), p.Hq, p.q_stride, p.r_stride, p.tau * 1.4426950408889634f};
    return p.d == 128 ? paged::launch_tc<128>(a, mk, mv, stream) : paged::launch_tc<64>(a, mk, mv, stream);
}

}  // namespace lla
