// Parallax attention over a paged bf16 cache for many query rows to a key head (prompts, chunks of
// prompts, cross attention, drafts over many shared heads): tcgen05 with 128-row tiles.
//
// Per block of 128 keys four products of 128 x 128 x d: S = Q K^T, T = R K^T, O1 += P V and O2 += P' V
// with P = 2^(l - m) and P' = P (T - s0) (the formulas of lla_paged_simt.cu).  S, T, O1 and O2 fill the
// 512 TMEM columns (d = 128), so S and T have one buffer each, and P and P' (bf16) overwrite the halves of S and T
// that they came from.  The products are issued as
//     S(j+1)  O2(j)  T(j+1)  O1(j+1)  S(j+2)  O2(j+1) ...
// : the softmax of S(j+1) runs under O2(j) and T(j+1), the weighting of T(j+1) under O1(j+1) and S(j+2).
// 512 tokens over 16,384 keys, 32 query / 4 key heads, d = 128: 189 us, 1.47 PFLOP/s (175 replayed from a graph on the same
// inputs; a block takes 2700 cycles, its products 2048); prompts of 700 to 4096 tokens, 16 heads: 269 us, 1.11 PFLOP/s
// (258 replayed; a tile's first and last block and its epilogue cost 4000 cycles).  At d = 64 the row warps bound it, 2300
// cycles a block: 144 and 195 us replayed.
//
// Eight warps hold the rows, a thread half of a row's columns.  The exponents are taken against the
// reference point of the blocks before while the maximum is taken beside them, and only the vote of a
// row's two warps on whether it grew stands between: the softmax of a block is one pass.  One warp feeds K
// and V through TMA rings (a box per page), one issues the products, two divide the work, publish the tiles
// and load the next tile's queries as soon as the last product that reads the present ones is done: the next
// tile's first products run under the epilogue.
#include <math.h>

#include "../../include/lla.h"
#include "lla_internal.h"
#include "lla_paged.h"
#include "paged_feed.h"
#include "paged_tc.cuh"

namespace lla {
namespace paged {
namespace {

using namespace tc;

constexpr int kRows = kTileRows;
constexpr int kSoft = 256;                     // threads that hold rows
constexpr int kLoad = 64;                      // threads that load queries and probes
constexpr int kThreads = kSoft + 64 + kLoad;   // 168 registers each at launch: 384 x 168 = 256 x 216 + 128 x 72

template <int D>
struct TcShape {
    static constexpr int kKeys = 128;                      // of a block
    static constexpr int kStages = D == 128 ? 2 : 4;       // of K and of V
    static constexpr int kCols = kKeys / 2;                // columns of S (and T) that a thread holds
    static constexpr int kTmem = 512;                      // columns: S, T, O1, O2 (a power of two)
    static constexpr int kRowTile = kRows * D * 2;         // bytes of Q or R: [D / 64][128 rows][128 B]
    static constexpr int kTile = kKeys * D * 2;            // bytes of a K or V block
    static constexpr size_t smem = (size_t)2 * kRowTile + (size_t)2 * kStages * kTile + 1024;
};

struct TcArgs {
    Work w;
    const __nv_bfloat16* q;
    const __nv_bfloat16* probe;
    __nv_bfloat16* out;
    int Hq, slices;                            // slices: head slices from page to page
    long long q_stride, r_stride;
    float scale;                               // tau log2(e)
    int row_boxes;                             // 128 is a multiple of G: a tile's rows are whole tokens
    float* lse;                                // [T, Hq], or null
};

constexpr int kRing = 4;                       // pieces published ahead

template <int D>
struct TcBars {
    uint64_t kfull[TcShape<D>::kStages], kempty[TcShape<D>::kStages];
    uint64_t vfull[TcShape<D>::kStages], vempty[TcShape<D>::kStages];
    uint64_t qfull, qfree, sfull, tfull, p1, p2, done, fin;
    uint64_t ready[kRing], free[kRing];        // of the published pieces
    Piece piece[kRing];                        // rows 0: no more
    uint32_t tmem;
    int err;
    float mx[2][kRows], s0[kRows];             // by column half: row maxima; centres
    float2 tot[2][kRows];                      // by column half: omega and A of a tile
};

// What feed_kv's two rings of copies are filled and drained through (paged_feed.h): one box to a lane.
template <int D>
struct KvRings {
    const CUtensorMap* map[2];                 // of K, of V
    uint32_t ring[2];
    TcBars<D>& b;
    int box, lane;
    // the block at hand: this lane's box, if it has one, and the boxes' bytes
    bool mine;
    int group, slice;
    uint32_t bytes;

    __device__ __forceinline__ uint64_t* full(int kv, int stage) { return kv ? &b.vfull[stage] : &b.kfull[stage]; }
    __device__ __forceinline__ bool wait_empty(int kv, int stage, int parity) {
        return __all_sync(0xffffffffu, mbar_wait(kv ? &b.vempty[stage] : &b.kempty[stage], parity, &b.err));
    }
    __device__ __forceinline__ void copy(int kv, int stage) {
        if (lane == 0) mbar_arrive_expect_tx(full(kv, stage), bytes);
        __syncwarp();
        if (mine) {
            const uint32_t dst = ring[kv] + (uint32_t)(stage * TcShape<D>::kTile + lane * box * D * 2);
            tma_load_rows(dst, map[kv], full(kv, stage), group, slice);
        }
        __syncwarp();
    }
    __device__ __forceinline__ void wait_full(int kv, int stage, int parity) { drain(full(kv, stage), parity); }
};

// K and V of a block go to rings of their own (K is given back a product earlier).
template <int D>
__device__ void feed_kv(const Work& w, Walk wk, const CUtensorMap* mk, const CUtensorMap* mv, int slices, uint32_t kring,
                        uint32_t vring, TcBars<D>& b) {
    constexpr int NS = TcShape<D>::kStages, kKeys = TcShape<D>::kKeys;
    const int lane = threadIdx.x & 31;
    const int box = min(1 << w.page_shift, kBoxRows), boxes = kKeys / box;     // <= 16
    KvRings<D> rings{{mk, mv}, {kring, vring}, b, box, lane, false, 0, 0, 0};
    RingCount<NS> n;
    bool ok = true;
    Piece p;
    while (ok && next_piece(w, wk, p)) {
        const int* row = w.table + (size_t)p.s * w.width;
        for (int j = p.j0; ok && j < p.j1; ++j) {
            const int key = j * kKeys + lane * box;
            rings.mine = lane < boxes && key < p.keys;
            rings.slice = (rings.mine ? checked_page(w, row, key) : 0) * slices + p.h;
            rings.group = (key & ((1 << w.page_shift) - 1)) >> 3;
            rings.bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, rings.mine)) * box * D * 2);
            ok = n.feed_block(rings);
        }
    }
    if (!ok || *(volatile int*)&b.err) n.drain(rings);    // copies in flight land before the CTA gives its memory back
}

// D[tmem] = A B^T, 128 x kKeys x D, both operands K-major in shared memory.
template <int D>
__device__ __forceinline__ void gemm_ss(uint32_t d, uint32_t a_addr, uint32_t b_addr) {
    constexpr int kKeys = TcShape<D>::kKeys;
    constexpr uint32_t ID = idesc_bf16(kRows, kKeys, false, false);
    const uint64_t a0 = sdesc_sw128(a_addr, 16, 1024), b0 = sdesc_sw128(b_addr, 16, D * 16);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const uint64_t ao = (uint64_t)(((ks >> 2) * (kRows * 128) + (ks & 3) * 32) >> 4);
        const uint64_t bo = (uint64_t)(((ks >> 2) * 1024 + (ks & 3) * 32) >> 4);
        if (ks == 0) umma_ss_c<false>(d, a0 + ao, b0 + bo, ID);
        else umma_ss_c<true>(d, a0 + ao, b0 + bo, ID);
    }
}
// D[tmem] (+)= P V, 128 x D x kKeys: P bf16 pairs in TMEM (each half of the keys in the first columns of the half
// its S or T was in), V [kKeys x D] read MN-major.
template <int D>
__device__ __forceinline__ void gemm_ts(uint32_t d, uint32_t p, uint32_t v_addr, bool acc) {
    constexpr int kKeys = TcShape<D>::kKeys, kHalf = kKeys / 32;      // k steps of a half
    constexpr uint32_t ID = idesc_bf16(kRows, D, false, true);
    const uint64_t b0 = sdesc_sw128(v_addr, 1024, D * 16);
    if (acc) umma_ts_c<true>(d, p, b0, ID);
    else umma_ts_c<false>(d, p, b0, ID);
#pragma unroll
    for (int ks = 1; ks < kKeys / 16; ++ks)
        umma_ts_c<true>(d, p + (ks / kHalf) * (kKeys / 2) + (ks % kHalf) * 8, b0 + (uint64_t)((ks * D * 32) >> 4), ID);
}

// The issuing warp.  All lanes run the loop and one elected lane issues: with everything that the products'
// descriptors are made of uniform across the warp the descriptors stay in uniform registers, which
// tcgen05.mma takes (issued from a branch of lane 0 each product's eight instructions took 570 to 830
// cycles to issue, more than the 512 it takes to run).
template <int D>
__device__ void issue(const Work& w, Walk wk, uint32_t tm, uint32_t qa, uint32_t ra, uint32_t kring, uint32_t vring,
                      TcBars<D>& b) {
    constexpr int NS = TcShape<D>::kStages, kTile = TcShape<D>::kTile, kKeys = TcShape<D>::kKeys;
    const uint32_t tS = tm, tT = tm + kKeys, tO1 = tm + 2 * kKeys, tO2 = tO1 + D;
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
            umma_commit(&b.sfull);
            gemm_ss<D>(tT, ra, kring + (n % NS) * kTile);
            umma_commit(&b.tfull);
            umma_commit(&b.kempty[n % NS]);
            if (nb == 1) umma_commit(&b.qfree);
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, mbar_wait(&b.vfull[n % NS], (n / NS) & 1, &b.err));
        for (int j = 0; ok && j < nb; ++j, ++n) {
            const int st = n % NS, sk = (n + 1) % NS;
            const bool more = j + 1 < nb;
            ok = __all_sync(0xffffffffu, mbar_wait(&b.p1, n & 1, &b.err));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) gemm_ts<D>(tO1, tS, vring + st * kTile, j > 0);
            __syncwarp();
            if (more) {
                ok = __all_sync(0xffffffffu, mbar_wait(&b.kfull[sk], ((n + 1) / NS) & 1, &b.err));
                if (!ok) break;
                if (elect_one()) {
                    gemm_ss<D>(tS, qa, kring + sk * kTile);
                    umma_commit(&b.sfull);
                }
                __syncwarp();
                // the next block's V, off the path from its P to its first product
                ok = __all_sync(0xffffffffu, mbar_wait(&b.vfull[sk], ((n + 1) / NS) & 1, &b.err));
                if (!ok) break;
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&b.p2, n & 1, &b.err));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                gemm_ts<D>(tO2, tT, vring + st * kTile, j > 0);
                umma_commit(&b.vempty[st]);
                if (more) {
                    gemm_ss<D>(tT, ra, kring + sk * kTile);
                    umma_commit(&b.tfull);
                    umma_commit(&b.kempty[sk]);
                    if (j + 2 == nb) umma_commit(&b.qfree);   // the last product that reads Q and R
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

// 16 bytes to shared memory without a register stop; zeros where `in` is false (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
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

// This thread's N columns of a row; the caller waits.
template <int N>
__device__ __forceinline__ void load_cols(uint32_t t, float (&x)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 32) tmem_ld32(t + c, *reinterpret_cast<float (*)[32]>(&x[c]));
}
template <int N>
__device__ __forceinline__ void store_cols(uint32_t t, const uint32_t (&x)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 16) tmem_st16(t + c, *reinterpret_cast<const uint32_t (*)[16]>(&x[c]));
    tmem_st_wait();
}

// 16-byte pieces of four neighbouring lanes, transposed: piece k of lane i and piece i of lane k change places.
__device__ __forceinline__ void transpose4(uint32_t (&y)[4][4]) {
    const bool b0 = threadIdx.x & 1, b1 = threadIdx.x & 2;
#pragma unroll
    for (int i = 0; i < 4; i += 2)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, b0 ? y[i][e] : y[i + 1][e], 1);
            y[i][e] = b0 ? got : y[i][e];
            y[i + 1][e] = b0 ? y[i + 1][e] : got;
        }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? y[i][e] : y[i + 2][e], 2);
            y[i][e] = b1 ? got : y[i][e];
            y[i + 2][e] = b1 ? y[i + 2][e] : got;
        }
}

// Or of x over the two warps of a row set (64 threads).
__device__ __forceinline__ bool pair_or(int id, bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 64, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"(id), "r"((uint32_t)x) : "memory");
    return r != 0;
}

// x <- p = 2^(scale x - ref), and p as bf16 pairs; the fp32 sum, and whether any p reached 2.
// The exponents' reference lies kHead above the maximum that set it, so a weight reaches 2 when a logit has
// grown kHead + 1 = 8 past that maximum, and that is a bit of its bf16 exponent: the maximum itself is taken only
// when the reference moves.  (Weights near 2^-kHead lose nothing: every sum is floating.)
constexpr float kHead = 7.f;
template <int N>
__device__ __forceinline__ void weigh(float (&x)[N], float scale, float ref, uint32_t (&pk)[N / 2], float& sum, bool& over) {
    const uint64_t sc2 = f2_pack(scale, scale), nr2 = f2_pack(-ref, -ref);
    uint64_t s0 = f2_pack(0.f, 0.f), s1 = s0;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        float u, v;
        f2_unpack(f2_fma(f2_pack(x[2 * i], x[2 * i + 1]), sc2, nr2), u, v);
        x[2 * i] = u = ex2(u);
        x[2 * i + 1] = v = ex2(v);
        if (i & 1) s1 = f2_add(s1, f2_pack(u, v));
        else s0 = f2_add(s0, f2_pack(u, v));
        // the value products take the weights in bf16 (half a step is 2^-8 of each); their sums and the normaliser
        // are fp32
        pk[i] = pack_bf16(u, v);
        bits |= pk[i];
    }
    float v;
    f2_unpack(f2_add(s0, s1), sum, v);
    sum += v;
    over = (bits & 0x40004000u) != 0;
}
template <int N>
__device__ __forceinline__ float top_of(const float (&x)[N]) {
    float a = x[0], b = x[1];
#pragma unroll
    for (int i = 2; i < N; i += 2) {
        a = fmaxf(a, x[i]);
        b = fmaxf(b, x[i + 1]);
    }
    return fmaxf(a, b);
}

// The two loading warps: publish the pieces, and bring each tile's queries and probes into shared memory once the
// products of the tile before have read theirs.  Where 128 is a multiple of G a tile's rows are the G heads of
// 128 / G tokens, a box of the token rows (rows behind the tile's last hold what follows, or zeros behind
// the tensor); else each row is copied by itself.  (Copied rows take a tile 6500 cycles, boxes 1500.)
template <int D>
__device__ void load_tiles(const TcArgs& a, Walk wk, const CUtensorMap* mq, const CUtensorMap* mr, uint32_t qa, uint32_t ra,
                           TcBars<D>& b) {
    const Work& w = a.w;
    const int t = threadIdx.x - (kThreads - kLoad), lane = threadIdx.x & 31;
    constexpr int kPieces = D / 8, kStep = kLoad / kPieces;      // 16-byte pieces of a row; rows at a time
    const int c = t % kPieces;
    bool ok = true, more = true;
    int tiles = 0;
    for (int k = 0; ok && more; ++k) {
        Piece p;
        more = next_piece(w, wk, p);
        if (!more) p.rows = 0;
        if (t < 32) {
            if (k >= kRing) ok = __all_sync(0xffffffffu, mbar_wait(&b.free[k % kRing], (k / kRing - 1) & 1, &b.err));
            if (!ok) break;
            if (lane == 0) {
                b.piece[k % kRing] = p;
                mbar_arrive(&b.ready[k % kRing]);
            }
            __syncwarp();
        }
        if (!more || p.j1 == p.j0) continue;
        if (tiles > 0) ok = __all_sync(0xffffffffu, mbar_wait(&b.qfree, (tiles - 1) & 1, &b.err));
        if (!ok) break;
        ++tiles;
        if (a.row_boxes) {
            if (lane == 0) {
                if (t == 0) {
                    mbar_arrive_expect_tx(&b.qfull, 2 * TcShape<D>::kRowTile);
                    const int token = p.q.token0 + over_g(w, p.row0);
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {
                        tma_load_4d(qa + x * (kRows * 128), mq, &b.qfull, x * 64, 0, p.h, token);
                        tma_load_4d(ra + x * (kRows * 128), mr, &b.qfull, x * 64, 0, p.h, token);
                    }
                } else {
                    mbar_arrive(&b.qfull);
                }
            }
            __syncwarp();
            continue;
        }
        const long long hc = (long long)p.h * w.G * D + c * 8;
#pragma unroll 4
        for (int rr = t / kPieces; rr < kRows; rr += kStep) {
            const bool in = rr < p.rows;
            const int f = in ? p.row0 + rr : 0, tk = over_g(w, f);
            const long long token = p.q.token0 + tk, col = hc + (f - tk * w.G) * D;
            const uint32_t to = (uint32_t)((c >> 3) * (kRows * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4));
            copy16(qa + to, a.q + token * a.q_stride + col, in);
            copy16(ra + to, a.probe + token * a.r_stride + col, in);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.qfull);
    }
    if (a.row_boxes && tiles > 0 && (!ok || *(volatile int*)&b.err)) drain(&b.qfull, (tiles - 1) & 1);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(TcArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mr) {
    using Sh = TcShape<D>;
    constexpr int NS = Sh::kStages, kTile = Sh::kTile, kKeys = Sh::kKeys, kCols = Sh::kCols, HD = D / 2;
    extern __shared__ unsigned char raw[];
    __shared__ long long scratch[40];
    __shared__ TcBars<D> b;
    unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t qa = smem_u32(base), ra = qa + Sh::kRowTile;
    unsigned char* vs = base + 2 * Sh::kRowTile + (size_t)NS * kTile;
    const uint32_t kring = qa + 2 * Sh::kRowTile, vring = kring + NS * kTile;
    const Work& w = a.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        tma_prefetch_desc(&mk);
        tma_prefetch_desc(&mv);
        if (a.row_boxes) {
            tma_prefetch_desc(&mq);
            tma_prefetch_desc(&mr);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&b.kfull[i], 1);
            mbar_init(&b.kempty[i], 1);
            mbar_init(&b.vfull[i], 1);
            mbar_init(&b.vempty[i], 1);
        }
        mbar_init(&b.qfull, kLoad / 32);
        mbar_init(&b.qfree, 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&b.ready[i], 1);
            mbar_init(&b.free[i], kSoft / 32);
        }
        mbar_init(&b.p1, kSoft / 32);
        mbar_init(&b.p2, kSoft / 32);
        mbar_init(&b.sfull, 1);
        mbar_init(&b.tfull, 1);
        mbar_init(&b.done, 1);
        mbar_init(&b.fin, 1);
        b.err = 0;
        mbar_fence_init();
    }
    if (warp == kSoft / 32) {
        tmem_alloc(&b.tmem, Sh::kTmem);
        tmem_relinquish();
    }
    cudaGridDependencySynchronize();           // the lengths may be the previous kernel's
    Walk wk = begin_walk(w, blockIdx.x, scratch);
    cudaTriggerProgrammaticLaunchCompletion();   // the merge waits for this grid's end all the same
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = b.tmem;

    if (warp >= kSoft / 32) {
        setmaxnreg_dec72();
        if (warp == kSoft / 32) feed_kv<D>(w, wk, &mk, &mv, a.slices, kring, vring, b);
        else if (warp == kSoft / 32 + 1)
            issue<D>(w, wk, __shfl_sync(0xffffffffu, tm, 0), __shfl_sync(0xffffffffu, qa, 0), __shfl_sync(0xffffffffu, ra, 0),
                     __shfl_sync(0xffffffffu, kring, 0), __shfl_sync(0xffffffffu, vring, 0), b);
        else
            load_tiles<D>(a, wk, &mq, &mr, qa, ra, b);
    } else {
        setmaxnreg_inc216();
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;      // column half, row
        const int pair = 1 + (warp & 3);                             // barrier of the row's two warps
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lanes + half * kCols, tT = tS + kKeys;
        const uint32_t tO1 = lanes + 2 * kKeys + half * HD, tO2 = tO1 + D;   // this half's output columns
        int n = 0, pieces = 0, k = 0;
        // The two warps of a row set agree on each piece before they use it, so that they pass the same barriers
        // whatever a wait gave.  Within a piece, after a wait that gave up, the others give up at once (they see the
        // flag) and every barrier is still passed: the CTA ends, with results that the error word disowns.
        for (;; ++k) {
            const bool got = mbar_wait(&b.ready[k % kRing], (k / kRing) & 1, &b.err);
            if (pair_or(pair, !got)) break;
            const Piece& p = b.piece[k % kRing];
            if (p.rows == 0) break;
            const int nb = p.j1 - p.j0;
            const int tk = over_g(w, min(p.row0 + r, p.row0 + p.rows - 1));
            float m = -INFINITY, om = 0.f, A = 0.f, s0 = 0.f;
            // rows behind the tile's last compute on whatever was loaded for them and are not written
            int limit = p.keys;
            if (r < p.rows && w.causal) limit = min(max(p.q.L - p.q.nq + tk + 1, 0), p.q.L);
            for (int j = 0; j < nb; ++j, ++n) {
                const int key0 = (p.j0 + j) * kKeys, in = limit - key0 - half * kCols;   // columns of this thread it sees
                const bool masked = !__all_sync(0xffffffffu, in >= kCols);
                const bool tail = p.keys < key0 + kKeys;
                // ---------------------------------------------------------------- S: the weights p
                mbar_wait(&b.sfull, n & 1, &b.err);
                tc_fence_after();
                uint32_t pk[kCols / 2];
                float x[kCols], ps, f = 1.f;
                bool grow = j == 0, over;
                auto scores = [&] {
                    load_cols(tS, x);
                    tmem_ld_wait();
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < kCols; ++i)
                            if (i >= in) x[i] = -INFINITY;
                    }
                };
                scores();
                if (j > 0) {
                    weigh(x, a.scale, m == -INFINITY ? 0.f : m, pk, ps, over);
                    grow = pair_or(pair, over && r < p.rows);   // rows that are not the tile's do not decide
                    if (grow) scores();        // S is still there
                }
                if (grow) {
                    const float top = top_of(x);
                    b.mx[half][r] = top;
                    named_bar_sync(pair, 64);
                    const float mn = fmaxf(m, fmaf(a.scale, fmaxf(top, b.mx[half ^ 1][r]), kHead));
                    f = mn == -INFINITY || j == 0 ? 1.f : ex2(m - mn);
                    m = mn;
                    om *= f;
                    A *= f;
                    weigh(x, a.scale, m == -INFINITY ? 0.f : m, pk, ps, over);
                    if (j > 0) {               // O1 of the blocks before (complete: S of this one came after it)
#pragma unroll 1
                        for (int c = 0; c < HD; c += 32) scale32(tO1 + c, f);
                    }
                }
                if (tail) {
                    // value rows behind the last key hold a page's rest or an earlier block; a zero weight does
                    // not remove a NaN, so they are cleared before the products read them
                    const int st = n % NS;
                    mbar_wait(&b.vfull[st], (n / NS) & 1, &b.err);
                    for (int e = tid; e < kKeys * (D / 8); e += kSoft) {
                        const int rr = e / (D / 8), c = e % (D / 8);
                        if (key0 + rr >= p.keys)
                            *reinterpret_cast<uint4*>(vs + (size_t)st * kTile + piece_off<D>(rr, c)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                store_cols(tS, pk);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p1);
                om += ps;

                // ------------------------------------------------------------- T: the weights p (t - s0)
                mbar_wait(&b.tfull, n & 1, &b.err);
                tc_fence_after();
                if (j > 0 && grow) {           // O2 of the blocks before (complete: T of this one came after it)
#pragma unroll 1
                    for (int c = 0; c < HD; c += 32) scale32(tO2 + c, f);
                }
                if (j == 0) {                  // centre: the softmax mean of t over the first keys
                    if (half == 0) {
                        float t[16], y[2] = {0.f, 0.f}, z[2] = {0.f, 0.f};
                        tmem_ld16(tT, t);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < in) {
                                z[i & 1] += x[i];
                                y[i & 1] = fmaf(x[i], t[i], y[i & 1]);
                            }
                        z[0] += z[1];
                        b.s0[r] = z[0] > 0.f ? (y[0] + y[1]) / z[0] : t[0];
                    }
                    named_bar_sync(pair, 64);
                    s0 = b.s0[r];
                }
                const uint64_t ns2 = f2_pack(-s0, -s0);
                uint64_t sum2 = f2_pack(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    float t[32];
                    tmem_ld32(tT + c, t);
                    tmem_ld_wait();
                    if (tail) {                // t of keys behind the last may be anything, a NaN too
                        const int left = p.keys - key0 - half * kCols - c;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i >= left) t[i] = s0;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t x2 = f2_mul(f2_pack(x[c + 2 * i], x[c + 2 * i + 1]),
                                                   f2_add(f2_pack(t[2 * i], t[2 * i + 1]), ns2));
                        sum2 = f2_add(sum2, x2);
                        float u, v;
                        f2_unpack(x2, u, v);
                        pk[c / 2 + i] = pack_bf16(u, v);
                    }
                }
                store_cols(tT, pk);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p2);
                float y, z;
                f2_unpack(sum2, y, z);
                A += y + z;
            }

            // where this lane stores: four lanes write 64 bytes of a row, of four rows one after another
            __nv_bfloat16* to[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rr = (r & ~3) + i, f2 = p.row0 + rr, t2 = over_g(w, f2);
                to[i] = rr < p.rows ? a.out + ((p.q.token0 + (long long)t2) * a.Hq + p.h * w.G + f2 - t2 * w.G) * D +
                                          half * HD + (lane & 3) * 8
                                    : nullptr;
            }
            if (nb > 0) {
                b.tot[half][r] = make_float2(om, A);
                named_bar_sync(pair, 64);
                om = b.tot[0][r].x + b.tot[1][r].x;
                A = b.tot[0][r].y + b.tot[1][r].y;
                mbar_wait(&b.done, pieces & 1, &b.err);
                tc_fence_after();
                ++pieces;
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
                if (p.slot < 0) {
                    uint32_t y[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = i * 8 + e * 2;
                            y[i][e] = pack_bf16(c1 * o1[k] - inv * o2[k], c1 * o1[k + 1] - inv * o2[k + 1]);
                        }
                    transpose4(y);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (to[k]) *reinterpret_cast<uint4*>(to[k] + c) = make_uint4(y[k][0], y[k][1], y[k][2], y[k][3]);
                } else if (r < p.rows) {
                    float4* d1 = part_sums(w, blockIdx.x, p.slot, D) + (size_t)((half * HD + c) / 4) * kRows + r;
                    float4* d2 = d1 + (size_t)(D / 4) * kRows;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        d1[i * kRows] = make_float4(o1[4 * i], o1[4 * i + 1], o1[4 * i + 2], o1[4 * i + 3]);
                        d2[i * kRows] = make_float4(o2[4 * i], o2[4 * i + 1], o2[4 * i + 2], o2[4 * i + 3]);
                    }
                }
            }
            if (r < p.rows && half == 0) {
                if (p.slot >= 0) part_stats(w, blockIdx.x, p.slot, D)[r] = make_float4(m, om, A, s0);
                else put_lse(w, a.lse, p.q.token0 + tk, p.h * w.G + p.row0 + r - tk * w.G, m, om);
            }
            tc_fence_before();                 // O is read: the next tile's products may write it (after p1)
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.free[k % kRing]);
        }
        // the last piece (its place is not used again) is the one that others may finish
        if (tid == 0) {
            const Piece& last = b.piece[(k + kRing - 1) % kRing];
            write_header(w, blockIdx.x, last, k > 0 && last.slot == 1 && !*(volatile int*)&b.err);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoft / 32) {
        __syncwarp();
        tmem_dealloc(tm, Sh::kTmem);
    }
    if (tid == 0 && b.err) atomicOr(w.err, (unsigned)kDevErrMbarTimeout);
}

template <int D>
cudaError_t launch_tc(const TcArgs& a, const CUtensorMap (&m)[4], cudaStream_t stream) {
    constexpr size_t smem = TcShape<D>::smem;
    cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(paged_tc_kernel<D>, dim3(a.w.ctas), kThreads, smem, stream, a, m[0], m[1], m[2], m[3]);
}

}  // namespace
}  // namespace paged

PagedSplit paged_tc_split(const PagedProblem& p, int sms) {
    (void)p;
    return PagedSplit{paged::kRows, paged::TcShape<128>::kKeys, sms, 2};
}

cudaError_t launch_paged_tc(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream, const char** why) {
    CUtensorMap m[4] = {};
    const bool boxes = paged::kRows % p.G == 0;
    if (!paged::make_cache_map(&m[0], p.k, p) || !paged::make_cache_map(&m[1], p.v, p) ||
        (boxes && (!paged::make_rows_map(&m[2], p.q, p.q_stride, p) || !paged::make_rows_map(&m[3], p.probe, p.r_stride, p)))) {
        *why = "tensor map of a paged call";
        return cudaErrorInvalidValue;
    }
    paged::TcArgs a{paged::make_work(p, sp), static_cast<const __nv_bfloat16*>(p.q), static_cast<const __nv_bfloat16*>(p.probe),
                    static_cast<__nv_bfloat16*>(p.out), p.Hq, (int)paged::slices_of_page(p), p.q_stride, p.r_stride,
                    p.tau * 1.4426950408889634f, boxes, p.lse};
    return p.d == 128 ? paged::launch_tc<128>(a, m, stream) : paged::launch_tc<64>(a, m, stream);
}

}  // namespace lla
