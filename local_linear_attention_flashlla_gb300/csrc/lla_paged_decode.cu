// Parallax attention over a paged bf16 cache for few query rows to a key head (a decode step, a few
// drafted tokens): reading the cache bounds it, 2 d bytes of K and of V for 8 d flops per row.  And over a paged
// fp32 cache (d = 32 or 64) for any number of rows.
//
// Eight query rows and their probes are stacked in one 16-row operand of mma.m16n8k16 (rows 0-7 the
// queries, 8-15 the probes of the same rows), so one product gives the logits and t = probe.k, and the
// accumulator layout puts both of a (row, key) pair in one thread.  The weights p and p (t - s0) are
// then, without any exchange, the two row halves of the second product's operand, whose accumulators
// hold O1 = sum p v and O2 = sum p (t - s0) v.  A 128-row tcgen05 tile would carry 8 to 32 useful
// rows and wait for its row warps (2300 cycles per 128 keys at d = 64); here the tensor pipe is busy 26 % of the
// time with eight rows.  64 sequences x 16 heads at 4096 keys: 321 us, 6.7 TB/s; 96 ragged sequences (100 to
// 16,000 keys, eight query heads to a key head, 16-row pages): 234 us, 6.4 TB/s (d = 64: 172 us, 6.2 TB/s, and 137).
//
// Up to 16 rows the value product takes each weight as two bf16 halves, in two products: outputs are then off from float64 by
// their own rounding alone (1.66e-3 of the norm), with bf16 weights by 2.4e-3.  That costs 320 us instead of 318 and 231 instead
// of 230 on these two, 16.6 instead of 16.0 on one sequence of 32,768 keys and 33.5 instead of 31.6 on 16 rows at d = 64 (the
// rest right after its half, in the same sums, 17.5 and 33.8).  With 17 to 32 rows the chain of products is what a warp waits
// for, 42.5 instead of 33.9 on 20 rows at d = 64 and 77 instead of 61 on 32 rows at d = 128: there, as on tcgen05 tiles (which would
// have six products to a block instead of four), the weights are bf16.
//
// A CTA has four computing warps and one that feeds 64-key blocks through a TMA ring (a box per page);
// two CTAs to an SM keep 192 KB of the cache in flight.  The four warps are one, two or four sets of
// eight rows by four, two or one parts of a block's keys, each with a running maximum of its own; the
// parts are joined once per tile, in the space of its last block (slices of an own 8 KB cost two barriers
// each, 1 us of the 10.5 that a tile of one block takes).  With two sets of rows in every warp instead the sums
// do not fit the registers: 32 sequences of 300 to 6000 keys, four key heads, 16 rows, 82 us at d = 128 where this
// took 56 with bf16 weights, and 37 against 31 at d = 64.  20 rows, d = 64: 34 us here, 42 on tcgen05 tiles; a warp then waits for its
// own chain of products and exponentials, and three or four CTAs to an SM (39 and 42 us) only add starts and parts.
// 32 rows at d = 128: 60 us, 62 on tcgen05 tiles; 48 rows at d = 64 would be two tiles, 42 us there.
//
// fp32: a cache row lies in the ring as a bf16 row of twice the columns would, and ldmatrix hands out its 32-bit
// words as it does pairs of bf16, so the first product only has other instructions: x y = xh yh + xh yl + xl yh,
// h and l the upper and lower 11 bits (three of m16n8k8 in tf32, fp32 sums).  What is left out and rounded is
// 3 2^-22 of a product, where an fp32 product has 2^-24 and the sums of d and of the keys more than either; outputs are
// as far from float64 as with fp32 products (2.8e-7 on the first case below).  The second product takes a step's keys
// in an order in which the accumulators are already its operand.  16 sequences of 1 to 97 tokens over 200 to 1024 keys,
// 4 heads, d = 32: 26.5 us (fp32 products on CUDA cores, which wait for shared memory, 35); 64 such sequences 76 (104),
// d = 64 148 (196); decode of 32 x 16 heads at 4096 keys, d = 32 and 64: 109 and 202 us (151 and 231), 4.9 and 5.3 TB/s;
// one row over 1000 keys, d = 64: 9.5 (7.5).  At d = 128 the ring leaves room for one CTA: 411 us where CUDA cores take
// 369, so they keep it.
#include <math.h>

#include "../../include/lla.h"
#include "lla_internal.h"
#include "lla_paged.h"
#include "paged_tc.cuh"

namespace lla {
namespace paged {
namespace {

constexpr int kKeys = 64;                      // keys of a block
constexpr int kWarps = 4;                      // computing warps
constexpr int kThreads = (kWarps + 1) * 32;

// RS sets of eight query rows in a tile: 1, 2 or 4.
template <typename T, int D, int RS>
struct DecShape {
    static constexpr int kWide = D * (int)sizeof(T) / 2;   // a row's bytes as bf16 columns
    static constexpr int kParts = kWarps / RS;             // warps that share a set's keys
    static constexpr int kShare = kKeys / kParts;          // keys of a block that a warp has
    // key tiles of a step and operand steps in registers: as many as the registers take (the others in shared memory)
    static constexpr int kTiles = (kWide >= 128 || sizeof(T) == 4) && RS == 4 ? 4 : kShare / 8;
    // (fp32 steps are split where they are used: in registers the compiler would keep the halves of all of them)
    static constexpr int kRegSteps = kWide == 128 && (RS > 1 || sizeof(T) == 4) ? 4 : sizeof(T) == 4 ? 0 : kWide / 16;
    // the value product takes the weights as two bf16 halves (2^-16 of each is left out); with four sets in bf16 alone (half a
    // step is 2^-8 of each): see above.  Its sums are fp32 in both.
    static constexpr bool kHalves = sizeof(T) == 2 && RS < 4;
    static constexpr int kStages = kWide == 128 ? 3 : 6;
    static constexpr int kTile = kKeys * kWide * 2;        // bytes of a K (or V) block
    static constexpr int kOperand = kWarps * (kWide / 16 - kRegSteps) * 512;
    static constexpr size_t smem = (size_t)kStages * 2 * kTile + kOperand + 1024;   // 1024: alignment of the ring
    static_assert(kWarps * 2 * 8 * D * 4 <= 2 * kTile, "a block's space takes the warps' sums");
};

struct DecArgs {
    Work w;
    const void* q;
    const void* probe;
    void* out;
    int Hq, slices;                            // slices: head slices from page to page
    long long q_stride, r_stride;
    float scale;                               // tau log2(e)
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x = hi + lo but for 2^-23 of it: hi has the upper 11 bits, rounded half away from zero, and what is left has 12 at most,
// of which the product reads 11 (the upper 19 bits of a word).  Rounding lo instead would be off by the same last bit, and
// an integer sum wraps around for some NaNs (0x7fffffff, which arithmetic produces, among them): here hi may, but lo is
// then the NaN of a subtraction, and for an infinity too.  Without lo's last bit in x itself, one operation more and
// lost half the time, 16 sequences of 200 to 1024 keys are off from float64 by 4.5e-7 where this is 2.8e-7.
__device__ __forceinline__ void split(uint32_t x, uint32_t& hi, uint32_t& lo) {
    hi = (x + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What two values packed as bf16 lost by it, packed as bf16.
__device__ __forceinline__ uint32_t rest_bf16(uint32_t packed, float lo, float hi) {
    return pack_bf16(lo - __uint_as_float(packed << 16), hi - __uint_as_float(packed & 0xffff0000u));
}

// c + x += a b over eight fp32 columns, as three products of halves.  The tensor core cuts its sums off instead of
// rounding them, so the two small products have a sum of their own, x, and the sums are short: a step's value product
// begins at zero (all in one sum, outputs over 1000 keys are off by 2.4e-6; like this by 3e-7).
__device__ __forceinline__ void product(float (&c)[4], float (&x)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    uint32_t ah[4], al[4], h0, l0, h1, l1;
#pragma unroll
    for (int i = 0; i < 4; ++i) split(a[i], ah[i], al[i]);
    split(b0, h0, l0);
    split(b1, h1, l1);
    mma1688(x, al, h0, h1);
    mma1688(x, ah, l0, l1);
    mma1688(c, ah, h0, h1);
}

__device__ __forceinline__ void put2(__nv_bfloat16* p, float x, float y) { *reinterpret_cast<uint32_t*>(p) = pack_bf16(x, y); }
__device__ __forceinline__ void put2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ void put4(__nv_bfloat16* p, float x, float y, float z, float w) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x, y), pack_bf16(z, w));
}
__device__ __forceinline__ void put4(float* p, float x, float y, float z, float w) {
    *reinterpret_cast<float4*>(p) = make_float4(x, y, z, w);
}

// The feeding warp: one block after another of this CTA's pieces, a box to a lane.
template <typename Sh>
__device__ void feed(const Work& w, Walk wk, const CUtensorMap* mk, const CUtensorMap* mv, int slices, uint32_t ring,
                     uint64_t* full, uint64_t* empty, volatile int* err) {
    constexpr int kStages = Sh::kStages, kTile = Sh::kTile, kRow = Sh::kWide * 2;
    const int lane = threadIdx.x & 31;
    const int box = min(1 << w.page_shift, kBoxRows);        // rows of a box
    const int boxes = kKeys / box;                           // <= 8
    int stage = 0, phase = 0, issued = 0;
    bool ok = true;
    Piece p;
    while (ok && next_piece(w, wk, p)) {
        const int* row = w.table + (size_t)p.s * w.width;
        for (int j = p.j0; j < p.j1; ++j) {
            const int key = j * kKeys + lane * box;          // first key of this lane's box
            const bool mine = lane < boxes && key < p.keys;
            const int page = mine ? checked_page(w, row, key) : 0;
            const int count = __popc(__ballot_sync(0xffffffffu, mine));
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[stage], phase ^ 1, err));
            if (!ok) break;
            if (lane == 0) tc::mbar_arrive_expect_tx(&full[stage], (uint32_t)(count * box * kRow * 2));
            __syncwarp();
            if (mine) {
                const uint32_t dst = ring + (uint32_t)(stage * 2 * kTile + lane * box * kRow);
                const int group = (key & ((1 << w.page_shift) - 1)) >> 3, slice = page * slices + p.h;
                tma_load_rows(dst, mk, &full[stage], group, slice);
                tma_load_rows(dst + kTile, mv, &full[stage], group, slice);
            }
            __syncwarp();
            ++issued;
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
    }
    if (!ok || *err)
        for (int t = max(issued - kStages, 0); t < issued; ++t) drain(&full[t % kStages], (t / kStages) & 1);
}

template <typename T, int D, int RS>
__global__ void __launch_bounds__(kThreads, 2)
    paged_decode_kernel(DecArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using Sh = DecShape<T, D, RS>;
    constexpr int kStages = Sh::kStages, kTile = Sh::kTile;
    constexpr int DB = Sh::kWide, KS = DB / 16;   // k steps of the first product
    constexpr int NT = D / 8;                  // column tiles of the second
    constexpr int NK = Sh::kTiles, KR = Sh::kRegSteps;
    constexpr int R = RS * 8;
    extern __shared__ unsigned char raw[];
    __shared__ long long scratch[40];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ int err;
    __shared__ float4 stats[kWarps][8];
    unsigned char* base = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t ring = tc::smem_u32(base);
    const Work& w = a.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // this lane's operand steps that registers do not hold
    uint4* qs = reinterpret_cast<uint4*>(base + (size_t)kStages * 2 * kTile) + warp * (KS - KR) * 32 + lane;

    if (tid == 0) {
        tc::tma_prefetch_desc(&mk);
        tc::tma_prefetch_desc(&mv);
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], kWarps);
        }
        err = 0;
        tc::mbar_fence_init();
    }
    cudaGridDependencySynchronize();           // the lengths may be the previous kernel's
    Walk wk = begin_walk(w, blockIdx.x, scratch);
    cudaTriggerProgrammaticLaunchCompletion();   // the merge waits for this grid's end all the same
    __syncthreads();

    if (warp == kWarps) {
        feed<Sh>(w, wk, &mk, &mv, a.slices, ring, full, empty, &err);
    } else {
        const int g = lane >> 2, c2 = (lane & 3) * 2;
        const int set = warp % RS, share0 = warp / RS * Sh::kShare;     // this warp's rows and keys of a block
        int stage = 0, phase = 0;
        bool shared = false, ok = true;
        Piece p;
        p.parts = 0; p.row0 = p.rows = p.h = 0; p.q.token0 = 0;
        // a warp whose wait gave up (ok false) computes nothing more, but passes every barrier of the join
        while (next_piece(w, wk, p)) {
            shared = p.slot == 1;
            const int r = set * 8 + g, fr = p.row0 + r, token = p.q.token0 + over_g(w, fr);
            const int head = p.h * w.G + (fr - over_g(w, fr) * w.G);
            const bool in = r < p.rows;
            // first operand, rows g: queries in registers 0 and 2, probes in 1 and 3
            uint32_t qf[KR > 0 ? KR : 1][4];
            int limit = 0;
            const uint32_t* gq = static_cast<const uint32_t*>(a.q);        // in words of 32 bits
            const uint32_t* gr = static_cast<const uint32_t*>(a.probe);
            if (in) {
                limit = w.causal ? min(max(p.q.L - p.q.nq + over_g(w, fr) + 1, 0), p.q.L) : p.q.L;
                gq += ((long long)token * a.q_stride + (long long)head * D) * (int)sizeof(T) / 4 + (lane & 3);
                gr += ((long long)token * a.r_stride + (long long)head * D) * (int)sizeof(T) / 4 + (lane & 3);
            }
            // keys that all of this warp's rows see
            const int all = __reduce_min_sync(0xffffffffu, in ? limit : 0x7fffffff);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t f[4] = {0u, 0u, 0u, 0u};
                if (in) {
                    f[0] = gq[k * 8];
                    f[1] = gr[k * 8];
                    f[2] = gq[k * 8 + 4];
                    f[3] = gr[k * 8 + 4];
                }
                if (k < KR) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) qf[KR > 0 ? k % KR : 0][i] = f[i];
                } else {
                    qs[(k - KR) * 32] = make_uint4(f[0], f[1], f[2], f[3]);
                }
            }
            float m = -INFINITY, om = 0.f, A = 0.f, s0 = 0.f;
            float o[NT][4];                    // per column pair: O1, O1, O2, O2
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
            bool first = true;
            for (int j = p.j0; ok && j < p.j1; ++j) {
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[stage], phase, &err));
                if (!ok) break;
                const uint32_t kt = ring + stage * 2 * kTile, vt = kt + kTile;
                const int behind = p.keys - j * kKeys;       // rows of the block that hold keys
                const int share1 = min(behind, share0 + Sh::kShare);
                if (set * 8 < p.rows && share0 < share1) {
                    if (share1 < share0 + Sh::kShare) {
                        // value rows behind the last key hold a page's rest or an earlier block, and a zero weight does not
                        // remove a NaN: they are cleared (by each of the warps that read them, to the same zeros)
                        for (int e = share1 * (DB / 8) + lane; e < (share0 + Sh::kShare) * (DB / 8); e += 32)
                            *reinterpret_cast<uint4*>(base + (vt - ring) + piece_off<DB>(e / (DB / 8), e % (DB / 8))) = make_uint4(0, 0, 0, 0);
                        tc::fence_proxy_async_smem();        // the ring's next copy is the async proxy's
                        __syncwarp();
                    }
#pragma unroll 1
                    for (int row0 = share0; row0 < share1; row0 += NK * 8) {
                        float s[NK][4], small[sizeof(T) == 4 ? NK : 1][4];
#pragma unroll
                        for (int n = 0; n < NK; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
                        for (int n = 0; n < (sizeof(T) == 4 ? NK : 0); ++n) small[n][0] = small[n][1] = small[n][2] = small[n][3] = 0.f;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            uint32_t f[4];
                            if (k < KR) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) f[i] = qf[KR > 0 ? k % KR : 0][i];
                            } else {
                                const uint4 x = qs[(k - KR) * 32];
                                f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
                            }
#pragma unroll
                            for (int n = 0; n < NK; n += 2) {
                                uint32_t b[4];
                                ldsm4(kt + piece_off<DB>(row0 + n * 8 + (lane & 7) + ((lane >> 4) << 3), k * 2 + ((lane >> 3) & 1)), b);
                                if constexpr (sizeof(T) == 2) {
                                    mma16816(s[n], f, b[0], b[1]);
                                    mma16816(s[n + 1], f, b[2], b[3]);
                                } else {
                                    product(s[n], small[n], f, b[0], b[1]);
                                    product(s[n + 1], small[n + 1], f, b[2], b[3]);
                                }
                            }
                        }
                        if constexpr (sizeof(T) == 4) {
#pragma unroll
                            for (int n = 0; n < NK; ++n)
#pragma unroll
                                for (int i = 0; i < 4; ++i) s[n][i] += small[n][i];
                        }
                        const int key0 = j * kKeys + row0;
                        if (key0 + NK * 8 > all) {           // some row does not see all of the step's keys
#pragma unroll
                            for (int n = 0; n < NK; ++n)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (key0 + n * 8 + c2 + e >= limit) {
                                        s[n][e] = -INFINITY;
                                        s[n][2 + e] = 0.f;
                                    }
                        }
                        float bm = -INFINITY;
#pragma unroll
                        for (int n = 0; n < NK; ++n) bm = fmaxf(bm, fmaxf(s[n][0], s[n][1]));
                        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
                        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2)) * a.scale;
                        // the reference point of the exponents follows the maximum only when that has grown by more than 8
                        // (weights to 2^8): most blocks then rescale nothing
                        if (__any_sync(0xffffffffu, bm > m + 8.f)) {
                            const float mn = fmaxf(m, bm);
                            const float f = mn == -INFINITY ? 1.f : tc::ex2(m - mn);
                            m = mn;
                            om *= f;
                            A *= f;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                o[n][0] *= f;
                                o[n][1] *= f;
                                o[n][2] *= f;
                                o[n][3] *= f;
                            }
                        }
                        const float mb = m == -INFINITY ? 0.f : m;
                        float ps = 0.f, pt = 0.f;
#pragma unroll
                        for (int n = 0; n < NK; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                s[n][e] = tc::ex2(fmaf(s[n][e], a.scale, -mb));
                                ps += s[n][e];
                                pt = fmaf(s[n][e], s[n][2 + e], pt);
                            }
                        if (first) {           // centre: the softmax mean of t over the first keys
                            float x = ps, y = pt;
                            x += __shfl_xor_sync(0xffffffffu, x, 1);
                            y += __shfl_xor_sync(0xffffffffu, y, 1);
                            x += __shfl_xor_sync(0xffffffffu, x, 2);
                            y += __shfl_xor_sync(0xffffffffu, y, 2);
                            s0 = x > 0.f ? y / x : 0.f;
                            first = false;
                        }
                        om += ps;
                        A += pt - s0 * ps;
                        if constexpr (sizeof(T) == 2) {
#pragma unroll
                            for (int kk = 0; kk < NK; kk += 2) {
                                uint32_t pf[4], rest[4];
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const float* y = s[kk + x];
                                    const float z0 = y[0] * (y[2] - s0), z1 = y[1] * (y[3] - s0);
                                    pf[2 * x] = pack_bf16(y[0], y[1]);
                                    pf[2 * x + 1] = pack_bf16(z0, z1);
                                    rest[2 * x] = rest_bf16(pf[2 * x], y[0], y[1]);
                                    rest[2 * x + 1] = rest_bf16(pf[2 * x + 1], z0, z1);
                                }
                                // four pairs of column tiles together: a product of the rests does not wait for the one
                                // before it in the same sums
                                constexpr int kPairs = 4;
#pragma unroll
                                for (int n0 = 0; n0 < NT / 2; n0 += kPairs) {
                                    uint32_t b[kPairs][4];
#pragma unroll
                                    for (int n = 0; n < kPairs; ++n)
                                        ldsm4t(vt + piece_off<DB>(row0 + kk * 8 + (lane & 15), (n0 + n) * 2 + (lane >> 4)), b[n]);
#pragma unroll
                                    for (int h = 0; h < (Sh::kHalves ? 2 : 1); ++h)
#pragma unroll
                                        for (int n = 0; n < kPairs; ++n) {
                                            mma16816(o[(n0 + n) * 2], h ? rest : pf, b[n][0], b[n][1]);
                                            mma16816(o[(n0 + n) * 2 + 1], h ? rest : pf, b[n][2], b[n][3]);
                                        }
                                }
                            }
                        } else {
                            // eight keys in the order 0 2 4 6 1 3 5 7, in which a lane has its two weights
                            uint32_t pf[NK][4];
#pragma unroll
                            for (int kk = 0; kk < NK; ++kk) {
                                const float* y = s[kk];
                                pf[kk][0] = __float_as_uint(y[0]);
                                pf[kk][1] = __float_as_uint(y[0] * (y[2] - s0));
                                pf[kk][2] = __float_as_uint(y[1]);
                                pf[kk][3] = __float_as_uint(y[1] * (y[3] - s0));
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float t[4] = {0.f, 0.f, 0.f, 0.f}, x[4] = {0.f, 0.f, 0.f, 0.f};
                                const int c = n * 8 + g;
                                const unsigned char* v = base + (vt - ring) + (c & 3) * 4;
#pragma unroll
                                for (int kk = 0; kk < NK; ++kk) {
                                    const int vr = row0 + kk * 8 + c2;
                                    product(t, x, pf[kk], *reinterpret_cast<const uint32_t*>(v + piece_off<DB>(vr, c >> 2)),
                                            *reinterpret_cast<const uint32_t*>(v + piece_off<DB>(vr + 1, c >> 2)));
                                }
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[n][i] += t[i] + x[i];
                            }
                        }
                    }
                }
                if (RS < 4 && j + 1 == p.j1) break;      // the last block's space serves the join before it is given back
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&empty[stage]);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
#pragma unroll
            for (int x = 1; x <= 2; x <<= 1) {
                om += __shfl_xor_sync(0xffffffffu, om, x);
                A += __shfl_xor_sync(0xffffffffu, A, x);
            }

            if constexpr (RS == 4) {
                // a warp has all keys of its rows
                if (!in) continue;
                if (p.slot < 0) {
                    const float inv = om != 0.f ? 1.f / om : 0.f, c1 = (1.f + A * inv) * inv;
                    T* out = static_cast<T*>(a.out) + ((long long)token * a.Hq + head) * D + c2;
#pragma unroll
                    for (int n = 0; n < NT; ++n) put2(out + n * 8, c1 * o[n][0] - inv * o[n][2], c1 * o[n][1] - inv * o[n][3]);
                } else {
                    float4* ps = part_sums(w, blockIdx.x, p.slot, D);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        *reinterpret_cast<float2*>(part_element(ps, R, D, 0, r, n * 8 + c2)) = make_float2(o[n][0], o[n][1]);
                        *reinterpret_cast<float2*>(part_element(ps, R, D, 1, r, n * 8 + c2)) = make_float2(o[n][2], o[n][3]);
                    }
                    if (c2 == 0) part_stats(w, blockIdx.x, p.slot, D)[r] = make_float4(m, om, A, s0);
                }
                continue;
            }

            // join the warps of a set: common maximum, centre of the first of them (it has the piece's first keys)
            if (c2 == 0) stats[warp][g] = make_float4(m, om, A, s0);
            tc::named_bar_sync(1, kWarps * 32);
            // the sums in the last block's space: [warp][O1, O2][row][column], columns swizzled by the row so that
            // neither the writes nor the reads collide; then a thread has four columns of a row
            float* sums = reinterpret_cast<float*>(base + (size_t)stage * 2 * kTile);
            auto place = [&](int x, int half, int row, int c) { return ((x * 2 + half) * 8 + row) * D + (c ^ ((row & 3) << 3)); };
            if (p.j0 < p.j1) {
                float mm = -INFINITY;
#pragma unroll
                for (int x = 0; x < Sh::kParts; ++x) mm = fmaxf(mm, stats[x * RS + set][g].x);
                const float f = m == -INFINITY ? (om == 0.f ? 0.f : om) : tc::ex2(m - mm);
                const float ds = s0 - stats[set][g].w;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    *reinterpret_cast<float2*>(sums + place(warp, 0, g, n * 8 + c2)) = make_float2(f * o[n][0], f * o[n][1]);
                    *reinterpret_cast<float2*>(sums + place(warp, 1, g, n * 8 + c2)) =
                        make_float2(f * fmaf(ds, o[n][0], o[n][2]), f * fmaf(ds, o[n][1], o[n][3]));
                }
                tc::named_bar_sync(1, kWarps * 32);
            }
#pragma unroll 1
            for (int e = tid; e < p.rows * (D / 4); e += kWarps * 32) {
                const int row = e / (D / 4), c = e % (D / 4) * 4, st = row / 8;
                float4 x1 = make_float4(0.f, 0.f, 0.f, 0.f), x2 = x1;
                float mm = -INFINITY, ow = 0.f, aw = 0.f;
                const float sref = stats[st][row % 8].w;
#pragma unroll
                for (int x = 0; x < Sh::kParts; ++x) mm = fmaxf(mm, stats[x * RS + st][row % 8].x);
                const float mb = mm == -INFINITY ? 0.f : mm;
#pragma unroll
                for (int x = 0; x < Sh::kParts; ++x) {
                    const float4 t = stats[x * RS + st][row % 8];
                    const float f = tc::ex2(t.x - mb);
                    ow = fmaf(f, t.y, ow);
                    aw = fmaf(f, fmaf(t.w - sref, t.y, t.z), aw);
                    if (p.j0 < p.j1) {
                        const float4 y = *reinterpret_cast<const float4*>(sums + place(x * RS + st, 0, row % 8, c));
                        const float4 z = *reinterpret_cast<const float4*>(sums + place(x * RS + st, 1, row % 8, c));
                        x1.x += y.x; x1.y += y.y; x1.z += y.z; x1.w += y.w;
                        x2.x += z.x; x2.y += z.y; x2.z += z.z; x2.w += z.w;
                    }
                }
                if (p.slot < 0) {
                    const int er = p.row0 + row, tk = over_g(w, er);
                    const float inv = ow != 0.f ? 1.f / ow : 0.f, c1 = (1.f + aw * inv) * inv;
                    put4(static_cast<T*>(a.out) + ((long long)(p.q.token0 + tk) * a.Hq + p.h * w.G + er - tk * w.G) * D + c,
                         c1 * x1.x - inv * x2.x, c1 * x1.y - inv * x2.y, c1 * x1.z - inv * x2.z, c1 * x1.w - inv * x2.w);
                } else {
                    float4* ps = part_sums(w, blockIdx.x, p.slot, D) + (size_t)(c / 4) * R + row;
                    ps[0] = x1;
                    ps[(size_t)(D / 4) * R] = x2;
                    if (c == 0) part_stats(w, blockIdx.x, p.slot, D)[row] = make_float4(mm, ow, aw, sref);
                }
            }
            tc::fence_proxy_async_smem();      // the space's next copy is the async proxy's
            tc::named_bar_sync(1, kWarps * 32);
            if (ok && p.j0 < p.j1) {
                if (lane == 0) tc::mbar_arrive(&empty[stage]);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (tid == 0) write_header(w, blockIdx.x, p, shared);
    }
    __syncthreads();
    if (tid == 0 && err) atomicOr(w.err, (unsigned)kDevErrMbarTimeout);
}

template <typename T, int D, int RS>
cudaError_t launch_one(const DecArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
    constexpr size_t smem = DecShape<T, D, RS>::smem;
    auto* kern = paged_decode_kernel<T, D, RS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(a.w.ctas), kThreads, smem, stream, a, mk, mv);
}

template <typename T, int D>
cudaError_t launch_dec(const DecArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
    switch (a.w.rows) {
        case 8: return launch_one<T, D, 1>(a, mk, mv, stream);
        case 16: return launch_one<T, D, 2>(a, mk, mv, stream);
        default: return launch_one<T, D, 4>(a, mk, mv, stream);
    }
}

}  // namespace
}  // namespace paged

bool paged_decode_fits(const PagedProblem& p, int path) {
    if (path == LLA_PATH_TENSOR) return (long long)p.max_new * p.G <= 32;
    return p.dtype == LLA_DTYPE_FP32 && (p.d == 32 || p.d == 64);
}

PagedSplit paged_decode_split(const PagedProblem& p, int sms) {
    const long long rows = (long long)p.max_new * p.G;
    return PagedSplit{rows <= 8 ? 8 : rows <= 16 ? 16 : 32, paged::kKeys, 2 * sms, 2};
}

cudaError_t launch_paged_decode(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream, const char** why) {
    CUtensorMap mk, mv;
    PagedProblem bytes = p;                    // as a bf16 cache of the same bytes
    if (p.dtype == LLA_DTYPE_FP32) {
        bytes.d *= 2;
        bytes.page_stride *= 2;
    }
    if (!paged::make_cache_map(&mk, p.k, bytes) || !paged::make_cache_map(&mv, p.v, bytes)) {
        *why = "tensor map of a paged cache";
        return cudaErrorInvalidValue;
    }
    paged::DecArgs a{paged::make_work(p, sp), p.q, p.probe, p.out, p.Hq, (int)paged::slices_of_page(p), p.q_stride, p.r_stride,
                     p.tau * 1.4426950408889634f};
    if (p.dtype == LLA_DTYPE_FP32)
        return p.d == 64 ? paged::launch_dec<float, 64>(a, mk, mv, stream) : paged::launch_dec<float, 32>(a, mk, mv, stream);
    return p.d == 128 ? paged::launch_dec<__nv_bfloat16, 128>(a, mk, mv, stream)
                      : paged::launch_dec<__nv_bfloat16, 64>(a, mk, mv, stream);
}

}  // namespace lla
