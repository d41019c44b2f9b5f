// paged_weigh (include/lla.h) for many query rows to a key head, bf16 with d in {64, 128}: tcgen05.
//
// A tile is 256 keys: two products of 128 keys x N query rows x d, S = K Q^T, for every block of up to 128 rows, the keys being
// the rows of the accumulator.  So a thread has a key, sums exp(scale s - lse) over its columns in registers, and the sum
// over query rows needs hardly any exchange; the keys stay in shared memory while query blocks pass.  128 x 128 x 128 takes
// the tensor pipe 512 cycles (576 with the last step, below) and its exponentials (32 a cycle) 512.  Two halves of the keys share each block of queries,
// which halves what comes from L2.
//
// A last step of 16 columns takes the logsumexp off inside the product: the keys have ones there, a query -lse / tau as four
// bf16 terms, together exact to 2^-32 of it.  They are made from a quotient in two parts (a rounded one was off by two units of
// 2^-24 in the worst case) and added last, so the sum is cut once, at the size of q.k: single weights of logits in the hundreds are within
// 1.0 unit of the logit's last place, 2.0 with the rounded quotient in three terms; the logsumexp read from shared memory by the
// weighing threads, 16 bytes for four columns beside the products' operands, is off by as much as the rounded quotient and takes 74 us
// for 70.7.
//
// Sixteen warps weigh (a thread a key and half of a block's columns), one copies keys and queries (TMA: a box per page, and per 64
// columns of a block's rows), one issues the products, two lay out each block's logsumexps and the keys that its rows see (and
// copy its rows where 128 is not a multiple of G).  The four accumulators, two for each half, fill TMEM.
//
// 512 tokens over 16,384 keys, 32/4 heads, d = 128: 70.6 us, 0.99 PFLOP/s, of which 10 are the start and the join of cut tiles.  The
// products alone take 64, some 1100 cycles each; copies and numbers alone 42.  The likely cause: both operands come from shared
// memory, 8 KB for every 64 cycles of the pipe, which is all that shared memory gives, beside the copies into it (N = 256, which reads a
// quarter less for the same work, took 57); no counter tells that from the issuing warp's own pace.  Tried there: eight weighing warps 76; exponentials partly on the FMA pipe 81 to
// 102; three stages of queries 75; N = 256 with one accumulator to a half 89 (products alone 57); 512 keys to a tile 88,
// with two or four issuing warps 81; an issuing warp to a half 80 (products alone 60).
#include <math.h>

#include "../../include/lla.h"
#include "lla_internal.h"
#include "lla_weigh.h"
#include "paged_tc.cuh"

namespace lla {
namespace weigh {
namespace {

using namespace tc;
using paged::drain;
using paged::elect_one;
using paged::kBoxRows;
using paged::kTileRows;

constexpr int kHalf = 128, kTile = 2 * kHalf;      // keys
constexpr int kSum = 512, kLoad = 64;              // threads that weigh, that lay out rows
constexpr int kThreads = kSum + 64 + kLoad;
constexpr int kK = 2, kQ = 2, kR = 4;              // stages of keys, of queries, of the rows' numbers
constexpr int kTail = 128 * 32;                    // bytes of an operand's last step: 16 columns, no swizzle

template <int D>
struct Shape {
    static constexpr int kKeyTile = kTile * D * 2, kRowTile = kTileRows * D * 2;
    static constexpr size_t smem = (size_t)kK * kKeyTile + (size_t)kQ * kRowTile + (kR + 1) * kTail + 1024;
};

struct Args {
    Work w;
    const __nv_bfloat16* q;
    const float* lse;
    int Hq, slices;                                // slices: head slices from page to page
    long long q_stride;
    float scale;                                   // tau log2(e)
    float inv, inv_low;                            // log2(e) / scale, in two parts
    int row_boxes;                                 // rows of a box where 128 is a multiple of G (a block's rows are whole tokens), else 0
};

struct Shared {
    uint64_t kfull[kK], kempty[kK], qfull[kQ], qempty[kQ], rfull[kR], rempty[kR];
    uint64_t sfull[2][2], sempty[2][2];            // by half and buffer
    uint64_t pfull[8], pempty[8];                  // of the sums that a second warp leaves
    uint64_t fin;
    uint32_t tmem;
    int err;
    int all[kR][2];                                // keys that all rows of the block see (by loading warp)
    alignas(16) int limit[kR][kTileRows];                      // keys a row sees
    float other[kTile];
};

// Offset of 16-byte piece c of row r in a last step: eight rows of a piece are one 128-byte block.
__device__ __forceinline__ uint32_t tail_off(int r, int c) { return (uint32_t)((r >> 3) * 256 + c * 128 + (r & 7) * 16); }
// Descriptor of such an operand: no swizzle; 128 bytes from piece to piece, 256 from eight rows to the next.
__device__ __forceinline__ uint64_t tail_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 16) | ((uint64_t)(256 >> 4) << 32) | (1ull << 46);
}
__device__ __forceinline__ int columns_of(int rows) { return (rows + 15) & ~15; }      // N of a product
__device__ __forceinline__ bool has_half(const Piece& p, int half) { return p.t * kTile + half * kHalf < p.q.L; }

// Keys and queries.  Copies in flight are waited for where a wait gave up: shared memory must not go back under them.
template <int D>
__device__ void feed(const Args& a, Walk wk, const CUtensorMap* mk, const CUtensorMap* mq, uint32_t kring, uint32_t qring, Shared& b) {
    using Sh = Shape<D>;
    const Work& w = a.w;
    const int lane = threadIdx.x & 31;
    const int box = min(1 << w.page_shift, kBoxRows), boxes = kTile / box;      // <= 32
    int nk = 0, nq = 0;
    bool ok = true;
    Piece p;
    while (ok && next_piece(w, wk, p)) {
        const int key = p.t * kTile + lane * box, st = nk % kK;
        const bool mine = lane < boxes && key < p.q.L;
        int page = 0;
        if (mine) {
            page = w.table[(size_t)p.s * w.width + (key >> w.page_shift)];
            if (page < 0 || page >= w.num_pages) page = w.num_pages;           // reads as zeros; its scores are not written
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&b.kempty[st], ((nk / kK) & 1) ^ 1, &b.err));
        if (!ok) break;
        const int count = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) mbar_arrive_expect_tx(&b.kfull[st], (uint32_t)(count * box * D * 2));
        __syncwarp();
        if (mine)
            paged::tma_load_rows(kring + (uint32_t)(st * Sh::kKeyTile + lane * box * D * 2), mk, &b.kfull[st],
                                 (key & ((1 << w.page_shift) - 1)) >> 3, page * a.slices + p.h);
        __syncwarp();
        ++nk;
        for (int j = p.b0; a.row_boxes && j < p.b1; ++j, ++nq) {
            const int sq = nq % kQ;
            ok = __all_sync(0xffffffffu, mbar_wait(&b.qempty[sq], ((nq / kQ) & 1) ^ 1, &b.err));
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&b.qfull[sq], (uint32_t)(a.row_boxes * D * 2));
                const int token = p.q.token0 + p.q.first + over_g(w, j * kTileRows);
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    paged::tma_load_4d(qring + sq * Sh::kRowTile + x * (kTileRows * 128), mq, &b.qfull[sq], x * 64, 0, p.h, token);
            }
            __syncwarp();
        }
    }
    if (!ok || *(volatile int*)&b.err) {
        for (int i = nk > kK ? nk - kK : 0; i < nk; ++i) drain(&b.kfull[i % kK], (i / kK) & 1);
        for (int i = nq > kQ ? nq - kQ : 0; i < nq; ++i) drain(&b.qfull[i % kQ], (i / kQ) & 1);
    }
}

// All lanes run the loop and one issues: what the descriptors are made of is uniform (lla_paged_tc.cu).
template <int D>
__device__ void issue(const Work& w, Walk wk, uint32_t tm, uint32_t kring, uint32_t qring, uint32_t tails, Shared& b) {
    using Sh = Shape<D>;
    int nk = 0, n = 0;
    bool ok = true;
    Piece p;
    while (ok && next_piece(w, wk, p)) {
        const int st = nk % kK;
        ok = __all_sync(0xffffffffu, mbar_wait(&b.kfull[st], (nk / kK) & 1, &b.err));
        if (!ok) break;
        const int b0 = __shfl_sync(0xffffffffu, p.b0, 0), b1 = __shfl_sync(0xffffffffu, p.b1, 0);
        const int rows = __shfl_sync(0xffffffffu, rows_of(w, p.q), 0);
        const bool second = __shfl_sync(0xffffffffu, (int)has_half(p, 1), 0);
        for (int j = b0; j < b1; ++j, ++n) {
            const int sq = n % kQ, sr = n % kR, buf = n & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(&b.qfull[sq], (n / kQ) & 1, &b.err) && mbar_wait(&b.rfull[sr], (n / kR) & 1, &b.err));
            if (!ok) break;
            const uint32_t id = idesc_bf16(kHalf, 16, false, false) - ((16u >> 3) << 17) +
                                ((uint32_t)(columns_of(min(rows - j * kTileRows, kTileRows)) >> 3) << 17);
            const uint64_t q0 = sdesc_sw128(qring + sq * Sh::kRowTile, 16, 1024);
            for (int half = 0; half < 2; ++half) {               // (both are waited for and committed, with products or without)
                ok = __all_sync(0xffffffffu, mbar_wait(&b.sempty[half][buf], ((n >> 1) & 1) ^ 1, &b.err));
                if (!ok) break;
                tc_fence_after();
                const uint64_t k0 = sdesc_sw128(kring + st * Sh::kKeyTile + half * (Sh::kKeyTile / 2), 16, D * 16);
                if (elect_one()) {
                    if (half == 0 || second) {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint64_t ko = (uint64_t)(((ks >> 2) * 1024 + (ks & 3) * 32) >> 4);
                            const uint64_t qo = (uint64_t)(((ks >> 2) * (kTileRows * 128) + (ks & 3) * 32) >> 4);
                            const uint32_t d = tm + (half * 2 + buf) * kTileRows;
                            if (ks == 0) umma_ss_c<false>(d, k0 + ko, q0 + qo, id);
                            else umma_ss_c<true>(d, k0 + ko, q0 + qo, id);
                        }
                        umma_ss_c<true>(tm + (half * 2 + buf) * kTileRows, tail_desc(tails + kR * kTail), tail_desc(tails + sr * kTail), id);
                    }
                    umma_commit(&b.sfull[half][buf]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (elect_one()) {
                umma_commit(&b.qempty[sq]);
                umma_commit(&b.rempty[sr]);
                if (j + 1 == b1) umma_commit(&b.kempty[st]);
            }
            __syncwarp();
        }
        ++nk;
    }
    __syncwarp();
    if (elect_one()) umma_commit(&b.fin);
    drain(&b.fin, 0);                                            // no product runs when TMEM is given back
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// Each block's numbers, and its rows where boxes cannot bring them.  The logsumexps come a block ahead: where a tile
// has one block their latency bounded it (64 x 8 key heads at 3000 to 4096 keys, 32 rows: 104 us, so 93).
template <int D>
__device__ void lay_out(const Args& a, Walk wk, uint32_t qring, unsigned char* tails, Shared& b) {
    const Work& w = a.w;
    const int t = threadIdx.x - (kThreads - kLoad), lane = threadIdx.x & 31, warp = t >> 5;
    constexpr int E = kTileRows / kLoad;
    Piece next;
    bool ok = true, more = next_piece(w, wk, next);
    int jn = next.b0;
    float yn[E];
    auto load = [&] {
        const int rows = rows_of(w, next.q);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int row = jn * kTileRows + i * kLoad + t;
            yn[i] = -INFINITY;
            if (more && row < rows) {
                const int tk = over_g(w, row);
                yn[i] = a.lse[(long long)(next.q.token0 + next.q.first + tk) * a.Hq + next.h * w.G + row - tk * w.G];
            }
        }
    };
    load();
    for (int n = 0; ok && more; ++n) {
        const Piece p = next;
        const int sr = n % kR, sq = n % kQ, row0 = jn * kTileRows, rows = rows_of(w, p.q), cols = columns_of(min(rows - row0, kTileRows));
        float y[E];
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = yn[i];
        if (++jn == next.b1) {
            more = next_piece(w, wk, next);
            jn = next.b0;
        }
        load();
        ok = __all_sync(0xffffffffu, mbar_wait(&b.rempty[sr], ((n / kR) & 1) ^ 1, &b.err));
        if (!ok) break;
        int all = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int r = i * kLoad + t;
            float v = 0.f, low = 0.f;                                    // -lse log2(e) / scale, and what v's rounding leaves
            int limit = 0;
            if (y[i] != -INFINITY) {                                     // -inf: a row without weights, or none
                v = -y[i] * a.inv;
                low = fmaf(-y[i], a.inv, -v) - y[i] * a.inv_low;
                limit = keys_seen(w, p.q, over_g(w, row0 + r));
            }
            const float hi = __bfloat162float(__float2bfloat16_rn(v)), left = fabsf(hi) < INFINITY ? v - hi : 0.f;
            const float mid = __bfloat162float(__float2bfloat16_rn(left)), rest = fabsf(hi) < INFINITY ? left - mid + low : 0.f;
            const float third = __bfloat162float(__float2bfloat16_rn(rest));
            *reinterpret_cast<uint4*>(tails + sr * kTail + tail_off(r, 0)) =
                make_uint4(paged::pack_bf16(hi, mid), paged::pack_bf16(third, rest - third), 0u, 0u);
            b.limit[sr][r] = limit;
            if (r < cols) all = min(all, limit);
        }
        all = __reduce_min_sync(0xffffffffu, all);
        if (lane == 0) b.all[sr][warp] = all;
        fence_proxy_async_smem();                // the products read the last step
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.rfull[sr]);
        if (!a.row_boxes) {
            ok = __all_sync(0xffffffffu, mbar_wait(&b.qempty[sq], ((n / kQ) & 1) ^ 1, &b.err));
            if (!ok) break;
            constexpr int kPieces = D / 8, kStep = kLoad / kPieces;
            const int c = t % kPieces;
            for (int r = t / kPieces; r < cols; r += kStep) {
                const int row = min(row0 + r, rows - 1), tk = over_g(w, row);
                const __nv_bfloat16* src = a.q + (p.q.token0 + p.q.first + tk) * a.q_stride +
                                           (long long)(p.h * w.G + row - tk * w.G) * D + c * 8;
                copy16(qring + sq * Shape<D>::kRowTile + (uint32_t)((c >> 3) * (kTileRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                       src, row0 + r < rows);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.qfull[sq]);
        }
    }
}

// Sum of 2^(scale x) over 32 columns, those with key < limit where MASK.
template <bool MASK>
__device__ __forceinline__ void weigh32(const float (&x)[32], const int* limit, int key, uint64_t sc2, uint64_t (&sum)[2]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float y[4];
        f2_unpack(f2_mul(f2_pack(x[4 * i], x[4 * i + 1]), sc2), y[0], y[1]);
        f2_unpack(f2_mul(f2_pack(x[4 * i + 2], x[4 * i + 3]), sc2), y[2], y[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = ex2(y[k]);
        if (MASK) {
            const int4 lim = *reinterpret_cast<const int4*>(limit + 4 * i);
            y[0] = key < lim.x ? y[0] : 0.f;
            y[1] = key < lim.y ? y[1] : 0.f;
            y[2] = key < lim.z ? y[2] : 0.f;
            y[3] = key < lim.w ? y[3] : 0.f;
        }
        sum[0] = f2_add(sum[0], f2_pack(y[0], y[1]));
        sum[1] = f2_add(sum[1], f2_pack(y[2], y[3]));
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_tc_kernel(Args a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mq) {
    using Sh = Shape<D>;
    extern __shared__ unsigned char raw[];
    __shared__ long long scratch[40];
    __shared__ __align__(16) Shared b;
    const uint32_t kring = smem_u32(raw) + ((1024u - (smem_u32(raw) & 1023u)) & 1023u), qring = kring + kK * Sh::kKeyTile;
    const uint32_t tails = qring + kQ * Sh::kRowTile;        // of the query stages, and of the keys behind them
    const Work& w = a.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        tma_prefetch_desc(&mk);
        if (a.row_boxes) tma_prefetch_desc(&mq);
        for (int i = 0; i < kK; ++i) {
            mbar_init(&b.kfull[i], 1);
            mbar_init(&b.kempty[i], 1);
        }
        for (int i = 0; i < kQ; ++i) {
            mbar_init(&b.qfull[i], a.row_boxes ? 1 : kLoad / 32);
            mbar_init(&b.qempty[i], 1);
        }
        for (int i = 0; i < kR; ++i) {
            mbar_init(&b.rfull[i], kLoad / 32);
            mbar_init(&b.rempty[i], kSum / 32 + 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&b.sfull[i >> 1][i & 1], 1);
            mbar_init(&b.sempty[i >> 1][i & 1], kSum / 64);            // warps of a half
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&b.pfull[i], 1);
            mbar_init(&b.pempty[i], 1);
        }
        mbar_init(&b.fin, 1);
        b.err = 0;
        mbar_fence_init();
    }
    {   // the last steps: ones for the keys, zeros in the second pieces of the queries
        unsigned char* t = raw + (tails - smem_u32(raw));
        for (int r = tid; r < 128; r += kThreads) {
            const uint32_t one = 0x3f80u;
            *reinterpret_cast<uint4*>(t + kR * kTail + tail_off(r, 0)) = make_uint4(one | one << 16, one | one << 16, 0u, 0u);
            for (int i = 0; i <= kR; ++i) *reinterpret_cast<uint4*>(t + i * kTail + tail_off(r, 1)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    }
    if (warp == kSum / 32) {
        tmem_alloc(&b.tmem, 512);
        tmem_relinquish();
    }
    cudaGridDependencySynchronize();
    Walk wk = begin_walk(w, scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = b.tmem;
    if (warp == kSum / 32) {
        feed<D>(a, wk, &mk, &mq, kring, qring, b);
    } else if (warp == kSum / 32 + 1) {
        issue<D>(w, wk, __shfl_sync(0xffffffffu, tm, 0), __shfl_sync(0xffffffffu, kring, 0), __shfl_sync(0xffffffffu, qring, 0),
                 __shfl_sync(0xffffffffu, tails, 0), b);
    } else if (warp > kSum / 32 + 1) {
        lay_out<D>(a, wk, qring, raw + (tails - smem_u32(raw)), b);
    } else {
        // warps w and w + 8 have the same keys, 64 columns of a block each; the first takes the sums of the second
        const int pair = warp & 7, half = pair >> 2, part = warp >> 3;
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16) + half * 2 * kTileRows + part * (kTileRows / 2);
        const uint64_t sc2 = f2_pack(a.scale, a.scale);
        int n = 0, pieces = 0;
        bool ok = true;
        Piece p;
        p.parts = p.s = p.h = p.t = 0;
        p.slot = -1;
        while (ok && next_piece(w, wk, p)) {
            const int in_tile = pair * 32 + lane, key = p.t * kTile + in_tile;
            const int last = min(p.t * kTile + half * kHalf + kHalf, p.q.L);      // behind the half's last key
            const bool live = has_half(p, half), whole = part == 0 && p.slot < 0 && key < p.q.L;
            const bool fresh = w.causal && key >= p.q.L - p.q.n;
            // page and old score, on their way while the rows are summed
            int page = -1;
            if (whole) page = w.table[(size_t)p.s * w.width + (key >> w.page_shift)];
            const bool there = page >= 0 && page < w.num_pages;
            const long long e = (((long long)page * w.Hkv + p.h) << w.page_shift) + (key & ((1 << w.page_shift) - 1));
            float old = 0.f;
            if (there && !fresh && w.decay != 0.f) old = w.scores[e];
            uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
            const int rows = rows_of(w, p.q);
            for (int j = p.b0; j < p.b1; ++j, ++n) {
                const int buf = n & 1, sr = n % kR, cols = columns_of(min(rows - j * kTileRows, kTileRows));
                ok = mbar_wait(&b.rfull[sr], (n / kR) & 1, &b.err);
                ok = mbar_wait(&b.sfull[half][buf], (n >> 1) & 1, &b.err) && ok;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (live) {
                    const bool open = last <= min(b.all[sr][0], b.all[sr][1]);    // every row sees all of the half's keys
#pragma unroll
                    for (int i = 0; i < kTileRows / 2; i += 32) {
                        const int c = part * (kTileRows / 2) + i;
                        if (c >= cols) break;
                        float x[32];
                        tmem_ld32(lanes + buf * kTileRows + i, x);
                        tmem_ld_wait();
                        // (columns behind the block's, where it has an odd number of sixteens, are old ones: masked)
                        if (open && c + 32 <= cols) weigh32<false>(x, &b.limit[sr][c], key, sc2, sum);
                        else weigh32<true>(x, &b.limit[sr][c], key, sc2, sum);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&b.sempty[half][buf]);
                    mbar_arrive(&b.rempty[sr]);
                }
            }
            if (!ok) break;
            float x, y, z;
            f2_unpack(f2_add(sum[0], sum[1]), x, y);
            z = x + y;
            if (part == 1) {
                ok = __all_sync(0xffffffffu, mbar_wait(&b.pempty[pair], (pieces & 1) ^ 1, &b.err));
                if (!ok) break;
                b.other[in_tile] = z;
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.pfull[pair]);
            } else {
                ok = __all_sync(0xffffffffu, mbar_wait(&b.pfull[pair], pieces & 1, &b.err));
                if (!ok) break;
                z += b.other[in_tile];
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.pempty[pair]);
                if (p.slot >= 0) part_of(w, blockIdx.x, p.slot)[in_tile] = z;
                else if (there) {
                    w.out[e] = !fresh && w.decay != 0.f ? fmaf(w.decay, old, z) : z;
                    if (fresh && w.positions) w.positions[e] = key + (w.dropped ? w.dropped[p.s] : 0);
                } else if (whole) {
                    atomicOr(w.err, (unsigned)kDevErrPagedArg);
                }
            }
            ++pieces;
        }
        if (tid == 0) w.hdr[blockIdx.x] = WeighHeader{ok && p.slot == 1 ? p.parts : 0, p.s, p.h, p.t};
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSum / 32) {
        __syncwarp();
        tmem_dealloc(tm, 512);
    }
    if (tid == 0 && b.err) atomicOr(w.err, (unsigned)kDevErrMbarTimeout);
}

template <int D>
cudaError_t launch_one(const Args& a, const CUtensorMap& mk, const CUtensorMap& mq, cudaStream_t stream) {
    constexpr size_t smem = Shape<D>::smem;
    cudaError_t e = cudaFuncSetAttribute(weigh_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return paged::launch_after(weigh_tc_kernel<D>, dim3(a.w.ctas), kThreads, smem, stream, a, mk, mq);
}

}  // namespace
}  // namespace weigh

bool weigh_tc_fits(const WeighProblem& p) {
    // 32 sequences of 300 to 6000 keys, four key heads (us, this kernel and lla_weigh.cu's): 12 rows d = 128 33 and 28, 20 rows 32 and
    // 49; at d = 64 16 rows 29 and 22, 20 rows 29 and 27; 64 x 8 key heads at 3000 to 4096 keys, 32 rows, d = 128 87 and 157
    return p.dtype == LLA_DTYPE_BF16 && ((p.d == 128 && most_rows(p) > 16) || (p.d == 64 && most_rows(p) > 32));
}

WeighSplit weigh_tc_split(const WeighProblem& p, int sms) {
    (void)p;
    return WeighSplit{weigh::kTile, paged::kTileRows, sms, 1};
}

cudaError_t launch_weigh_tc(const WeighProblem& p, const WeighSplit& sp, cudaStream_t stream, const char** why) {
    PagedProblem c{};                              // what the tensor maps are made of
    c.T = p.T; c.Hq = p.Hq; c.Hkv = p.Hkv; c.G = p.G; c.d = p.d; c.page_shift = p.page_shift; c.num_pages = p.num_pages;
    c.page_stride = p.page_stride;
    CUtensorMap mk = {}, mq = {};
    // a box: no more rows than any sequence has (32 rows beside 256 keys: 21.2 us with 128, 20.9)
    int boxes = paged::kTileRows % p.G ? 0 : paged::kTileRows;
    while (boxes / 2 >= most_rows(p) && boxes / 2 >= 16 && boxes / 2 >= p.G) boxes /= 2;
    if (!paged::make_cache_map(&mk, p.k, c) || (boxes && !paged::make_rows_map(&mq, p.q, p.q_stride, c, boxes))) {
        *why = "tensor map of a paged call";
        return cudaErrorInvalidValue;
    }
    const float scale = p.tau * 1.4426950408889634f;
    const double inv = 1.4426950408889634074 / scale;
    weigh::Args a{weigh::make_work(p, sp), static_cast<const __nv_bfloat16*>(p.q), p.lse, p.Hq, (int)paged::slices_of_page(c),
                  p.q_stride, scale, (float)inv, (float)(inv - (double)(float)inv), boxes};
    return p.d == 128 ? weigh::launch_one<128>(a, mk, mq, stream) : weigh::launch_one<64>(a, mk, mq, stream);
}

}  // namespace lla
