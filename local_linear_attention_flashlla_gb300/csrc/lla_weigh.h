// Shared by the translation units of paged_weigh (include/lla.h): the problem, and the division of its work.
//
// A tile is KT keys of a (sequence, key head); its work is the blocks of RB query rows that see any of them, and a unit is one
// of these (and `extra` more for a tile's start and end).  All units of a call, in the order (sequence, key head, tile,
// block), are dealt to the CTAs in contiguous ranges of equal length.  A key's score is the sum over its tile's blocks: a
// tile that a range border cuts leaves partial sums, KT floats, which weigh_join_kernel adds in the order of the CTAs.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "lla_paged.h"

namespace lla {

struct WeighProblem {
    const void* q;            // [T, Hq, d], token stride q_stride elements
    const float* lse;         // [T, Hq]
    const void* k;            // [num_pages, Hkv, page, d], page stride page_stride elements
    const float* scores;      // [num_pages, Hkv, page]
    float* out;               // the same, or scores
    int* positions;           // or null
    const int* dropped;       // or null
    const int* table;
    const int* cu_q;
    const int* kv_lens;
    const int* granted;       // or null
    int T, S, Hq, Hkv, G, d, page_shift, num_pages, width, max_new, last, causal, dtype;
    long long q_stride, page_stride;
    float tau, decay;
    unsigned* err;
    void* ws;
};

// The most rows that count which a sequence has to a key head.
inline long long most_rows(const WeighProblem& p) { return (long long)(p.last > 0 && p.last < p.max_new ? p.last : p.max_new) * p.G; }

struct WeighHeader {
    int parts;      // 0: this CTA starts no tile that others finish; else CTAs that share it
    int s, h, tile;
};

struct WeighSplit {
    int keys, rows, ctas, extra;      // KT, RB (KT a multiple of RB, powers of two), CTAs
};
inline size_t weigh_workspace_bytes(const WeighSplit& sp) {
    return (size_t)kPagedMaxCtas * sizeof(WeighHeader) + (size_t)sp.ctas * 2 * sp.keys * sizeof(float);
}

// bf16, d in {64, 128}, many rows: lla_weigh_tc.cu.  Everything else: lla_weigh.cu.
bool weigh_tc_fits(const WeighProblem& p);
WeighSplit weigh_tc_split(const WeighProblem& p, int sms);
cudaError_t launch_weigh_tc(const WeighProblem& p, const WeighSplit& sp, cudaStream_t stream, const char** why);
WeighSplit weigh_mma_split(const WeighProblem& p, int sms);
cudaError_t launch_weigh_mma(const WeighProblem& p, const WeighSplit& sp, cudaStream_t stream);
cudaError_t launch_weigh_join(const WeighProblem& p, const WeighSplit& sp, cudaStream_t stream);

#ifdef __CUDACC__
namespace weigh {

struct Work {
    const int* table;
    const int* cu_q;
    const int* kv_lens;
    const float* scores;
    float* out;
    int* positions;
    const int* dropped;
    int T, S, Hkv, G, width, page_shift, num_pages, max_new, last, causal;
    int ctas;
    signed char extra, keys_shift, rows_shift;      // (three ints: 64 x 8 key heads with 32 rows 92 us for 87)
    float decay;
    paged::Divisor g;
    const int* granted;       // or null
    WeighHeader* hdr;         // [kPagedMaxCtas], then parts [ctas][2][KT]: slot 0 a tile that an earlier CTA starts, 1 one that others finish
    unsigned* err;
};

inline Work make_work(const WeighProblem& p, const WeighSplit& sp) {
    Work w;
    w.table = p.table; w.cu_q = p.cu_q; w.kv_lens = p.kv_lens; w.granted = p.granted;
    w.scores = p.scores; w.out = p.out; w.positions = p.positions;
    w.dropped = p.dropped; w.T = p.T; w.S = p.S; w.Hkv = p.Hkv; w.G = p.G; w.width = p.width; w.page_shift = p.page_shift;
    w.num_pages = p.num_pages; w.max_new = p.max_new; w.last = p.last; w.causal = p.causal;
    w.ctas = sp.ctas; w.extra = (signed char)sp.extra; w.keys_shift = (signed char)paged::log2_up(sp.keys); w.rows_shift = (signed char)paged::log2_up(sp.rows);
    w.decay = p.decay;
    w.g = paged::make_divisor(p.G);
    w.hdr = static_cast<WeighHeader*>(p.ws);
    w.err = p.err;
    return w;
}

__device__ __forceinline__ int over_g(const Work& w, int x) { return (int)paged::over(w.g, (unsigned)x); }

// A sequence, cut to what the tensors hold (and reported where it had to be), without rows where it was refused: its tokens from
// token0 on, those that count from token0 + first on (the last `last` of them), rows = (n - first) G of them to a key head.
struct Seq {
    int token0, n, first, L;
};
__device__ __forceinline__ Seq load_seq(const Work& w, int s) {
    const int c0 = w.cu_q[s], c1 = w.cu_q[s + 1], kv = w.kv_lens[s];
    const bool refused = w.granted && w.granted[s] == 0;
    Seq q;
    q.token0 = min(max(c0, 0), w.T);
    const int end = min(max(c1, q.token0), w.T);
    q.n = min(end - q.token0, w.max_new);
    q.L = min(max(kv, 0), w.width << w.page_shift);
    q.first = w.last > 0 ? max(q.n - w.last, 0) : 0;
    if (q.token0 != c0 || q.token0 + q.n != c1 || q.L != kv) atomicOr(w.err, (unsigned)kDevErrPagedArg);
    if (refused) q.n = 0;                            // no rows: no tiles
    return q;
}
__device__ __forceinline__ int rows_of(const Work& w, const Seq& q) { return (q.n - q.first) * w.G; }
__device__ __forceinline__ int tiles_of(const Work& w, const Seq& q) {
    return q.n > 0 ? (q.L + (1 << w.keys_shift) - 1) >> w.keys_shift : 0;
}
__device__ __forceinline__ int blocks_of(const Work& w, const Seq& q) {
    return (rows_of(w, q) + (1 << w.rows_shift) - 1) >> w.rows_shift;
}
// Keys that counted token i sees.
__device__ __forceinline__ int keys_seen(const Work& w, const Seq& q, int i) {
    return w.causal ? min(max(q.L - q.n + q.first + i + 1, 0), q.L) : q.L;
}
// The first block that holds a row which sees any key of tile t (t < tiles): in causal attention token i, counted from
// the first that counts, sees key t KT if i >= t KT - off, off = L - n + first.  KT is a multiple of RB, so the block is
// floor((t KT - off) G / RB) = t (KT / RB) G + floor(-off G / RB).
__device__ __forceinline__ int first_block(const Work& w, const Seq& q, int t) {
    if (!w.causal) return 0;
    const long long row = ((long long)(t << w.keys_shift) - (q.L - q.n + q.first)) * w.G;
    if (row <= 0) return 0;
    const int blocks = blocks_of(w, q);
    const long long b = row >> w.rows_shift;
    return b < blocks ? (int)b : blocks - 1;         // (not reached: the last row sees every key)
}
__device__ __forceinline__ int tile_units(const Work& w, const Seq& q, int t) {
    return blocks_of(w, q) - first_block(w, q, t) + w.extra;
}
// Units of the first x tiles of a key head.
__device__ __forceinline__ long long units_before(const Work& w, const Seq& q, int x) {
    long long u = (long long)x * (blocks_of(w, q) + w.extra);
    if (w.causal) {
        const long long off = q.L - q.n + q.first;
        const long long t1 = off < 0 ? 0 : (off >> w.keys_shift) + 1;       // the first tile whose first key lies behind off
        if (x > t1) {
            const long long per = (long long)w.G << (w.keys_shift - w.rows_shift);
            u -= per * ((long long)x * (x - 1) / 2 - t1 * (t1 - 1) / 2) + (x - t1) * ((-off * w.G) >> w.rows_shift);
        }
    }
    return u;
}
__device__ __forceinline__ long long head_units(const Work& w, const Seq& q) { return units_before(w, q, tiles_of(w, q)); }

// A CTA's place in the order of units.
struct Walk {
    long long u, end, share;
    int over;                 // the first `over` ranges have one unit more
    int s, h, t, j;           // sequence, key head, tile, unit of the tile
    Seq q;
};

constexpr int kMostWarps = 20;

// Range of CTA blockIdx.x and the tile it begins in.  Every thread of the block calls it; sh: 40 long longs; blockDim.x is
// a multiple of 32 and at most 32 kMostWarps.
__device__ inline Walk begin_walk(const Work& w, long long* sh) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, cta = blockIdx.x;
    const int per = (w.S + nt - 1) / nt, s0 = min(tid * per, w.S), s1 = min(s0 + per, w.S);
    Walk k;
    k.s = k.h = k.t = k.j = 0;
    k.u = k.end = 0;
    k.q.token0 = k.q.n = k.q.first = k.q.L = 0;
    long long mine = 0, total;
    for (int s = s0; s < s1; ++s) {
        k.q = load_seq(w, s);
        mine += head_units(w, k.q) * w.Hkv;
    }
    long long pre = paged::block_scan<kMostWarps>(mine, sh, &total) - mine;
    const int active = (int)(total < w.ctas ? total : w.ctas);
    if (cta >= active) return k;
    k.share = paged::div_units(total, active);
    k.over = (int)(total - k.share * active);
    k.u = cta * k.share + min(cta, k.over);
    k.end = k.u + k.share + (cta < k.over);
    int* at = reinterpret_cast<int*>(sh + 32);
    if (k.u >= pre && k.u < pre + mine) {
        int s = s0;
        for (; s + 1 < s1; ++s) {
            const long long u = head_units(w, load_seq(w, s)) * w.Hkv;
            if (k.u < pre + u) break;
            pre += u;
        }
        sh[36] = pre;
        at[0] = s;
    }
    __syncthreads();
    k.s = at[0];
    k.q = load_seq(w, k.s);
    long long rem = k.u - sh[36];
    const long long unit = head_units(w, k.q);
    if (unit > 0) {
        k.h = (int)paged::div_units(rem, unit);
        rem -= k.h * unit;
        int lo = 0;                                  // the last tile with units_before <= rem: 32 probes at a time
        const int tiles = tiles_of(w, k.q);
        for (int range = tiles; range > 1;) {
            const int step = (range + 31) >> 5, probe = lo + lane * step;
            const bool yes = lane * step < range && units_before(w, k.q, probe) <= rem;
            lo += (__popc(__ballot_sync(0xffffffffu, yes)) - 1) * step;
            range = min(step, tiles - lo);
        }
        k.t = lo;
        k.j = (int)(rem - units_before(w, k.q, lo));
    }
    if (k.j <= w.extra) {                            // within the extra units: the tile is this CTA's from its start
        k.u -= k.j;
        k.j = 0;
    }
    return k;
}

// The next piece: blocks [b0, b1) of a tile.  slot: -1 the whole tile, else the slot of its partial sums.
struct Piece {
    int s, h, t, b0, b1, slot, parts;
    Seq q;
};
__device__ __forceinline__ bool next_piece(const Work& w, Walk& k, Piece& p) {
    if (k.u >= k.end) return false;
    const int units = tile_units(w, k.q, k.t), f = first_block(w, k.q, k.t);
    const long long left = k.end - k.u;
    const int take = (int)(left < units - k.j ? left : units - k.j);
    if (k.j == 0 && take <= w.extra) return false;   // the border lies in the tile's extra units: the next CTA's
    p.s = k.s; p.h = k.h; p.t = k.t; p.q = k.q;
    p.b0 = f + max(k.j - w.extra, 0);
    p.b1 = f + k.j + take - w.extra;
    const bool first = k.j == 0, last = k.j + take == units;
    p.slot = first && last ? -1 : first ? 1 : 0;
    p.parts = 0;
    if (p.slot == 1) {
        const long long u = k.u + units - 1, big = k.over * (k.share + 1);     // the tile's last unit, and whose it is
        const int cta = u < big ? (int)paged::div_units(u, k.share + 1) : k.over + (int)paged::div_units(u - big, k.share);
        p.parts = cta - (int)blockIdx.x + 1;
    }
    k.u += take;
    k.j += take;
    if (k.j == units) {
        k.j = 0;
        if (++k.t == tiles_of(w, k.q)) {
            k.t = 0;
            if (++k.h == w.Hkv) {
                k.h = 0;
                if (k.u < k.end) {
                    do {
                        if (++k.s >= w.S) {          // lengths that changed during the call
                            k.end = k.u;
                            break;
                        }
                        k.q = load_seq(w, k.s);
                    } while (tiles_of(w, k.q) == 0);
                }
            }
        }
    }
    return true;
}

// Score of key `key` of a tile whose rows gave it the weight x.
__device__ __forceinline__ void put_score(const Work& w, const Seq& q, int s, int h, int key, float x) {
    if (key >= q.L) return;
    const int page = w.table[(size_t)s * w.width + (key >> w.page_shift)];
    if (page < 0 || page >= w.num_pages) {
        atomicOr(w.err, (unsigned)kDevErrPagedArg);
        return;
    }
    const long long e = (((long long)page * w.Hkv + h) << w.page_shift) + (key & ((1 << w.page_shift) - 1));
    const bool fresh = w.causal && key >= q.L - q.n;
    if (!fresh && w.decay != 0.f) x = fmaf(w.decay, w.scores[e], x);
    w.out[e] = x;
    if (fresh && w.positions) w.positions[e] = key + (w.dropped ? w.dropped[s] : 0);
}

__device__ __forceinline__ float* part_of(const Work& w, int cta, int slot) {
    return reinterpret_cast<float*>(w.hdr + kPagedMaxCtas) + (((size_t)cta * 2 + slot) << w.keys_shift);
}

}  // namespace weigh
#endif

}  // namespace lla
