// Shared by the paged-cache translation units: the problem description, the division of ragged
// (sequence, key head, row tile) work among a fixed number of CTAs, and the partial results of tiles
// that several CTAs share.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lla {

// lla_paged_parallax arguments after validation (include/lla.h describes them).
struct PagedProblem {
    const void* q;            // [T, Hq, d], token stride q_stride
    const void* probe;        // [T, Hq, d], token stride r_stride
    const void* k;            // [num_pages, Hkv, page, d], page stride page_stride
    const void* v;
    const int* table;         // [S, width]
    const int* cu_q;          // [S + 1]
    const int* kv_lens;       // [S]
    void* out;                // [T, Hq, d] contiguous
    float* lse;               // [T, Hq], or null
    int T, S, Hq, Hkv, G, d, page_shift, num_pages, width, max_new;
    long long q_stride, r_stride, page_stride;   // elements
    float tau;
    int causal, dtype;
    unsigned* err;            // device error word
    void* ws;                 // partial results (paged_workspace_bytes)
};

// A row tile of a (sequence, key head): rows [tile R, (tile + 1) R) of its nq * G query rows, where
// row r is token r / G and query head h G + r % G.  A tile's work is its key blocks; a unit is one of
// them.  All units of a call, in the order (sequence, key head, tile, block), are dealt to the CTAs in
// contiguous ranges of equal length, whatever the lengths of the sequences: a tile that a range border
// cuts is finished by merging its parts (paged_merge).
struct PartHeader {
    int parts;      // 0: this CTA starts no tile that others finish; else CTAs that share it
    int row0;       // first row (in the flat row space of its sequence: token * G + head in group)
    int rows;       // rows of the tile
    int token0;     // row of q / out that holds token 0 of the sequence
    int head;       // key head
    int pad[3];
};

constexpr int kPagedMaxCtas = 1024;

// Partials: per CTA two slots (0: the tile whose earlier blocks another CTA has, 1: the tile whose
// later blocks another CTA has); a slot holds rows x { m, omega, A, s0 } and rows x 2 x d sums.
inline size_t paged_part_floats(int rows, int d) { return (size_t)rows * (4 + 2 * (size_t)d); }
inline size_t paged_workspace_bytes(int ctas, int rows, int d) {
    return (size_t)kPagedMaxCtas * sizeof(PartHeader) + (size_t)ctas * 2 * paged_part_floats(rows, d) * sizeof(float);
}

// How a path divides the work: rows of a tile, keys of a block (powers of two, rows <= keys), CTAs.
struct PagedSplit {
    int rows, keys, ctas;
    int extra;      // units charged for a tile beside its blocks: what a tile costs before its first block and after its last
};

// bf16, d in {64, 128}, at most 32 query rows to a key head (max_new * G); fp32, d in {32, 64}: lla_paged_decode.cu.
bool paged_decode_fits(const PagedProblem& p, int path);
PagedSplit paged_decode_split(const PagedProblem& p, int sms);
cudaError_t launch_paged_decode(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream, const char** why);
// bf16, d in {64, 128}, any number of rows: lla_paged_tc.cu.
PagedSplit paged_tc_split(const PagedProblem& p, int sms);
cudaError_t launch_paged_tc(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream, const char** why);
PagedSplit paged_simt_split(const PagedProblem& p, int sms);
cudaError_t launch_paged_simt(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream);
cudaError_t launch_paged_merge(const PagedProblem& p, const PagedSplit& sp, cudaStream_t stream);

#ifdef __CUDACC__
namespace paged {

// Launches with programmatic stream serialisation: the grid may be set up while the kernel before it still
// runs, and waits for that kernel's end in cudaGridDependencySynchronize before it reads anything.
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Division of x < 2^31 by a number known on the host: multiplication with the rounded-up reciprocal (T. Granlund and
// P. Montgomery, Division by Invariant Integers using Multiplication, 1994).
struct Divisor {
    unsigned mul, shift;
};
inline int log2_up(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}
inline Divisor make_divisor(int d) {
    const unsigned s = (unsigned)log2_up(d);
    return Divisor{(unsigned)((((1ull << 32) * ((1ull << s) - (unsigned)d)) / (unsigned)d) + 1), s};
}

// What a kernel needs of the problem, by value.
struct Work {
    const int* table;
    const int* cu_q;
    const int* kv_lens;
    int T, S, Hkv, G, width, page_shift, num_pages, max_new, causal;
    int rows, keys, ctas, extra;
    int keys_shift, rows_shift;       // their log2; rows <= keys
    Divisor g, m;                     // G, and keys / rows * G
    PartHeader* hdr;
    float* part;
    unsigned* err;
};

inline Work make_work(const PagedProblem& p, const PagedSplit& sp) {
    Work w;
    w.table = p.table; w.cu_q = p.cu_q; w.kv_lens = p.kv_lens;
    w.T = p.T; w.S = p.S; w.Hkv = p.Hkv; w.G = p.G; w.width = p.width; w.page_shift = p.page_shift;
    w.num_pages = p.num_pages; w.max_new = p.max_new; w.causal = p.causal;
    w.rows = sp.rows; w.keys = sp.keys; w.ctas = sp.ctas;
    w.extra = sp.extra;
    w.keys_shift = log2_up(sp.keys);
    w.rows_shift = log2_up(sp.rows);
    w.g = make_divisor(p.G);
    w.m = make_divisor(sp.keys / sp.rows * p.G);
    w.hdr = static_cast<PartHeader*>(p.ws);
    w.part = reinterpret_cast<float*>(static_cast<char*>(p.ws) + (size_t)kPagedMaxCtas * sizeof(PartHeader));
    w.err = p.err;
    return w;
}

__device__ __forceinline__ unsigned over(const Divisor& d, unsigned x) {
    return (__umulhi(d.mul, x) + x) >> d.shift;
}
__device__ __forceinline__ int over_g(const Work& w, int x) { return (int)over(w.g, (unsigned)x); }

// a / b for 0 <= a, 0 < b; a 32-bit division where both fit (they nearly always do).
__device__ __forceinline__ long long div_units(long long a, long long b) {
    if (((unsigned long long)(a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
    return a / b;
}

// A sequence as the kernels see it: lengths outside what the tensors hold are cut to it and reported
// through the device error word, so that no later index can leave them.
struct Seq {
    int token0, nq, L;
};

__device__ __forceinline__ Seq load_seq(const Work& w, int s) {
    const int c0 = w.cu_q[s], c1 = w.cu_q[s + 1], kv = w.kv_lens[s];
    Seq q;
    q.token0 = min(max(c0, 0), w.T);
    const int end = min(max(c1, q.token0), w.T);
    q.nq = min(end - q.token0, w.max_new);
    q.L = min(max(kv, 0), w.width << w.page_shift);
    if (q.token0 != c0 || q.token0 + q.nq != c1 || q.L != kv) atomicOr(w.err, (unsigned)kDevErrPagedArg);
    return q;
}

// sum_{x < X} floor(x / m) = m q (q - 1) / 2 + q r, X = q m + r, for m = keys / rows * G.
__device__ inline long long quotient_sum(const Work& w, unsigned X) {
    const unsigned m = (unsigned)((w.keys >> w.rows_shift) * w.G), q = over(w.m, X), r = X - q * m;
    return (long long)((unsigned long long)q * (q - 1) / 2 * m + (unsigned long long)q * r);
}

__device__ __forceinline__ int tiles_of(const Work& w, const Seq& q) { return (q.nq * w.G + w.rows - 1) >> w.rows_shift; }

// Keys that the rows of tile i see, at most (the last row's); 0 if none.
__device__ __forceinline__ int tile_keys(const Work& w, const Seq& q, int i) {
    if (!w.causal) return q.L;
    const int last = over_g(w, min((i + 1) * w.rows, q.nq * w.G) - 1);
    return min(max(q.L - q.nq + last + 1, 0), q.L);
}

// Units charged for tile i: its blocks (>= 1: a tile without keys still has its rows to write) and the extra ones,
// which come first.  A causal sequence
// with fewer keys than tokens is charged as if it had as many.
__device__ __forceinline__ int tile_units(const Work& w, const Seq& q, int i) {
    if (!w.causal) return max(1, (q.L + w.keys - 1) >> w.keys_shift) + w.extra;
    const int last = over_g(w, min((i + 1) * w.rows, q.nq * w.G) - 1);
    return ((max(q.L - q.nq, 0) + last) >> w.keys_shift) + 1 + w.extra;
}

// Units of the first n tiles of one key head (n <= tiles).
__device__ inline long long units_before(const Work& w, const Seq& q, int n) {
    if (n == 0) return 0;
    if (!w.causal) return (long long)n * tile_units(w, q, 0);
    const int tiles = tiles_of(w, q);
    long long u = 0;
    int full = n;
    if (n == tiles) {
        u = tile_units(w, q, n - 1);
        --full;
    }
    if (full > 0) {
        // tile i: floor((c0 G + rows (i + 1) - 1) / (keys G)) + 1 = floor((i + b) / (keys / rows G)) + 1 units, rows and
        // keys being powers of two
        const unsigned b = ((unsigned)max(q.L - q.nq, 0) * w.G + w.rows - 1) >> w.rows_shift;
        u += (long long)full * (1 + w.extra) + quotient_sum(w, b + full) - quotient_sum(w, b);
    }
    return u;
}

// Units of one key head of a sequence.
__device__ __forceinline__ long long head_units(const Work& w, const Seq& q) {
    return q.nq > 0 ? units_before(w, q, tiles_of(w, q)) : 0;
}

// A position in the order of units.
struct Walk {
    int cta;              // whose range it is (a CTA, or a pair of them)
    long long u, end;     // next unit of this CTA, end of its range
    long long share;      // units of a CTA's range; the first `over` ranges have one more
    int over, active;     // active: CTAs that have work
    int s, h, i, j;       // sequence, key head, tile, block
    Seq q;
};

// First unit of range c, and the range that holds unit u.
__device__ __forceinline__ long long range_start(const Walk& k, int c) { return c * k.share + min(c, k.over); }
__device__ __forceinline__ int range_of(const Walk& k, long long u) {
    const long long big = k.over * (k.share + 1);        // units of the longer ranges
    return u < big ? (int)div_units(u, k.share + 1) : k.over + (int)div_units(u - big, k.share);
}

// A range border within a tile's extra units counts as lying before the tile: who ends there leaves the tile, who
// begins there takes all of it, so that no piece is without blocks for that reason.
__device__ __forceinline__ void snap_start(const Work& w, Walk& k) {
    if (k.j <= w.extra) {
        k.u -= k.j;
        k.j = 0;
    }
}

constexpr int kMostWarps = 12;       // of a block that divides work

// Inclusive sum of v over the block's threads in thread order; *all: the block's total.  sh: 32 long longs.  NW: the most warps.
template <int NW = kMostWarps>
__device__ __forceinline__ long long block_scan(long long v, long long* sh, long long* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    long long sum = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const long long t = i < nw ? sh[i] : 0;
        if (i < warp) v += t;
        sum += t;
    }
    *all = sum;
    __syncthreads();
    return v;
}

// Units of the longest tile of a sequence.
__device__ __forceinline__ int longest_tile(const Work& w, const Seq& q) {
    return q.nq > 0 ? tile_units(w, q, tiles_of(w, q) - 1) : 0;
}

// log2 of the least units worth a CTA: a tile of B units cut into parts of m takes m blocks one after another (0.7 us
// each for decode tiles) and the join of B / m parts (0.08 us each), least at m = sqrt(B / 9); a power of two
// beside it.  One sequence, two key heads, one token: 200 to 1000 keys 8.3 us where m = 4 takes 10 and m = 8
// takes 9 to 13; 8000 keys 11.0 where m = 1 takes 15; 32,768 keys 16.3 where m = 4 takes 18.  The other kernels' blocks
// and joins both cost more: 64 tokens over 500 keys (128-row tiles) 16.6 us where m = 4 takes 19, a prompt of 300 tokens
// 15.8 and 14.7, 32 rows over 500 keys on CUDA cores 10.3 where m = 2 takes 13.6, over 4000 keys 20.5 and 18.5.
__device__ __forceinline__ int least_shift(int longest) { return (32 - __clz(longest / 9 | 1)) / 2; }

// CTA cta's range of `total` units; false: it has none.
__device__ __forceinline__ bool set_range(const Work& w, Walk& k, int cta, long long total, int longest) {
    const int shift = least_shift(longest);
    const long long most = (total + (1 << shift) - 1) >> shift;
    k.active = (int)(most < w.ctas ? most : w.ctas);
    if (cta >= k.active) return false;
    k.share = div_units(total, k.active);
    k.over = (int)(total - k.share * k.active);
    k.u = range_start(k, cta);
    k.end = range_start(k, cta + 1);
    return true;
}

// The tile and block of a walk whose next unit is the rem-th of its sequence, `unit` units to a key head.
__device__ __forceinline__ Walk find_tile(const Work& w, Walk k, long long rem, long long unit) {
    const int lane = threadIdx.x & 31, tiles = tiles_of(w, k.q);
    k.h = (int)div_units(rem, unit);
    rem -= k.h * unit;
    if (tiles > 1) {
        int lo = 0;                                // the last tile with units_before <= rem: 32 probes at a time
        for (int range = tiles; range > 1;) {
            const int step = (range + 31) >> 5, probe = lo + lane * step;
            const bool yes = lane * step < range && units_before(w, k.q, probe) <= rem;
            lo += (__popc(__ballot_sync(0xffffffffu, yes)) - 1) * step;
            range = min(step, tiles - lo);
        }
        k.i = lo;
        rem -= units_before(w, k.q, lo);
    }
    k.j = (int)rem;
    snap_start(w, k);
    return k;
}

// Range of CTA `cta` and the tile it begins in.  Every thread of the block calls it; the shared scratch is
// 40 long longs.  active = 0: no units at all.  blockDim.x is a multiple of 32.  A thread sums a run of
// consecutive sequences, so that one scan finds the total and, with it, whose sequence the range begins in.
__device__ inline Walk begin_walk(const Work& w, int cta, long long* sh) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
    const int per = (w.S + nt - 1) / nt, s0 = min(tid * per, w.S), s1 = min(s0 + per, w.S);
    Walk k;
    k.cta = cta;
    k.s = k.h = k.i = k.j = 0;
    k.q.token0 = k.q.nq = k.q.L = 0;
    k.u = k.end = 0;
    int longest = 0;
    long long mine = 0, unit = 0, total;           // unit: of a key head of the last sequence looked at
    if (w.S <= 32) {
        // a lane to a sequence, every warp for itself: no barrier
        Seq q;
        q.token0 = q.nq = q.L = 0;
        if (lane < w.S) {
            q = load_seq(w, lane);
            unit = head_units(w, q);
            mine = unit * w.Hkv;
            longest = longest_tile(w, q);
        }
        long long inc = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        total = __shfl_sync(0xffffffffu, inc, 31);
        if (!set_range(w, k, cta, total, (int)__reduce_max_sync(0xffffffffu, (unsigned)longest))) return k;
        const unsigned here = __ballot_sync(0xffffffffu, k.u >= inc - mine && k.u < inc);
        const int s = __ffs((int)here) - 1;
        k.s = s;
        k.q.token0 = __shfl_sync(0xffffffffu, q.token0, s);
        k.q.nq = __shfl_sync(0xffffffffu, q.nq, s);
        k.q.L = __shfl_sync(0xffffffffu, q.L, s);
        unit = __shfl_sync(0xffffffffu, unit, s);
        return find_tile(w, k, k.u - __shfl_sync(0xffffffffu, inc - mine, s), unit);
    }
    for (int s = s0; s < s1; ++s) {
        k.q = load_seq(w, s);
        unit = head_units(w, k.q);
        mine += unit * w.Hkv;
        longest = max(longest, longest_tile(w, k.q));
    }
    unsigned* most = reinterpret_cast<unsigned*>(sh + kMostWarps);        // a warp's longest tile, behind the scan's sums
    longest = (int)__reduce_max_sync(0xffffffffu, (unsigned)longest);
    if (lane == 0) most[tid >> 5] = (unsigned)longest;
    long long pre = block_scan(mine, sh, &total) - mine;
    for (int i = 0; i < (nt + 31) >> 5; ++i) longest = max(longest, (int)most[i]);
    if (!set_range(w, k, cta, total, longest)) return k;
    int* at = reinterpret_cast<int*>(sh + 32);     // sequence, token0, nq, L
    if (k.u >= pre && k.u < pre + mine) {
        int s = s0;
        if (per > 1) {
            for (; s + 1 < s1; ++s) {
                const long long u = head_units(w, load_seq(w, s)) * w.Hkv;
                if (k.u < pre + u) break;
                pre += u;
            }
            k.q = load_seq(w, s);
            unit = head_units(w, k.q);
        }
        sh[36] = pre;
        sh[37] = unit;
        at[0] = s;
        at[1] = k.q.token0;
        at[2] = k.q.nq;
        at[3] = k.q.L;
    }
    __syncthreads();
    k.s = at[0];
    k.q.token0 = at[1];
    k.q.nq = at[2];
    k.q.L = at[3];
    return find_tile(w, k, k.u - sh[36], sh[37]);
}

// The CTA's next piece of work: blocks [j0, j1) of a tile.
struct Piece {
    int s, h, i;
    Seq q;
    int row0, rows;       // flat rows of the tile
    int keys;             // keys that the tile's last row sees
    int j0, j1;           // blocks that hold any of them
    int slot;             // -1: the whole tile is this CTA's; 0, 1: partial slot
    int parts;            // slot 1: CTAs that share the tile
};

__device__ __forceinline__ bool next_piece(const Work& w, Walk& k, Piece& p) {
    if (k.u >= k.end) return false;
    const int units = tile_units(w, k.q, k.i);
    const long long left = k.end - k.u;
    const int take = (int)(left < units - k.j ? left : units - k.j);
    if (k.j == 0 && take <= w.extra) return false;       // the border lies in the tile's extra units
    p.s = k.s; p.h = k.h; p.i = k.i; p.q = k.q;
    p.row0 = k.i * w.rows;
    p.rows = min(w.rows, k.q.nq * w.G - p.row0);
    p.keys = tile_keys(w, k.q, k.i);
    const int nb = (p.keys + w.keys - 1) >> w.keys_shift;
    p.j0 = min(max(k.j - w.extra, 0), nb);
    p.j1 = min(max(k.j + take - w.extra, 0), nb);
    const bool first = k.j == 0, last = k.j + take == units;
    p.slot = first && last ? -1 : first ? 1 : 0;
    p.parts = 0;
    if (p.slot == 1) {
        const long long tile_end = k.u + units;      // first unit behind the tile (k.j is 0)
        p.parts = range_of(k, tile_end - 1) - k.cta + 1;
    }
    k.u += take;
    k.j += take;
    if (k.j == units) {
        k.j = 0;
        if (++k.i == tiles_of(w, k.q)) {
            k.i = 0;
            if (++k.h == w.Hkv) {
                k.h = 0;
                if (k.u < k.end) {
                    do {
                        if (++k.s >= w.S) {           // lengths that changed during the call
                            k.end = k.u;
                            break;
                        }
                        k.q = load_seq(w, k.s);
                    } while (k.q.nq == 0);
                }
            }
        }
    }
    return true;
}

// A slot's parts: { m, omega, A, s0 } of each row, then the sums as float4 [2][d / 4][rows] (O1, then O2):
// the threads of a warp have a row each where it matters, and consecutive rows are consecutive in memory.
__device__ __forceinline__ float4* part_stats(const Work& w, int cta, int slot, int d) {
    return reinterpret_cast<float4*>(w.part) + ((size_t)cta * 2 + slot) * ((size_t)w.rows * (1 + d / 2));
}
__device__ __forceinline__ float4* part_sums(const Work& w, int cta, int slot, int d) {
    return part_stats(w, cta, slot, d) + w.rows;
}
// Element of the sums (half 0: O1, 1: O2) of a row's column.
__device__ __forceinline__ float* part_element(float4* sums, int rows, int d, int half, int row, int col) {
    return reinterpret_cast<float*>(sums + (size_t)(half * (d / 4) + col / 4) * rows + row) + col % 4;
}

// A row's logsumexp of its scaled logits, from its exponents' reference point (log2) and its weights' sum; a row that
// sees no key has m = -inf and om = 0, and gets -inf.
__device__ __forceinline__ void put_lse(const Work& w, float* lse, long long token, int head, float m, float om) {
    if (lse) lse[token * (w.Hkv * w.G) + head] = (m + log2f(om)) * 0.6931471805599453f;
}

// This CTA's header: written once by every CTA, with the tile that it starts and others finish (its
// last piece) or none.
__device__ __forceinline__ void write_header(const Work& w, int cta, const Piece& p, bool shared) {
    PartHeader h;
    h.parts = shared ? p.parts : 0;
    h.row0 = p.row0;
    h.rows = p.rows;
    h.token0 = p.q.token0;
    h.head = p.h;
    h.pad[0] = h.pad[1] = h.pad[2] = 0;
    w.hdr[cta] = h;
}

}  // namespace paged
#endif

}  // namespace lla
