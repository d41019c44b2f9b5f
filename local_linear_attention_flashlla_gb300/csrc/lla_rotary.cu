// Rotary positions of the heads' rows, with RMS normalisation and a gain before them, and the gradient of both.
//
//   u = gain x / sqrt(mean(x^2) + eps),   y = m Rot(position f) u on the first `rot` columns, y = u on the others
//   g = m Rot(-position f) dy,   h = g gain,   dx = rs (h - x rs^2 mean(h x)),   dgain = sum over rows of g x rs
//
// A frequency is a 64-bit fixed-point fraction of a turn per position, so position times frequency modulo one turn is an
// integer product whose overflow is the modulus: the angle of position 2^30 is as exact as that of position 1 (fp32
// products would be off by 2^-24 of the whole angle, thousands of turns).  Its upper 32 bits make the fp32 argument.
//
// Both directions are bound by the bytes of the rows: every row is read and written once, 16 bytes a lane at a time.  A
// lane holds two 16-byte pieces of a row, those whose columns turn together (half a rotary dimension apart, or
// neighbours), and a token's lanes compute its sines once for all heads that they take.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/lla.h"
#include "lla_internal.h"
#include "lla_paged.h"
#include "rotary_angle.h"

namespace lla {
namespace rotary {
namespace {

constexpr int kMost = LLA_ROTARY_MOST;      // tensors of a call
constexpr int kThreads = 256, kWarps = kThreads / 32;

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

struct Rows {
    const char* x;
    const char* dy;
    char* out;
    const float* gain;
    float* dgain;
    long long xs[3], dys[3], os[3];          // batch, head and position strides in bytes
    int heads;
};

struct Args {
    Rows rows[kMost];
    const int* positions;                    // [n], or [B, n]
    long long position_stride;               // 0 or n
    const long long* turns;                  // [rot / 2]: turns per position, 2^-64 of one each
    const int* cu_q;                         // [S + 1] and [S], or null
    const int* shift;
    float* part;                             // backward: [blocks][count][d] sums for the gains' gradients
    int count, B, n, S, rot, heads, split;   // heads: of all tensors; split: of them to a warp
    float magnitude, eps;                    // eps < 0: no normalisation
};

template <typename T>
struct Vec {
    static constexpr int N = 16 / (int)sizeof(T);      // elements of a piece
};

__device__ __forceinline__ void unpack(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// Sine and cosine of t 2^-32 turns.  The nearest quarter turn is taken off in integers, exactly; what is left, at most an eighth of
// a turn, has polynomials in x^2 of least largest absolute error (Remez): degree 7 for the sine, 8 for the cosine
// (2^-28.7 and 2^-29.1 with their coefficients in fp32), with the sums' fp32 roundings 2^-23.3 each.
__device__ __forceinline__ void sincos_turn(int t, float& s, float& c) {
    const unsigned q = ((unsigned)t + 0x20000000u) >> 30;                       // quarter turns, modulo 4
    const float x = (float)(int)((unsigned)t - (q << 30)) * 0x1.921fb6p-30f;    // 2 pi 2^-32
    const float z = x * x;
    float ps = fmaf(z, -0x1.98da66p-13f, 0x1.1105b4p-7f);
    ps = fmaf(z, ps, -0x1.555540p-3f);
    ps = fmaf(x * z, ps, x);
    float pc = fmaf(z, 0x1.993430p-16f, -0x1.6c087ep-10f);
    pc = fmaf(z, pc, 0x1.55553ep-5f);
    pc = fmaf(z, pc, -0.5f);
    pc = fmaf(z, pc, 1.f);
    const float ss = q & 1 ? pc : ps, cc = q & 1 ? ps : pc;
    s = q & 2 ? -ss : ss;
    c = (q + 1) & 2 ? -cc : cc;
}

// How a row's pieces lie in its lanes, and how its columns pair up.
//   kHalves  columns c and c + rot / 2 turn together, and half a rotary dimension is a whole number of pieces: a lane
//            holds two such pieces (or two neighbouring ones behind the rotary columns)
//   kPairs   columns 2 c and 2 c + 1 turn together: two neighbouring pieces
//   kStaged  as kHalves for any other rot: two neighbouring pieces, partners through shared memory
enum Form { kHalves, kPairs, kStaged };

template <typename T, int D, int F>
struct Lane {
    static constexpr int N = Vec<T>::N, NV = D / N, L = NV / 2;       // pieces and lanes of a row
    static constexpr int G = 32 / L;                                  // rows (tokens) of a warp
    static constexpr int A = F == kStaged ? 2 * N : N;                // angles of a lane
    static_assert(NV >= 2, "two pieces to a lane");
    int lane, piece[2];
    float c[A], s[A];

    static __device__ __forceinline__ int piece_of(int l, int p, int rot) {
        const int h = rot / 2 / N;
        return F != kHalves || l >= h ? 2 * l + p : l + p * h;       // behind the rotary columns: 2 h + 2 (l - h) + p
    }
    __device__ __forceinline__ void place(int l, int rot) {
        lane = l;
        piece[0] = piece_of(l, 0, rot);
        piece[1] = piece_of(l, 1, rot);
    }
    // sines and cosines of the lane's angles, times the magnitude; columns that do not turn have 1 and 0
    __device__ __forceinline__ void angles(const Args& a, long long position) {
#pragma unroll
        for (int i = 0; i < A; ++i) {
            int f = lane * N + i;
            if (F == kStaged) {
                f = lane * 2 * N + i;
                if (f >= a.rot / 2) f -= a.rot / 2;
                if (lane * 2 * N + i >= a.rot) f = a.rot;
            }
            c[i] = 1.f;
            s[i] = 0.f;
            if (2 * f < a.rot) {
                sincos_turn(turn_of(position, a.turns[f]), s[i], c[i]);
                c[i] *= a.magnitude;
                s[i] *= a.magnitude;
            }
        }
    }
    // y = m Rot x (sign 1) or m Rot^T x (sign -1), in place; stage: the row's D floats (kStaged)
    __device__ __forceinline__ void turn(float (&x)[2][N], float sign, int rot, float* stage) const {
        if (F == kHalves) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float u = x[0][i], v = x[1][i], t = sign * s[i];
                x[0][i] = fmaf(u, c[i], -v * t);
                x[1][i] = fmaf(v, c[i], u * t);
            }
        } else if (F == kPairs) {
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    const int k = p * (N / 2) + i;
                    const float u = x[p][2 * i], v = x[p][2 * i + 1], t = sign * s[k];
                    x[p][2 * i] = fmaf(u, c[k], -v * t);
                    x[p][2 * i + 1] = fmaf(v, c[k], u * t);
                }
        } else {
            __syncwarp();
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < N; ++i) stage[(lane * 2 + p) * N + i] = x[p][i];
            __syncwarp();
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int col = (lane * 2 + p) * N + i;
                    if (col < rot) {
                        const int k = p * N + i;
                        const bool low = col < rot / 2;
                        const float other = stage[low ? col + rot / 2 : col - rot / 2], t = sign * s[k % A];
                        x[p][i] = fmaf(x[p][i], c[k % A], low ? -other * t : other * t);
                    }
                }
        }
    }
};

// The position of token t of batch b, moved by what was evicted of its sequence.
__device__ __forceinline__ long long position_of(const Args& a, int b, int t) {
    long long p = a.positions[b * a.position_stride + t];
    if (a.shift) {
        int lo = 0, hi = a.S - 1;            // the last sequence that begins at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu_q[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        if (a.cu_q[lo] <= t && t < a.cu_q[lo + 1]) p += a.shift[lo];
    }
    return p;
}

template <int W>
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// A warp's tokens and heads.  The kWarps items of a block are neighbouring groups of tokens and the same `split` heads: what a
// block reads at a time is one run of a head's rows where these lie position after position.
struct Item {
    int b, t, h0, h1;
    bool in;
};
__device__ __forceinline__ int splits_of(const Args& a) { return (a.heads + a.split - 1) / a.split; }
template <int G>
__device__ __forceinline__ Item item_of(const Args& a, long long w, int group) {
    const int splits = splits_of(a);
    const long long run = w / (kWarps * splits);             // of kWarps groups
    const int split = (int)(w / kWarps - run * splits);
    const long long token = (run * kWarps + w % kWarps) * G + group, tokens = (long long)a.B * a.n;
    Item it;
    it.in = token < tokens;
    const long long k = it.in ? token : tokens - 1;          // lanes without a token take part in the shuffles only
    it.b = (int)(k / a.n);
    it.t = (int)(k - (long long)it.b * a.n);
    it.h0 = split * a.split;
    it.h1 = min(it.h0 + a.split, a.heads);
    return it;
}

// A warp has one item; the rows of U heads are loaded to registers together.  Train shape (16 + 16 heads of 128, 8 x 4096): 90 us, 6.0
// TB/s, 0.89 of a plain copy's bandwidth.  Tried there: three blocks to an SM 108 to 139, a persistent kernel with
// the rows through shared memory, as the gradient's, 96, and 117 to 123 with three blocks.  The same in fp32: 163 us, 0.98; staged
// (rot 100 of 128) 275.
template <typename T, int D, int F>
__global__ void __launch_bounds__(kThreads, 2) rotary_kernel(const __grid_constant__ Args a) {
    using Ln = Lane<T, D, F>;
    constexpr int N = Ln::N, L = Ln::L, G = Ln::G;
    constexpr int U = 4;                     // heads whose rows are on their way together
    __shared__ float staged[F == kStaged ? kWarps * G * D : 1];
    const int warp = threadIdx.x >> 5, ln = threadIdx.x & 31;
    float* stage = staged + (F == kStaged ? (warp * G + ln / L) * D : 0);
    const long long w = (long long)blockIdx.x * kWarps + warp;
    Ln l;
    l.place(ln % L, a.rot);
    cudaGridDependencySynchronize();
    const Item it = item_of<G>(a, w, ln / L);
    if (!__any_sync(0xffffffffu, it.in)) return;
    l.angles(a, position_of(a, it.b, it.t));
    const bool norm = a.eps >= 0.f;
    int first = 0;                           // the tensor's first head
#pragma unroll 1
    for (int i = 0; i < a.count; first += a.rows[i].heads, ++i) {
        const Rows& r = a.rows[i];
        const int h0 = max(it.h0 - first, 0), h1 = min(it.h1 - first, r.heads);
        if (h0 >= h1) continue;
        float gain[2][N];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int e = 0; e < N; ++e) gain[p][e] = r.gain ? r.gain[l.piece[p] * N + e] : 1.f;
        const char* x = r.x + it.b * r.xs[0] + it.t * r.xs[2];
        char* out = r.out + it.b * r.os[0] + it.t * r.os[2];
#pragma unroll 1
        for (int h = h0; h < h1; h += U) {
            uint4 raw[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u < h1) {
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        raw[u][p] = *reinterpret_cast<const uint4*>(x + (h + u) * r.xs[1] + l.piece[p] * 16);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h + u >= h1) break;
                float v[2][N];
                unpack(raw[u][0], v[0]);
                unpack(raw[u][1], v[1]);
                if (norm) {
                    float q = 0.f;
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int e = 0; e < N; ++e) q = fmaf(v[p][e], v[p][e], q);
                    const float rs = rsqrtf(sum_lanes<L>(q) * (1.f / D) + a.eps);
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int e = 0; e < N; ++e) v[p][e] *= rs * gain[p][e];
                }
                l.turn(v, 1.f, a.rot, stage);
                if (it.in) {
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        *reinterpret_cast<uint4*>(out + (h + u) * r.os[1] + l.piece[p] * 16) = pack(v[p]);
                }
            }
        }
    }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A warp's rows one after another: work items, in them the tensors, in them the heads.
template <int G>
struct Cursor {
    long long w;
    int i, first, h, h1;                     // tensor, its first head; head in the tensor, and behind its last of the item
    Item it;
    bool more;
    const char *dy, *x;                      // this lane's row; x only where it is normalised
    __device__ __forceinline__ void enter(const Args& a) {       // the first tensor from i on that has heads of the item
        for (; i < a.count; first += a.rows[i++].heads) {
            const Rows& r = a.rows[i];
            h = max(it.h0 - first, 0);
            h1 = min(it.h1 - first, r.heads);
            if (h < h1) {
                dy = r.dy + it.b * r.dys[0] + it.t * r.dys[2] + h * r.dys[1];
                x = r.x + it.b * r.xs[0] + it.t * r.xs[2] + h * r.xs[1];
                return;
            }
        }
        more = false;
    }
    __device__ __forceinline__ void begin(const Args& a, long long item, long long items, int group) {
        w = item;
        more = w < items;
        if (!more) return;
        it = item_of<G>(a, w, group);
        i = first = 0;
        enter(a);
    }
    __device__ __forceinline__ void step(const Args& a, long long stride, long long items, int group) {
        if (++h < h1) {
            dy += a.rows[i].dys[1];
            x += a.rows[i].xs[1];
            return;
        }
        first += a.rows[i++].heads;
        enter(a);
        if (!more) begin(a, w + stride, items, group);
    }
};

// The rows come through shared memory, kStages of them to a warp: no barrier of the block, and loads stay in flight under the
// arithmetic.  Where dy has K = 2 pieces of 16 bytes to one of x, a lane reads two neighbouring ones; the copies are shared out so
// that neighbouring lanes copy neighbouring pieces (whole 32-byte sectors), and piece C of the warp's rows lies in slot
// C ^ (C >> 3 & 1), which keeps eight lanes' writes and eight lanes' reads of every second piece in eight different slots.  Train
// shape, fp32 dy: 168 us, 6.4 TB/s, 0.96 of a plain copy's bandwidth (bf16 dy 129, 0.94; all in fp32 262, 0.92; staged, rot 100, 421); each lane copying its own pieces 217, the copies shared out
// without the swap of slots 229, rows through registers 226.  A warp goes through work items, its sums for the gains' gradients
// in shared memory; a block's sums leave in the order of its warps, and rotary_gain_kernel adds the blocks' in theirs: no
// atomics, the same bits every run.
constexpr int kStages = 4;
template <typename T, typename Y>
constexpr int stage_bytes() { return 32 * 16 * (2 * Vec<T>::N / Vec<Y>::N + 2); }

template <typename T, typename Y, int D, int F>
__global__ void __launch_bounds__(kThreads, 2) rotary_backward_kernel(const __grid_constant__ Args a, long long items) {
    using Ln = Lane<T, D, F>;
    constexpr int N = Ln::N, L = Ln::L, G = Ln::G, M = Vec<Y>::N, K = N / M, kStage = stage_bytes<T, Y>();
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ float staged[F == kStaged ? kWarps * G * D : 1];
    __shared__ __align__(16) float gains[kMost][D];
    const int warp = threadIdx.x >> 5, ln = threadIdx.x & 31, group = ln / L;
    float* stage = staged + (F == kStaged ? (warp * G + group) * D : 0);
    const unsigned char* mine = ring + warp * kStages * kStage;          // 512 bytes to a piece of every lane: 2 K of dy, 2 of x
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
    float* sums = reinterpret_cast<float*>(ring + kWarps * kStages * kStage);     // [warp][tensor][D], behind the stages
    float* own = sums + warp * a.count * D;
    const bool norm = a.eps >= 0.f;
    const long long stride = (long long)gridDim.x * kWarps, w0 = (long long)blockIdx.x * kWarps + warp;
    for (int e = ln; e < a.count * D; e += 32) own[e] = 0.f;
    Ln l;
    l.place(ln % L, a.rot);
    cudaGridDependencySynchronize();
    for (int e = threadIdx.x; e < a.count * D; e += kThreads) gains[e / D][e % D] = a.rows[e / D].gain ? a.rows[e / D].gain[e % D] : 1.f;
    __syncthreads();
    Cursor<G> ahead;
    ahead.begin(a, w0, items, group);
    // what this lane copies of dy: of the L K pieces that the row's lanes read in turn, number k L + lane
    auto slot = [](int c) { return (K == 2 ? c ^ (c >> 3 & 1) : c) * 16; };
    int from[2][K], to[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = k * L + ln % L;
        to[k] = slot(group * L * K + c);
#pragma unroll
        for (int p = 0; p < 2; ++p) from[p][k] = (Ln::piece_of(c / K, p, a.rot) * K + c % K) * 16;
    }
    auto fetch = [&](int st) {
        if (ahead.more) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
#pragma unroll
                for (int k = 0; k < K; ++k) copy16(base + st * kStage + p * K * 512 + to[k], ahead.dy + from[p][k]);
                if (norm) copy16(base + st * kStage + (2 * K + p) * 512 + ln * 16, ahead.x + l.piece[p] * 16);
            }
            ahead.step(a, stride, items, group);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    int st = 0;
    Item next = item_of<G>(a, w0, group);
    long long position = w0 < items ? position_of(a, next.b, next.t) : 0;
    for (long long w = w0; w < items; w += stride) {
        const Item it = next;
        l.angles(a, position);
        if (w + stride < items) {            // the next item's position is on its way under this one's rows
            next = item_of<G>(a, w + stride, group);
            position = position_of(a, next.b, next.t);
        }
        int first = 0;
#pragma unroll 1
        for (int i = 0; i < a.count; first += a.rows[i].heads, ++i) {
            const Rows& r = a.rows[i];
            const int h0 = max(it.h0 - first, 0), h1 = min(it.h1 - first, r.heads);
            if (h0 >= h1) continue;
            float dgain[2][N];
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int e = 0; e < N; ++e) dgain[p][e] = 0.f;
            char* out = r.out + it.b * r.os[0] + it.t * r.os[2] + h0 * r.os[1];
#pragma unroll 1
            for (int h = h0; h < h1; ++h, out += r.os[1]) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
                __syncwarp();                                    // other lanes' copies; and the row before is read
                const unsigned char* row = mine + st * kStage;
                float g[2][N], v[2][N];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        float y[M];
                        unpack(*reinterpret_cast<const uint4*>(row + p * K * 512 + slot(ln * K + k)), y);
#pragma unroll
                        for (int e = 0; e < M; ++e) g[p][k * M + e] = y[e];
                    }
                    if (norm) unpack(*reinterpret_cast<const uint4*>(row + (2 * K + p) * 512 + ln * 16), v[p]);
                }
                fetch(st == 0 ? kStages - 1 : st - 1);           // the stage of the row before
                st = st + 1 == kStages ? 0 : st + 1;
                l.turn(g, -1.f, a.rot, stage);
                if (norm) {
                    float q = 0.f, m = 0.f;
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int e = 0; e < N; ++e) q = fmaf(v[p][e], v[p][e], q);
                    const float rs = rsqrtf(sum_lanes<L>(q) * (1.f / D) + a.eps);
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            v[p][e] *= rs;                              // the unit row
                            if (it.in) dgain[p][e] = fmaf(g[p][e], v[p][e], dgain[p][e]);
                            g[p][e] *= gains[i][l.piece[p] * N + e];
                            m = fmaf(g[p][e], v[p][e], m);
                        }
                    m = sum_lanes<L>(m) * (1.f / D);
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int e = 0; e < N; ++e) g[p][e] = rs * fmaf(-v[p][e], m, g[p][e]);
                }
                if (it.in) {
#pragma unroll
                    for (int p = 0; p < 2; ++p) *reinterpret_cast<uint4*>(out + l.piece[p] * 16) = pack(g[p]);
                }
            }
            if (r.dgain) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        float d = dgain[p][e];
#pragma unroll
                        for (int o = L; o < 32; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                        if (ln < L) own[i * D + l.piece[p] * N + e] += d;
                    }
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.part) return;
    __syncthreads();
    for (int e = threadIdx.x; e < a.count * D; e += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) t += sums[k * a.count * D + e];
        a.part[(long long)blockIdx.x * a.count * D + e] = t;
    }
}

// dgain[i][c] = sum over blocks: a block of 32 x 32 threads has a tensor's 32 columns, a warp every 32nd block's row.
__global__ void __launch_bounds__(1024) rotary_gain_kernel(const __grid_constant__ Args a, int blocks, int D) {
    __shared__ float sh[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5, i = blockIdx.y;
    cudaGridDependencySynchronize();
    if (!a.rows[i].dgain) return;
    float t = 0.f;
    if (c < D)
        for (int b = k; b < blocks; b += 32) t += a.part[((long long)b * a.count + i) * D + c];
    sh[k][threadIdx.x & 31] = t;
    __syncthreads();
    t = sum_lanes<32>(sh[threadIdx.x & 31][k]);
    if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + k < D) a.rows[i].dgain[blockIdx.x * 32 + k] = t;
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

// Two blocks' shared memory fits an SM, but for bf16 rows with fp32 dy where they are staged (one tensor of d = 16 still fits) or are four
// tensors of d = 128: there the second half of the grid follows the first (train shape's rows as four tensors 192 us, as two 168).
constexpr int kBackwardBlocksPerSm = 2;
constexpr int kMostBlocks = 1024;
size_t part_bytes(int count, int d) { return (size_t)kMostBlocks * count * d * sizeof(float); }

int rows_of_warp(int es, int d) { return 32 / (d * es / 32); }

// Heads to a warp: as many as leave the device 32 warps an SM, so that a token's sines serve several rows, and 16 at most (train
// shape: 8 97 us, 16 90, 32 91; gradient 241, 217, 227 then; 1 to a warp, whose start nothing hides, 303 and 611).
void divide(Args& a, int es, int d, int sms) {
    const long long groups = ((long long)a.B * a.n + rows_of_warp(es, d) - 1) / rows_of_warp(es, d);
    const long long each = groups * a.heads / ((long long)sms * 32);
    a.split = (int)(each < 1 ? 1 : each > 16 ? 16 : each);
    if (a.split > a.heads) a.split = a.heads;
}

template <typename T, int D>
cudaError_t launch_forward(const Args& a, int form, unsigned blocks, cudaStream_t s) {
    switch (form) {
        case kHalves: return paged::launch_after(rotary_kernel<T, D, kHalves>, dim3(blocks), kThreads, 0, s, a);
        case kPairs: return paged::launch_after(rotary_kernel<T, D, kPairs>, dim3(blocks), kThreads, 0, s, a);
        default: return paged::launch_after(rotary_kernel<T, D, kStaged>, dim3(blocks), kThreads, 0, s, a);
    }
}
template <typename T, typename Y, int D, int F>
cudaError_t launch_backward_form(const Args& a, unsigned blocks, long long items, cudaStream_t s) {
    constexpr size_t rows = (size_t)kWarps * kStages * stage_bytes<T, Y>(), sums = (size_t)kWarps * D * sizeof(float);   // of a tensor
    const size_t smem = rows + a.count * sums;
    cudaError_t e = cudaFuncSetAttribute(rotary_backward_kernel<T, Y, D, F>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(rows + kMost * sums));
    if (e != cudaSuccess) return e;
    return paged::launch_after(rotary_backward_kernel<T, Y, D, F>, dim3(blocks), kThreads, smem, s, a, items);
}
template <typename T, typename Y, int D>
cudaError_t launch_backward(const Args& a, int form, unsigned blocks, long long items, cudaStream_t s) {
    switch (form) {
        case kHalves: return launch_backward_form<T, Y, D, kHalves>(a, blocks, items, s);
        case kPairs: return launch_backward_form<T, Y, D, kPairs>(a, blocks, items, s);
        default: return launch_backward_form<T, Y, D, kStaged>(a, blocks, items, s);
    }
}
template <typename T>
cudaError_t forward_of(const Args& a, int d, int form, unsigned blocks, cudaStream_t s) {
    switch (d) {
        case 16: return launch_forward<T, 16>(a, form, blocks, s);
        case 32: return launch_forward<T, 32>(a, form, blocks, s);
        case 64: return launch_forward<T, 64>(a, form, blocks, s);
        default: return launch_forward<T, 128>(a, form, blocks, s);
    }
}
template <typename T, typename Y>
cudaError_t backward_of(const Args& a, int d, int form, unsigned blocks, long long items, cudaStream_t s) {
    switch (d) {
        case 16: return launch_backward<T, Y, 16>(a, form, blocks, items, s);
        case 32: return launch_backward<T, Y, 32>(a, form, blocks, items, s);
        case 64: return launch_backward<T, Y, 64>(a, form, blocks, items, s);
        default: return launch_backward<T, Y, 128>(a, form, blocks, items, s);
    }
}

bool strides_ok(const long long* s, int ve) { return s[0] % ve == 0 && s[1] % ve == 0 && s[2] % ve == 0; }

// Checks of both calls; fills a.  dy_es: 0 in the forward pass.
int check(Args& a, int dtype, const lla_rotary_rows* rows, int count, int B, int n, int d, const int* positions,
          long long position_stride, const long long* turns, int rot, float magnitude, float eps, const int* cu_q,
          const int* shift, int S, int dy_es) {
    if (dtype != LLA_DTYPE_BF16 && dtype != LLA_DTYPE_FP32) return failf(LLA_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (!rows || !positions || !turns) return failf(LLA_ERR_INVALID_ARG, "null pointer");
    if (count < 1 || count > kMost) return failf(LLA_ERR_INVALID_ARG, "count must be in [1, %d] (got %d)", kMost, count);
    if (d != 16 && d != 32 && d != 64 && d != 128)
        return failf(LLA_ERR_INVALID_ARG, "head dim d must be 16, 32, 64 or 128 (got %d)", d);
    if (B < 1 || n < 1 || (long long)B * n > (1LL << 30)) return failf(LLA_ERR_INVALID_ARG, "B and n must be >= 1 and B*n <= 2^30");
    if (rot < 2 || rot > d || rot % 2) return failf(LLA_ERR_INVALID_ARG, "rot must be even and in [2, d] (got %d)", rot);
    if (!(fabsf(magnitude) < INFINITY) || magnitude == 0.f) return failf(LLA_ERR_INVALID_ARG, "magnitude must be finite and not 0");
    if (!(fabsf(eps) < INFINITY)) return failf(LLA_ERR_INVALID_ARG, "eps must be finite (negative: no normalisation)");
    if (position_stride != 0 && position_stride != n) return failf(LLA_ERR_INVALID_ARG, "position_stride must be 0 or n");
    if (!aligned(positions, 4) || !aligned(turns, 8) || !aligned(cu_q, 4) || !aligned(shift, 4))
        return failf(LLA_ERR_INVALID_ARG, "integer pointers must be aligned to their type");
    if ((cu_q != nullptr) != (shift != nullptr)) return failf(LLA_ERR_INVALID_ARG, "cu_q and shift go together");
    if (shift && (B != 1 || S < 1)) return failf(LLA_ERR_INVALID_ARG, "shift needs B = 1 and S >= 1");
    const int es = dtype == LLA_DTYPE_BF16 ? 2 : 4;
    a.heads = 0;
    for (int i = 0; i < count; ++i) {
        const lla_rotary_rows& r = rows[i];
        const bool reads_x = dy_es == 0 || eps >= 0.f;
        if (!r.out || (reads_x && !r.x) || (dy_es && !r.dy)) return failf(LLA_ERR_INVALID_ARG, "null tensor pointer (tensor %d)", i);
        if (r.heads < 1 || r.heads > 65535) return failf(LLA_ERR_INVALID_ARG, "heads must be in [1, 65535] (tensor %d)", i);
        if (!aligned(r.out, 16) || (reads_x && !aligned(r.x, 16)) || (dy_es && !aligned(r.dy, 16)) || !aligned(r.gain, 4) || !aligned(r.dgain, 4))
            return failf(LLA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned, gains 4-byte (tensor %d)", i);
        if (!strides_ok(r.out_stride, 16 / es) || (reads_x && !strides_ok(r.x_stride, 16 / es)) || (dy_es && !strides_ok(r.dy_stride, 16 / dy_es)))
            return failf(LLA_ERR_INVALID_ARG, "strides must be multiples of 16 bytes (tensor %d)", i);
        if (eps < 0.f && (r.gain || r.dgain)) return failf(LLA_ERR_INVALID_ARG, "a gain goes with the normalisation, eps >= 0 (tensor %d)", i);
        Rows& o = a.rows[i];
        o.x = static_cast<const char*>(r.x);
        o.dy = static_cast<const char*>(r.dy);
        o.out = static_cast<char*>(r.out);
        o.gain = r.gain;
        o.dgain = dy_es ? r.dgain : nullptr;
        o.heads = r.heads;
        for (int k = 0; k < 3; ++k) {
            o.xs[k] = r.x_stride[k] * es;
            o.os[k] = r.out_stride[k] * es;
            o.dys[k] = r.dy_stride[k] * (dy_es ? dy_es : es);
        }
        a.heads += r.heads;
    }
    a.positions = positions; a.position_stride = position_stride; a.turns = turns; a.cu_q = cu_q; a.shift = shift;
    a.part = nullptr; a.count = count; a.B = B; a.n = n; a.S = S; a.rot = rot; a.magnitude = magnitude; a.eps = eps;
    return LLA_OK;
}

int form_of(int rot, int interleaved, int es) {
    return interleaved ? kPairs : rot / 2 % (16 / es) == 0 ? kHalves : kStaged;
}

}  // namespace
}  // namespace rotary
}  // namespace lla

namespace lr = lla::rotary;

extern "C" {

int lla_rotary(int dtype, const lla_rotary_rows* rows, int count, int B, int n, int d, const int* positions,
               long long position_stride, const long long* turns, int rot, int interleaved, float magnitude, float eps,
               const int* cu_q, const int* shift, int S, void* stream) {
    lla::set_error(LLA_OK, "");
    lr::Args a{};
    const int st = lr::check(a, dtype, rows, count, B, n, d, positions, position_stride, turns, rot, magnitude, eps, cu_q, shift, S, 0);
    if (st != LLA_OK) return st;
    const int sms = lr::sm_count(), es = dtype == LLA_DTYPE_BF16 ? 2 : 4;
    if (sms < 1) return lr::failf(LLA_ERR_CUDA, "lla_rotary: no device");
    lr::divide(a, es, d, sms);
    const int G = lr::rows_of_warp(es, d);
    const long long blocks = ((long long)B * n + G * lr::kWarps - 1) / (G * lr::kWarps) * ((a.heads + a.split - 1) / a.split);
    if (blocks > INT_MAX) return lr::failf(LLA_ERR_INVALID_ARG, "problem too large");
    const int form = lr::form_of(rot, interleaved, es);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = es == 2 ? lr::forward_of<__nv_bfloat16>(a, d, form, (unsigned)blocks, s)
                                  : lr::forward_of<float>(a, d, form, (unsigned)blocks, s);
    if (e != cudaSuccess) return lr::cuda_failf(e, "lla_rotary launch");
    return LLA_OK;
}

size_t lla_rotary_backward_workspace_size(int count, int d) {
    if (count < 1 || count > lr::kMost || (d != 16 && d != 32 && d != 64 && d != 128)) return 0;
    return lr::part_bytes(count, d);
}

int lla_rotary_backward(int dtype, int dy_dtype, const lla_rotary_rows* rows, int count, int B, int n, int d,
                        const int* positions, long long position_stride, const long long* turns, int rot, int interleaved,
                        float magnitude, float eps, const int* cu_q, const int* shift, int S, void* workspace,
                        size_t workspace_bytes, void* stream) {
    lla::set_error(LLA_OK, "");
    if (dy_dtype != LLA_DTYPE_FP32 && dy_dtype != dtype)
        return lr::failf(LLA_ERR_INVALID_ARG, "dy must have the rows' dtype or be fp32");
    lr::Args a{};
    const int es = dtype == LLA_DTYPE_BF16 ? 2 : 4, ys = dy_dtype == LLA_DTYPE_BF16 ? 2 : 4;
    const int st = lr::check(a, dtype, rows, count, B, n, d, positions, position_stride, turns, rot, magnitude, eps, cu_q, shift, S, ys);
    if (st != LLA_OK) return st;
    bool gains = false;
    for (int i = 0; i < count; ++i) gains |= a.rows[i].dgain != nullptr;
    const size_t need = gains ? lr::part_bytes(count, d) : 0;
    if (workspace && need) {
        if (workspace_bytes < need) return lr::failf(LLA_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
        if (!lr::aligned(workspace, 256)) return lr::failf(LLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    }
    const int sms = lr::sm_count();
    if (sms < 1) return lr::failf(LLA_ERR_CUDA, "lla_rotary_backward: no device");
    lr::divide(a, es, d, sms);
    const int G = lr::rows_of_warp(es, d);
    long long blocks = ((long long)B * n + G * lr::kWarps - 1) / (G * lr::kWarps) * ((a.heads + a.split - 1) / a.split);
    const long long items = blocks * lr::kWarps;
    const long long most = lr::kBackwardBlocksPerSm * sms < lr::kMostBlocks ? lr::kBackwardBlocksPerSm * sms : lr::kMostBlocks;
    if (blocks > most) blocks = most;
    const int form = lr::form_of(rot, interleaved, es);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* ws = workspace;
    cudaError_t e = cudaSuccess;
    if (need && !ws && (e = cudaMallocAsync(&ws, need, s)) != cudaSuccess) return lr::cuda_failf(e, "cudaMallocAsync(workspace)");
    a.part = need ? static_cast<float*>(ws) : nullptr;
    if (es == 4) e = lr::backward_of<float, float>(a, d, form, (unsigned)blocks, items, s);
    else if (ys == 4) e = lr::backward_of<__nv_bfloat16, float>(a, d, form, (unsigned)blocks, items, s);
    else e = lr::backward_of<__nv_bfloat16, __nv_bfloat16>(a, d, form, (unsigned)blocks, items, s);
    if (e == cudaSuccess && need)
        e = lla::paged::launch_after(lr::rotary_gain_kernel, dim3((d + 31) / 32, count), 1024, 0, s, a, (int)blocks, d);
    if (need && !workspace) {
        const cudaError_t e2 = cudaFreeAsync(ws, s);
        if (e == cudaSuccess && e2 != cudaSuccess) return lr::cuda_failf(e2, "cudaFreeAsync(workspace)");
    }
    if (e != cudaSuccess) return lr::cuda_failf(e, "lla_rotary_backward launch");
    return LLA_OK;
}

}  // extern "C"
