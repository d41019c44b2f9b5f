// Shared by the tensor-core kernels over paged bf16 caches: the cache's tensor map, TMA loads of page
// boxes, and waits for copies in flight.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lla_paged.h"
#include "tc_host.h"
#include "tc_ptx.cuh"

namespace lla {
namespace paged {

constexpr int kBoxRows = 64;       // a box holds up to this many rows of one page and head

// A block of rows lies in shared memory as [rows / 8][d / 64][8 rows][128 B], 128-byte swizzle: groups of eight
// rows, in them the 64-column halves.  So the rows of a page are one run whatever the page size, and one TMA
// box brings them in; the groups are d * 16 bytes apart, the halves 1024, for tcgen05's descriptors and for
// ldmatrix alike.  (A box per half and page took the TMA unit about 70 cycles each, 3250 a block with 16-row pages,
// where the products need 2048.)
template <int D>
__device__ __forceinline__ uint32_t piece_off(int r, int c) {          // 16-byte piece c of row r
    return (uint32_t)((r >> 3) * (D * 16) + (c >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Head slices of a cache: pages are a whole number of them apart (checked by the caller), so (page, head) is one
// coordinate, page * slices_of_page + head.
inline long long slices_of_page(const PagedProblem& p) { return p.page_stride / ((1LL << p.page_shift) * p.d); }

// The cache as (64 columns, row of a group, half, group of the page, slice); a slice behind the last reads as zeros.
inline bool make_cache_map(CUtensorMap* map, const void* cache, const PagedProblem& p) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const int page = 1 << p.page_shift;
    const long long slices = (p.num_pages - 1) * slices_of_page(p) + p.Hkv;
    cuuint64_t dims[5] = {64, 8, (cuuint64_t)(p.d / 64), (cuuint64_t)(page / 8), (cuuint64_t)slices};
    cuuint64_t strides[4] = {(cuuint64_t)p.d * 2, 128, (cuuint64_t)p.d * 16, (cuuint64_t)page * p.d * 2};
    cuuint32_t box[5] = {64, 8, (cuuint32_t)(p.d / 64), (cuuint32_t)((page < kBoxRows ? page : kBoxRows) / 8), 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(cache), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One box: the rows of `slice` from group `group` on.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int group, int slice) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %3, %3, %4, %5}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(0), "r"(group), "r"(slice)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// Bounded wait for a copy in flight, whatever the error flag says: shared memory must not be given back
// under it.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = tc::globaltimer_ns();
    while (!tc::mbar_try_wait(bar, parity))
        if (tc::globaltimer_ns() - t0 > 2000000000ull) break;
}

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

// The page that holds a key of sequence row `row`, checked: an id outside the cache is reported and
// replaced by one past the last, which the map reads as zeros.
__device__ __forceinline__ int checked_page(const Work& w, const int* row, int key) {
    int page = row[key >> w.page_shift];
    if (page < 0 || page >= w.num_pages) {
        atomicOr(w.err, (unsigned)kDevErrPagedArg);
        page = w.num_pages;
    }
    return page;
}

}  // namespace paged
}  // namespace lla
