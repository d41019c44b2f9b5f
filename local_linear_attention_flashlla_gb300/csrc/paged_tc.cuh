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

constexpr int kBoxRows = 64;       // a box holds up to this many rows of one page and head, 64 columns wide

// [P, Hkv, page, d] bf16 cache, pages page_stride elements apart; 128-byte swizzle.  Coordinates
// (column, row of the page, key head, page); a page past the last reads as zeros.
inline bool make_cache_map(CUtensorMap* map, const void* cache, const PagedProblem& p) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const int page = 1 << p.page_shift;
    cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)page, (cuuint64_t)p.Hkv, (cuuint64_t)p.num_pages};
    cuuint64_t strides[3] = {(cuuint64_t)p.d * 2, (cuuint64_t)page * p.d * 2, (cuuint64_t)p.page_stride * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)(page < kBoxRows ? page : kBoxRows), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(cache), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
