// attn_map.cuh -- a paged cache as a TMA tensor: boxes of slots of one page and
// one head.
#pragma once

#include "attn.cuh"
#include "tc_common.cuh"
#include "tma_host.cuh"

namespace gdr {

// The layout of a box in shared memory: rows of 16-bit values in blocks of 64
// columns under the 128-byte swizzle; 8-bit rows as they are, or (kPageSwizzled)
// under the swizzle of their length (64 or 128 bytes).
enum PageLayout { kPagePlain = 0, kPageSwizzled = 1 };

// [page][head][slot][column], boxes of `box` slots.  False if the driver
// rejects the map.
inline bool page_map(CUtensorMap *map, const AttnProblem &p, const void *base,
                     const int64_t (&st)[3], int D, int box, PageLayout layout) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const bool raw = cache_quantised(p.c.dtype);
    const uint64_t es = raw ? 1 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)p.c.page_size, (cuuint64_t)p.c.H,
                                (cuuint64_t)p.c.n_pages};
    const cuuint64_t strides[3] = {st[1] * es, st[2] * es, st[0] * es};
    const cuuint32_t bx[4] = {raw ? (cuuint32_t)D : 64u, (cuuint32_t)box, 1, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const auto type = raw                   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                      : p.dtype == GDR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const auto swizzle = raw && layout == kPagePlain ? CU_TENSOR_MAP_SWIZZLE_NONE
                         : raw && D == 64            ? CU_TENSOR_MAP_SWIZZLE_64B
                                                     : CU_TENSOR_MAP_SWIZZLE_128B;
    return enc(map, type, 4, const_cast<void *>(base), dims, strides, bx, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The scales of a box are copied in 16-byte units.
inline bool scales_aligned16(const PagedCache &c) {
    return ((reinterpret_cast<uintptr_t>(c.ks) | reinterpret_cast<uintptr_t>(c.vs)) & 15u) == 0;
}

__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int column,
                                         int slot, int head, int page) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(column), "r"(slot),
        "r"(head), "r"(page)
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace gdr
