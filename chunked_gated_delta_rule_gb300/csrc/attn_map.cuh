// attn_map.cuh -- what the tensor-core kernels share: a paged cache as a TMA
// tensor (boxes of slots of one page and one head), and its 8-bit values as FP16.
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

// The scale s that a row of values is weighed with, 2^(t + log2 s - m): its own,
// but no smaller than 2^-100, so that the sum of the 2^(t + log2 s - m) / s stays
// finite.  A row of zeros has none, and any will do that neither loses its weight
// in that sum (below 2^-126 beside the largest) nor drives the others out of FP16.
constexpr float kLeastScale = 0x1p-100f, kScaleOfZeros = 0x1p-60f;
__device__ __forceinline__ float weighed_scale(float s) {
    return s < kLeastScale ? (s == 0.f ? kScaleOfZeros : kLeastScale) : s;
}

// Four 8-bit values (FMT 1: E4M3, 2: integers) as FP16, exact.
template <int FMT>
__device__ __forceinline__ void widen4(uint32_t x, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == 1) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(x));
    } else {
        const uint32_t u = x ^ 0x80808080u;  // x + 128, the low bits of 1024 + x + 128
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 c = __floats2half2_rn(1152.f, 1152.f);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&a), c);
        const __half2 z = __hsub2(*reinterpret_cast<const __half2 *>(&b), c);
        lo = *reinterpret_cast<const uint32_t *>(&y);
        hi = *reinterpret_cast<const uint32_t *>(&z);
    }
}

}  // namespace gdr
