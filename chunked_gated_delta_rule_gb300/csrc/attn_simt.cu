// attn_simt.cu -- attention over a paged cache on CUDA cores, in FP32: the
// route of FP32 tensors and of every shape and stride that the tensor-core
// kernels do not take.
//
// One warp a (token, query head) row.  The warp walks the row's visible
// positions 32 at a time: lane j forms the score of position j (its own key,
// the query broadcast from shared memory), the lanes join maximum and sum,
// and the values are added with lanes across the columns.  Each key is read
// once for every query row that sees it, so the kernel is bound by L1 and L2
// and by FP32 products, not by memory; the tensor-core kernels are the fast
// route.  Measured, 16 query heads on 2 of 256 columns: 512 new tokens over 4K
// 29.6 ms (FP32 the same), 32 decodes over up to 4K 6.1 ms, one over 16K 14.8 ms
// (its axis is not split); elementary library products take 1.6, 2.6 and 1.5 ms.  A position that a row does not see is never multiplied into it, so
// what a masked place holds (infinities, NaN) cannot reach it.
#include <cuda_fp8.h>

#include "attn.cuh"
#include "gdr_launch.cuh"

namespace gdr {
namespace {

constexpr int kAWarps = 4;
constexpr int kAMaxD = 256;

template <typename Tio, typename Tc>
__global__ void __launch_bounds__(32 * kAWarps) k_attn_simt(AttnProblem p) {
    __shared__ float sq[kAWarps][kAMaxD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tokens = rows_packed(p.r) ? p.r.T : p.r.N * p.r.T;
    const int64_t row = (int64_t)blockIdx.x * kAWarps + warp;
    if (row >= tokens * p.Hq) return;
    const int64_t t = row / p.Hq;
    const int h = (int)(row - t * p.Hq), hk = h / p.G;
    const int64_t n = find_seq(p.r, t);
    int64_t t0, len;
    seq_span(p.r, n, t0, len);
    const int64_t kv = cached_len(p.c, n, p.r.status);
    int lo = 0, hi = 0;
    if (t >= t0 && t < t0 + len) visible(p, (int)kv, (int)(kv - len + (t - t0)), lo, hi);
    if (row == 0) check_offsets(p.r);

    const Tio *q = reinterpret_cast<const Tio *>(p.q) + tok_at(p.sq, t, h);
    for (int d = lane; d < p.K; d += 32) sq[warp][d] = (float)q[d] * p.scale;
    __syncwarp();

    float m = -INFINITY, l = 0.f;
    float acc[kAMaxD / 32] = {};
    for (int j0 = lo; j0 < hi; j0 += 32) {
        const int j = j0 + lane;
        int64_t ko = 0, vo = 0;
        float s = -INFINITY, vs = 1.f;
        bool live = j < hi;
        if (live) {
            const int pi = j / p.c.page_size, slot = j - pi * p.c.page_size;
            const int page = page_of(p.c, n, pi, p.r.status);
            live = page >= 0;
            if (live) {
                ko = page_at(p.c.kst, page, slot, hk);
                vo = page_at(p.c.vst, page, slot, hk);
                const Tc *k = reinterpret_cast<const Tc *>(p.c.k) + ko;
                s = 0.f;
                for (int d = 0; d < p.K; ++d) s = fmaf(sq[warp][d], (float)k[d], s);
                if constexpr (sizeof(Tc) == 1) {
                    const int64_t at = scale_at(p.c, page, slot, hk);
                    s *= p.c.ks[at];
                    vs = p.c.vs[at];
                }
            }
        }
        float mt = s;
        for (int d = 16; d; d >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, d));
        const float mn = fmaxf(m, mt), mu = mn == -INFINITY ? 0.f : mn;
        const float fix = __expf(m - mu);
        const float w = live ? __expf(s - mu) : 0.f;
        m = mn;
        float lt = w;
        for (int d = 16; d; d >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, d);
        l = fmaf(l, fix, lt);
#pragma unroll
        for (int i = 0; i < kAMaxD / 32; ++i) acc[i] *= fix;
        const float wv = w * vs;
        const unsigned lives = __ballot_sync(0xffffffffu, live);
        for (int jj = 0; jj < 32; ++jj) {
            const float wj = __shfl_sync(0xffffffffu, wv, jj);
            const int64_t oj = __shfl_sync(0xffffffffu, vo, jj);
            if (!(lives >> jj & 1)) continue;
            const Tc *v = reinterpret_cast<const Tc *>(p.c.v) + oj;
#pragma unroll
            for (int i = 0; i < kAMaxD / 32; ++i) {
                const int d = i * 32 + lane;
                if (d < p.V) acc[i] = fmaf(wj, (float)v[d], acc[i]);
            }
        }
    }
    // NaN scores leave m untouched (fmaxf) but make l NaN, and with it the row
    const bool empty = l == 0.f;
    const float inv = empty ? 0.f : 1.f / l;
    Tio *o = reinterpret_cast<Tio *>(p.o) + tok_at(p.so, t, h);
#pragma unroll
    for (int i = 0; i < kAMaxD / 32; ++i) {
        const int d = i * 32 + lane;
        if (d < p.V) o[d] = (Tio)(acc[i] * inv);
    }
    if (p.lse && lane == 0)
        p.lse[t * p.Hq + h] = empty ? -INFINITY : (m == -INFINITY ? 0.f : m) + logf(l);
}

template <typename Tio, typename Tc>
cudaError_t launch(const AttnProblem &p, cudaStream_t st) {
    const int64_t rows = (rows_packed(p.r) ? p.r.T : p.r.N * p.r.T) * p.Hq;
    const int64_t blocks = (rows + kAWarps - 1) / kAWarps;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    k_attn_simt<Tio, Tc><<<(unsigned)blocks, 32 * kAWarps, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename Tio>
cudaError_t launch_fmt(const AttnProblem &p, cudaStream_t st) {
    if (p.c.dtype == GDR_E4M3) return launch<Tio, __nv_fp8_e4m3>(p, st);
    if (p.c.dtype == GDR_I8) return launch<Tio, int8_t>(p, st);
    return launch<Tio, Tio>(p, st);
}

}  // namespace

cudaError_t attn_simt(const AttnProblem &p, cudaStream_t st) {
    if (p.dtype == GDR_BF16) return launch_fmt<__nv_bfloat16>(p, st);
    if (p.dtype == GDR_F16) return launch_fmt<__half>(p, st);
    return launch_fmt<float>(p, st);
}

}  // namespace gdr
