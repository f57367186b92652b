// cache.cu -- new keys and values into a paged cache, quantised on the way,
// and back.
//
// An 8-bit cache holds, for every (token, head) row x, the values
//   q = rn(x / s),  s = max|x| * (1 / qmax)   (q = 0 where s = 0),
// qmax = 448 for E4M3 and 127 for 8-bit integers, and s in FP32; it stands
// for q s.  The division is IEEE's and the product with 1 / qmax one FP32
// product, so the bits follow from the formula alone.  max|x| keeps s finite
// and normal for every row of 16-bit values that holds one above 2^-117; a row
// with a NaN or an infinity has no scale: it is stored as q = 0, s = NaN and
// reads back as NaN.
//
// Both directions should be bound by memory and are, once the instructions a
// value are few: with the compiler's division, checks and conversions value by
// value they were 39 to write one and 17 to read one (64K tokens x 8 heads to
// E4M3 and back: 337 us).  So
//   * the quotients come from one reciprocal a row: r = rn(1 / s), p = rn(x r),
//     then twice p <- rn(p - r (p s - x)), products and sums fused (with the signs
//     so, a zero keeps its own).  The first
//     step makes p faithful (p is within two units in the last place at the
//     start), and a faithful p is then rounded correctly (Markstein, "Computation
//     of elementary functions on the IBM RISC System/6000 processor", 1990), as
//     long as x - p s does not underflow; rows with s < 2^-60 take the division.
//     (A quotient below 2^-10 is stored as 0 whatever its last bits.)
//   * the largest magnitude is taken of the bits, two 16-bit values at once: the
//     bits of magnitudes are in their order, and those of infinities and NaNs lie
//     above all others;
//   * a row is the work of the 2 to 32 lanes that hold 8 values of it each, as
//     16-byte loads of 16-bit types, kPasses rows at once.  Where a warp's rows
//     live (sequence, length, page: one load behind the other) is looked up 32
//     at a time, a lane a row; warps do not wait for each other.
#include <cuda_fp8.h>

#include "gdr_launch.cuh"
#include "paged.cuh"

namespace gdr {
namespace {

constexpr int kCThreads = 256;
constexpr int kPasses = 2;
constexpr int kBlocksPerSm = 6;
constexpr int kWarps = kCThreads / 32;

struct RowArgs {
    PagedCache c;
    TokenRows r;
    const void *k, *v;  // the call's rows (written by the reader)
    TokStride sk, sv;
    int K, V, lanes;    // lanes a row: a power of two, 8 lanes >= max(K, V)
    int64_t rows;       // tokens x heads
    int chunk;          // rows that a warp looks up at once, at most 32
};

// Where a row of the block lives, in elements: in the call's tensors, in the
// pages and among the scales; live: it has a place in the cache.
struct Place {
    int64_t k, v, kc, vc, scale;
    int live;
};

// Eight values as they lie in memory.
template <typename T>
struct alignas(16) Eight {
    T e[8];
    template <bool VEC>
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC) {
            using W = typename std::conditional<sizeof(T) == 1, uint2, uint4>::type;
#pragma unroll
            for (int i = 0; i < (int)(sizeof(e) / sizeof(W)); ++i)
                reinterpret_cast<W *>(e)[i] = reinterpret_cast<const W *>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = p[i];
        }
    }
    template <bool VEC>
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (VEC) {
            using W = typename std::conditional<sizeof(T) == 1, uint2, uint4>::type;
#pragma unroll
            for (int i = 0; i < (int)(sizeof(e) / sizeof(W)); ++i)
                reinterpret_cast<W *>(p)[i] = reinterpret_cast<const W *>(e)[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = e[i];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(e) / 4; ++i) reinterpret_cast<uint32_t *>(e)[i] = 0;
    }
    __device__ __forceinline__ void widen(float (&x)[8]) const {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(e);
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else if constexpr (std::is_same<T, __nv_fp8_e4m3>::value) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h;
                asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
                    : "=r"(h)
                    : "r"(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]));
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (float)e[i];
        }
    }
    // The bits of the largest magnitude, as a float's.
    __device__ __forceinline__ uint32_t most() const {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(e);
        if constexpr (sizeof(T) == 2) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            m = max(m & 0xffffu, m >> 16);
            if constexpr (std::is_same<T, __half>::value)
                return m >= 0x7c00u ? 0x7f800000u : __float_as_uint(__half2float(__ushort_as_half((uint16_t)m)));
            return m << 16;
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        }
    }
    // The values nearest to x (ties to even; E4M3 saturates, 8-bit integers are
    // within range).
    __device__ __forceinline__ void narrow(const float (&x)[8]) {
        uint32_t *w = reinterpret_cast<uint32_t *>(e);
        if constexpr (std::is_same<T, __nv_fp8_e4m3>::value) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                asm("{\n\t.reg .b16 a, b;\n\t"
                    "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
                    "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\tmov.b32 %0, {a, b};\n\t}"
                    : "=r"(w[i])
                    : "f"(x[4 * i]), "f"(x[4 * i + 1]), "f"(x[4 * i + 2]), "f"(x[4 * i + 3]));
        } else if constexpr (std::is_same<T, int8_t>::value) {
            // x + 1.5 2^23: the sum's unit is 1, its low byte the integer
            uint32_t b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(x[i] + 12582912.f);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                                   __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        } else if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = x[i];
        }
    }
};

// The places of the warp's `n` <= 32 rows from `first` on (token-major, then
// head): none before position 0, past the table or in a page outside the cache.
__device__ __forceinline__ void find_places(const RowArgs &a, int64_t first, int n, Place *places) {
    const int H = a.c.H, r = threadIdx.x & 31;
    const int64_t t0 = first >> 31 ? first / H : (uint32_t)first / (uint32_t)H;
    const int h0 = (int)(first - t0 * H);
    {
        const int d = (h0 + r) / H, h = h0 + r - d * H;
        const int64_t t = t0 + d;
        // the warp looks its first row's sequence up together, then every lane
        // steps to its own
        int64_t seq = find_seq(a.r, t0);
        if (r >= n) return;
        int64_t begin = row_bound(a.r, seq), end = row_bound(a.r, seq + 1);
        int len = a.c.kv_lens[seq];
        while (t >= end && seq + 1 < a.r.N) {
            begin = end;
            end = row_bound(a.r, ++seq + 1);
            len = a.c.kv_lens[seq];
        }
        int page = -1, slot = 0;
        if (rows_packed(a.r) && (begin < 0 || t < begin || t >= end || end > a.r.T)) {
            report(a.r.status, GDR_ERR_SEQLENS);
        } else {
            const int64_t pos = (int64_t)len - (end - t);
            if (len < 0 || len > a.c.max_pages * a.c.page_size) {  // no token has a place
                report(a.r.status, GDR_ERR_INDEX);
            } else if (pos >= 0) {
                const unsigned pi = (unsigned)pos / (unsigned)a.c.page_size;
                slot = (int)((unsigned)pos - pi * (unsigned)a.c.page_size);
                page = page_of(a.c, seq, (int)pi, a.r.status);
            }
        }
        Place &x = places[r];
        x.k = tok_at(a.sk, t, h);
        x.v = tok_at(a.sv, t, h);
        x.live = page >= 0;
        x.kc = page_at(a.c.kst, page, slot, h);
        x.vc = page_at(a.c.vst, page, slot, h);
        x.scale = scale_at(a.c, page, slot, h);
    }
}

template <typename Tc>
__device__ constexpr float inv_qmax() {
    return std::is_same<Tc, int8_t>::value ? 1.0f / 127.0f : 1.0f / 448.0f;
}

// A lane's part of a row: quantised by the row's scale (all lanes of the row
// come here), or as it is.
template <typename Tin, typename Tc, bool VEC>
__device__ __forceinline__ void write_row(const Eight<Tin> &x, bool live, Tc *dst, float *scale, int lanes,
                                          bool first_lane) {
    if constexpr (sizeof(Tc) == 1) {
        uint32_t m = x.most();
        for (int d = lanes >> 1; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        // a row with a NaN or an infinity has none
        const float s = m >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                         : __uint_as_float(m) * inv_qmax<Tc>();
        if (!live) return;
        if (first_lane) *scale = s;
        float f[8];
        x.widen(f);
        if (s >= 0x1p-60f) {
            const float r = __frcp_rn(s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float q = f[i] * r;
                q = fmaf(fmaf(q, s, -f[i]), -r, q);
                f[i] = fmaf(fmaf(q, s, -f[i]), -r, q);
            }
        } else {
            // a scale of a few of FP32's least units may be a third too small
            constexpr float kMost = std::is_same<Tc, int8_t>::value ? 127.f : 448.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = s > 0.f ? fminf(fmaxf(__fdiv_rn(f[i], s), -kMost), kMost) : 0.f;
        }
        Eight<Tc> y;
        y.narrow(f);
        y.template store<VEC>(dst);
    } else {
        if (live) x.template store<VEC>(dst);
    }
}

// Both kernels: a warp takes every so-manieth chunk of rows.  The table of offsets
// is looked over by a warp that calls of few rows leave idle.
template <typename Tin, typename Tc, bool VEC>
__global__ void __launch_bounds__(kCThreads, kBlocksPerSm) k_cache_write(RowArgs a) {
    __shared__ Place s_places[kWarps][32];
    Place *places = s_places[threadIdx.x >> 5];
    const int groups = 32 / a.lanes, group = (threadIdx.x & 31) / a.lanes;
    const int sub = threadIdx.x & (a.lanes - 1), d = sub * 8;
    const int64_t warp = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (warp == kWarps - 1) check_offsets(a.r);
    for (int64_t first = warp * a.chunk; first < a.rows; first += (int64_t)gridDim.x * kWarps * a.chunk) {
        const int n = (int)(a.rows - first < a.chunk ? a.rows - first : a.chunk);
        __syncwarp();
        find_places(a, first, n, places);
        __syncwarp();
        for (int r0 = 0; r0 < n; r0 += groups * kPasses) {
            Eight<Tin> x[kPasses], y[kPasses];
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = r0 + i * groups + group;
                const bool live = r < n && places[r].live;
                x[i].zero();
                y[i].zero();
                if (live && d < a.K)
                    x[i].template load<VEC>(reinterpret_cast<const Tin *>(a.k) + places[r].k + d);
                if (live && d < a.V)
                    y[i].template load<VEC>(reinterpret_cast<const Tin *>(a.v) + places[r].v + d);
            }
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = r0 + i * groups + group;
                const Place &at = places[r < n ? r : 0];
                const bool live = r < n && at.live;
                write_row<Tin, Tc, VEC>(x[i], live && d < a.K, reinterpret_cast<Tc *>(a.c.k) + at.kc + d,
                                        a.c.ks + at.scale, a.lanes, sub == 0);
                write_row<Tin, Tc, VEC>(y[i], live && d < a.V, reinterpret_cast<Tc *>(a.c.v) + at.vc + d,
                                        a.c.vs + at.scale, a.lanes, sub == 0);
            }
        }
    }
}

template <typename Tout, typename Tc, bool VEC>
__device__ __forceinline__ void read_row(const Eight<Tc> &x, float scale, Tout *dst) {
    if constexpr (sizeof(Tc) == 1) {
        float f[8];
        x.widen(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= scale;
        Eight<Tout> y;
        y.narrow(f);
        y.template store<VEC>(dst);
    } else {
        x.template store<VEC>(dst);
    }
}

template <typename Tout, typename Tc, bool VEC>
__global__ void __launch_bounds__(kCThreads, kBlocksPerSm) k_cache_read(RowArgs a) {
    __shared__ Place s_places[kWarps][32];
    Place *places = s_places[threadIdx.x >> 5];
    const int groups = 32 / a.lanes, group = (threadIdx.x & 31) / a.lanes;
    const int sub = threadIdx.x & (a.lanes - 1), d = sub * 8;
    const int64_t warp = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (warp == kWarps - 1) check_offsets(a.r);
    Tout *ko = const_cast<Tout *>(reinterpret_cast<const Tout *>(a.k));
    Tout *vo = const_cast<Tout *>(reinterpret_cast<const Tout *>(a.v));
    for (int64_t first = warp * a.chunk; first < a.rows; first += (int64_t)gridDim.x * kWarps * a.chunk) {
        const int n = (int)(a.rows - first < a.chunk ? a.rows - first : a.chunk);
        __syncwarp();
        find_places(a, first, n, places);
        __syncwarp();
        for (int r0 = 0; r0 < n; r0 += groups * kPasses) {
            Eight<Tc> x[kPasses], y[kPasses];
            float sk[kPasses], sv[kPasses];
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = r0 + i * groups + group;
                const Place &at = places[r < n ? r : 0];
                const bool live = r < n && at.live;
                sk[i] = sv[i] = 1.f;
                x[i].zero();  // a token without a place
                y[i].zero();
                if constexpr (sizeof(Tc) == 1) {
                    if (live) {
                        sk[i] = a.c.ks[at.scale];
                        sv[i] = a.c.vs[at.scale];
                    }
                }
                if (live && d < a.K)
                    x[i].template load<VEC>(reinterpret_cast<const Tc *>(a.c.k) + at.kc + d);
                if (live && d < a.V)
                    y[i].template load<VEC>(reinterpret_cast<const Tc *>(a.c.v) + at.vc + d);
            }
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = r0 + i * groups + group;
                if (r >= n) continue;
                if (d < a.K) read_row<Tout, Tc, VEC>(x[i], sk[i], ko + places[r].k + d);
                if (d < a.V) read_row<Tout, Tc, VEC>(y[i], sv[i], vo + places[r].v + d);
            }
        }
    }
}

// 8-element groups of every row start on a multiple of their own size.
bool rows_vec(const void *p, int64_t s0, int64_t s1, int64_t s2, int es) {
    const int w = es == 1 ? 8 : 16;
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(s0 * es) | (uintptr_t)(s1 * es) |
             (uintptr_t)(s2 * es)) & (uintptr_t)(w - 1)) == 0;
}

template <typename Tio, typename Tc>
cudaError_t launch_rows(bool write, bool vec, const RowArgs &a, cudaStream_t st) {
    const int64_t most = (int64_t)device_sms() * kBlocksPerSm;
    const int64_t blocks = (a.rows + (int64_t)a.chunk * kWarps - 1) / ((int64_t)a.chunk * kWarps);
    const dim3 g((unsigned)(blocks < most ? blocks : most));
    if (write) {
        if (vec) k_cache_write<Tio, Tc, true><<<g, kCThreads, 0, st>>>(a);
        else k_cache_write<Tio, Tc, false><<<g, kCThreads, 0, st>>>(a);
    } else {
        if (vec) k_cache_read<Tio, Tc, true><<<g, kCThreads, 0, st>>>(a);
        else k_cache_read<Tio, Tc, false><<<g, kCThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

template <typename Tio>
cudaError_t launch_fmt(bool write, bool vec, const RowArgs &a, cudaStream_t st) {
    if (a.c.dtype == GDR_E4M3) return launch_rows<Tio, __nv_fp8_e4m3>(write, vec, a, st);
    if (a.c.dtype == GDR_I8) return launch_rows<Tio, int8_t>(write, vec, a, st);
    return launch_rows<Tio, Tio>(write, vec, a, st);
}

}  // namespace

cudaError_t cache_rows(bool write, const PagedCache &c, const TokenRows &r, int dtype,
                       const void *k, const void *v, const TokStride &sk, const TokStride &sv,
                       int K, int V, cudaStream_t st) {
    RowArgs a{c, r, k, v, sk, sv, K, V, 2, 0, 32};
    a.rows = (rows_packed(r) ? r.T : r.N * r.T) * c.H;
    if (a.rows == 0) return cudaSuccess;
    while (a.lanes * 8 < K || a.lanes * 8 < V) a.lanes *= 2;
    // many rows: a full warp of look-ups; few: fewer rows a warp, on more SMs
    const int64_t warps = (int64_t)device_sms() * kBlocksPerSm * kWarps;
    while (a.chunk > 4 && a.rows < warps * a.chunk) a.chunk /= 2;
    const int es = dtype == GDR_F32 ? 4 : 2, ec = cache_quantised(c.dtype) ? 1 : es;
    const bool vec = rows_vec(k, sk.t, sk.h, 0, es) && rows_vec(v, sv.t, sv.h, 0, es) &&
                     rows_vec(c.k, c.kst[0], c.kst[1], c.kst[2], ec) &&
                     rows_vec(c.v, c.vst[0], c.vst[1], c.vst[2], ec);
    if (dtype == GDR_BF16) return launch_fmt<__nv_bfloat16>(write, vec, a, st);
    if (dtype == GDR_F16) return launch_fmt<__half>(write, vec, a, st);
    return launch_fmt<float>(write, vec, a, st);
}

}  // namespace gdr
