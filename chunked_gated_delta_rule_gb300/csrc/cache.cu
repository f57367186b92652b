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
// Both directions are bound by memory: each row is loaded, reduced and stored
// by the 2 to 32 lanes that hold 8 values of it each (16-byte loads of 16-bit
// types), a row's key and value by the same lanes with both loads issued
// before either is used.
#include <cuda_fp8.h>

#include "gdr_launch.cuh"
#include "paged.cuh"

namespace gdr {
namespace {

constexpr int kCThreads = 256;

struct RowArgs {
    PagedCache c;
    TokenRows r;
    const void *k, *v;  // the call's rows (written by the reader)
    TokStride sk, sv;
    int K, V, lanes;    // lanes a row: a power of two, 8 lanes >= max(K, V)
    int64_t rows;       // tokens x heads
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
    if constexpr (VEC && sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)e[i];
    } else if constexpr (VEC && sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)p[i];
    }
}

template <typename T>
__device__ __forceinline__ T from_float(float x) { return (T)x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ int8_t from_float<int8_t>(float x) {
    return (int8_t)max(-127, min(127, __float2int_rn(x)));
}
template <>
__device__ __forceinline__ __nv_fp8_e4m3 from_float<__nv_fp8_e4m3>(float x) {
    return __nv_fp8_e4m3(x);  // round to nearest even, saturating
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
    if constexpr (VEC && sizeof(T) <= 2) {
        __align__(16) T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = from_float<T>(x[i]);
        if constexpr (sizeof(T) == 2) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(e);
        else *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(e);
    } else if constexpr (VEC) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = from_float<T>(x[i]);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8_cache(const T *p, float (&x)[8]) {
    if constexpr (VEC && sizeof(T) == 1) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)e[i];
    } else {
        load8<T, VEC>(p, x);
    }
}

// Where row i (token-major, then head) lives: false when it has no place
// (before position 0, past the table, a page outside the cache).
__device__ __forceinline__ bool row_place(const RowArgs &a, int64_t i, int64_t &t, int &h,
                                          int &page, int &slot) {
    const bool live = i < a.rows;
    // the warp looks its first row's sequence up together, then every lane
    // steps to its own (a warp's rows span at most 16 tokens)
    const int64_t i0 = __shfl_sync(0xffffffffu, i, 0);
    const int H = a.c.H;
    const int64_t ti0 = (i0 < a.rows ? i0 : a.rows - 1) / H;
    int64_t n = find_seq(a.r, ti0);
    if (!live) return false;
    t = i / H;
    h = (int)(i - t * H);
    int64_t end = row_bound(a.r, n + 1);
    while (t >= end && n + 1 < a.r.N) end = row_bound(a.r, ++n + 1);
    if (rows_packed(a.r) && (t < row_bound(a.r, n) || t >= end || end > a.r.T)) {
        report(a.r.status, GDR_ERR_SEQLENS);
        return false;
    }
    const int64_t pos = (int64_t)a.c.kv_lens[n] - (end - t);
    if (pos < 0) return false;
    if (pos >= a.c.max_pages * a.c.page_size) {
        report(a.r.status, GDR_ERR_INDEX);
        return false;
    }
    const unsigned pi = (unsigned)pos / (unsigned)a.c.page_size;
    slot = (int)((unsigned)pos - pi * (unsigned)a.c.page_size);
    page = page_of(a.c, n, (int)pi, a.r.status);
    return page >= 0;
}

// max|x| over a row's lanes; NaN if the row holds a NaN or an infinity.
__device__ __forceinline__ float row_scale(const float (&x)[8], int lanes, float inv_qmax) {
    float m = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m = fmaxf(m, fabsf(x[i]));
        bad |= !isfinite(x[i]);
    }
    if (bad) m = INFINITY;
    for (int d = lanes >> 1; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    return isfinite(m) ? m * inv_qmax : __int_as_float(0x7fc00000);
}

template <typename Tc>
__device__ constexpr float inv_qmax() {
    return sizeof(Tc) > 1 ? 1.f : std::is_same<Tc, int8_t>::value ? 1.0f / 127.0f : 1.0f / 448.0f;
}

template <typename Tc, bool VEC>
__device__ __forceinline__ void write_row(float (&x)[8], bool live, Tc *dst, float *scale, int lanes,
                                          bool first_lane, bool in_row) {
    if constexpr (sizeof(Tc) == 1) {
        const float s = row_scale(x, lanes, inv_qmax<Tc>());
        const bool divide = s > 0.f;  // false for 0 and NaN
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = divide ? __fdiv_rn(x[i], s) : 0.f;
        if (live && first_lane) *scale = s;
    }
    if (live && in_row) store8<Tc, VEC>(dst, x);
}

template <typename Tin, typename Tc, bool VEC>
__global__ void __launch_bounds__(kCThreads) k_cache_write(RowArgs a) {
    const int sub = threadIdx.x & (a.lanes - 1), d = sub * 8;
    const int64_t i = (int64_t)blockIdx.x * (kCThreads / a.lanes) + threadIdx.x / a.lanes;
    int64_t t = 0;
    int h = 0, page = 0, slot = 0;
    const bool live = row_place(a, i, t, h, page, slot);
    float x[8] = {}, y[8] = {};
    if (live && d < a.K)
        load8<Tin, VEC>(reinterpret_cast<const Tin *>(a.k) + tok_at(a.sk, t, h) + d, x);
    if (live && d < a.V)
        load8<Tin, VEC>(reinterpret_cast<const Tin *>(a.v) + tok_at(a.sv, t, h) + d, y);
    const int64_t so = scale_at(a.c, page, slot, h);
    write_row<Tc, VEC>(x, live, reinterpret_cast<Tc *>(a.c.k) + page_at(a.c.kst, page, slot, h) + d,
                       a.c.ks + so, a.lanes, sub == 0, d < a.K);
    write_row<Tc, VEC>(y, live, reinterpret_cast<Tc *>(a.c.v) + page_at(a.c.vst, page, slot, h) + d,
                       a.c.vs + so, a.lanes, sub == 0, d < a.V);
}

template <typename Tout, typename Tc, bool VEC>
__global__ void __launch_bounds__(kCThreads) k_cache_read(RowArgs a) {
    const int sub = threadIdx.x & (a.lanes - 1), d = sub * 8;
    const int64_t i = (int64_t)blockIdx.x * (kCThreads / a.lanes) + threadIdx.x / a.lanes;
    int64_t t = 0;
    int h = 0, page = 0, slot = 0;
    const bool live = row_place(a, i, t, h, page, slot);
    if (i >= a.rows) return;
    t = i / a.c.H;
    h = (int)(i - t * a.c.H);
    float x[8] = {}, y[8] = {};
    if (live) {
        float sk = 1.f, sv = 1.f;
        if constexpr (sizeof(Tc) == 1) {
            const int64_t so = scale_at(a.c, page, slot, h);
            sk = a.c.ks[so];
            sv = a.c.vs[so];
        }
        if (d < a.K)
            load8_cache<Tc, VEC>(reinterpret_cast<const Tc *>(a.c.k) +
                                     page_at(a.c.kst, page, slot, h) + d, x);
        if (d < a.V)
            load8_cache<Tc, VEC>(reinterpret_cast<const Tc *>(a.c.v) +
                                     page_at(a.c.vst, page, slot, h) + d, y);
        if constexpr (sizeof(Tc) == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] *= sk;
                y[e] *= sv;
            }
        }
    }
    Tout *ko = const_cast<Tout *>(reinterpret_cast<const Tout *>(a.k));
    Tout *vo = const_cast<Tout *>(reinterpret_cast<const Tout *>(a.v));
    if (d < a.K) store8<Tout, VEC>(ko + tok_at(a.sk, t, h) + d, x);
    if (d < a.V) store8<Tout, VEC>(vo + tok_at(a.sv, t, h) + d, y);
}

// 8-element groups of every row start on a multiple of their own size.
bool rows_vec(const void *p, int64_t s0, int64_t s1, int64_t s2, int es) {
    const int w = es == 1 ? 8 : 16;
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(s0 * es) | (uintptr_t)(s1 * es) |
             (uintptr_t)(s2 * es)) & (uintptr_t)(w - 1)) == 0;
}

template <typename Tio, typename Tc>
cudaError_t launch_rows(bool write, bool vec, const RowArgs &a, cudaStream_t st) {
    const int64_t per = kCThreads / a.lanes, blocks = (a.rows + per - 1) / per;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 g((unsigned)blocks);
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
    RowArgs a{c, r, k, v, sk, sv, K, V, 2, 0};
    a.rows = (rows_packed(r) ? r.T : r.N * r.T) * c.H;
    if (a.rows == 0) return cudaSuccess;
    while (a.lanes * 8 < K || a.lanes * 8 < V) a.lanes *= 2;
    const int es = dtype == GDR_F32 ? 4 : 2, ec = cache_quantised(c.dtype) ? 1 : es;
    const bool vec = rows_vec(k, sk.t, sk.h, 0, es) && rows_vec(v, sv.t, sv.h, 0, es) &&
                     rows_vec(c.k, c.kst[0], c.kst[1], c.kst[2], ec) &&
                     rows_vec(c.v, c.vst[0], c.vst[1], c.vst[2], ec);
    if (dtype == GDR_BF16) return launch_fmt<__nv_bfloat16>(write, vec, a, st);
    if (dtype == GDR_F16) return launch_fmt<__half>(write, vec, a, st);
    return launch_fmt<float>(write, vec, a, st);
}

}  // namespace gdr
