// norm.cu -- root-mean-square norm of rows, with the residual's addition in
// front of it and an 8-bit output behind it, and its gradients.
//
//   r = x + res (rounded to the inputs' type: what the next layers see)
//   y = r rstd w,   rstd = 1 / sqrt(mean(r^2) + eps)
//   8 bits: s = max|y| (1 / 448) or max|y| (1 / 127) over the row or each `group` columns,
//   q = round(y / s) (0 where s = 0; s = NaN, q = 0 where y is not finite), as the paged
//   cache stores its rows.
//   dx = rstd (w dy - n mean(w dy n)) + dres with n = r rstd;  dw = sum over rows of dy n.
//
// Bound by memory: each value is read once and written once, r stays in
// registers between the sum of squares and the product.  A row of up to 1024
// values (32 of a thread) is a warp's, which waits for no other, as long as there
// are rows enough to fill the device.  Wider rows take a block of as few warps as
// hold them, and few rows one of more.
//
// BF16, 64K rows of 2048 with a residual into E4M3 with scales a 128 columns: 150 us (940 MB,
// 6.3 TB/s, 0.93 of what a copy reaches).  16K rows of 4096: forward 77 us, backward 102 and its
// sums 12 (537 MB each; 7.0 TB/s, some of it left in L2, and 5.3: three rows and the sums leave a
// thread 128 registers, so few rows are under way while others are summed).
#include <cuda_fp8.h>

#include "layer.cuh"

namespace gdr {
namespace {

constexpr int kWarpRows = 4;  // rows of a block whose warps take one each
constexpr int kMaxBlock = 512, kMaxNarrow = 1024;  // threads of a row
constexpr int kBwdThreads = 512;                   // of the backward on an SM: their registers fill it

template <typename T, int V, bool WARP>
constexpr int most_threads() {
    return WARP ? 32 * kWarpRows : V * sizeof(T) < 16 ? kMaxNarrow : kMaxBlock;
}

// Sums over the threads of a row, a warp or the block (sh: 32 pairs), of two values at once.
__device__ __forceinline__ float2 warp_sum(float2 x) {
#pragma unroll
    for (int i = 16; i; i >>= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, i);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, i);
    }
    return x;
}
template <bool WARP>
__device__ __forceinline__ float2 row_sum(float2 x, float2 *sh) {
    x = warp_sum(x);
    if constexpr (WARP) return x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
    __syncthreads();  // sh may still be read
    if (lane == 0) sh[warp] = x;
    __syncthreads();
    return warp_sum(lane < n ? sh[lane] : make_float2(0.f, 0.f));
}
// The largest of magnitudes, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
    for (int k = 1; k < LANES; k <<= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, k));
    return x;
}
template <bool WARP>
__device__ __forceinline__ float row_max(float x, float2 *sh) {
    x = lanes_max<32>(x);
    if constexpr (WARP) return x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
    __syncthreads();
    if (lane == 0) sh[warp].x = x;
    __syncthreads();
    return lanes_max<32>(lane < n ? sh[lane].x : 0.f);
}

template <typename T, int V>
__device__ __forceinline__ void load_weights(const NormArgs &a, int c, F2 (&w)[kPairs<V>]) {
    if (!a.w.p || c >= a.D) {
#pragma unroll
        for (int j = 0; j < kPairs<V>; ++j) w[j] = f2(1.f);
    } else if (a.w.f32) {
        Row<float, V> r;
        r.load((const float *)a.w.p + c, 16, V);
        widen2<float, V>(r, w);
    } else {
        Row<T, V> r;
        r.load((const T *)a.w.p + c, 16, V);
        widen2<T, V>(r, w);
    }
}

// V values y as 8-bit values, stored at p: round(y / s) from one reciprocal, whose product with y,
// corrected twice, is the rounded quotient (Markstein, 1990) unless y - p s underflows, which the
// division is for.
template <int V, bool E4M3>
__device__ __forceinline__ void store8(uint8_t *p, const F2 (&y)[kPairs<V>], float s) {
    constexpr int P = kPairs<V>;
    uint32_t w[(V + 3) / 4] = {};
    if (s > 0.f) {  // not NaN
        const float inv = __frcp_rn(s);
        const F2 s2 = f2(s), r = f2(inv), nr = f2(-inv), m1 = f2(-1.f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float lo, hi;
            if (s >= 0x1p-60f) {
                const F2 minus = y[i] * m1;
                F2 q = y[i] * r;
                q = fma2(nr, fma2(q, s2, minus), q);
                q = fma2(nr, fma2(q, s2, minus), q);
                split(q, lo, hi);
            } else {
                // a scale of a few of FP32's least units may be a third too small
                constexpr float kMost = E4M3 ? 448.f : 127.f;
                split(y[i], lo, hi);
                lo = fminf(fmaxf(__fdiv_rn(lo, s), -kMost), kMost);
                hi = fminf(fmaxf(__fdiv_rn(hi, s), -kMost), kMost);
            }
            uint32_t two;
            if constexpr (E4M3) {
                two = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
            } else {
                two = (__float2int_rn(lo) & 0xff) | (__float2int_rn(hi) & 0xff) << 8;
            }
            w[i / 2] |= two << 16 * (i % 2);
        }
    }
    if constexpr (V == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else if constexpr (V == 4) *reinterpret_cast<uint32_t *>(p) = w[0];
    else if constexpr (V == 2) *reinterpret_cast<uint16_t *>(p) = (uint16_t)w[0];
    else *p = (uint8_t)w[0];
}

__device__ __forceinline__ float scale_of(float most, float inv_max) {
    return most < __uint_as_float(0x7f800000u) ? __fmul_rn(most, inv_max) : __uint_as_float(0x7fffffffu);
}

// Where a thread's i-th vector of V values lies in its row (D: none).  A warp's neighbouring
// vectors cover 128 columns, those of a scale: half a warp's at once, or kRun of them in turn.
template <int V, bool WARP>
struct Columns {
    static constexpr int kRun = V >= 4 ? 1 : 4 / V;
    int lane, warp, warps;
    __device__ __forceinline__ Columns()
        : lane(threadIdx.x & 31), warp(WARP ? 0 : threadIdx.x >> 5), warps(WARP ? 1 : blockDim.x >> 5) {}
    __device__ __forceinline__ int first(int i) const {  // of the warp
        return (((i / kRun) * warps + warp) * kRun + i % kRun) * 32 * V;
    }
    __device__ __forceinline__ int operator()(int i) const { return first(i) + lane * V; }
};

// OUT: 0 the call's type, 1 E4M3, 2 8-bit integers, GROUP: with a scale each 128 columns.  V: values of a thread's load; D is a multiple.
template <typename T, int V, int NV, bool WARP, int OUT, bool GROUP>
__global__ void __launch_bounds__(most_threads<T, V, WARP>()) k_norm(NormArgs a) {
    constexpr int P = kPairs<V>;
    __shared__ float2 sh[32];
    const Columns<V, WARP> col;
    const int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.rows) return;  // whole warps
    const int D = (int)a.D;
    Row<T, V> r[NV];
    F2 sum2 = f2(0.f);
    {
        const T *x = (const T *)a.x + row * a.xs, *res = (const T *)a.res + row * a.ress;
        Row<T, V> s[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            r[i].load(x + c, 16, c < D ? V : 0);
            if (a.res) s[i].load(res + c, 16, c < D ? V : 0);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (col.first(i) >= D) continue;
            F2 f[P];
            widen2<T, V>(r[i], f);
            if (a.res) {
                F2 g[P];
                widen2<T, V>(s[i], g);
#pragma unroll
                for (int j = 0; j < P; ++j) f[j] = f[j] + g[j];
                narrow2<T, V>(f, r[i]);
                const int c = col(i);
                if (c < D) r[i].store((T *)a.r + row * a.rs + c, 16, V);
                widen2<T, V>(r[i], f);
            }
#pragma unroll
            for (int j = 0; j < P; ++j) sum2 = fma2(f[j], f[j], sum2);
        }
    }
    const float sum = row_sum<WARP>(make_float2(both(sum2), 0.f), sh).x;
    const F2 rstd = f2(rsqrtf(sum / (float)D + a.eps));
    auto normed = [&](int i, F2(&y)[P]) {
        F2 w[P];
        widen2<T, V>(r[i], y);
        load_weights<T, V>(a, col(i), w);
#pragma unroll
        for (int j = 0; j < P; ++j) y[j] = y[j] * rstd * w[j];
    };
    auto largest = [](const F2(&y)[P], float m) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float lo, hi;
            split(y[j], lo, hi);
            m = max_nan(m, fabsf(lo));
            if (V > 1) m = max_nan(m, fabsf(hi));
        }
        return m;
    };
    if constexpr (OUT == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            if (col.first(i) >= D) continue;
            F2 y[P];
            normed(i, y);
            if (c < D) store2<T, V>((T *)a.y + row * a.ys + c, y);
        }
    } else {
        // values past D are zeros and, in a row without a finite rstd, NaN: they do not count
        const float inv_max = OUT == 1 ? 1.f / 448.f : 1.f / 127.f;
        constexpr int kRun = Columns<V, WARP>::kRun;
        F2 y[NV][P];
        float most = 0.f;
        if constexpr (!GROUP) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (col.first(i) >= D) continue;
                normed(i, y[i]);
                if (col(i) < D) most = largest(y[i], most);
            }
            most = row_max<WARP>(most, sh);
            if (threadIdx.x % (WARP ? 32 : kMaxNarrow) == 0) a.scale[row] = scale_of(most, inv_max);
        }
#pragma unroll
        for (int i0 = 0; i0 < NV; i0 += kRun) {
            if (col.first(i0) >= D) continue;
            if constexpr (GROUP) {
                most = 0.f;
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    normed(i0 + k, y[i0 + k]);
                    if (col(i0 + k) < D) most = largest(y[i0 + k], most);
                }
                most = lanes_max<(V >= 4 ? 128 / V : 32)>(most);
            }
            const float s = scale_of(most, inv_max);
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                const int c = col(i0 + k);
                if (c >= D) continue;
                store8<V, OUT == 1>((uint8_t *)a.y + row * a.ys + c, y[i0 + k], s);
                if (GROUP && c % 128 == 0) a.scale[row * ((D + 127) / 128) + c / 128] = s;
            }
        }
    }
}

// A block takes rows blockIdx, blockIdx + gridDim, ... (WARP: its warps each one) and holds the
// sums of dy n of its columns; part gets those of the whole block.
template <typename T, int V, int NV, bool WARP>
__global__ void __launch_bounds__(most_threads<T, V, WARP>()) k_norm_bwd(NormArgs a) {
    constexpr int P = kPairs<V>;
    extern __shared__ float acc[];  // WARP: [kWarpRows][D]
    __shared__ float2 sh[32];
    const Columns<V, WARP> col;
    const int64_t step = WARP ? (int64_t)gridDim.x * kWarpRows : gridDim.x;
    const int D = (int)a.D;
    F2 dw[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j) dw[i][j] = f2(0.f);
    for (int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
         row < a.rows; row += step) {
        Row<T, V> r[NV], dy[NV], dr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            const int valid = c < D ? V : 0;
            r[i].load((const T *)a.r + row * a.rs + c, 16, valid);
            dy[i].load((const T *)a.dy + row * a.dys + c, 16, valid);
            if (a.dres) dr[i].load((const T *)a.dres + row * a.dress + c, 16, valid);
            else dr[i].zero();
        }
        F2 sum2 = f2(0.f), dot2 = f2(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F2 f[P], g[P], w[P];
            widen2<T, V>(r[i], f);
            widen2<T, V>(dy[i], g);
            load_weights<T, V>(a, col(i), w);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                sum2 = fma2(f[j], f[j], sum2);
                dot2 = fma2(f[j], g[j] * w[j], dot2);
            }
        }
        const float2 sums = row_sum<WARP>(make_float2(both(sum2), both(dot2)), sh);
        const float rstd = rsqrtf(sums.x / (float)D + a.eps);
        const F2 rs = f2(rstd), k = f2(-sums.y * rstd / (float)D);  // -mean(w dy n)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            F2 f[P], g[P], w[P], e[P];
            widen2<T, V>(r[i], f);
            widen2<T, V>(dy[i], g);
            widen2<T, V>(dr[i], e);
            load_weights<T, V>(a, c, w);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const F2 n = f[j] * rs;
                dw[i][j] = fma2(g[j], n, dw[i][j]);
                e[j] = fma2(rs, fma2(n, k, g[j] * w[j]), e[j]);
            }
            if (c < D) store2<T, V>((T *)a.dx + row * D + c, e);
        }
    }
    if (!a.dw) return;
    float *to = WARP ? acc + (threadIdx.x >> 5) * D : a.part + (int64_t)blockIdx.x * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = col(i);
        if (c < D) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                float lo, hi;
                split(dw[i][j], lo, hi);
                to[c + 2 * j] = lo;
                if (V > 1) to[c + 2 * j + 1] = hi;
            }
        }
    }
    if constexpr (WARP) {  // the block's warps join their sums
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += blockDim.x) {
            float s = acc[c];
#pragma unroll
            for (int k = 1; k < kWarpRows; ++k) s += acc[k * D + c];
            a.part[(int64_t)blockIdx.x * D + c] = s;
        }
    }
}

__global__ void __launch_bounds__(kColumnThreads) k_norm_weight(NormArgs a, int64_t blocks) {
    const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    pdl_wait();
    const float s = column_sum(a.part + c, a.D, blocks, c < a.D);
    if (threadIdx.x < 32 && c < a.D) a.dw[c] = s;
}

// Threads of a row (32: a warp) and vectors of a thread.  A row takes as few warps as hold it with
// `most` vectors a thread (E4M3, 16K rows of 4096 / 5120: 88 / 107 us with 4 vectors, 126 / 186 with 8,
// 100 / 171 with 2); with few rows it is spread over more, up to a vector each, until they fill the
// device (64 / 1024 / 4096 rows of 2048 into E4M3: 12 / 14 / 24 us, 18 / 18 / 30 without).  Narrow loads
// (rows off 16 bytes) have a block a row and 4 or 16 of them a thread.
struct Shape {
    int threads, nv;
};
Shape shape_of(int64_t rows, int64_t D, int vec, int es, int most) {
    const int64_t all = D / vec;
    int threads = 32;
    auto need = [&] { return (all + threads - 1) / threads; };
    if (vec * es < 16) {
        threads = 64;
        while (threads < kMaxNarrow && need() > 4) threads *= 2;
        return Shape{threads, need() > 4 ? 16 : 4};
    }
    if (need() > most) threads = (int)((all + 32 * most - 1) / (32 * most)) * 32;
    while (need() > 1 && 2 * threads <= kMaxBlock && rows * threads < (int64_t)device_sms() * 1024) threads *= 2;
    int k = 1;
    while (k < need()) k *= 2;
    return Shape{threads, k};
}
// Vectors of a thread at most: 32 values, so that 512 threads hold a row of 16384.
constexpr int most_of(int es) { return es == 2 ? 4 : 8; }

// Calls f(V, NV, WARP) as constants.
template <typename T, int MOST, typename F>
cudaError_t with_shape(const NormArgs &a, const Shape &s, F f) {
    constexpr std::integral_constant<bool, true> warp{};
    constexpr std::integral_constant<bool, false> block{};
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 4> four{};
    constexpr std::integral_constant<int, 16> sixteen{};
    if (a.vec == 1) return s.nv == 4 ? f(one, four, block) : f(one, sixteen, block);
    if constexpr (sizeof(T) == 2) {
        constexpr std::integral_constant<int, 2> two{};
        if (a.vec == 2) return s.nv == 4 ? f(two, four, block) : f(two, sixteen, block);
    }
    constexpr std::integral_constant<int, 16 / (int)sizeof(T)> wide{};
    auto go = [&](auto nv) { return s.threads == 32 ? f(wide, nv, warp) : f(wide, nv, block); };
    if (s.nv == 1) return go(one);
    if (s.nv == 2) return go(std::integral_constant<int, 2>{});
    if (MOST == 4 || s.nv == 4) return go(four);
    return go(std::integral_constant<int, MOST>{});
}

template <typename T, int OUT, bool GROUP>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t st) {
    constexpr int kMost = most_of(sizeof(T));
    const Shape s = shape_of(a.rows, a.D, a.vec, sizeof(T), kMost);
    return with_shape<T, kMost>(a, s, [&](auto v, auto nv, auto w) {
        constexpr bool WARP = decltype(w)::value;
        const unsigned grid = (unsigned)(WARP ? (a.rows + kWarpRows - 1) / kWarpRows : a.rows);
        k_norm<T, decltype(v)::value, decltype(nv)::value, WARP, OUT, GROUP>
            <<<grid, WARP ? 32 * kWarpRows : s.threads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t launch_norm_bwd(const NormArgs &a, int64_t blocks, cudaStream_t st) {
    constexpr int kMost = most_of(sizeof(T));
    const Shape s = shape_of(a.rows, a.D, a.vec, sizeof(T), kMost);
    return with_shape<T, kMost>(a, s, [&](auto v, auto nv, auto w) {
        constexpr bool WARP = decltype(w)::value;
        k_norm_bwd<T, decltype(v)::value, decltype(nv)::value, WARP>
            <<<(unsigned)blocks, WARP ? 32 * kWarpRows : s.threads,
               WARP ? kWarpRows * (size_t)a.D * sizeof(float) : 0, st>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t norm_fwd(const NormArgs &a, int dtype, int out_dtype, cudaStream_t st) {
    auto go = [&](auto t) {
        using T = decltype(t);
        if (out_dtype == GDR_E4M3) return a.group ? launch_norm<T, 1, true>(a, st) : launch_norm<T, 1, false>(a, st);
        if (out_dtype == GDR_I8) return a.group ? launch_norm<T, 2, true>(a, st) : launch_norm<T, 2, false>(a, st);
        return launch_norm<T, 0, false>(a, st);
    };
    if (dtype == GDR_BF16) return go(__nv_bfloat16{});
    if (dtype == GDR_F16) return go(__half{});
    return go(float{});
}

// Blocks of the backward pass: as many as the device holds at once, or as there are rows.
int64_t norm_bwd_blocks(int64_t rows, int64_t D, int vec, int dtype) {
    const int es = dtype == GDR_F32 ? 4 : 2;
    const Shape s = shape_of(rows, D, vec, es, most_of(es));
    const int64_t all = s.threads == 32 ? (rows + kWarpRows - 1) / kWarpRows : rows;
    const int block = s.threads == 32 ? 32 * kWarpRows : s.threads;
    const int64_t fit = (int64_t)device_sms() * (block < kBwdThreads ? kBwdThreads / block : 1);
    return all < fit ? all : fit;
}

cudaError_t norm_bwd(const NormArgs &a, int dtype, int64_t blocks, cudaStream_t st) {
    if (dtype == GDR_BF16) return launch_norm_bwd<__nv_bfloat16>(a, blocks, st);
    if (dtype == GDR_F16) return launch_norm_bwd<__half>(a, blocks, st);
    return launch_norm_bwd<float>(a, blocks, st);
}

cudaError_t norm_weight_grad(const NormArgs &a, int64_t blocks, cudaStream_t st) {
    return launch_pdl(k_norm_weight, dim3((unsigned)((a.D + 31) / 32)), dim3(kColumnThreads), 0, st, a, blocks);
}

}  // namespace gdr
