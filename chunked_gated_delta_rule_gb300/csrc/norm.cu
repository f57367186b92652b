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
// registers between the sum of squares and the product.  A warp takes a row
// alone, without waiting for others, as long as there are rows enough to fill
// the device; with fewer rows a block takes one.
#include <cuda_fp8.h>

#include "layer.cuh"

namespace gdr {
namespace {

constexpr int kWarpRows = 4;  // rows of a block whose warps take one each
constexpr int kMaxBlock = 512, kMaxNarrow = 1024;  // threads of a row

template <typename T, int V, bool WARP>
constexpr int most_threads() {
    return WARP ? 32 * kWarpRows : V * sizeof(T) < 16 ? kMaxNarrow : kMaxBlock;
}

// Sum over the threads of a row: a warp, or the block (sh: 32 floats).
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
    return x;
}
template <bool WARP>
__device__ __forceinline__ float row_sum(float x, float *sh) {
    x = warp_sum(x);
    if constexpr (WARP) return x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
    __syncthreads();  // sh may still be read
    if (lane == 0) sh[warp] = x;
    __syncthreads();
    return warp_sum(lane < n ? sh[lane] : 0.f);
}
template <bool WARP>
__device__ __forceinline__ uint32_t row_max(uint32_t x, float *sh) {
    x = __reduce_max_sync(0xffffffffu, x);
    if constexpr (WARP) return x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
    __syncthreads();
    if (lane == 0) sh[warp] = __uint_as_float(x);
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < n ? __float_as_uint(sh[lane]) : 0u);
}

template <typename T, int V>
__device__ __forceinline__ void load_weights(const NormArgs &a, int64_t c, float (&w)[V]) {
    if (!a.w.p || c >= a.D) {
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = 1.f;
    } else if (a.w.f32) {
        Row<float, V> r;
        r.load((const float *)a.w.p + c, 16, V);
        r.widen(w);
    } else {
        Row<T, V> r;
        r.load((const T *)a.w.p + c, 16, V);
        r.widen(w);
    }
}

// round(y / s), from one reciprocal: its product with y, corrected twice, is the rounded quotient
// (Markstein, 1990) unless y - p s underflows, which the division is for.
__device__ __forceinline__ float quotient(float y, float s, float inv) {
    if (s < 0x1p-60f) return s > 0.f ? __fdiv_rn(y, s) : 0.f;
    float p = y * inv;
    p = fmaf(-inv, fmaf(p, s, -y), p);
    return fmaf(-inv, fmaf(p, s, -y), p);
}

// V values y as 8-bit values, stored at p.
template <int V, bool E4M3>
__device__ __forceinline__ void store8(uint8_t *p, const float (&y)[V], float s) {
    const float inv = s >= 0x1p-60f ? __frcp_rn(s) : 0.f;
    uint32_t w[(V + 3) / 4] = {};
    if (s == s) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float lo = quotient(y[i], s, inv), hi = i + 1 < V ? quotient(y[i + 1 < V ? i + 1 : i], s, inv) : 0.f;
            uint32_t two;
            if constexpr (E4M3) {
                two = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
            } else {
                two = (__float2int_rn(lo) & 0xff) | (__float2int_rn(hi) & 0xff) << 8;
            }
            w[i / 4] |= two << 8 * (i % 4);
        }
    }
    if constexpr (V == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else if constexpr (V == 4) *reinterpret_cast<uint32_t *>(p) = w[0];
    else if constexpr (V == 2) *reinterpret_cast<uint16_t *>(p) = (uint16_t)w[0];
    else *p = (uint8_t)w[0];
}

__device__ __forceinline__ float scale_of(uint32_t most, float inv_max) {
    return most >= 0x7f800000u ? __uint_as_float(0x7fffffffu)
                               : __fmul_rn(__uint_as_float(most), inv_max);
}

// Where a thread's i-th vector of V values lies in its row (D: none).  A warp's neighbouring
// vectors cover 128 columns, those of a scale: half a warp's at once, or kRun of them in turn.
template <int V, bool WARP>
struct Columns {
    static constexpr int kRun = V >= 4 ? 1 : 4 / V;
    int lane, warp, warps;
    __device__ __forceinline__ Columns()
        : lane(threadIdx.x & 31), warp(WARP ? 0 : threadIdx.x >> 5), warps(WARP ? 1 : blockDim.x >> 5) {}
    __device__ __forceinline__ int64_t operator()(int i) const {
        return (int64_t)((((i / kRun) * warps + warp) * kRun + i % kRun) * 32 + lane) * V;
    }
};

// OUT: 0 the call's type, 1 E4M3, 2 8-bit integers.  V: values of a thread's load; D is a multiple.
template <typename T, int V, int NV, bool WARP, int OUT>
__global__ void __launch_bounds__(most_threads<T, V, WARP>()) k_norm(NormArgs a) {
    __shared__ float sh[32];
    const Columns<V, WARP> col;
    const int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.rows) return;  // whole warps
    const int64_t D = a.D;
    Row<T, V> r[NV];
    float sum = 0.f;
    {
        Row<T, V> s[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = col(i);
            r[i].load((const T *)a.x + row * a.xs + c, 16, c < D ? V : 0);
            if (a.res) s[i].load((const T *)a.res + row * a.ress + c, 16, c < D ? V : 0);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[V];
            r[i].widen(f);
            if (a.res) {
                float g[V];
                s[i].widen(g);
#pragma unroll
                for (int j = 0; j < V; ++j) f[j] += g[j];
                r[i].narrow(f);
                const int64_t c = col(i);
                if (c < D) r[i].store((T *)a.r + row * a.rs + c, 16, V);
                r[i].widen(f);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) sum = fmaf(f[j], f[j], sum);
        }
    }
    sum = row_sum<WARP>(sum, sh);
    const float rstd = rsqrtf(sum / (float)D + a.eps);
    auto normed = [&](int i, float(&y)[V]) {
        float w[V];
        r[i].widen(y);
        load_weights<T, V>(a, col(i), w);
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = y[j] * rstd * w[j];
    };
    auto largest = [](const float(&y)[V], uint32_t m) {
#pragma unroll
        for (int j = 0; j < V; ++j) m = max(m, __float_as_uint(y[j]) & 0x7fffffffu);
        return m;
    };
    if constexpr (OUT == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = col(i);
            float y[V];
            normed(i, y);
            Row<T, V> out;
            out.narrow(y);
            if (c < D) out.store((T *)a.y + row * a.ys + c, 16, V);
        }
    } else {
        // a row without a finite rstd has NaN where its values are zeros past D: masked by c < D
        const float inv_max = OUT == 1 ? 1.f / 448.f : 1.f / 127.f;
        const int64_t groups = a.group ? (D + 127) / 128 : 1;
        uint32_t most = 0;
        if (!a.group) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float y[V];
                normed(i, y);
                if (col(i) < D) most = largest(y, most);
            }
            most = row_max<WARP>(most, sh);
        }
        constexpr int kRun = Columns<V, WARP>::kRun;
#pragma unroll
        for (int i0 = 0; i0 < NV; i0 += kRun) {
            float y[kRun][V];
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                normed(i0 + k, y[k]);
                if (col(i0 + k) < D) m = largest(y[k], m);
            }
            if (a.group) {
#pragma unroll
                for (int k = 1; k < 32 && k < 128 / V; k <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
                most = m;
            }
            const float s = scale_of(most, inv_max);
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                const int64_t c = col(i0 + k);
                if (c >= D) continue;
                store8<V, OUT == 1>((uint8_t *)a.y + row * a.ys + c, y[k], s);
                if (a.group ? c % 128 == 0 : c == 0) a.scale[row * groups + (a.group ? c / 128 : 0)] = s;
            }
        }
    }
}

// A block takes rows blockIdx, blockIdx + gridDim, ... (WARP: its warps each one) and holds the
// sums of dy n of its columns; part gets those of the whole block.
template <typename T, int V, int NV, bool WARP>
__global__ void __launch_bounds__(most_threads<T, V, WARP>()) k_norm_bwd(NormArgs a) {
    extern __shared__ float acc[];  // WARP: [kWarpRows][D]
    __shared__ float sh[32];
    const Columns<V, WARP> col;
    const int64_t step = WARP ? (int64_t)gridDim.x * kWarpRows : gridDim.x, D = a.D;
    float dw[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
    for (int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
         row < a.rows; row += step) {
        Row<T, V> r[NV], dy[NV], dr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = col(i);
            const int valid = c < D ? V : 0;
            r[i].load((const T *)a.r + row * a.rs + c, 16, valid);
            dy[i].load((const T *)a.dy + row * a.dys + c, 16, valid);
            if (a.dres) dr[i].load((const T *)a.dres + row * a.dress + c, 16, valid);
            else dr[i].zero();
        }
        float sum = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[V], g[V], w[V];
            r[i].widen(f);
            dy[i].widen(g);
            load_weights<T, V>(a, col(i), w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                sum = fmaf(f[j], f[j], sum);
                dot = fmaf(f[j], g[j] * w[j], dot);
            }
        }
        sum = row_sum<WARP>(sum, sh);
        dot = row_sum<WARP>(dot, sh);
        const float rstd = rsqrtf(sum / (float)D + a.eps);
        const float k = dot * rstd / (float)D;  // mean(w dy n)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = col(i);
            float f[V], g[V], w[V], e[V];
            r[i].widen(f);
            dy[i].widen(g);
            dr[i].widen(e);
            load_weights<T, V>(a, c, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float n = f[j] * rstd;
                dw[i][j] = fmaf(g[j], n, dw[i][j]);
                e[j] = fmaf(rstd, fmaf(-n, k, g[j] * w[j]), e[j]);
            }
            Row<T, V> out;
            out.narrow(e);
            if (c < D) out.store((T *)a.dx + row * D + c, 16, V);
        }
    }
    if (!a.dw) return;
    float *to = WARP ? acc + (threadIdx.x >> 5) * D : a.part + blockIdx.x * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = col(i);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c < D) to[c + j] = dw[i][j];
    }
    if constexpr (WARP) {  // the block's warps join their sums
        __syncthreads();
        for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
            float s = acc[c];
#pragma unroll
            for (int k = 1; k < kWarpRows; ++k) s += acc[k * D + c];
            a.part[blockIdx.x * D + c] = s;
        }
    }
}

__global__ void __launch_bounds__(256) k_norm_weight(NormArgs a, int64_t blocks) {
    __shared__ float sum[8][33];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    pdl_wait();
    float s = 0.f;
    if (c < a.D)
        for (int64_t b = strand; b < blocks; b += 8) s += a.part[b * a.D + c];
    sum[strand][lane] = s;
    __syncthreads();
    if (strand || c >= a.D) return;
    for (int j = 1; j < 8; ++j) s += sum[j][lane];
    a.dw[c] = s;
}

// Threads of a row (32: a warp) and vectors of a thread.  With rows enough a
// warp takes up to `most` vectors; else a row is spread over more threads until
// they fill the device or hold a vector each.  Narrow loads (rows off 16 bytes)
// have a block a row and 4 or 16 of them a thread.
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
    while (need() > most) threads *= 2;
    while (need() > 1 && threads < kMaxBlock && rows * threads < (int64_t)device_sms() * 1024) threads *= 2;
    int k = 1;
    while (k < need()) k *= 2;
    return Shape{threads, k};
}
constexpr int kMostFwd = 8;  // 16384 values: 512 threads of 8 vectors of 4 values
// Backward a thread holds three rows and the sums: 32 values of each at most.
constexpr int most_bwd(int es) { return es == 2 ? 4 : 8; }

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

template <typename T, int OUT>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t st) {
    const Shape s = shape_of(a.rows, a.D, a.vec, sizeof(T), kMostFwd);
    return with_shape<T, kMostFwd>(a, s, [&](auto v, auto nv, auto w) {
        constexpr bool WARP = decltype(w)::value;
        const unsigned grid = (unsigned)(WARP ? (a.rows + kWarpRows - 1) / kWarpRows : a.rows);
        k_norm<T, decltype(v)::value, decltype(nv)::value, WARP, OUT>
            <<<grid, WARP ? 32 * kWarpRows : s.threads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t launch_norm_bwd(const NormArgs &a, int64_t blocks, cudaStream_t st) {
    constexpr int kMost = most_bwd(sizeof(T));
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
        if (out_dtype == GDR_E4M3) return launch_norm<T, 1>(a, st);
        if (out_dtype == GDR_I8) return launch_norm<T, 2>(a, st);
        return launch_norm<T, 0>(a, st);
    };
    if (dtype == GDR_BF16) return go(__nv_bfloat16{});
    if (dtype == GDR_F16) return go(__half{});
    return go(float{});
}

// Blocks of the backward pass: as many as the device holds at once, or as there are rows.
int64_t norm_bwd_blocks(int64_t rows, int64_t D, int vec, int dtype) {
    const int es = dtype == GDR_F32 ? 4 : 2;
    const Shape s = shape_of(rows, D, vec, es, most_bwd(es));
    const int64_t all = s.threads == 32 ? (rows + kWarpRows - 1) / kWarpRows : rows;
    const int block = s.threads == 32 ? 32 * kWarpRows : s.threads;
    const int64_t fit = (int64_t)device_sms() * (1024 / block);
    return all < fit ? all : fit;
}

cudaError_t norm_bwd(const NormArgs &a, int dtype, int64_t blocks, cudaStream_t st) {
    if (dtype == GDR_BF16) return launch_norm_bwd<__nv_bfloat16>(a, blocks, st);
    if (dtype == GDR_F16) return launch_norm_bwd<__half>(a, blocks, st);
    return launch_norm_bwd<float>(a, blocks, st);
}

cudaError_t norm_weight_grad(const NormArgs &a, int64_t blocks, cudaStream_t st) {
    return launch_pdl(k_norm_weight, dim3((unsigned)((a.D + 31) / 32)), dim3(256), 0, st, a, blocks);
}

}  // namespace gdr
