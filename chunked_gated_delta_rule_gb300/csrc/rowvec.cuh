// rowvec.cuh -- what the operators over rows of channels share (short
// convolution, selective scan, norm): a thread's consecutive values of a row in
// any of the three types, parameters in either type, the sequence that a token
// belongs to, and sigmoid and softplus.
#pragma once

#include <type_traits>

#include "paged.cuh"

namespace gdr {

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __bfloat162float(x);
    else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
    else return x;
}
template <typename T>
__device__ __forceinline__ T from_f32(float x) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(x);
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
    else return x;
}

// V consecutive values as they lie in memory.  `bytes` is what their address is a
// multiple of (the same for a whole call, so the branch is uniform): wide loads
// and stores need 16, or all the values' bytes where those are fewer.  Values
// from `valid` on are zeros and are not touched in memory.
template <typename T, int V>
struct Row {
    static constexpr int kBytes = V * (int)sizeof(T), kNeed = kBytes < 16 ? kBytes : 16;
    static constexpr int kWords = (kBytes + 3) / 4;
    static_assert(kBytes <= 32 && (kBytes & (kBytes - 1)) == 0, "up to two 16-byte loads");
    uint32_t w[kWords];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const T *p, int bytes, int valid) {
        if (valid >= V && bytes >= kNeed) {
            if constexpr (kBytes % 16 == 0) {
#pragma unroll
                for (int i = 0; i < kWords / 4; ++i) {
                    const uint4 x = reinterpret_cast<const uint4 *>(p)[i];
                    w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
                }
            } else if constexpr (kBytes == 8) {
                const uint2 x = *reinterpret_cast<const uint2 *>(p);
                w[0] = x.x; w[1] = x.y;
            } else if constexpr (kBytes == 4) {
                w[0] = *reinterpret_cast<const uint32_t *>(p);
            } else {
                w[0] = *reinterpret_cast<const uint16_t *>(p);
            }
        } else {
            zero();
            T *e = reinterpret_cast<T *>(w);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < valid) e[i] = p[i];
        }
    }
    __device__ __forceinline__ void store(T *p, int bytes, int valid) const {
        if (valid >= V && bytes >= kNeed) {
            if constexpr (kBytes % 16 == 0) {
#pragma unroll
                for (int i = 0; i < kWords / 4; ++i)
                    reinterpret_cast<uint4 *>(p)[i] =
                        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            } else if constexpr (kBytes == 8) {
                *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
            } else if constexpr (kBytes == 4) {
                *reinterpret_cast<uint32_t *>(p) = w[0];
            } else {
                *reinterpret_cast<uint16_t *>(p) = (uint16_t)w[0];
            }
        } else {
            const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < valid) p[i] = e[i];
        }
    }
    __device__ __forceinline__ void widen(float (&x)[V]) const {
        if constexpr (V > 1 && std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = to_f32(e[i]);
        }
    }
    // Rounded to nearest, ties to even.
    __device__ __forceinline__ void narrow(const float (&x)[V]) {
        if constexpr (std::is_same<T, float>::value) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(x[i]);
        } else if constexpr (V == 1) {
            const T y = from_f32<T>(x[0]);
            w[0] = *reinterpret_cast<const uint16_t *>(&y);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&y);
                } else {
                    const __half2 y = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&y);
                }
            }
        }
    }
};

// A parameter tensor in the call's type or in FP32.
struct Param {
    const void *p;
    int f32;
};
template <typename T>
__device__ __forceinline__ float param_at(const Param &a, int64_t i) {
    return a.f32 ? reinterpret_cast<const float *>(a.p)[i]
                 : to_f32(reinterpret_cast<const T *>(a.p)[i]);
}

// Largest of 16, 8, 4, 2 that divides all the given byte counts and addresses.
inline int common_bytes(std::initializer_list<uint64_t> of) {
    uint64_t all = 16;
    for (uint64_t x : of) all |= x;
    return (int)(all & (~all + 1));
}
inline uint64_t addr(const void *p) { return (uint64_t)reinterpret_cast<uintptr_t>(p); }

__device__ __forceinline__ int64_t total_tokens(const TokenRows &r) {
    return rows_packed(r) ? r.T : r.N * r.T;
}

// Sum of the n values p[0], p[step], ..: a block takes 32 of them side by side (thread l + 32 k the
// k-th strand of column l), a row of each strand at once, the strands joined in their order.
// Threads 0 to 31 get the sums.
constexpr int kColumnThreads = 512;
__device__ __forceinline__ float column_sum(const float *p, int64_t step, int64_t n, bool in) {
    constexpr int kStrands = kColumnThreads / 32;
    __shared__ float sum[kStrands][33];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    float s = 0.f;
    if (in) {
#pragma unroll 8
        for (int64_t i = strand; i < n; i += kStrands) s += p[i * step];
    }
    sum[strand][lane] = s;
    __syncthreads();
    if (strand == 0)
#pragma unroll
        for (int k = 1; k < kStrands; ++k) s += sum[k][lane];
    return s;
}

__device__ __forceinline__ bool same_in_warp(int64_t x) {
    return __all_sync(0xffffffffu, x == __shfl_sync(0xffffffffu, x, 0));
}

// The sequence n = [s, e) that holds token t, found by a warp whose lanes all look for the same
// one (`together`: every lane takes part), or by a thread on its own.  A token that none holds lies
// in a hole: n = -1, and the hole reaches to e.
struct Seq {
    int64_t n, s, e;
};
__device__ __forceinline__ Seq seq_at(const TokenRows &r, int64_t t, bool together) {
    if (!rows_packed(r)) {
        const int64_t n = t / r.T;
        return Seq{n, n * r.T, (n + 1) * r.T};
    }
    int64_t lo = 0, hi = r.N;
    if (together) {
        lo = find_seq(r, t);
    } else {
        while (hi - lo > 1) {  // the last n with cu[n] <= t
            const int64_t mid = (lo + hi) >> 1;
            if (row_bound(r, mid) <= t) lo = mid;
            else hi = mid;
        }
    }
    const int64_t s = row_bound(r, lo), e = row_bound(r, lo + 1);
    if (s >= 0 && s <= t && t < e && e <= r.T) return Seq{lo, s, e};
    return Seq{-1, t, lo == r.N - 1 && t >= e ? r.T : t + 1};
}

// Row of a state pool that sequence n has, or -1 (reported).
__device__ __forceinline__ int64_t state_row(const int32_t *idx, int64_t n_states, int64_t n,
                                             int32_t *status) {
    const int64_t row = idx ? (int64_t)idx[n] : n;
    if (row >= 0 && row < n_states) return row;
    report(status, GDR_ERR_INDEX);
    return -1;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two FP32 values in a register pair, worked on by one instruction.  It takes the FMA pipe for two
// cycles, as two single ones do (2.1 cycles a scheduler either way, measured alone), so what it saves
// is the second one's issue slot, which others take meanwhile (with one integer operation beside it 2.4
// cycles, with two 2.9): the scan's inner loop takes 5.5 cycles a state with pairs and 6.2 without (8
// states of a channel, measured alone).
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void split(F2 a, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 ex2(F2 a) {
    float lo, hi;
    split(a, lo, hi);
    return f2(ex2(lo), ex2(hi));
}
__device__ __forceinline__ float both(F2 a) {
    float lo, hi;
    split(a, lo, hi);
    return lo + hi;
}

// V values as pairs (one value: a pair with nothing beside it).
template <int V>
constexpr int kPairs = (V + 1) / 2;

template <typename T, int V>
__device__ __forceinline__ void widen2(const Row<T, V> &r, F2 (&x)[kPairs<V>]) {
    float f[V];
    r.widen(f);
    if constexpr (V == 1) {
        x[0] = f2(f[0], 0.f);
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) x[j] = f2(f[2 * j], f[2 * j + 1]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void narrow2(const F2 (&x)[kPairs<V>], Row<T, V> &r) {
    float f[2 * kPairs<V>], g[V];
#pragma unroll
    for (int j = 0; j < kPairs<V>; ++j) split(x[j], f[2 * j], f[2 * j + 1]);
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = f[j];
    r.narrow(g);
}
template <typename T, int V>
__device__ __forceinline__ void store2(T *p, const F2 (&x)[kPairs<V>]) {
    Row<T, V> r;
    narrow2<T, V>(x, r);
    r.store(p, 16, V);
}

// 1 / (1 + e^-x)
__device__ __forceinline__ F2 sigmoid2(F2 x) {
    float a, b;
    split(ex2(x * f2(-kLog2e)) + f2(1.f), a, b);
    return f2(rcp(a), rcp(b));
}
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

}  // namespace gdr
