// conv.cu -- the short causal convolution along a sequence, one filter of W
// taps for each channel, its gradients, and its form for single tokens.
//
//   u[t, c] = b[c] + sum_k w[c, k] x[t - (W - 1) + k, c],   y = u or u sigmoid(u)
//
// The W - 1 inputs before a sequence's first token come from its row of h0, the
// last W - 1 inputs of what came before, or are zeros.  Backward, with du = dy
// (du/dy): dx[p] = sum_k w[k] du[p + (W - 1) - k] within the sequence, dw[k] =
// sum_t du[t] x[t - (W - 1) + k], db = sum_t du[t].
//
// Bound by memory: 2 W + 4 operations a value against the 4 bytes that it moves
// forward.  A thread takes 16 bytes of neighbouring channels and walks a run of
// tokens with the last W - 1 inputs in registers, so every row is read once but
// for the W - 1 before a run.  Sequences lie behind one another: a thread looks
// up which one its run starts in and goes from there.
#include "layer.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;  // rows that a thread has in flight

// Channels of a thread: 16 bytes, where rows start at multiples of that and C is
// a multiple; else one.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

template <typename T, int W, int V>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int64_t c, float (&w)[W][V],
                                          float (&b)[V]) {
    float flat[V * W];
    if (V % 4 == 0 && a.w_bytes >= 16) {  // a multiple of 16 bytes lies at a multiple of 16
        if (a.w.f32) {
#pragma unroll
            for (int i = 0; i < V * W / 4; ++i) {
                const float4 f = reinterpret_cast<const float4 *>((const float *)a.w.p + c * W)[i];
                flat[4 * i] = f.x; flat[4 * i + 1] = f.y; flat[4 * i + 2] = f.z; flat[4 * i + 3] = f.w;
            }
        } else {
            constexpr int P = V < kVec<T> ? V : kVec<T>;
#pragma unroll
            for (int i = 0; i < V * W / P; ++i) {
                Row<T, P> r;
                float f[P];
                r.load((const T *)a.w.p + c * W + i * P, 16, P);
                r.widen(f);
#pragma unroll
                for (int j = 0; j < P; ++j) flat[i * P + j] = f[j];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) flat[i] = param_at<T>(a.w, c * W + i);
    }
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) w[k][j] = flat[j * W + k];
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = a.b.p ? param_at<T>(a.b, c + j) : 0.f;
}

// The W - 1 inputs before token t of sequence [s, ..), oldest first; those before s from row
// `row` of h0.
template <typename T, int W, int V>
__device__ __forceinline__ void load_window(const ConvArgs &a, int64_t t, int64_t s, int64_t row,
                                            int64_t c, float (&win)[W - 1][V]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int64_t p = t - (W - 1) + k;
        Row<T, V> r;
        if (p >= s) r.load((const T *)a.x + p * a.xs + c, 16, V);
        else if (a.h0)
            r.load((const T *)a.h0 + (row * (W - 1) + (W - 1) + (p - s)) * a.C + c, 16, V);
        else r.zero();
        r.widen(win[k]);
    }
}

template <int W, int V>
__device__ __forceinline__ void taps(const float (&w)[W][V], const float (&b)[V],
                                     const float (&win)[W - 1][V], const float (&x)[V],
                                     float (&u)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        u[j] = fmaf(w[W - 1][j], x[j], b[j]);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) u[j] = fmaf(w[k][j], win[k][j], u[j]);
    }
}
template <int W, int V>
__device__ __forceinline__ void shift(float (&win)[W - 1][V], const float (&x)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) win[k][j] = win[k + 1][j];
        win[W - 2][j] = x[j];
    }
}

template <typename T, int W, int V>
__device__ __forceinline__ void one_token(const ConvArgs &a, const Row<T, V> &r, int64_t t,
                                          int64_t c, const float (&w)[W][V],
                                          const float (&b)[V], float (&win)[W - 1][V]) {
    float x[V], u[V];
    r.widen(x);
    taps<W, V>(w, b, win, x, u);
    shift<W, V>(win, x);
    if (a.silu) {
#pragma unroll
        for (int j = 0; j < V; ++j) u[j] *= sigmoid_f(u[j]);
    }
    Row<T, V> y;
    y.narrow(u);
    y.store((T *)a.y + t * a.ys + c, 16, V);
}

// A thread: V channels of a run of tokens.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads) k_conv(ConvArgs a) {
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t total = total_tokens(a.r), run = id / nv, c = id % nv * V;
    int64_t t = run * a.run;
    if (blockIdx.x == 0 && threadIdx.x < 32) check_offsets(a.r);
    if (t >= total) return;
    const int64_t t1 = min(t + a.run, total);
    float w[W][V], b[V], win[W - 1][V];
    load_taps<T, W, V>(a, c, w, b);
    Seq q{-1, 0, t};
    while (t < t1) {
        q = seq_at(a.r, t);
        int64_t row = 0;
        if (q.n >= 0 && a.h0) row = state_row(a.idx, a.n_states, q.n, a.r.status);
        const int64_t end = min(q.e, t1);
        if (q.n < 0 || row < 0) {  // nobody's tokens
            Row<T, V> zero;
            zero.zero();
            for (; t < end; ++t) zero.store((T *)a.y + t * a.ys + c, 16, V);
            continue;
        }
        load_window<T, W, V>(a, t, q.s, row, c, win);
        for (; t + kAhead <= end; t += kAhead) {
            Row<T, V> r[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                r[i].load((const T *)a.x + (t + i) * a.xs + c, 16, V);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) one_token<T, W, V>(a, r[i], t + i, c, w, b, win);
        }
        for (; t < end; ++t) {
            Row<T, V> r;
            r.load((const T *)a.x + t * a.xs + c, 16, V);
            one_token<T, W, V>(a, r, t, c, w, b, win);
        }
    }
}

// The last W - 1 inputs of every sequence into its row of ht, after k_conv (ht may be h0: a
// row's reader is its writer).
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads) k_conv_state(ConvArgs a) {
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t n = id / nv, c = id % nv * V;
    pdl_wait();
    if (n >= a.r.N) return;
    int64_t s, len;
    seq_span(a.r, n, s, len);
    const int64_t row = state_row(a.idx, a.n_states, n, a.r.status);
    if (row < 0) return;
    float win[W - 1][V];
    load_window<T, W, V>(a, s + len, s, row, c, win);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        Row<T, V> r;
        r.narrow(win[k]);
        r.store((T *)a.ht + (row * (W - 1) + k) * a.C + c, 16, V);
    }
}

// A thread: V channels of a whole sequence, for sequences of few tokens, from and into its row
// of the states.  One thread behind the last sequence clears what no sequence holds.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads) k_conv_step(ConvArgs a) {
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t n = id / nv, c = id % nv * V;
    if (blockIdx.x == 0 && threadIdx.x < 32) check_offsets(a.r);
    if (n > a.r.N) return;
    Row<T, V> zero;
    zero.zero();
    if (n == a.r.N) {
        if (!rows_packed(a.r)) return;
        const int64_t first = min(max(row_bound(a.r, 0), (int64_t)0), a.r.T);
        for (int64_t t = 0; t < first; ++t) zero.store((T *)a.y + t * a.ys + c, 16, V);
        for (int64_t t = max(row_bound(a.r, n), (int64_t)0); t < a.r.T; ++t)
            zero.store((T *)a.y + t * a.ys + c, 16, V);
        return;
    }
    int64_t s, len, row = 0;
    seq_span(a.r, n, s, len);
    if (a.h0 || a.ht) row = state_row(a.idx, a.n_states, n, a.r.status);
    if (row < 0) {
        for (int64_t t = s; t < s + len; ++t) zero.store((T *)a.y + t * a.ys + c, 16, V);
        return;
    }
    float w[W][V], b[V], win[W - 1][V];
    load_taps<T, W, V>(a, c, w, b);
    load_window<T, W, V>(a, s, s, row, c, win);
    for (int64_t t = s; t < s + len; ++t) {
        Row<T, V> r;
        r.load((const T *)a.x + t * a.xs + c, 16, V);
        one_token<T, W, V>(a, r, t, c, w, b, win);
    }
    if (a.ht) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            Row<T, V> r;
            r.narrow(win[k]);
            r.store((T *)a.ht + (row * (W - 1) + k) * a.C + c, 16, V);
        }
    }
}

// du of one token from its inputs and dy.
template <int W, int V>
__device__ __forceinline__ void grad_u(bool silu, const float (&w)[W][V], const float (&b)[V],
                                       const float (&win)[W - 1][V], const float (&x)[V],
                                       float (&du)[V]) {
    if (!silu) return;
    float u[V];
    taps<W, V>(w, b, win, x, u);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float g = sigmoid_f(u[j]);
        du[j] *= g * fmaf(u[j], 1.f - g, 1.f);
    }
}

// A thread: V channels of a run of tokens [t0, t1), going W - 1 tokens past it (a token's
// gradient needs the W - 1 after it), with the sums that these still lack in registers.  dw and
// db of the run go to part[run][(W + 1) C].
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads) k_conv_bwd(ConvArgs a) {
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t total = total_tokens(a.r), run = id / nv, c = id % nv * V;
    const int64_t t0 = run * a.run;
    if (blockIdx.x == 0 && threadIdx.x < 32) check_offsets(a.r);
    if (t0 >= total) return;
    const int64_t t1 = min(t0 + a.run, total);
    float w[W][V], b[V], dw[W + 1][V];
    load_taps<T, W, V>(a, c, w, b);
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[k][j] = 0.f;

    int64_t t = t0;
    while (t < t1) {
        const Seq q = seq_at(a.r, t);
        const int64_t row = q.n;
        if (q.n < 0) {
            Row<T, V> zero;
            zero.zero();
            for (const int64_t end = min(q.e, t1); t < end; ++t)
                zero.store((T *)a.dx + t * a.C + c, 16, V);
            continue;
        }
        float win[W - 1][V], pend[W][V];  // pend[k]: dx of token t - k, so far
        load_window<T, W, V>(a, t, q.s, row, c, win);
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) pend[k][j] = 0.f;
        const int64_t mine = min(q.e, t1), stop = min(q.e, t1 + W - 1), first = t;
        auto token = [&](const Row<T, V> &rx, const Row<T, V> &rd, int64_t p) {
            float x[V], du[V];
            rx.widen(x);
            rd.widen(du);
            grad_u<W, V>(a.silu, w, b, win, x, du);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (p < mine) {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) dw[k][j] = fmaf(du[j], win[k][j], dw[k][j]);
                    dw[W - 1][j] = fmaf(du[j], x[j], dw[W - 1][j]);
                    dw[W][j] += du[j];
                }
#pragma unroll
                for (int k = W - 1; k > 0; --k) pend[k][j] = fmaf(w[W - 1 - k][j], du[j], pend[k - 1][j]);
                pend[0][j] = w[W - 1][j] * du[j];
            }
            shift<W, V>(win, x);
            if (p - (W - 1) >= first) {
                Row<T, V> r;
                r.narrow(pend[W - 1]);
                r.store((T *)a.dx + (p - (W - 1)) * a.C + c, 16, V);
            }
        };
        constexpr int kU = 4;
        for (; t + kU <= stop; t += kU) {
            Row<T, V> rx[kU], rd[kU];
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                rx[i].load((const T *)a.x + (t + i) * a.xs + c, 16, V);
                rd[i].load((const T *)a.dy + (t + i) * a.ys + c, 16, V);
            }
#pragma unroll
            for (int i = 0; i < kU; ++i) token(rx[i], rd[i], t + i);
        }
        for (; t < stop; ++t) {
            Row<T, V> rx, rd;
            rx.load((const T *)a.x + t * a.xs + c, 16, V);
            rd.load((const T *)a.dy + t * a.ys + c, 16, V);
            token(rx, rd, t);
        }
        if (stop == q.e) {  // the sequence's last tokens: what is pending is whole but for dht
#pragma unroll
            for (int k = W - 2; k >= 0; --k) {
                const int64_t p = q.e - 1 - k;
                if (p < first || p >= mine) continue;
                if (a.dht) {
                    Row<T, V> r;
                    float d[V];
                    r.load((const T *)a.dht + (row * (W - 1) + W - 2 - k) * a.C + c, 16, V);
                    r.widen(d);
#pragma unroll
                    for (int j = 0; j < V; ++j) pend[k][j] += d[j];
                }
                Row<T, V> r;
                r.narrow(pend[k]);
                r.store((T *)a.dx + p * a.C + c, 16, V);
            }
        }
        t = mine;
    }
    float *part = a.part + run * (W + 1) * a.C;
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int k = 0; k <= W; ++k) part[k * a.C + c + j] = dw[k][j];
    }
}

// Gradient of the states that the sequences started from: dh0[k] = sum over the first tokens
// q <= k of w[k - q] du[q], and dht where the sequence is shorter than the window.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads) k_conv_dh0(ConvArgs a) {
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t n = id / nv, c = id % nv * V;
    if (n >= a.r.N) return;
    int64_t s, len;
    seq_span(a.r, n, s, len);
    float w[W][V], b[V], win[W - 1][V], d[W - 1][V];
    load_taps<T, W, V>(a, c, w, b);
    load_window<T, W, V>(a, s, s, n, c, win);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
#pragma unroll
        for (int j = 0; j < V; ++j) d[k][j] = 0.f;
        if (a.dht && k >= len) {
            Row<T, V> r;
            r.load((const T *)a.dht + (n * (W - 1) + k - len) * a.C + c, 16, V);
            r.widen(d[k]);
        }
    }
#pragma unroll
    for (int q = 0; q < W - 1; ++q) {
        if (q >= len) break;
        Row<T, V> rx, rd;
        float x[V], du[V];
        rx.load((const T *)a.x + (s + q) * a.xs + c, 16, V);
        rd.load((const T *)a.dy + (s + q) * a.ys + c, 16, V);
        rx.widen(x);
        rd.widen(du);
        grad_u<W, V>(a.silu, w, b, win, x, du);
        shift<W, V>(win, x);
#pragma unroll
        for (int k = q; k < W - 1; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) d[k][j] = fmaf(w[k - q][j], du[j], d[k][j]);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        Row<T, V> r;
        r.narrow(d[k]);
        r.store((T *)a.dh0 + (n * (W - 1) + k) * a.C + c, 16, V);
    }
}

// dw[c, k] and db[c]: the sums of the runs, in their order within each of 8 strands.
__global__ void __launch_bounds__(256) k_conv_params(ConvArgs a, int64_t runs, int W) {
    __shared__ float sum[8][33];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane, cols = (W + 1) * a.C;
    pdl_wait();
    float s = 0.f;
    if (i < cols)
        for (int64_t r = strand; r < runs; r += 8) s += a.part[r * cols + i];
    sum[strand][lane] = s;
    __syncthreads();
    if (strand || i >= cols) return;
    for (int j = 1; j < 8; ++j) s += sum[j][lane];
    const int64_t k = i / a.C, c = i % a.C;
    if (k < W) a.dw[c * W + k] = s;
    else if (a.db) a.db[c] = s;
}

unsigned blocks_for(int64_t threads) { return (unsigned)((threads + kThreads - 1) / kThreads); }

template <typename F>
cudaError_t by_type(const ConvArgs &a, int W, int dtype, F f) {
    auto of = [&](auto t, auto v) {
        if (W == 2) return f(t, std::integral_constant<int, 2>{}, v);
        if (W == 3) return f(t, std::integral_constant<int, 3>{}, v);
        return f(t, std::integral_constant<int, 4>{}, v);
    };
    auto type = [&](auto t) {
        if (a.wide) return of(t, std::integral_constant<int, kVec<decltype(t)>>{});
        return of(t, std::integral_constant<int, 1>{});
    };
    if (dtype == GDR_BF16) return type(__nv_bfloat16{});
    if (dtype == GDR_F16) return type(__half{});
    return type(float{});
}

}  // namespace

cudaError_t conv_fwd(const ConvArgs &a, int W, int dtype, bool step, cudaStream_t st) {
    return by_type(a, W, dtype, [&](auto t, auto w, auto v) {
        constexpr int Wc = decltype(w)::value, V = decltype(v)::value;
        using T = decltype(t);
        if (step) k_conv_step<T, Wc, V><<<blocks_for((a.r.N + 1) * (a.C / V)), kThreads, 0, st>>>(a);
        else k_conv<T, Wc, V><<<blocks_for(a.runs * (a.C / V)), kThreads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t conv_state(const ConvArgs &a, int W, int dtype, cudaStream_t st) {
    return by_type(a, W, dtype, [&](auto t, auto w, auto v) {
        constexpr int V = decltype(v)::value;
        return launch_pdl(k_conv_state<decltype(t), decltype(w)::value, V>,
                          dim3(blocks_for(a.r.N * (a.C / V))), dim3(kThreads), 0, st, a);
    });
}

cudaError_t conv_bwd(const ConvArgs &a, int W, int dtype, cudaStream_t st) {
    return by_type(a, W, dtype, [&](auto t, auto w, auto v) {
        constexpr int V = decltype(v)::value < 4 ? 1 : 4;  // of 8 the registers would be too many
        k_conv_bwd<decltype(t), decltype(w)::value, V>
            <<<blocks_for(a.runs * (a.C / V)), kThreads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t conv_dh0(const ConvArgs &a, int W, int dtype, cudaStream_t st) {
    return by_type(a, W, dtype, [&](auto t, auto w, auto v) {
        constexpr int V = decltype(v)::value;
        k_conv_dh0<decltype(t), decltype(w)::value, V>
            <<<blocks_for(a.r.N * (a.C / V)), kThreads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t conv_params(const ConvArgs &a, int W, cudaStream_t st) {
    const int64_t cols = (W + 1) * a.C;
    return launch_pdl(k_conv_params, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, st, a, a.runs,
                      W);
}

}  // namespace gdr
