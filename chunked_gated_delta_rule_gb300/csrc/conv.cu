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
// forward.  A thread takes neighbouring channels and walks a run of tokens with
// the last W - 1 inputs in registers, so every row is read once but for the W - 1
// before a run.  The rows to come are on their way to shared memory meanwhile, each
// thread's to places of its own: in registers they would leave too few threads to
// keep the memory busy.  Sequences lie behind one another: a thread looks up which
// one its run starts in and goes from there.
//
// 64K tokens x 2048 channels x 4 taps in BF16: forward 92 us (537 MB, 5.8 TB/s, 0.86 of
// what a copy reaches), backward 159 us and its sums 8 us (805 MB, 5.1 TB/s): there the
// issue slots are 56% taken, by W + 1 products for u and the sigmoid, W for dx and W + 1
// for the weights.  256 single tokens x 6144 channels: 14 us, a chain of look-ups and rows.
#include "layer.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 4;  // tokens that a thread asks for at once

// Channels of a thread: 16 bytes, where rows start at multiples of that and C is
// a multiple; else one.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

template <typename T, int W, int V>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int64_t c, F2 (&w)[W][kPairs<V>],
                                          F2 (&b)[kPairs<V>]) {
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
    for (int j = 0; j < kPairs<V>; ++j) {
        const int hi = 2 * j + 1 < V ? 2 * j + 1 : 2 * j;
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][j] = f2(flat[2 * j * W + k], flat[hi * W + k]);
        b[j] = a.b.p ? f2(param_at<T>(a.b, c + 2 * j), param_at<T>(a.b, c + hi)) : f2(0.f);
    }
}

// The W - 1 inputs before token t of sequence [s, ..), oldest first; those before s from row
// `row` of h0.
template <typename T, int W, int V>
__device__ __forceinline__ void load_window(const ConvArgs &a, int64_t t, int64_t s, int64_t row,
                                            int64_t c, F2 (&win)[W - 1][kPairs<V>]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int64_t p = t - (W - 1) + k;
        Row<T, V> r;
        if (p >= s) r.load((const T *)a.x + p * a.xs + c, 16, V);
        else if (a.h0) r.load((const T *)a.h0 + (row * (W - 1) + (W - 1) + (p - s)) * a.C + c, 16, V);
        else r.zero();
        widen2<T, V>(r, win[k]);
    }
}

template <int W, int P>
__device__ __forceinline__ void taps(const F2 (&w)[W][P], const F2 (&b)[P], const F2 (&win)[W - 1][P],
                                     const F2 (&x)[P], F2 (&u)[P]) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
        u[j] = fma2(w[W - 1][j], x[j], b[j]);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) u[j] = fma2(w[k][j], win[k][j], u[j]);
    }
}
template <int W, int P>
__device__ __forceinline__ void shift(F2 (&win)[W - 1][P], const F2 (&x)[P]) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) win[k][j] = win[k + 1][j];
        win[W - 2][j] = x[j];
    }
}

template <typename T, int W, int V>
__device__ __forceinline__ void one_token(const ConvArgs &a, const Row<T, V> &r, int64_t t, int64_t c,
                                          const F2 (&w)[W][kPairs<V>], const F2 (&b)[kPairs<V>],
                                          F2 (&win)[W - 1][kPairs<V>]) {
    constexpr int P = kPairs<V>;
    F2 x[P], u[P];
    widen2<T, V>(r, x);
    taps<W, P>(w, b, win, x, u);
    shift<W, P>(win, x);
    if (a.silu) {
#pragma unroll
        for (int j = 0; j < P; ++j) u[j] = u[j] * sigmoid2(u[j]);
    }
    store2<T, V>((T *)a.y + t * a.ys + c, u);
}

// Rows of N tensors on their way to shared memory, in batches of kAhead tokens.  A thread reads only
// what it has asked for, so it waits for its own copies and for nobody else.  Single values
// (V = 1) are loaded when they are wanted.
template <typename T, int V, int N>
struct Feed {
    static constexpr bool kRing = V > 1;
    static constexpr int kSlot = kThreads * V * (int)sizeof(T);  // a row of every thread
    static constexpr int kBatch = kAhead * N * kSlot;
    // batches that are on their way or worked on, within 48 KB
    static constexpr int kDepth = kBatch <= 12288 ? 4 : 3;
    static constexpr int kBytes = kRing ? kDepth * kBatch : 16;

    uint8_t *const ring;    // the thread's place in the first slot
    const T *next[N];       // rows of the next batch to ask for
    const int64_t stride[N];
    int put = 0, get = 0;   // batches, in bytes from ring
    int64_t left = 0;       // batches to ask for

    __device__ __forceinline__ void ask() {
        if constexpr (kRing) {
            if (left > 0) {
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint32_t to = (uint32_t)__cvta_generic_to_shared(ring) + put + n * kSlot;
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        if constexpr (V * sizeof(T) == 16)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * N * kSlot),
                                         "l"(next[n]) : "memory");
                        else
                            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + i * N * kSlot),
                                         "l"(next[n]), "n"(V * sizeof(T)) : "memory");
                        next[n] += stride[n];
                    }
                }
                put = put + kBatch == kBytes ? 0 : put + kBatch;
                --left;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    // `batches` batches of the rows from p[n] on.
    __device__ __forceinline__ void start(const T *const (&p)[N], int64_t batches) {
#pragma unroll
        for (int n = 0; n < N; ++n) next[n] = p[n];
        left = batches;
        put = get = 0;
#pragma unroll
        for (int k = 0; k < kDepth - 1; ++k) ask();
    }
    // The rows of the next batch; the place of the one before it is free for another.
    __device__ __forceinline__ void take(Row<T, V> (&r)[kAhead][N]) {
        if constexpr (kRing) asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if constexpr (kRing) {
                    r[i][n].load(reinterpret_cast<const T *>(ring + get + (i * N + n) * kSlot), 16, V);
                } else {
                    r[i][n].load(next[n], 16, V);
                    next[n] += stride[n];
                }
            }
        get = get + kBatch == kBytes ? 0 : get + kBatch;
        ask();
    }
};

// A thread: V channels of a run of tokens.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads, kConvThreads / kThreads) k_conv(ConvArgs a) {
    constexpr int P = kPairs<V>;
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t total = total_tokens(a.r), run = id / nv, c = id % nv * V;
    int64_t t = run * a.run;
    const bool together = same_in_warp(run);
    pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x < 32) check_offsets(a.r);
    if (t >= total) return;
    const int64_t t1 = min(t + a.run, total);
    using F = Feed<T, V, 1>;
    __shared__ __align__(16) uint8_t ring[F::kBytes];
    F feed{ring + (F::kRing ? threadIdx.x * V * sizeof(T) : 0), {}, {a.xs}};
    F2 w[W][P], b[P], win[W - 1][P];
    load_taps<T, W, V>(a, c, w, b);
    while (t < t1) {
        const Seq q = seq_at(a.r, t, together);
        int64_t row = 0;
        if (q.n >= 0 && (a.h0 || a.ht)) row = state_row(a.idx, a.n_states, q.n, a.r.status);
        const int64_t end = min(q.e, t1);
        if (q.n < 0 || row < 0) {  // nobody's tokens
            Row<T, V> zero;
            zero.zero();
            for (; t < end; ++t) zero.store((T *)a.y + t * a.ys + c, 16, V);
            continue;
        }
        load_window<T, W, V>(a, t, q.s, row, c, win);
        const int64_t batches = (end - t) / kAhead;
        feed.start({(const T *)a.x + t * a.xs + c}, batches);
        for (int64_t k = 0; k < batches; ++k) {
            Row<T, V> r[kAhead][1];
            feed.take(r);
#pragma unroll
            for (int i = 0; i < kAhead; ++i, ++t) one_token<T, W, V>(a, r[i][0], t, c, w, b, win);
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
    F2 win[W - 1][kPairs<V>];
    load_window<T, W, V>(a, s + len, s, row, c, win);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store2<T, V>((T *)a.ht + (row * (W - 1) + k) * a.C + c, win[k]);
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
    F2 w[W][kPairs<V>], b[kPairs<V>], win[W - 1][kPairs<V>];
    load_taps<T, W, V>(a, c, w, b);
    load_window<T, W, V>(a, s, s, row, c, win);
    for (int64_t t = s; t < s + len; ++t) {
        Row<T, V> r;
        r.load((const T *)a.x + t * a.xs + c, 16, V);
        one_token<T, W, V>(a, r, t, c, w, b, win);
    }
    if (a.ht) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) store2<T, V>((T *)a.ht + (row * (W - 1) + k) * a.C + c, win[k]);
    }
}

// du of one token from its inputs and dy.
template <int W, int P>
__device__ __forceinline__ void grad_u(bool silu, const F2 (&w)[W][P], const F2 (&b)[P],
                                       const F2 (&win)[W - 1][P], const F2 (&x)[P], F2 (&du)[P]) {
    if (!silu) return;
    F2 u[P];
    taps<W, P>(w, b, win, x, u);
#pragma unroll
    for (int j = 0; j < P; ++j) {  // g (1 + u (1 - g)), g = sigmoid(u)
        const F2 g = sigmoid2(u[j]);
        du[j] = du[j] * (g * fma2(u[j], fma2(g, f2(-1.f), f2(1.f)), f2(1.f)));
    }
}

// A thread: V channels of a run of tokens [t0, t1), going W - 1 tokens past it (a token's
// gradient needs the W - 1 after it), with the sums that these still lack in registers.  dw and
// db of the run go to part[run][(W + 1) C].
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads, kConvThreads / kThreads) k_conv_bwd(ConvArgs a) {
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t total = total_tokens(a.r), run = id / nv, c = id % nv * V;
    const int64_t t0 = run * a.run;
    const bool together = same_in_warp(run);
    pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x < 32) check_offsets(a.r);
    if (t0 >= total) return;
    const int64_t t1 = min(t0 + a.run, total);
    constexpr int P = kPairs<V>;
    using F = Feed<T, V, 2>;
    __shared__ __align__(16) uint8_t ring[F::kBytes];
    F feed{ring + (F::kRing ? threadIdx.x * V * sizeof(T) : 0), {}, {a.xs, a.ys}};
    F2 w[W][P], b[P], dw[W + 1][P];
    load_taps<T, W, V>(a, c, w, b);
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int j = 0; j < P; ++j) dw[k][j] = f2(0.f);

    int64_t t = t0;
    while (t < t1) {
        const Seq q = seq_at(a.r, t, together);
        const int64_t row = q.n;
        if (q.n < 0) {
            Row<T, V> zero;
            zero.zero();
            for (const int64_t end = min(q.e, t1); t < end; ++t)
                zero.store((T *)a.dx + t * a.C + c, 16, V);
            continue;
        }
        F2 win[W - 1][P], pend[W][P];  // pend[k]: dx of token t - k, so far
        load_window<T, W, V>(a, t, q.s, row, c, win);
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int j = 0; j < P; ++j) pend[k][j] = f2(0.f);
        const int64_t mine = min(q.e, t1), stop = min(q.e, t1 + W - 1), first = t;
        const int own = (int)(mine - t);  // tokens of the run: at most a few hundred
        T *out = (T *)a.dx + (t - (W - 1)) * a.C + c;
        int at = 0;  // tokens done
        auto token = [&](const Row<T, V> &rx, const Row<T, V> &rd) {
            F2 x[P], du[P];
            widen2<T, V>(rx, x);
            widen2<T, V>(rd, du);
            grad_u<W, P>(a.silu, w, b, win, x, du);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (at < own) {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) dw[k][j] = fma2(du[j], win[k][j], dw[k][j]);
                    dw[W - 1][j] = fma2(du[j], x[j], dw[W - 1][j]);
                    dw[W][j] = dw[W][j] + du[j];
                }
#pragma unroll
                for (int k = W - 1; k > 0; --k) pend[k][j] = fma2(w[W - 1 - k][j], du[j], pend[k - 1][j]);
                pend[0][j] = w[W - 1][j] * du[j];
            }
            shift<W, P>(win, x);
            if (at >= W - 1) store2<T, V>(out, pend[W - 1]);
            out += a.C;
            ++at;
        };
        const int64_t batches = (stop - t) / kAhead;
        feed.start({(const T *)a.x + t * a.xs + c, (const T *)a.dy + t * a.ys + c}, batches);
        for (int64_t k = 0; k < batches; ++k) {
            Row<T, V> r[kAhead][2];
            feed.take(r);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) token(r[i][0], r[i][1]);
        }
        for (t += batches * kAhead; t < stop; ++t) {
            Row<T, V> rx, rd;
            rx.load((const T *)a.x + t * a.xs + c, 16, V);
            rd.load((const T *)a.dy + t * a.ys + c, 16, V);
            token(rx, rd);
        }
        if (stop == q.e) {  // the sequence's last tokens: what is pending is whole but for dht
#pragma unroll
            for (int k = W - 2; k >= 0; --k) {
                const int64_t p = q.e - 1 - k;
                if (p < first || p >= mine) continue;
                if (a.dht) {
                    Row<T, V> r;
                    F2 d[P];
                    r.load((const T *)a.dht + (row * (W - 1) + W - 2 - k) * a.C + c, 16, V);
                    widen2<T, V>(r, d);
#pragma unroll
                    for (int j = 0; j < P; ++j) pend[k][j] = pend[k][j] + d[j];
                }
                store2<T, V>((T *)a.dx + p * a.C + c, pend[k]);
            }
        }
        t = mine;
    }
    float *part = a.part + run * (W + 1) * a.C;
#pragma unroll
    for (int k = 0; k <= W; ++k) store2<float, V>(part + k * a.C + c, dw[k]);
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
    constexpr int P = kPairs<V>;
    F2 w[W][P], b[P], win[W - 1][P], d[W - 1][P];
    load_taps<T, W, V>(a, c, w, b);
    load_window<T, W, V>(a, s, s, n, c, win);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        Row<T, V> r;
        r.zero();
        if (a.dht && k >= len) r.load((const T *)a.dht + (n * (W - 1) + k - len) * a.C + c, 16, V);
        widen2<T, V>(r, d[k]);
    }
#pragma unroll
    for (int q = 0; q < W - 1; ++q) {
        if (q >= len) break;
        Row<T, V> rx, rd;
        F2 x[P], du[P];
        rx.load((const T *)a.x + (s + q) * a.xs + c, 16, V);
        rd.load((const T *)a.dy + (s + q) * a.ys + c, 16, V);
        widen2<T, V>(rx, x);
        widen2<T, V>(rd, du);
        grad_u<W, P>(a.silu, w, b, win, x, du);
        shift<W, P>(win, x);
#pragma unroll
        for (int k = q; k < W - 1; ++k)
#pragma unroll
            for (int j = 0; j < P; ++j) d[k][j] = fma2(w[k - q][j], du[j], d[k][j]);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store2<T, V>((T *)a.dh0 + (n * (W - 1) + k) * a.C + c, d[k]);
}

// dw[c, k] and db[c]: the sums of the runs.
__global__ void __launch_bounds__(kColumnThreads) k_conv_params(ConvArgs a, int W) {
    const int64_t i = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31), cols = (W + 1) * a.C;
    pdl_wait();
    const float s = column_sum(a.part + i, cols, a.runs, i < cols);
    if (threadIdx.x >= 32 || i >= cols) return;
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
    return launch_pdl(k_conv_params, dim3((unsigned)((cols + 31) / 32)), dim3(kColumnThreads), 0, st, a, W);
}

}  // namespace gdr
