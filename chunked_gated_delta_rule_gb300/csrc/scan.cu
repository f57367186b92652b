// scan.cu -- the selective state-space scan: for every channel c and state s
//
//   d_t = softplus(dt_t + bias),   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t
//   y_t = <C_t, h_t> + D x_t,      out = y silu(z)
//
// with B_t and C_t shared by the channels of a group.  FP32 states and sums.
//
// Every (token, channel, state) takes one exponential (its decay depends on all
// three) and five FP32 operations: the exponentials bound it, not the memory.
// So the scan runs along the tokens as it is written, each state's chain in a
// register, and whatever else a token needs is kept off the inner loop: a tile
// of tokens is staged in shared memory with d_t and d_t x_t computed once a
// channel, and the D and z terms are added when a tile's sums are written out.
// The sums over a channel's states take part of a shuffle a token: LPC tokens
// are folded at once.
//
// With too few (sequence, channel) chains to fill the device the sequences are
// cut into pieces: a first pass leaves each piece's end from a zero start, and
// the sum of its time steps (the piece's decay is exp(A sum d), so no products
// of decays are kept); a join turns the ends into starts; a second pass runs
// the pieces from those.  That doubles the exponentials.
#include "scan.cuh"

namespace gdr {
namespace {

// Tokens of a tile, and channels that a loading thread takes of one token.
template <int LPC>
struct FwdLay : Lay<LPC> {
    static constexpr int kT = 8 * LPC < 32 ? 8 * LPC : 32;
    static constexpr int kV = kT * Lay<LPC>::kC / kNT;
    static constexpr int kBC = kT * LPC * 2;                       // 4-state vectors of B and C
    static constexpr int kBCper = (kBC + kNT - 1) / kNT;
};

// The sums of LPC tokens over a channel's LPC lanes: lane q ends with token q's.
template <int LPC>
__device__ __forceinline__ float fold(float (&v)[LPC], int q) {
#pragma unroll
    for (int m = LPC / 2; m >= 1; m >>= 1) {
        const bool up = q & m;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float keep = up ? v[i + m] : v[i], send = up ? v[i] : v[i + m];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
    return v[0];
}

// SUM: leave a piece's end from a zero start (E) and the sum of its time steps (sd).  Else: the
// outputs, from E (pieces) or from h0 (whole sequences), and the last state into ht.
template <typename T, int LPC, bool SUM>
__global__ void __launch_bounds__(kNT) k_scan(ScanArgs a, int tiles) {
    using L = FwdLay<LPC>;
    constexpr int kT = L::kT, V = L::kV, kC = L::kC;
    __shared__ float2 sdx[kT][kC];  // time step and its product with x; the sums over states
    __shared__ float4 sbc[2][kT][LPC];
    const int tid = threadIdx.x, q = tid % LPC, cl = tid / LPC;
    const int64_t slot = blockIdx.x / tiles;
    const Tile tile = tile_of<LPC>(a, (int)(blockIdx.x % tiles));
    const int tr = tid / (kC / V), cv = tid % (kC / V) * V;
    pdl_wait();
    if (!SUM && slot == a.slots) {  // tokens of no sequence
        if (!rows_packed(a.r)) return;
        Row<T, V> zero;
        zero.zero();
        const int valid = max(0, min(V, tile.valid - cv));
        const int64_t first = min(max(row_bound(a.r, 0), (int64_t)0), a.r.T);
        for (int64_t t = tr; t < first; t += kT)
            zero.store((T *)a.y + t * a.ys + tile.c0 + cv, a.bytes, valid);
        for (int64_t t = max(row_bound(a.r, a.r.N), (int64_t)0) + tr; t < a.r.T; t += kT)
            zero.store((T *)a.y + t * a.ys + tile.c0 + cv, a.bytes, valid);
        return;
    }
    if (!(SUM && a.piece == 0) && blockIdx.x == 0 && tid < 32) check_offsets(a.r);
    const Piece p = piece_of(a, slot);
    if (p.n < 0) return;
    int64_t row = 0;
    if (!SUM && (a.h0 || a.ht)) row = state_row(a.idx, a.n_states, p.n, a.r.status);
    const int64_t c = tile.c0 + cl;
    const bool mine = cl < tile.valid;

    float A2[kPS], h[kPS];
#pragma unroll
    for (int i = 0; i < kPS; ++i) {
        const int s = q * kPS + i;
        const bool in = mine && s < a.S;
        A2[i] = in ? a.A[c * a.S + s] * kLog2e : 0.f;
        h[i] = 0.f;
        if (!SUM && in && row >= 0) {
            if (a.piece) h[i] = a.E[(slot * a.C + c) * a.S + s];
            else if (a.h0) h[i] = a.h0[(row * a.C + c) * a.S + s];
        }
    }
    float bias[V], skip[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const bool in = cv + j < tile.valid;
        bias[j] = a.dt_bias && in ? a.dt_bias[tile.c0 + cv + j] : 0.f;
        skip[j] = !SUM && a.D && in ? a.D[tile.c0 + cv + j] : 0.f;
    }

    Row<T, V> nx, nd, nz;
    Row<T, 4> nbc[L::kBCper];
    auto fetch = [&](int at) {
        const int64_t t0 = p.t0 + at;
        const int len = p.len - at;
        load_row<T, V>(nx, a.x, a.xs, t0, tr, len, tile, cv, a.bytes);
        load_row<T, V>(nd, a.dt, a.dts, t0, tr, len, tile, cv, a.bytes);
        if (!SUM && a.z) load_row<T, V>(nz, a.z, a.zs, t0, tr, len, tile, cv, a.bytes);
#pragma unroll
        for (int k = 0; k < L::kBCper; ++k) {
            const int id = k * kNT + tid, which = id / (kT * LPC), t = id / LPC % kT, v = id % LPC;
            if (id < (SUM ? kT * LPC : L::kBC))
                load_bc<T>(nbc[k], which ? a.Cm : a.Bm, which ? a.cs : a.bs, tile.g, t0, t, len, 4 * v,
                           a.S, a.bc_bytes);
        }
    };
    fetch(0);
    float total = 0.f;
    for (int at = 0; at < p.len; at += kT) {
        Row<T, V> cx = nx, cz = nz;
        {
            float x[V], d[V];
            nx.widen(x);
            nd.widen(d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                // past the end a time step of zero leaves the states as they are
                const float dt = at + tr < p.len ? time_step(a, d[j] + bias[j]) : 0.f;
                sdx[tr][cv + j] = make_float2(dt, dt * x[j]);
            }
        }
#pragma unroll
        for (int k = 0; k < L::kBCper; ++k) {
            const int id = k * kNT + tid;
            if (id < (SUM ? kT * LPC : L::kBC)) {
                float f[4];
                nbc[k].widen(f);
                sbc[id / (kT * LPC)][id / LPC % kT][id % LPC] = make_float4(f[0], f[1], f[2], f[3]);
            }
        }
        __syncthreads();
        if (at + kT < p.len) fetch(at + kT);
#pragma unroll 2
        for (int t0 = 0; t0 < kT; t0 += LPC) {
            float y[LPC];
#pragma unroll
            for (int k = 0; k < LPC; ++k) {
                const float2 d = sdx[t0 + k][cl];
                const float4 B = sbc[0][t0 + k][q];
                const float b[4] = {B.x, B.y, B.z, B.w};
#pragma unroll
                for (int i = 0; i < kPS; ++i) h[i] = fmaf(ex2(d.x * A2[i]), h[i], d.y * b[i]);
                if constexpr (SUM) {
                    total += d.x;
                } else {
                    const float4 C = sbc[1][t0 + k][q];
                    y[k] = fmaf(h[0], C.x, fmaf(h[1], C.y, fmaf(h[2], C.z, h[3] * C.w)));
                }
            }
            if constexpr (!SUM) {
                const float sum = fold<LPC>(y, q);
                __syncwarp();
                sdx[t0 + q][cl].x = sum;
            }
        }
        __syncthreads();
        if constexpr (!SUM) {
            // the next tile's time steps go where this thread reads its sums
            const int valid = at + tr < p.len ? max(0, min(V, tile.valid - cv)) : 0;
            float x[V], y[V];
            cx.widen(x);
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = fmaf(skip[j], x[j], sdx[tr][cv + j].x);
            if (a.z) {
                float z[V];
                cz.widen(z);
#pragma unroll
                for (int j = 0; j < V; ++j) y[j] *= z[j] * sigmoid_f(z[j]);
            }
            Row<T, V> out;
            out.narrow(y);
            if (row < 0) out.zero();
            out.store((T *)a.y + (p.t0 + at + tr) * a.ys + tile.c0 + cv, a.bytes, valid);
        }
    }
    if (!mine) return;
    if constexpr (SUM) {
        if (q == 0) a.sd[slot * a.C + c] = total;
    }
    float *to = SUM ? a.E + (slot * a.C + c) * a.S
                    : (a.ht && p.last && row >= 0 ? a.ht + (row * a.C + c) * a.S : nullptr);
    if (to) {
#pragma unroll
        for (int i = 0; i < kPS; ++i)
            if (q * kPS + i < a.S) to[q * kPS + i] = h[i];
    }
}

// Ends of pieces into their starts, in place: h <- exp(A sd) h + E.  Backward (blockIdx.y = 1):
// the gradients that enter the pieces' starts into those that reach their ends.
__global__ void __launch_bounds__(256) k_scan_join(ScanArgs a) {
    const int64_t per = a.C * a.S, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t n = id / per, i = id % per, c = i / a.S;
    pdl_wait();
    if (n >= a.r.N) return;
    int64_t s, len;
    seq_span(a.r, n, s, len);
    const int64_t L = a.piece, first = s / L + n, pieces = max((int64_t)1, (len + L - 1) / L);
    const float A2 = a.A[i] * kLog2e;
    constexpr int kU = 8;  // pieces whose loads are in flight
    if (blockIdx.y == 0) {
        float h = 0.f;
        if (a.h0) {
            const int64_t row = state_row(a.idx, a.n_states, n, a.r.status);
            if (row >= 0) h = a.h0[row * per + i];
        }
        for (int64_t j = 0; j < pieces; j += kU) {
            float e[kU], d[kU];
#pragma unroll
            for (int k = 0; k < kU; ++k)
                if (j + k < pieces) {
                    e[k] = a.E[(first + j + k) * per + i];
                    d[k] = a.sd[(first + j + k) * a.C + c];
                }
#pragma unroll
            for (int k = 0; k < kU; ++k)
                if (j + k < pieces) {
                    a.E[(first + j + k) * per + i] = h;
                    h = fmaf(ex2(A2 * d[k]), h, e[k]);
                }
        }
        return;
    }
    float g = a.dht ? a.dht[n * per + i] : 0.f;
    for (int64_t j = pieces - 1; j >= 0; j -= kU) {
        float e[kU], d[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k)
            if (j - k >= 0) {
                e[k] = a.R[(first + j - k) * per + i];
                d[k] = a.sd[(first + j - k) * a.C + c];
            }
#pragma unroll
        for (int k = 0; k < kU; ++k)
            if (j - k >= 0) {
                a.R[(first + j - k) * per + i] = g;
                g = fmaf(ex2(A2 * d[k]), g, e[k]);
            }
    }
    if (a.dh0) a.dh0[n * per + i] = g;
}

// Sequences of few tokens, a thread four states of a channel as above but straight from memory:
// what counts is the states' row, read and written once.
template <typename T, int LPC>
__global__ void __launch_bounds__(kNT) k_scan_step(ScanArgs a, int tiles) {
    const int tid = threadIdx.x, q = tid % LPC, cl = tid / LPC;
    const int64_t n = blockIdx.x / tiles;
    const Tile tile = tile_of<LPC>(a, (int)(blockIdx.x % tiles));
    const int64_t c = tile.c0 + cl;
    if (blockIdx.x == 0 && tid < 32) check_offsets(a.r);
    const bool mine = cl < tile.valid;
    T *y = (T *)a.y + c;
    if (n == a.r.N) {  // tokens of no sequence
        if (!rows_packed(a.r) || !mine || q) return;
        const int64_t first = min(max(row_bound(a.r, 0), (int64_t)0), a.r.T);
        for (int64_t t = 0; t < first; ++t) y[t * a.ys] = from_f32<T>(0.f);
        for (int64_t t = max(row_bound(a.r, n), (int64_t)0); t < a.r.T; ++t)
            y[t * a.ys] = from_f32<T>(0.f);
        return;
    }
    int64_t s, len, row = 0;
    seq_span(a.r, n, s, len);
    if (a.h0 || a.ht) row = state_row(a.idx, a.n_states, n, a.r.status);
    if (row < 0) {
        if (mine && q == 0)
            for (int64_t t = s; t < s + len; ++t) y[t * a.ys] = from_f32<T>(0.f);
        return;
    }
    const int s0 = q * kPS;
    const int have = mine ? max(0, min(kPS, a.S - s0)) : 0;
    float A2[kPS], h[kPS];
    {
        Row<float, 4> ra, rh;
        ra.load(a.A + c * a.S + s0, a.S % 4 ? 4 : a.out_bytes, have);
        rh.zero();
        if (a.h0) rh.load(a.h0 + (row * a.C + c) * a.S + s0, a.S % 4 ? 4 : a.out_bytes, have);
        ra.widen(A2);
        rh.widen(h);
    }
#pragma unroll
    for (int i = 0; i < kPS; ++i) A2[i] *= kLog2e;
    const float bias = a.dt_bias && mine ? a.dt_bias[c] : 0.f, skip = a.D && mine ? a.D[c] : 0.f;
    for (int64_t t = s; t < s + len; ++t) {
        Row<T, 4> rb, rc;
        rb.load((const T *)a.Bm + t * a.bs[0] + tile.g * a.bs[1] + s0, a.bc_bytes, have);
        rc.load((const T *)a.Cm + t * a.cs[0] + tile.g * a.cs[1] + s0, a.bc_bytes, have);
        float x = 0.f, d = 0.f, z = 0.f, b[4], cc[4];
        if (mine) {
            x = to_f32(((const T *)a.x)[t * a.xs + c]);
            d = time_step(a, to_f32(((const T *)a.dt)[t * a.dts + c]) + bias);
            if (a.z) z = to_f32(((const T *)a.z)[t * a.zs + c]);
        }
        rb.widen(b);
        rc.widen(cc);
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kPS; ++i) {
            h[i] = fmaf(ex2(d * A2[i]), h[i], d * x * b[i]);
            v = fmaf(h[i], cc[i], v);
        }
#pragma unroll
        for (int m = LPC / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        v = fmaf(skip, x, v);
        if (a.z) v *= z * sigmoid_f(z);
        if (mine && q == 0) y[t * a.ys] = from_f32<T>(v);
    }
    if (a.ht && have) {
        Row<float, 4> r;
        r.narrow(h);
        r.store(a.ht + (row * a.C + c) * a.S + s0, a.S % 4 ? 4 : a.out_bytes, have);
    }
}

}  // namespace

int scan_tile(int S) { return kNT / (S <= 4 ? 1 : S <= 8 ? 2 : S <= 16 ? 4 : S <= 32 ? 8 : 16); }
int64_t scan_tiles(int64_t C, int S, int G) {
    const int64_t per = C / G, kC = scan_tile(S);
    return G * ((per + kC - 1) / kC);
}

cudaError_t scan_step(const ScanArgs &a, int dtype, cudaStream_t st) {
    const int64_t tiles = scan_tiles(a.C, a.S, a.G);
    return scan_type(dtype, [&](auto t) {
        return scan_lanes(a.S, [&](auto l) {
            k_scan_step<decltype(t), decltype(l)::value>
                <<<(unsigned)((a.r.N + 1) * tiles), kNT, 0, st>>>(a, (int)tiles);
            return cudaGetLastError();
        });
    });
}

cudaError_t scan_pieces(const ScanArgs &a, int dtype, bool summary, cudaStream_t st) {
    const int64_t tiles = scan_tiles(a.C, a.S, a.G);
    return scan_type(dtype, [&](auto t) {
        return scan_lanes(a.S, [&](auto l) {
            using T = decltype(t);
            constexpr int LPC = decltype(l)::value;
            if (summary) {
                k_scan<T, LPC, true><<<(unsigned)(a.slots * tiles), kNT, 0, st>>>(a, (int)tiles);
                return cudaGetLastError();
            }
            const dim3 grid((unsigned)((a.slots + 1) * tiles));
            if (a.piece) return launch_pdl(k_scan<T, LPC, false>, grid, dim3(kNT), 0, st, a, (int)tiles);
            k_scan<T, LPC, false><<<grid, kNT, 0, st>>>(a, (int)tiles);
            return cudaGetLastError();
        });
    });
}

cudaError_t scan_join(const ScanArgs &a, bool backward, cudaStream_t st) {
    const int64_t all = a.r.N * a.C * a.S;
    return launch_pdl(k_scan_join, dim3((unsigned)((all + 255) / 256), backward ? 2 : 1), dim3(256), 0,
                      st, a);
}

}  // namespace gdr
