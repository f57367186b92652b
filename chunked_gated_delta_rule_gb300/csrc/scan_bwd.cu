// scan_bwd.cu -- gradients of the selective scan.  With a_t = exp(d_t A) and
// dv = dout silu(z):
//
//   dh_t = dv_t C_t + a_{t+1} dh_{t+1}   (dht behind the last token)
//   e_t  = dh_t a_t h_{t-1}
//   dC = sum_c dv h,   dB = sum_c dh d x,   dD = sum_t dv x
//   dx = d <dh, B> + D dv,   dd = <e, A> + x <dh, B>,   dA = sum_t d e
//   ddt = dd sigmoid(dt + bias),   dz = dout (<C, h> + D x) silu'(z)
//
// Pieces of kScanBwdPiece tokens, all at once, whatever the sequences:
//   1. one sweep leaves each piece's end from a zero start (E), its sum of time
//      steps, and the gradient that its outputs send to its start (R): with P the
//      product of the decays so far, R = sum_t P_t C_t dv_t;
//   2. the join turns ends into starts, forward for E and backward for R;
//   3. the main pass runs the piece forward from its start, keeping the state in
//      front of every 8 tokens, then backward 8 tokens at a time: their decays and
//      states are formed again in registers and the gradients follow from the last
//      to the first.
//   4. sums over channels (dB, dC) and over pieces (dA, dD, dbias), in a fixed order.
// The exponentials are taken three times, which bounds the pass together with
// the sums across lanes: over a channel's states for dx, dd and <C, h>, over the
// channels for dB and dC.  Both fold several tokens, or the eight values of a
// thread, at once, so that a shuffle carries a value that is still wanted.
#include "scan.cuh"

namespace gdr {
namespace {

constexpr int kU = 8;                          // tokens formed again at once
constexpr int kKeep = kScanBwdPiece / kU;      // states kept of a piece

template <int LPC>
struct BwdLay : Lay<LPC> {
    static constexpr int kT = LPC == 1 ? 8 : 16;  // tokens of a tile
    static constexpr int kVals = kT * Lay<LPC>::kC;
    static constexpr int kV = kVals / kNT >= 2 ? kVals / kNT : 2;
    static constexpr int kLoad = kVals / kV;      // threads that load rows
    static constexpr int kRows = Lay<LPC>::kC / kV;      // ... of one token
    static constexpr int kBC = kT * LPC * 2;
    static constexpr int kBCper = (kBC + kNT - 1) / kNT;
};

// dv = dout silu(z), or dout.
template <int V>
__device__ __forceinline__ void gate_grad(const float (&g)[V], const float (&z)[V], bool gated,
                                          float (&dv)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) dv[j] = gated ? g[j] * z[j] * sigmoid_f(z[j]) : g[j];
}

// Stages tokens [t0, t0 + kT) of the piece: time steps and their products with x, dv, B and C.
template <typename T, int LPC>
struct Stage {
    using L = BwdLay<LPC>;
    static constexpr int kT = L::kT, V = L::kV, kC = L::kC;
    Row<T, V> x, dt, z, dy;
    Row<T, 4> bc[L::kBCper];

    template <bool GRAD>
    __device__ __forceinline__ void fetch(const ScanArgs &a, const Tile &tile, int64_t t0, int len) {
        const int tid = threadIdx.x, tr = tid / L::kRows, cv = tid % L::kRows * V;
        if (tid < L::kLoad) {
            load_row<T, V>(x, a.x, a.xs, t0, tr, len, tile, cv, a.bytes);
            load_row<T, V>(dt, a.dt, a.dts, t0, tr, len, tile, cv, a.bytes);
            if constexpr (GRAD) {
                load_row<T, V>(dy, a.dy, a.ys, t0, tr, len, tile, cv, a.bytes);
                if (a.z) load_row<T, V>(z, a.z, a.zs, t0, tr, len, tile, cv, a.bytes);
            }
        }
#pragma unroll
        for (int k = 0; k < L::kBCper; ++k) {
            const int id = k * kNT + tid, which = id / (kT * LPC), t = id / LPC % kT, v = id % LPC;
            if (id < (GRAD ? L::kBC : kT * LPC))
                load_bc<T>(bc[k], which ? a.Cm : a.Bm, which ? a.cs : a.bs, tile.g, t0, t, len, 4 * v,
                           a.S, a.bc_bytes);
        }
    }
    template <bool GRAD>
    __device__ __forceinline__ void put(const ScanArgs &a, const float (&bias)[V], int len,
                                        float2 (*sdx)[kC], float (*sdv)[kC], float4 (*sbc)[kT][LPC]) {
        const int tid = threadIdx.x, tr = tid / L::kRows, cv = tid % L::kRows * V;
        if (tid < L::kLoad) {
            float fx[V], fd[V];
            x.widen(fx);
            dt.widen(fd);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = tr < len ? time_step(a, fd[j] + bias[j]) : 0.f;
                sdx[tr][cv + j] = make_float2(d, d * fx[j]);
            }
            if constexpr (GRAD) {
                float g[V], fz[V], dv[V];
                dy.widen(g);
                if (a.z) z.widen(fz);
                gate_grad<V>(g, fz, a.z != nullptr, dv);
#pragma unroll
                for (int j = 0; j < V; ++j) sdv[tr][cv + j] = dv[j];
            }
        }
#pragma unroll
        for (int k = 0; k < L::kBCper; ++k) {
            const int id = k * kNT + tid;
            if (id < (GRAD ? L::kBC : kT * LPC)) {
                float f[4];
                bc[k].widen(f);
                sbc[id / (kT * LPC)][id / LPC % kT][id % LPC] = make_float4(f[0], f[1], f[2], f[3]);
            }
        }
    }
};

template <int LPC>
__device__ __forceinline__ void load_A2(const ScanArgs &a, int64_t c, bool mine, int q, float (&A2)[kPS]) {
#pragma unroll
    for (int i = 0; i < kPS; ++i) {
        const int s = q * kPS + i;
        A2[i] = mine && s < a.S ? a.A[c * a.S + s] * kLog2e : 0.f;
    }
}
template <int V>
__device__ __forceinline__ void load_channel(const float *p, const Tile &tile, int cv, float (&f)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = p && cv + j < tile.valid ? p[tile.c0 + cv + j] : 0.f;
}

// 1. E, sd and R of a piece.
template <typename T, int LPC>
__global__ void __launch_bounds__(kNT) k_scan_bwd_sum(ScanArgs a, int tiles) {
    using L = BwdLay<LPC>;
    constexpr int kT = L::kT, V = L::kV, kC = L::kC;
    __shared__ float2 sdx[kT][kC];
    __shared__ float sdv[kT][kC];
    __shared__ float4 sbc[2][kT][LPC];
    const int tid = threadIdx.x, q = tid % LPC, cl = tid / LPC;
    const int64_t slot = blockIdx.x / tiles;
    const Tile tile = tile_of<LPC>(a, (int)(blockIdx.x % tiles));
    if (blockIdx.x == 0 && tid < 32) check_offsets(a.r);
    const Piece p = piece_of(a, slot);
    if (p.n < 0) return;
    const int64_t c = tile.c0 + cl;
    const bool mine = cl < tile.valid;
    float A2[kPS], h[kPS], P[kPS], R[kPS], bias[V], total = 0.f;
    load_A2<LPC>(a, c, mine, q, A2);
    load_channel<V>(a.dt_bias, tile, tid % L::kRows * V, bias);
#pragma unroll
    for (int i = 0; i < kPS; ++i) {
        h[i] = R[i] = 0.f;
        P[i] = 1.f;
    }
    Stage<T, LPC> s;
    s.template fetch<true>(a, tile, p.t0, p.len);
    for (int at = 0; at < p.len; at += kT) {
        s.template put<true>(a, bias, p.len - at, sdx, sdv, sbc);
        __syncthreads();
        if (at + kT < p.len) s.template fetch<true>(a, tile, p.t0 + at + kT, p.len - at - kT);
#pragma unroll 4
        for (int t = 0; t < kT; ++t) {
            const float2 d = sdx[t][cl];
            const float dv = sdv[t][cl];
            const float4 B = sbc[0][t][q], C = sbc[1][t][q];
            const float b[4] = {B.x, B.y, B.z, B.w}, cc[4] = {C.x, C.y, C.z, C.w};
#pragma unroll
            for (int i = 0; i < kPS; ++i) {
                const float w = ex2(d.x * A2[i]);
                h[i] = fmaf(w, h[i], d.y * b[i]);
                P[i] *= w;
                R[i] = fmaf(P[i], cc[i] * dv, R[i]);
            }
            total += d.x;
        }
        __syncthreads();
    }
    if (!mine) return;
    if (q == 0) a.sd[slot * a.C + c] = total;
#pragma unroll
    for (int i = 0; i < kPS; ++i)
        if (q * kPS + i < a.S) {
            a.E[(slot * a.C + c) * a.S + q * kPS + i] = h[i];
            a.R[(slot * a.C + c) * a.S + q * kPS + i] = R[i];
        }
}

// Sums of v[token] over a channel's LPC lanes.  A lane ends with kU / LPC tokens (at least one),
// those from first_token<LPC>(q) on.
template <int LPC>
__device__ __forceinline__ void fold_states(float (&v)[kU], int q) {
    int n = kU;
#pragma unroll
    for (int m = LPC / 2; m >= 1; m >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = q & m;
#pragma unroll
            for (int i = 0; i < kU / 2; ++i)
                if (i < n) {
                    const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
        }
    }
}
template <int LPC>
__device__ __forceinline__ int first_token(int q) {
    return LPC <= kU ? q * (kU / LPC) : q / (LPC / kU);
}

// Sums of v[8] (four states of B, four of C) over the warp's 32 / LPC channels.  A lane ends
// with 8 / channels of them (at least one), from first_value<LPC>(channel) on.
template <int LPC>
__device__ __forceinline__ void fold_channels(float (&v)[8], int lane) {
    int n = 8;
#pragma unroll
    for (int m = 16; m >= LPC; m >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = lane & m;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) {
                    const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
        }
    }
}

template <int LPC>
constexpr size_t bwd_smem() {
    using L = BwdLay<LPC>;
    return sizeof(float4) * kKeep * kNT + sizeof(float2) * L::kT * L::kC + sizeof(float) * L::kT * L::kC +
           sizeof(float4) * 2 * L::kT * LPC + sizeof(float) * (kNT / 32) * L::kT * 2 * L::kS;
}

// 3. The gradients of a piece.  At the end E's slot holds its part of dA.
template <typename T, int LPC>
__global__ void __launch_bounds__(kNT, 2) k_scan_bwd(ScanArgs a, int tiles) {
    using L = BwdLay<LPC>;
    constexpr int kT = L::kT, V = L::kV, kC = L::kC, kS = L::kS;
    extern __shared__ float4 smem[];
    float4(*keep)[kNT] = reinterpret_cast<float4(*)[kNT]>(smem);
    float4(*sbc)[kT][LPC] = reinterpret_cast<float4(*)[kT][LPC]>(smem + kKeep * kNT);
    float2(*sdx)[kC] = reinterpret_cast<float2(*)[kC]>(smem + kKeep * kNT + 2 * kT * LPC);
    float(*sdv)[kC] = reinterpret_cast<float(*)[kC]>(sdx + kT);
    float(*red)[kT][2 * kS] = reinterpret_cast<float(*)[kT][2 * kS]>(sdv + kT);
    const int tid = threadIdx.x, q = tid % LPC, cl = tid / LPC, lane = tid & 31, warp = tid >> 5;
    const int64_t slot = blockIdx.x / tiles;
    const int tile_id = (int)(blockIdx.x % tiles);
    const Tile tile = tile_of<LPC>(a, tile_id);
    const int tr = tid / L::kRows, cv = tid % L::kRows * V;
    const int64_t all = total_tokens(a.r);
    float *part = a.part + (int64_t)tile_id * all * 2 * a.S;
    T *dx = (T *)a.dx, *ddt = (T *)a.ddt, *dz = (T *)a.dz;
    pdl_wait();
    if (slot == a.slots) {  // tokens of no sequence
        if (!rows_packed(a.r)) return;
        Row<T, V> zero;
        zero.zero();
        const int valid = max(0, min(V, tile.valid - cv));
        auto clear = [&](int64_t from, int64_t to) {
            if (tid < L::kLoad)
                for (int64_t t = from + tr; t < to; t += kT) {
                    zero.store(dx + t * a.C + tile.c0 + cv, a.out_bytes, valid);
                    zero.store(ddt + t * a.C + tile.c0 + cv, a.out_bytes, valid);
                    if (a.z) zero.store(dz + t * a.C + tile.c0 + cv, a.out_bytes, valid);
                }
            for (int64_t i = from * 2 * a.S + tid; i < to * 2 * a.S; i += kNT) part[i] = 0.f;
        };
        clear(0, min(max(row_bound(a.r, 0), (int64_t)0), a.r.T));
        clear(max(row_bound(a.r, a.r.N), (int64_t)0), a.r.T);
        return;
    }
    const Piece p = piece_of(a, slot);
    const int64_t c = tile.c0 + cl, at_state = (slot * a.C + c) * a.S + q * kPS;
    const bool mine = cl < tile.valid;
    const int len = p.n < 0 ? 0 : p.len;
    float A[kPS], A2[kPS], h[kPS], dh[kPS], dA[kPS], bias[V], skip[V], dD[V], db[V];
#pragma unroll
    for (int i = 0; i < kPS; ++i) {
        const bool in = mine && q * kPS + i < a.S;
        A[i] = in ? a.A[c * a.S + q * kPS + i] : 0.f;
        A2[i] = A[i] * kLog2e;
        h[i] = in && len ? a.E[at_state + i] : 0.f;
        dh[i] = in && len ? a.R[at_state + i] : 0.f;
        dA[i] = 0.f;
    }
    load_channel<V>(a.dt_bias, tile, cv, bias);
    load_channel<V>(a.D, tile, cv, skip);
#pragma unroll
    for (int j = 0; j < V; ++j) dD[j] = db[j] = 0.f;

    Stage<T, LPC> s;
    if (len) s.template fetch<false>(a, tile, p.t0, len);
    for (int at = 0; at < len; at += kT) {
        s.template put<false>(a, bias, len - at, sdx, sdv, sbc);
        __syncthreads();
        if (at + kT < len) s.template fetch<false>(a, tile, p.t0 + at + kT, len - at - kT);
        else s.template fetch<true>(a, tile, p.t0 + at, len - at);  // the backward's first
#pragma unroll
        for (int u = 0; u < kT; u += kU) {
            keep[(at + u) / kU][tid] = make_float4(h[0], h[1], h[2], h[3]);
#pragma unroll
            for (int t = u; t < u + kU; ++t) {
                const float2 d = sdx[t][cl];
                const float4 B = sbc[0][t][q];
                const float b[4] = {B.x, B.y, B.z, B.w};
#pragma unroll
                for (int i = 0; i < kPS; ++i) h[i] = fmaf(ex2(d.x * A2[i]), h[i], d.y * b[i]);
            }
        }
        __syncthreads();
    }
    for (int at = (len - 1) / kT * kT; at >= 0 && len; at -= kT) {
        Row<T, V> cx = s.x, cd = s.dt, cz = s.z, cy = s.dy;
        s.template put<true>(a, bias, len - at, sdx, sdv, sbc);
        __syncthreads();
        if (at) s.template fetch<true>(a, tile, p.t0 + at - kT, len - at + kT);
#pragma unroll 1
        for (int u = kT - kU; u >= 0; u -= kU) {
            float w[kU][kPS], hs[kU][kPS], v[kU], hb[kU], ea[kU], h0[kPS];
            const float4 k0 = keep[(at + u) / kU][tid];
            h0[0] = k0.x; h0[1] = k0.y; h0[2] = k0.z; h0[3] = k0.w;
#pragma unroll
            for (int t = 0; t < kU; ++t) {
                const float2 d = sdx[u + t][cl];
                const float4 B = sbc[0][u + t][q], C = sbc[1][u + t][q];
                const float b[4] = {B.x, B.y, B.z, B.w}, cc[4] = {C.x, C.y, C.z, C.w};
                v[t] = 0.f;
#pragma unroll
                for (int i = 0; i < kPS; ++i) {
                    w[t][i] = ex2(d.x * A2[i]);
                    hs[t][i] = fmaf(w[t][i], t ? hs[t - 1][i] : h0[i], d.y * b[i]);
                    v[t] = fmaf(hs[t][i], cc[i], v[t]);
                }
            }
#pragma unroll
            for (int t = kU - 1; t >= 0; --t) {
                const float2 d = sdx[u + t][cl];
                const float dv = sdv[u + t][cl];
                const float4 B = sbc[0][u + t][q], C = sbc[1][u + t][q];
                const float b[4] = {B.x, B.y, B.z, B.w}, cc[4] = {C.x, C.y, C.z, C.w};
                float bc[8];
                hb[t] = ea[t] = 0.f;
#pragma unroll
                for (int i = 0; i < kPS; ++i) {
                    dh[i] = fmaf(dv, cc[i], dh[i]);
                    bc[i] = dh[i] * d.y;
                    bc[4 + i] = dv * hs[t][i];
                    hb[t] = fmaf(dh[i], b[i], hb[t]);
                    dh[i] *= w[t][i];
                    const float e = dh[i] * (t ? hs[t - 1][i] : h0[i]);
                    ea[t] = fmaf(e, A[i], ea[t]);
                    dA[i] = fmaf(e, d.x, dA[i]);
                }
                fold_channels<LPC>(bc, lane);
                // the channel's number among the warp's 32 / LPC names the values a lane has
                constexpr int kCh = 32 / LPC, kHas = kCh >= 8 ? 1 : 8 / kCh, kDup = kCh > 8 ? kCh / 8 : 1;
                const int ch = lane / LPC;
                if (ch % kDup == 0) {
#pragma unroll
                    for (int i = 0; i < kHas; ++i) {
                        const int idx = ch / kDup * kHas + i;  // B's four, C's four
                        red[warp][u + t][idx / 4 * kS + q * kPS + idx % 4] = bc[i];
                    }
                }
            }
            fold_states<LPC>(v, q);
            fold_states<LPC>(hb, q);
            fold_states<LPC>(ea, q);
            __syncwarp();
            constexpr int kMine = kU / LPC >= 1 ? kU / LPC : 1;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int t = u + first_token<LPC>(q) + i;
                if (LPC <= kU || q % (LPC / kU ? LPC / kU : 1) == 0) {
                    sdx[t][cl] = make_float2(hb[i], ea[i]);
                    sdv[t][cl] = v[i];
                }
            }
        }
        __syncthreads();
        if (tid < L::kLoad && at + tr < len) {
            const int valid = max(0, min(V, tile.valid - cv));
            float x[V], raw[V], g[V], z[V], dv[V], ox[V], ot[V], oz[V];
            cx.widen(x);
            cd.widen(raw);
            cy.widen(g);
            if (a.z) cz.widen(z);
            gate_grad<V>(g, z, a.z != nullptr, dv);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 r = sdx[tr][cv + j];  // <dh, B>, <e, A>
                const float pre = raw[j] + bias[j], d = time_step(a, pre);
                ox[j] = fmaf(r.x, d, dv[j] * skip[j]);
                ot[j] = fmaf(r.x, x[j], r.y);
                if (a.softplus) ot[j] *= sigmoid_f(pre);
                dD[j] = fmaf(dv[j], x[j], dD[j]);
                db[j] += ot[j];
                if (a.z) {
                    const float sg = sigmoid_f(z[j]);
                    oz[j] = g[j] * fmaf(skip[j], x[j], sdv[tr][cv + j]) * sg * fmaf(z[j], 1.f - sg, 1.f);
                }
            }
            const int64_t to = (p.t0 + at + tr) * a.C + tile.c0 + cv;
            Row<T, V> r;
            r.narrow(ox);
            r.store(dx + to, a.out_bytes, valid);
            r.narrow(ot);
            r.store(ddt + to, a.out_bytes, valid);
            if (a.z) {
                r.narrow(oz);
                r.store(dz + to, a.out_bytes, valid);
            }
        }
        for (int i = tid; i < kT * 2 * kS; i += kNT) {
            const int t = i / (2 * kS), w = i / kS % 2, st = i % kS;
            if (at + t >= len || st >= a.S) continue;
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < kNT / 32; ++k) sum += red[k][t][w * kS + st];
            part[((p.t0 + at + t) * 2 + w) * a.S + st] = sum;
        }
        __syncthreads();
    }
    if (mine) {
#pragma unroll
        for (int i = 0; i < kPS; ++i)
            if (q * kPS + i < a.S) a.E[at_state + i] = dA[i];
    }
    // dD and dbias: the sums of the loading threads' rows, one behind the other
    float(*sum)[2][kC] = reinterpret_cast<float(*)[2][kC]>(smem);
    __syncthreads();
    if (tid < L::kLoad) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sum[tr][0][cv + j] = dD[j];
            sum[tr][1][cv + j] = db[j];
        }
    }
    __syncthreads();
    for (int i = tid; i < 2 * kC; i += kNT) {
        const int w = i / kC, ch = i % kC;
        if (ch >= tile.valid) continue;
        float f = 0.f;
        for (int t = 0; t < kT; ++t) f += sum[t][w][ch];
        a.pd[(slot * 2 + w) * a.C + tile.c0 + ch] = f;
    }
}

// 4a. dB and dC of a token, group and state: the sums of the group's tiles.
template <typename T>
__global__ void __launch_bounds__(256) k_scan_bwd_bc(ScanArgs a, int tiles) {
    const int64_t all = total_tokens(a.r), per = 2 * (int64_t)a.S, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    pdl_wait();
    if (id >= all * a.G * per) return;
    const int64_t t = id / (a.G * per);
    const int g = (int)(id / per % a.G), w = (int)(id / a.S % 2), s = (int)(id % a.S), n = tiles / a.G;
    float f = 0.f;
    const float *p = a.part + ((int64_t)g * n * all + t) * per + w * a.S + s;
    for (int k = 0; k < n; ++k) f += p[(int64_t)k * all * per];
    T *to = (T *)(w ? a.dCm : a.dBm);
    to[(t * a.G + g) * a.S + s] = from_f32<T>(f);
}

// 4b. dA, dD and dbias: the sums of the slots, in eight strands.
__global__ void __launch_bounds__(256) k_scan_bwd_params(ScanArgs a) {
    __shared__ float sum[8][33];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    const int64_t states = a.C * a.S, cols = states + 2 * a.C, i = (int64_t)blockIdx.x * 32 + lane;
    pdl_wait();
    const float *p = i < states ? a.E + i : a.pd + (i - states);
    const int64_t step = i < states ? states : 2 * a.C;
    float f = 0.f;
    if (i < cols)
        for (int64_t k = strand; k < a.slots; k += 8) f += p[k * step];
    sum[strand][lane] = f;
    __syncthreads();
    if (strand || i >= cols) return;
    for (int j = 1; j < 8; ++j) f += sum[j][lane];
    if (i < states) a.dA[i] = f;
    else if (i < states + a.C) { if (a.dD) a.dD[i - states] = f; }
    else if (a.dbias) a.dbias[i - states - a.C] = f;
}

}  // namespace

cudaError_t scan_bwd_summary(const ScanArgs &a, int dtype, cudaStream_t st) {
    const int64_t tiles = scan_tiles(a.C, a.S, a.G);
    return scan_type(dtype, [&](auto t) {
        return scan_lanes(a.S, [&](auto l) {
            k_scan_bwd_sum<decltype(t), decltype(l)::value>
                <<<(unsigned)(a.slots * tiles), kNT, 0, st>>>(a, (int)tiles);
            return cudaGetLastError();
        });
    });
}

cudaError_t scan_bwd(const ScanArgs &a, int dtype, cudaStream_t st) {
    const int64_t tiles = scan_tiles(a.C, a.S, a.G);
    return scan_type(dtype, [&](auto t) {
        return scan_lanes(a.S, [&](auto l) {
            using T = decltype(t);
            constexpr int LPC = decltype(l)::value;
            constexpr size_t smem = bwd_smem<LPC>();
            static std::atomic<uint64_t> done{0};
            cudaError_t e = once_a_device(done, [] {
                return cudaFuncSetAttribute(k_scan_bwd<T, LPC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            (int)smem);
            });
            if (e != cudaSuccess) return e;
            return launch_pdl(k_scan_bwd<T, LPC>, dim3((unsigned)((a.slots + 1) * tiles)), dim3(kNT), smem,
                              st, a, (int)tiles);
        });
    });
}

cudaError_t scan_bwd_bc(const ScanArgs &a, int dtype, cudaStream_t st) {
    const int64_t tiles = scan_tiles(a.C, a.S, a.G);
    const int64_t all = rows_packed(a.r) ? a.r.T : a.r.N * a.r.T, outs = all * a.G * 2 * a.S;
    return scan_type(dtype, [&](auto t) {
        return launch_pdl(k_scan_bwd_bc<decltype(t)>, dim3((unsigned)((outs + 255) / 256)), dim3(256), 0, st,
                          a, (int)tiles);
    });
}

cudaError_t scan_bwd_params(const ScanArgs &a, cudaStream_t st) {
    const int64_t cols = a.C * a.S + 2 * a.C;
    return launch_pdl(k_scan_bwd_params, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, st, a);
}

}  // namespace gdr
