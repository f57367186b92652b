// scan.cu -- the selective state-space scan: for every channel c and state s
//
//   d_t = softplus(dt_t + bias),   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t
//   y_t = <C_t, h_t> + D x_t,      out = y silu(z)
//
// with B_t and C_t shared by the channels of a group.  FP32 states and sums.
//
// Every (token, channel, state) takes one exponential (its decay depends on all
// three) and four FP32 operations, and no matrix product does them: instructions
// and their latencies bound it, not the memory.  So the scan runs along the tokens
// as it is written, each state's chain in a register, and whatever else a token
// needs is kept off the inner loop: a tile of tokens is staged in shared memory
// with d_t and d_t x_t computed once a channel, and the D and z terms are added
// when a tile's sums are written out.  The sums over a channel's states take part
// of a shuffle a token: LPC tokens are folded at once.
//
// With too few (sequence, channel) chains to fill the device the sequences are
// cut into pieces: a first pass leaves each piece's end from a zero start, and
// the sum of its time steps (the piece's decay is exp(A sum d), so no products
// of decays are kept); a join turns the ends into starts; a second pass runs
// the pieces from those.  That takes the exponentials twice.  One sequence of 16K
// tokens x 2048 channels x 16 states: 109, 9 and 168 us; the passes take about 8 and
// 12.5 cycles a scheduler for 32 states, the loop alone would take 5.5.  No unit is
// full (issue slots 59 and 60%, the FMA pipe 56 and 53%, exponentials 58 and 41%):
// with four warps a scheduler (128 registers a thread) a warp mostly waits for the
// result of its own last instruction, for a pipe that another has, and in the second
// pass for shared memory.
#include "scan.cuh"

namespace gdr {
namespace {

constexpr int kPS = 8;  // states of a thread

// Channels of a block, tokens of a tile, channels that a loading thread takes of one token.
template <int LPC>
struct Lay {
    static constexpr int kC = kNT / LPC;
    static constexpr int kT = LPC == 1 ? 8 : 16;
    static constexpr int kV = kT * kC / kNT, kRows = kC / kV;
    static constexpr int kBC = kT * LPC * 2;  // vectors of kPS states of B and C
    static constexpr int kBCper = (kBC + kNT - 1) / kNT;
};

// SUM: leave a piece's end from a zero start (E) and the sum of its time steps (sd).  Else: the
// outputs, from E (pieces) or from h0 (whole sequences), and the last state into ht.
template <typename T, int LPC, bool SUM>
__global__ void __launch_bounds__(kNT, 4) k_scan(ScanArgs a, Tiles tiles) {
    using L = Lay<LPC>;
    constexpr int kT = L::kT, V = L::kV, kC = L::kC;
    using O = Order<V, L::kRows>;
    __shared__ float2 sdx[kT][kC + O::kPad];  // time step and its product with x; the sums over states
    __shared__ float4 sbc[2][kT][2][LPC];  // lanes' halves side by side, so that eight lanes read all banks
    const int tid = threadIdx.x, q = tid % LPC, cl = tid / LPC;
    const uint32_t slot_id = blockIdx.x / tiles.all;
    const int64_t slot = slot_id;
    const Tile tile = tile_of<kC>(tiles, blockIdx.x - slot_id * tiles.all);
    const int tr = tid / L::kRows, lv = tid % L::kRows, cv = lv * V;
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
    if ((SUM || !a.piece) && blockIdx.x == 0 && tid < 32) check_offsets(a.r);
    const Piece p = piece_of(a, slot);
    if (p.n < 0) return;
    int64_t row = 0;
    if (!SUM && (a.h0 || a.ht)) row = state_row(a.idx, a.n_states, p.n, a.r.status);
    const int ch = O::channel(cl);
    const int64_t c = tile.c0 + ch, at_state = c * a.S + q * kPS;
    const bool mine = ch < tile.valid;

    F2 A2[kPS / 2], h[kPS / 2];
    {
        const float *from = SUM || row < 0 ? nullptr
                            : a.piece      ? a.E + slot * a.C * a.S
                            : a.h0         ? a.h0 + row * a.C * a.S
                                           : nullptr;
        float fa[kPS], fh[kPS];
#pragma unroll
        for (int i = 0; i < kPS; ++i) {
            const bool in = mine && q * kPS + i < a.S;
            fa[i] = in ? times_log2e(a.A[at_state + i]) : 0.f;
            fh[i] = in && from ? from[at_state + i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kPS / 2; ++i) {
            A2[i] = f2(fa[2 * i], fa[2 * i + 1]);
            h[i] = f2(fh[2 * i], fh[2 * i + 1]);
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
    Row<T, kPS> nbc[L::kBCper];
    constexpr int kLoadBC = SUM ? kT * LPC : L::kBC;
    auto fetch = [&](int at) {
        const int64_t t0 = p.t0 + at;
        const int len = p.len - at;
        load_row<T, V>(nx, a.x, a.xs, t0, tr, len, tile, cv, a.bytes);
        load_row<T, V>(nd, a.dt, a.dts, t0, tr, len, tile, cv, a.bytes);
        if (!SUM && a.z) load_row<T, V>(nz, a.z, a.zs, t0, tr, len, tile, cv, a.bytes);
#pragma unroll
        for (int k = 0; k < L::kBCper; ++k) {
            const int id = k * kNT + tid, which = id / (kT * LPC), t = id / LPC % kT, v = id % LPC;
            if (id < kLoadBC)
                load_bc<T, kPS>(nbc[k], which ? a.Cm : a.Bm, which ? a.cs : a.bs, tile.g, t0, t, len,
                                kPS * v, a.S, a.bc_bytes);
        }
    };
    fetch(0);
    float total = 0.f;
    for (int at = 0; at < p.len; at += kT) {
        const Row<T, V> cx = nx, cz = nz;
        {
            float x[V], raw[V], d[V];
            nx.widen(x);
            nd.widen(raw);
            time_steps<V>(a, raw, bias, d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (at + tr >= p.len) d[j] = 0.f;  // past the end the states stay as they are
                sdx[tr][O::place(lv, j)] = make_float2(d[j], d[j] * x[j]);
            }
        }
#pragma unroll
        for (int k = 0; k < L::kBCper; ++k) {
            const int id = k * kNT + tid;
            if (id < kLoadBC) {
                float f[kPS];
                nbc[k].widen(f);
                float4 *to = &sbc[id / (kT * LPC)][id / LPC % kT][0][id % LPC];
                to[0] = make_float4(f[0], f[1], f[2], f[3]);
                to[LPC] = make_float4(f[4], f[5], f[6], f[7]);
            }
        }
        __syncthreads();
        if (at + kT < p.len) fetch(at + kT);
#pragma unroll
        for (int t0 = 0; t0 < kT; t0 += LPC) {
            float y[LPC];
#pragma unroll
            for (int k = 0; k < LPC; ++k) {
                const float2 d = sdx[t0 + k][cl];
                const F2 dd = f2(d.x), dx = f2(d.y);
                const ulonglong2 *B = reinterpret_cast<const ulonglong2 *>(&sbc[0][t0 + k][0][q]);
                const ulonglong2 *C = reinterpret_cast<const ulonglong2 *>(&sbc[1][t0 + k][0][q]);
                const ulonglong2 b0 = B[0], b1 = B[LPC];
                const F2 b[4] = {{b0.x}, {b0.y}, {b1.x}, {b1.y}};
#pragma unroll
                for (int i = 0; i < kPS / 2; ++i) h[i] = fma2(decay(dd, A2[i]), h[i], dx * b[i]);
                if constexpr (SUM) {
                    total += d.x;
                } else {
                    const ulonglong2 c0 = C[0], c1 = C[LPC];
                    y[k] = both(fma2(h[0], F2{c0.x}, h[1] * F2{c0.y}) +
                                fma2(h[2], F2{c1.x}, h[3] * F2{c1.y}));
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
            for (int j = 0; j < V; ++j) y[j] = fmaf(skip[j], x[j], sdx[tr][O::place(lv, j)].x);
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
    float *to = SUM ? a.E + slot * a.C * a.S : (a.ht && p.last && row >= 0 ? a.ht + row * a.C * a.S : nullptr);
    if (to) {
#pragma unroll
        for (int i = 0; i < kPS / 2; ++i) {
            float lo, hi;
            split(h[i], lo, hi);
            if (q * kPS + 2 * i < a.S) to[at_state + 2 * i] = lo;
            if (q * kPS + 2 * i + 1 < a.S) to[at_state + 2 * i + 1] = hi;
        }
    }
}

// Ends of pieces into their starts, in place: h <- exp(A sd) h + E.  Backward (blockIdx.y = 1):
// the gradients that enter the pieces' starts into those that reach their ends.  A thread has V
// states of a channel (4, where S is a multiple), and the loads of several pieces in flight: the
// pieces of a sequence follow one another, so what counts is what is asked for at once.
template <int V>
__global__ void __launch_bounds__(128) k_scan_join(ScanArgs a) {
    const int per = (int)(a.C * a.S) / V;  // below 2^31
    const int64_t id = (int64_t)blockIdx.x * 128 + threadIdx.x;
    const int64_t n = id / per, states = a.C * a.S;
    const int at = (int)(id % per) * V, c = at / a.S;
    pdl_wait();
    if (n >= a.r.N) return;
    int64_t s, len;
    seq_span(a.r, n, s, len);
    const int64_t L = a.piece, first = s / L + n, pieces = max((int64_t)1, (len + L - 1) / L);
    const bool back = blockIdx.y;
    float *const part = (back ? a.R : a.E) + first * states + at;
    const float *const sd = a.sd + first * a.C + c;
    float A2[V], h[V];
    Row<float, V> r;
    r.load(a.A + at, a.st_bytes, V);
    r.widen(A2);
#pragma unroll
    for (int k = 0; k < V; ++k) A2[k] = times_log2e(A2[k]);
    r.zero();
    if (back) {
        if (a.dht) r.load(a.dht + n * states + at, a.st_bytes, V);
    } else if (a.h0) {
        const int64_t row = state_row(a.idx, a.n_states, n, a.r.status);
        if (row >= 0) r.load(a.h0 + row * states + at, a.st_bytes, V);
    }
    r.widen(h);
    constexpr int kU = 8;
    for (int64_t j = 0; j < pieces; j += kU) {
        Row<float, V> e[kU];
        float d[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k)
            if (j + k < pieces) {
                const int64_t i = back ? pieces - 1 - j - k : j + k;
                e[k].load(part + i * states, 16, V);
                d[k] = sd[i * a.C];
            }
#pragma unroll
        for (int k = 0; k < kU; ++k)
            if (j + k < pieces) {
                const int64_t i = back ? pieces - 1 - j - k : j + k;
                float f[V];
                e[k].widen(f);
                r.narrow(h);
                r.store(part + i * states, 16, V);
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = fmaf(decay(A2[v], d[k]), h[v], f[v]);
            }
    }
    if (back && a.dh0) {
        r.narrow(h);
        r.store(a.dh0 + n * states + at, a.st_bytes, V);
    }
}

// Sequences of few tokens, straight from memory: what counts is the states' row, read and
// written once.  A warp has 32 channels of a sequence: a lane four states of LPC of them (lane l
// those of channels i (32 / LPC) + l / LPC), and with its own token values of channel l, whose time
// step it forms for the others.  What bounds it is a warp's chain of loads (the state's index, the
// states, all before the first product), so blocks an SM count more than a few spilled registers, and
// what does not wait for the index is asked for before it.  256 sequences x 4096 channels, cold, of 8 /
// 16 / 32 / 64 states: 26 / 37 / 55 / 113 us (states alone at the memory's rate 10 / 20 / 40 / 79); as many
// blocks as fit of themselves, and the loads in their order: 28 / 42 / 59 / 126.
constexpr int step_blocks(int lpc) { return lpc <= 2 ? 7 : lpc == 4 ? 6 : lpc == 8 ? 4 : 2; }
template <typename T, int LPC>
__global__ void __launch_bounds__(kNT, step_blocks(LPC)) k_scan_step(ScanArgs a, Tiles tiles) {
    constexpr int kCh = 32 / LPC;
    const int lane = threadIdx.x & 31, q = lane % LPC, cl = lane / LPC;
    const uint32_t id = blockIdx.x * (kNT / 32) + (threadIdx.x >> 5), seq = id / tiles.all;
    const int64_t n = seq;
    if (blockIdx.x == 0 && threadIdx.x < 32) check_offsets(a.r);
    if (n > a.r.N) return;
    const Tile tile = tile_of<32>(tiles, id - seq * tiles.all);
    const bool mine = lane < tile.valid;
    T *y = (T *)a.y + tile.c0 + lane;
    if (n == a.r.N) {  // tokens of no sequence
        if (!rows_packed(a.r) || !mine) return;
        const int64_t first = min(max(row_bound(a.r, 0), (int64_t)0), a.r.T);
        for (int64_t t = 0; t < first; ++t) y[t * a.ys] = from_f32<T>(0.f);
        for (int64_t t = max(row_bound(a.r, n), (int64_t)0); t < a.r.T; ++t)
            y[t * a.ys] = from_f32<T>(0.f);
        return;
    }
    int64_t s, len;
    seq_span(a.r, n, s, len);
    const int s0 = q * 4, wide = a.S % 4 ? 4 : a.st_bytes;
    const int64_t at_state = (tile.c0 + cl) * a.S + s0;
    const float bias = a.dt_bias && mine ? a.dt_bias[tile.c0 + lane] : 0.f;
    const float skip = a.D && mine ? a.D[tile.c0 + lane] : 0.f;
    auto run = [&](auto whole) {
        // whole: all 32 channels, all states of every lane, 16-byte loads
        constexpr bool W = decltype(whole)::value;
        const int states = W ? 4 : max(0, min(4, a.S - s0)), bytes = W ? 16 : wide;
        auto have = [&](int i) { return W || i * kCh + cl < tile.valid ? states : 0; };
        const int step = kCh * a.S;
        Row<T, 4> rb, rc;
        T rx, rd, rz;
        auto fetch = [&](int64_t t) {
            rb.load((const T *)a.Bm + t * a.bs[0] + tile.g * a.bs[1] + s0, W ? 16 : a.bc_bytes, states);
            rc.load((const T *)a.Cm + t * a.cs[0] + tile.g * a.cs[1] + s0, W ? 16 : a.bc_bytes, states);
            rx = rd = rz = from_f32<T>(0.f);
            if (W || mine) {
                rx = ((const T *)a.x)[t * a.xs + tile.c0 + lane];
                rd = ((const T *)a.dt)[t * a.dts + tile.c0 + lane];
                if (a.z) rz = ((const T *)a.z)[t * a.zs + tile.c0 + lane];
            }
        };
        // what does not wait for the row's number is asked for before it
        if (len > 0) fetch(s);
        Row<float, 4> A[LPC], h[LPC];
#pragma unroll
        for (int i = 0; i < LPC; ++i) A[i].load(a.A + at_state + i * step, bytes, have(i));
        const int64_t row = a.h0 || a.ht ? state_row(a.idx, a.n_states, n, a.r.status) : 0;
        if (row < 0) {
            if (mine)
                for (int64_t t = s; t < s + len; ++t) y[t * a.ys] = from_f32<T>(0.f);
            return;
        }
        const int64_t row_state = row * a.C * a.S + at_state;
#pragma unroll
        for (int i = 0; i < LPC; ++i) {
            h[i].zero();
            if (a.h0) h[i].load(a.h0 + row_state + i * step, bytes, have(i));
        }
        float A2[LPC][4];
#pragma unroll
        for (int i = 0; i < LPC; ++i) {
            A[i].widen(A2[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) A2[i][k] = times_log2e(A2[i][k]);
        }
        for (int64_t t = s; t < s + len; ++t) {
            const float x = to_f32(rx), z = to_f32(rz);
            float d = to_f32(rd) + bias, b[4], cc[4], v[LPC];
            rb.widen(b);
            rc.widen(cc);
            if (t + 1 < s + len) fetch(t + 1);
            if (a.softplus) {
                float unused;
                split(softplus2(f2(d)), d, unused);
            }
            const F2 b01 = f2(b[0], b[1]), b23 = f2(b[2], b[3]), c01 = f2(cc[0], cc[1]), c23 = f2(cc[2], cc[3]);
            const float dx = d * x;
#pragma unroll
            for (int i = 0; i < LPC; ++i) {
                const F2 di = f2(__shfl_sync(0xffffffffu, d, i * kCh + cl));
                const F2 dxi = f2(__shfl_sync(0xffffffffu, dx, i * kCh + cl));
                float h4[4];
                h[i].widen(h4);
                const F2 h01 = fma2(decay(di, f2(A2[i][0], A2[i][1])), f2(h4[0], h4[1]), dxi * b01);
                const F2 h23 = fma2(decay(di, f2(A2[i][2], A2[i][3])), f2(h4[2], h4[3]), dxi * b23);
                v[i] = both(fma2(h01, c01, h23 * c23));
                split(h01, h4[0], h4[1]);
                split(h23, h4[2], h4[3]);
                h[i].narrow(h4);
            }
            // lane q of a channel's lanes has the sum of the q-th of its channels
            float sum = __shfl_sync(0xffffffffu, fold<LPC>(v, q), lane % kCh * LPC + lane / kCh);
            sum = fmaf(skip, x, sum);
            if (a.z) sum *= z * sigmoid_f(z);
            if (W || mine) y[t * a.ys] = from_f32<T>(sum);
        }
        if (!a.ht) return;
#pragma unroll
        for (int i = 0; i < LPC; ++i) h[i].store(a.ht + row_state + i * step, bytes, have(i));
    };
    if (tile.valid == 32 && a.S == 4 * LPC && wide >= 16 && a.bc_bytes >= 4 * (int)sizeof(T)) run(std::true_type{});
    else run(std::false_type{});
}

}  // namespace

// Channels of a block of k_scan.
int scan_channels(int S) { return kNT / (S <= 8 ? 1 : S <= 16 ? 2 : S <= 32 ? 4 : 8); }

cudaError_t scan_step(const ScanArgs &a, int dtype, cudaStream_t st) {
    const Tiles tiles = tiles_of(a, 32);
    const int64_t warps = kNT / 32;
    return scan_type(dtype, [&](auto t) {
        return scan_lanes(a.S, 4, [&](auto l) {
            k_scan_step<decltype(t), decltype(l)::value>
                <<<(unsigned)(((a.r.N + 1) * tiles.all + warps - 1) / warps), kNT, 0, st>>>(a, tiles);
            return cudaGetLastError();
        });
    });
}

cudaError_t scan_pieces(const ScanArgs &a, int dtype, bool summary, cudaStream_t st) {
    const Tiles tiles = tiles_of(a, scan_channels(a.S));
    return scan_type(dtype, [&](auto t) {
        return scan_lanes(a.S, kPS, [&](auto l) {
            using T = decltype(t);
            constexpr int LPC = decltype(l)::value;
            if constexpr (LPC <= 8) {  // S is at most 64
                if (summary) {
                    k_scan<T, LPC, true><<<(unsigned)(a.slots * tiles.all), kNT, 0, st>>>(a, tiles);
                    return cudaGetLastError();
                }
                const dim3 grid((unsigned)((a.slots + 1) * tiles.all));
                if (a.piece)
                    return launch_pdl(k_scan<T, LPC, false>, grid, dim3(kNT), 0, st, a, tiles);
                k_scan<T, LPC, false><<<grid, kNT, 0, st>>>(a, tiles);
            }
            return cudaGetLastError();
        });
    });
}

cudaError_t scan_join(const ScanArgs &a, bool backward, cudaStream_t st) {
    const int V = a.S % 4 ? 1 : 4;
    const int64_t all = a.r.N * a.C * a.S / V;
    const dim3 grid((unsigned)((all + 127) / 128), backward ? 2 : 1);
    if (V == 4) return launch_pdl(k_scan_join<4>, grid, dim3(128), 0, st, a);
    return launch_pdl(k_scan_join<1>, grid, dim3(128), 0, st, a);
}

}  // namespace gdr
