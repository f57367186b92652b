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
//      product of the decays so far, R = sum_t P_t C_t dv_t; and every 8 tokens the
//      state and the sum of the time steps so far;
//   2. the join turns ends into starts, forward for E and backward for R;
//   3. the main pass goes back through the piece 4 tokens at a time: what was left
//      of the states, and what the piece's start adds to them (its decay follows
//      from the sum of the time steps), are the states in front of them, theirs are
//      formed again in registers, and the gradients follow from the last token to
//      the first.
//   4. sums over channels (dB, dC) and over pieces (dA, dD, dbias), in a fixed order.
// What bounds the main pass is the number of instructions, a third of them for the
// sums across lanes: over a channel's states for dx, dd and <C, h>, over the
// channels for dB and dC.  A thread therefore has two channels of four states (the
// channels' sums begin in its registers), and lanes fold eight values at once, so
// that a shuffle carries a value that is still wanted.  The decays are formed a
// second time on the way back: an exponential costs less than the registers.  Rows
// are on their way to shared memory while a tile is worked on, and four blocks fit an
// SM with 9 to 32 states (three with up to 8 or over 32 in 16 bits, two in FP32: there
// shared memory is what limits them).  8 x 2048 tokens x 2048 channels x 16 states: 680
// us; with three blocks and a forward sweep of its own in place of what the first pass
// leaves, 846.  Issue slots are 65% taken and no pipe more than 46%, shared memory 69%:
// as in the forward scan, what is left are latencies that four warps a scheduler leave.
#include "scan.cuh"

namespace gdr {
namespace {

constexpr int kU = kScanBwdKeep;           // tokens from one kept state to the next
constexpr int kG = 4;                      // tokens whose states are in registers at once
constexpr int kKeep = kScanBwdPiece / kU;  // of a piece; the first is the piece's start
constexpr int kWarps = kNT / 32;

// CH channels and STATES states of a thread: channels of a block, tokens of a tile, and what a
// loading thread takes of it.
template <int LPC, int CH, int STATES, int TOKENS>
struct Lay {
    static constexpr int kC = CH * kNT / LPC, kS = STATES * LPC;
    static constexpr int kT = TOKENS;
    static constexpr int kV = kT * kC / kNT;
    static constexpr int kRows = kC / kV;     // loading threads of one token
    static constexpr int kVec = STATES;       // states of a vector of B or C
    static constexpr int kBC = kT * LPC * 2;
    static constexpr int kBCper = (kBC + kNT - 1) / kNT;
    using O = Order<kV, kRows>;
    static constexpr int kPitch = kC + O::kPad;  // of a row of shared memory
    static_assert(kV <= 8 && kV >= 2, "");
};

template <int LPC>
using Ends = Lay<LPC, 1, 8, LPC == 1 ? 8 : 16>;
// Few tokens a tile: a thread's own rows of two tiles then take little shared memory.
template <int LPC>
using Main = Lay<LPC, 2, 4, LPC == 16 ? 16 : kU>;

// dv = dout silu(z), or dout.
template <int V>
__device__ __forceinline__ void gate_grad(const float (&g)[V], const float (&z)[V], bool gated,
                                          float (&dv)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) dv[j] = gated ? g[j] * z[j] * sigmoid_f(z[j]) : g[j];
}

// Stages tokens [t0, t0 + kT) of the piece: time steps and their products with x, dv, B and C.
template <typename T, typename L>
struct Stage {
    static constexpr int kT = L::kT, V = L::kV, kP = L::kPitch, LPC = L::kS / L::kVec;
    using O = typename L::O;
    Row<T, V> x, dt, z, dy;
    Row<T, L::kVec> bc[L::kBCper];

    __device__ __forceinline__ void fetch(const ScanArgs &a, const Tile &tile, int64_t t0, int len) {
        const int tid = threadIdx.x, tr = tid / L::kRows, cv = tid % L::kRows * V;
        load_row<T, V>(x, a.x, a.xs, t0, tr, len, tile, cv, a.bytes);
        load_row<T, V>(dt, a.dt, a.dts, t0, tr, len, tile, cv, a.bytes);
        load_row<T, V>(dy, a.dy, a.ys, t0, tr, len, tile, cv, a.bytes);
        if (a.z) load_row<T, V>(z, a.z, a.zs, t0, tr, len, tile, cv, a.bytes);
        fetch_bc(a, tile, t0, len);
    }
    __device__ __forceinline__ void fetch_bc(const ScanArgs &a, const Tile &tile, int64_t t0, int len) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int k = 0; k < L::kBCper; ++k) {
            const int id = k * kNT + tid, which = id / (kT * LPC), t = id / LPC % kT, v = id % LPC;
            if (id < L::kBC)
                load_bc<T, L::kVec>(bc[k], which ? a.Cm : a.Bm, which ? a.cs : a.bs, tile.g, t0, t, len,
                                    L::kVec * v, a.S, a.bc_bytes);
        }
    }
    // sbc: [2][kT][kS], a row's vectors' first four states behind one another, then their last; bias: of the tile's channels, in the order of their places
    __device__ __forceinline__ void put(const ScanArgs &a, const float *bias, int len, float2 (*sdx)[kP],
                                        float (*sdv)[kP], float *sbc) const {
        const int tid = threadIdx.x, tr = tid / L::kRows, lv = tid % L::kRows;
        float fx[V], raw[V], fb[V], d[V];
        x.widen(fx);
        dt.widen(raw);
#pragma unroll
        for (int j = 0; j < V; ++j) fb[j] = bias[O::place(lv, j)];
        time_steps<V>(a, raw, fb, d);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (tr >= len) d[j] = 0.f;  // past the end the states stay as they are
            sdx[tr][O::place(lv, j)] = make_float2(d[j], d[j] * fx[j]);
        }
        float g[V], fz[V], dv[V];
        dy.widen(g);
        if (a.z) z.widen(fz);
        gate_grad<V>(g, fz, a.z != nullptr, dv);
#pragma unroll
        for (int j = 0; j < V; ++j) sdv[tr][O::place(lv, j)] = dv[j];
#pragma unroll
        for (int k = 0; k < L::kBCper; ++k) {
            const int id = k * kNT + tid;
            if (id < L::kBC) {
                float f[L::kVec];
                bc[k].widen(f);
#pragma unroll
                for (int i = 0; i < L::kVec; i += 4)
                    *reinterpret_cast<float4 *>(sbc + id / LPC * L::kS + i * LPC + id % LPC * 4) =
                        make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
            }
        }
    }
};

// The rows of a tile on their way to shared memory, each thread's to places of its own: there they
// are when the tile is staged, and again when its gradients are written.
template <typename T, typename L>
struct Rows {
    static constexpr int V = L::kV;
    using R = Row<T, V>;
    struct alignas(R::kBytes < 16 ? R::kBytes : 16) Slot {
        uint8_t b[R::kBytes];
    };
    Slot own[4][kNT];  // x, dt, dy, z

    __device__ __forceinline__ void ask(const ScanArgs &a, const Tile &tile, int64_t t0, int len) {
        const int tid = threadIdx.x, tr = tid / L::kRows, cv = tid % L::kRows * V;
        const int valid = tr < len ? max(0, min(V, tile.valid - cv)) : 0;
        const void *const base[4] = {a.x, a.dt, a.dy, a.z};
        const int64_t stride[4] = {a.xs, a.dts, a.ys, a.zs};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n == 3 && !a.z) break;
            const T *from = (const T *)base[n] + (t0 + tr) * stride[n] + tile.c0 + cv;
            if (valid == V && a.bytes >= R::kNeed) {
                constexpr int kCopy = R::kNeed;
                const uint32_t to = (uint32_t)__cvta_generic_to_shared(&own[n][tid]);
#pragma unroll
                for (int i = 0; i < R::kBytes / kCopy; ++i) {
                    if constexpr (kCopy == 16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16 * i),
                                     "l"((const uint8_t *)from + 16 * i) : "memory");
                    else
                        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(kCopy)
                                     : "memory");
                }
            } else {
                R r;
                r.load(from, a.bytes, valid);
                r.store(reinterpret_cast<T *>(&own[n][tid]), 16, V);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ R row(int n) const {
        R r;
        r.load(reinterpret_cast<const T *>(&own[n][threadIdx.x]), 16, V);
        return r;
    }
};

// The bias of the tile's channels in the order of their places, and D behind it.
template <typename L>
__device__ __forceinline__ void load_channels(const ScanArgs &a, const Tile &tile, float *to) {
    for (int i = threadIdx.x; i < L::kC; i += kNT) {
        const int ch = L::O::channel(i);
        to[i] = a.dt_bias && ch < tile.valid ? a.dt_bias[tile.c0 + ch] : 0.f;
        to[L::kC + i] = a.D && ch < tile.valid ? a.D[tile.c0 + ch] : 0.f;
    }
}

// K neighbouring states of a channel from s0 on; zeros past S, where `in` does not hold, and without
// an address.
template <int K>
__device__ __forceinline__ void load_states(const float *p, int s0, int S, bool in, F2 (&to)[K / 2]) {
    Row<float, K> r;
    r.load(p, S % 4 ? 4 : 16, p && in ? max(0, min(K, S - s0)) : 0);
    widen2<float, K>(r, to);
}
template <int K>
__device__ __forceinline__ void store_states(float *p, int s0, int S, const F2 (&from)[K / 2]) {
    Row<float, K> r;
    narrow2<float, K>(from, r);
    r.store(p, S % 4 ? 4 : 16, max(0, min(K, S - s0)));
}
template <int K>
__device__ __forceinline__ void load_A2(const ScanArgs &a, int64_t at, int s0, bool in, F2 (&to)[K / 2]) {
    float f[K];
#pragma unroll
    for (int i = 0; i < K; ++i) f[i] = in && s0 + i < a.S ? times_log2e(a.A[at + i]) : 0.f;
#pragma unroll
    for (int i = 0; i < K / 2; ++i) to[i] = f2(f[2 * i], f[2 * i + 1]);
}

// 1. E, sd and R of a piece.  A thread has eight states of a channel.
template <typename T, int LPC>
__global__ void __launch_bounds__(kNT) k_scan_bwd_ends(ScanArgs a, Tiles tiles) {
    using L = Ends<LPC>;
    constexpr int kT = L::kT, kC = L::kC, P = 4;
    __shared__ __align__(16) float2 sdx[kT][L::kPitch];
    __shared__ float sdv[kT][L::kPitch], sch[2 * kC];
    __shared__ __align__(16) float sbc[2 * kT * L::kS];
    const int tid = threadIdx.x, q = tid % LPC, cl = tid / LPC;
    const uint32_t slot_id = blockIdx.x / tiles.all;
    const int64_t slot = slot_id;
    const Tile tile = tile_of<kC>(tiles, blockIdx.x - slot_id * tiles.all);
    if (blockIdx.x == 0 && tid < 32) check_offsets(a.r);
    const Piece p = piece_of(a, slot);
    if (p.n < 0) return;
    const int ch = L::O::channel(cl);
    const int64_t c = tile.c0 + ch, at_state = c * a.S + q * 8;
    const bool mine = ch < tile.valid;
    F2 A2[P], h[P], D[P], R[P];
    float total = 0.f;
    load_A2<8>(a, at_state, q * 8, mine, A2);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        h[i] = R[i] = f2(0.f);
        D[i] = f2(1.f);
    }
    Stage<T, L> s;
    s.fetch(a, tile, p.t0, p.len);
    load_channels<L>(a, tile, sch);
    __syncthreads();
    for (int at = 0; at < p.len; at += kT) {
        s.put(a, sch, p.len - at, sdx, sdv, sbc);
        __syncthreads();
        if (at + kT < p.len) s.fetch(a, tile, p.t0 + at + kT, p.len - at - kT);
#pragma unroll 4
        for (int t = 0; t < kT; ++t) {
            if (t % kU == 0 && at + t && mine) {
                const int64_t k = slot * kKeep + (at + t) / kU;
                store_states<8>(a.keep + k * a.C * a.S + at_state, q * 8, a.S, h);
                if (q == 0) a.keep_d[k * a.C + c] = total;
            }
            const float2 d = sdx[t][cl];
            const F2 dd = f2(d.x), dx = f2(d.y), dv = f2(sdv[t][cl]);
            const ulonglong2 *B = reinterpret_cast<const ulonglong2 *>(sbc + t * L::kS + q * 4);
            const ulonglong2 *C = reinterpret_cast<const ulonglong2 *>(sbc + (kT + t) * L::kS + q * 4);
            const ulonglong2 b0 = B[0], b1 = B[LPC], c0 = C[0], c1 = C[LPC];
            const F2 b[P] = {{b0.x}, {b0.y}, {b1.x}, {b1.y}}, cc[P] = {{c0.x}, {c0.y}, {c1.x}, {c1.y}};
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const F2 w = decay(dd, A2[i]);
                h[i] = fma2(w, h[i], dx * b[i]);
                D[i] = D[i] * w;
                R[i] = fma2(D[i], cc[i] * dv, R[i]);
            }
            total += d.x;
        }
        __syncthreads();
    }
    if (!mine) return;
    if (q == 0) a.sd[slot * a.C + c] = total;
    store_states<8>(a.E + slot * a.C * a.S + at_state, q * 8, a.S, h);
    store_states<8>(a.R + slot * a.C * a.S + at_state, q * 8, a.S, R);
}

// Sums of eight values over a channel's LPC lanes.  A lane ends with 8 / LPC of them (at least
// one), those from first_of<LPC>(q) on; with LPC = 16 two lanes end with the same.
template <int LPC>
__device__ __forceinline__ void fold_states(float (&v)[8], int q) {
    int n = 8;
#pragma unroll
    for (int m = LPC / 2; m >= 1; m >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = q & m;
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
__device__ __forceinline__ int first_of(int q) {
    return LPC <= 8 ? q * (8 / LPC) : q / 2;
}

// Sums of eight values (four states of B, four of C) over the warp's 32 / LPC lanes of one state.
// A lane ends with 8 / lanes of them (at least one).
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

template <typename T, int LPC>
struct Smem {
    using L = Main<LPC>;
    float sbc[2 * L::kT * L::kS];
    float2 sdx[L::kT][L::kPitch];      // time step, and its product with x
    float2 res[L::kT][L::kPitch];      // <dh, B>, <e, A> / ln 2
    float sdv[L::kT][L::kPitch];       // dv, then <C, h>
    float red[kWarps][L::kT][2 * L::kS];
    float sch[2 * L::kC];
    // a thread's own
    Rows<T, L> rows[2];                // of this tile and the next
    float acc[2][L::kV][kNT];          // dD and dbias of the channels that it loads
    float4 start[2][kNT];              // what its states start from in the piece
    float4 base[2][kNT];               // ... and in front of the last kept place
    float4 kept[2][2][kNT];            // what was kept in front of the tile's last kU tokens, and the next's
    float kept_d[2][2][kNT];
};

// Four states of two channels, forward by a token; y: <C, h> of the two.
template <bool OUT>
__device__ __forceinline__ void step(const float4 &d, const ulonglong2 &B, const ulonglong2 &C,
                                     const F2 (&A2)[2][2], F2 (&h)[2][2], float *y) {
    const float dd[2] = {d.x, d.z}, dx[2] = {d.y, d.w};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const F2 dk = f2(dd[k]), xk = f2(dx[k]);
        h[k][0] = fma2(decay(dk, A2[k][0]), h[k][0], xk * F2{B.x});
        h[k][1] = fma2(decay(dk, A2[k][1]), h[k][1], xk * F2{B.y});
        if constexpr (OUT) y[k] = both(fma2(h[k][0], F2{C.x}, h[k][1] * F2{C.y}));
    }
}

__device__ __forceinline__ void put_own(float4 &to, const F2 (&x)[2]) {
    *reinterpret_cast<ulonglong2 *>(&to) = make_ulonglong2(x[0].v, x[1].v);
}
__device__ __forceinline__ void take_own(const float4 &from, F2 (&x)[2]) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&from);
    x[0] = F2{v.x};
    x[1] = F2{v.y};
}

// 3. The gradients of a piece.  At the end E's slot holds its part of dA.
template <typename T, int LPC>
__global__ void __launch_bounds__(kNT, 4) k_scan_bwd(ScanArgs a, Tiles tiles) {
    using L = Main<LPC>;
    constexpr int kT = L::kT, V = L::kV, kC = L::kC, kS = L::kS;
    extern __shared__ __align__(16) uint8_t raw_smem[];
    Smem<T, LPC> &sm = *reinterpret_cast<Smem<T, LPC> *>(raw_smem);
    const int tid = threadIdx.x, q = tid % LPC, cl = tid / LPC, lane = tid & 31, warp = tid >> 5;
    const uint32_t slot_id = blockIdx.x / tiles.all, tile_id = blockIdx.x - slot_id * tiles.all;
    const int64_t slot = slot_id;
    const Tile tile = tile_of<kC>(tiles, tile_id);
    const int tr = tid / L::kRows, lv = tid % L::kRows, cv = lv * V;
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
    const int len = p.n < 0 ? 0 : p.len;
    const int s0 = q * 4;
    int64_t at_state[2];
    bool mine[2];
    F2 A2[2][2], dh[2][2], dA[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int ch = L::O::channel(2 * cl + k);
        at_state[k] = (tile.c0 + ch) * a.S + s0;
        mine[k] = ch < tile.valid;
        load_A2<4>(a, at_state[k], s0, mine[k], A2[k]);
        F2 start[2];
        load_states<4>(a.E + slot * a.C * a.S + at_state[k], s0, a.S, mine[k] && len, start);
        put_own(sm.start[k][tid], start);
        load_states<4>(a.R + slot * a.C * a.S + at_state[k], s0, a.S, mine[k] && len, dh[k]);
        dA[k][0] = dA[k][1] = f2(0.f);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) sm.acc[0][j][tid] = sm.acc[1][j][tid] = 0.f;
    load_channels<L>(a, tile, sm.sch);
    auto B_at = [&](int t) { return *reinterpret_cast<const ulonglong2 *>(sm.sbc + t * kS + s0); };
    auto C_at = [&](int t) { return *reinterpret_cast<const ulonglong2 *>(sm.sbc + (kT + t) * kS + s0); };
    auto d_at = [&](int t) { return *reinterpret_cast<const float4 *>(&sm.sdx[t][2 * cl]); };

    // What was kept in front of token `at` (none before the first) on its way: the states without what
    // the piece started from, and the sum of the time steps up to there.
    const int have = max(0, min(4, a.S - s0));
    auto ask_kept = [&](int stage, int at) {
        if (at <= 0) return;
        const int64_t i = slot * kKeep + at / kU;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float *from = a.keep + i * a.C * a.S + at_state[k];
            const float *from_d = a.keep_d + i * a.C + tile.c0 + L::O::channel(2 * cl + k);
            if (mine[k] && have == 4 && a.S % 4 == 0) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::
                             "r"((uint32_t)__cvta_generic_to_shared(&sm.kept[stage][k][tid])), "l"(from) : "memory");
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::
                             "r"((uint32_t)__cvta_generic_to_shared(&sm.kept_d[stage][k][tid])), "l"(from_d) : "memory");
            } else {
                Row<float, 4> x;
                x.load(from, 4, mine[k] ? have : 0);
                x.store(reinterpret_cast<float *>(&sm.kept[stage][k][tid]), 16, 4);
                sm.kept_d[stage][k][tid] = mine[k] ? *from_d : 0.f;
            }
        }
    };

    Stage<T, L> s;
    const int last = (len - 1) / kT * kT;
    int now = 0;
    if (len) {
        ask_kept(0, last + kT - kU);
        sm.rows[0].ask(a, tile, p.t0 + last, len - last);
        s.fetch_bc(a, tile, p.t0 + last, len - last);
    }
    __syncthreads();
    for (int at = last; at >= 0 && len; at -= kT, now ^= 1) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        s.x = sm.rows[now].row(0);
        s.dt = sm.rows[now].row(1);
        s.dy = sm.rows[now].row(2);
        if (a.z) s.z = sm.rows[now].row(3);
        s.put(a, sm.sch, len - at, sm.sdx, sm.sdv, sm.sbc);
        __syncthreads();
        if (at) {
            ask_kept(now ^ 1, at - kU);  // the last kU tokens of the tile before this
            sm.rows[now ^ 1].ask(a, tile, p.t0 + at - kT, len - at + kT);
            s.fetch_bc(a, tile, p.t0 + at - kT, len - at + kT);
        }
#pragma unroll 1
        for (int u = kT - kG; u >= 0; u -= kG) {
            F2 hs[kG][2][2], before[2][2];
            const int from = at + u - u % kU;
            if (u % kU && from) {
                if (u < kT - kU) {  // of a tile of more than kU tokens: the first of them
                    ask_kept(now, from);
                    asm volatile("cp.async.wait_all;" ::: "memory");
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    F2 f[2];
                    take_own(sm.kept[now][k][tid], f);
                    take_own(sm.start[k][tid], before[k]);
                    const F2 d = f2(sm.kept_d[now][k][tid]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) before[k][j] = fma2(decay(d, A2[k][j]), before[k][j], f[j]);
                    put_own(sm.base[k][tid], before[k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) take_own(from ? sm.base[k][tid] : sm.start[k][tid], before[k]);
            }
            if (u % kU) {
#pragma unroll
                for (int t = kG; t > 0; --t) step<false>(d_at(u - t), B_at(u - t), ulonglong2{}, A2, before, nullptr);
            }
            float y[2 * kG], hb[2 * kG], ea[2 * kG];  // of token t and channel k in 2 t + k
#pragma unroll
            for (int t = 0; t < kG; ++t) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j) hs[t][k][j] = t ? hs[t ? t - 1 : 0][k][j] : before[k][j];
                step<true>(d_at(u + t), B_at(u + t), C_at(u + t), A2, hs[t], y + 2 * t);
            }
            if (a.z) fold_states<LPC>(y, q);
            // so that nothing of the way there is kept in registers for the way back
            asm volatile("" ::: "memory");
#pragma unroll
            for (int t = kG - 1; t >= 0; --t) {
                const float4 d = d_at(u + t);
                const float2 dv2 = *reinterpret_cast<const float2 *>(&sm.sdv[u + t][2 * cl]);
                const ulonglong2 B = B_at(u + t), C = C_at(u + t);
                const F2 b[2] = {{B.x}, {B.y}}, cc[2] = {{C.x}, {C.y}};
                const float ds[2] = {d.x, d.z}, dxs[2] = {d.y, d.w}, dvs[2] = {dv2.x, dv2.y};
                F2 dB[2], dC[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const F2 dd = f2(ds[k]), dx2 = f2(dxs[k]), dv = f2(dvs[k]);
                    F2 e[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        F2 &g = dh[k][j];
                        g = fma2(dv, cc[j], g);
                        dB[j] = k ? fma2(g, dx2, dB[j]) : g * dx2;
                        dC[j] = k ? fma2(dv, hs[t][k][j], dC[j]) : dv * hs[t][k][j];
                        e[j] = g * b[j];
                    }
                    hb[2 * t + k] = both(e[0] + e[1]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        F2 &g = dh[k][j];
                        g = g * decay(dd, A2[k][j]);
                        e[j] = g * (t ? hs[t ? t - 1 : 0][k][j] : before[k][j]);
                        dA[k][j] = fma2(e[j], dd, dA[k][j]);
                    }
                    ea[2 * t + k] = both(fma2(e[0], A2[k][0], e[1] * A2[k][1]));
                }
                float bc[8];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    split(dB[j], bc[2 * j], bc[2 * j + 1]);
                    split(dC[j], bc[4 + 2 * j], bc[5 + 2 * j]);
                }
                fold_channels<LPC>(bc, lane);
                // the lane's number among those of its states names the values that it has
                constexpr int kCh = 32 / LPC, kHas = kCh >= 8 ? 1 : 8 / kCh, kDup = kCh > 8 ? kCh / 8 : 1;
                const int ch = lane / LPC;
                if (ch % kDup == 0) {
#pragma unroll
                    for (int i = 0; i < kHas; ++i) {
                        const int idx = ch / kDup * kHas + i;  // B's four, C's four
                        sm.red[warp][u + t][idx / 4 * kS + s0 + idx % 4] = bc[i];
                    }
                }
            }
            fold_states<LPC>(hb, q);
            fold_states<LPC>(ea, q);
            __syncwarp();  // dv of these tokens has been read
#pragma unroll
            for (int i = 0; i < (LPC <= 8 ? 8 / LPC : 1); ++i) {
                const int idx = first_of<LPC>(q) + i, t = u + idx / 2, place = 2 * cl + idx % 2;
                if (LPC <= 8 || q % 2 == 0) {
                    sm.res[t][place] = make_float2(hb[i], ea[i]);
                    if (a.z) sm.sdv[t][place] = y[i];
                }
            }
        }
        __syncthreads();
        if (at + tr < len) {
            const int valid = max(0, min(V, tile.valid - cv));
            float x[V], raw[V], g[V], z[V], dv[V], ox[V], ot[V], oz[V];
            sm.rows[now].row(0).widen(x);
            sm.rows[now].row(1).widen(raw);
            sm.rows[now].row(2).widen(g);
            if (a.z) sm.rows[now].row(3).widen(z);
            gate_grad<V>(g, z, a.z != nullptr, dv);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int at_j = L::O::place(lv, j);
                const float2 r = sm.res[tr][at_j];
                const float skip = sm.sch[kC + at_j];
                ox[j] = fmaf(r.x, sm.sdx[tr][at_j].x, dv[j] * skip);
                ot[j] = fmaf(r.x, x[j], r.y * kLn2);
                if (a.softplus) ot[j] *= sigmoid_f(raw[j] + sm.sch[at_j]);
                sm.acc[0][j][tid] = fmaf(dv[j], x[j], sm.acc[0][j][tid]);
                sm.acc[1][j][tid] += ot[j];
                if (a.z) {
                    const float sg = sigmoid_f(z[j]);
                    oz[j] = g[j] * fmaf(skip, x[j], sm.sdv[tr][at_j]) * sg * fmaf(z[j], 1.f - sg, 1.f);
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
            for (int k = 0; k < kWarps; ++k) sum += sm.red[k][t][w * kS + st];
            part[((p.t0 + at + t) * 2 + w) * a.S + st] = sum;
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (mine[k]) store_states<4>(a.E + slot * a.C * a.S + at_state[k], s0, a.S, dA[k]);
    // dD and dbias: the sums of the loading threads' rows, one behind the other
    __syncthreads();
    for (int i = tid; i < 2 * kC; i += kNT) {
        const int w = i / kC, ch = i % kC;
        if (ch >= tile.valid) continue;
        float f = 0.f;
#pragma unroll
        for (int t = 0; t < kT; ++t) f += sm.acc[w][ch % V][t * L::kRows + ch / V];
        a.pd[(slot * 2 + w) * a.C + tile.c0 + ch] = f;
    }
}

// 4a. dB and dC of a token, group and state: the sums of the group's tiles.
template <typename T>
__global__ void __launch_bounds__(256) k_scan_bwd_bc(ScanArgs a, Tiles tiles) {
    const int64_t all = total_tokens(a.r), per = 2 * (int64_t)a.S, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    pdl_wait();
    if (id >= all * a.G * per) return;
    const int64_t t = id / (a.G * per);
    const int g = (int)(id / per % a.G), w = (int)(id / a.S % 2), s = (int)(id % a.S), n = (int)tiles.group;
    float f = 0.f;
    const float *p = a.part + ((int64_t)g * n * all + t) * per + w * a.S + s;
    for (int k = 0; k < n; ++k) f += p[(int64_t)k * all * per];
    T *to = (T *)(w ? a.dCm : a.dBm);
    to[(t * a.G + g) * a.S + s] = from_f32<T>(f);
}

// 4b. dA, dD and dbias: the sums of the slots.
__global__ void __launch_bounds__(kColumnThreads) k_scan_bwd_params(ScanArgs a) {
    const int64_t states = a.C * a.S, cols = states + 2 * a.C;
    const int64_t i = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    pdl_wait();
    const float f = column_sum(i < states ? a.E + i : a.pd + (i - states), i < states ? states : 2 * a.C,
                               a.slots, i < cols);
    if (threadIdx.x >= 32 || i >= cols) return;
    if (i < states) a.dA[i] = f;
    else if (i < states + a.C) { if (a.dD) a.dD[i - states] = f; }
    else if (a.dbias) a.dbias[i - states - a.C] = f;
}

}  // namespace

// Channels of a block of the main pass.
int scan_bwd_channels(int S) { return 2 * kNT / (S <= 8 ? 2 : S <= 16 ? 4 : S <= 32 ? 8 : 16); }

cudaError_t scan_bwd_ends(const ScanArgs &a, int dtype, cudaStream_t st) {
    return scan_type(dtype, [&](auto t) {
        return scan_lanes(a.S, 8, [&](auto l) {
            constexpr int LPC = decltype(l)::value;
            if constexpr (LPC <= 8) {  // S is at most 64
                using T = decltype(t);
                const Tiles tiles = tiles_of(a, Ends<LPC>::kC);
                k_scan_bwd_ends<T, LPC><<<(unsigned)(a.slots * tiles.all), kNT, 0, st>>>(a, tiles);
            }
            return cudaGetLastError();
        });
    });
}

cudaError_t scan_bwd(const ScanArgs &a, int dtype, cudaStream_t st) {
    const Tiles tiles = tiles_of(a, scan_bwd_channels(a.S));
    return scan_type(dtype, [&](auto t) {
        return scan_lanes(a.S, 4, [&](auto l) {
            using T = decltype(t);
            constexpr int LPC = decltype(l)::value < 2 ? 2 : decltype(l)::value;
            constexpr size_t smem = sizeof(Smem<T, LPC>);
            static std::atomic<uint64_t> done{0};
            cudaError_t e = once_a_device(done, [] {
                return cudaFuncSetAttribute(k_scan_bwd<T, LPC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            (int)smem);
            });
            if (e != cudaSuccess) return e;
            return launch_pdl(k_scan_bwd<T, LPC>, dim3((unsigned)((a.slots + 1) * tiles.all)), dim3(kNT), smem,
                              st, a, tiles);
        });
    });
}

cudaError_t scan_bwd_bc(const ScanArgs &a, int dtype, cudaStream_t st) {
    const Tiles tiles = tiles_of(a, scan_bwd_channels(a.S));
    const int64_t all = rows_packed(a.r) ? a.r.T : a.r.N * a.r.T, outs = all * a.G * 2 * a.S;
    return scan_type(dtype, [&](auto t) {
        return launch_pdl(k_scan_bwd_bc<decltype(t)>, dim3((unsigned)((outs + 255) / 256)), dim3(256), 0, st,
                          a, tiles);
    });
}

cudaError_t scan_bwd_params(const ScanArgs &a, cudaStream_t st) {
    const int64_t cols = a.C * a.S + 2 * a.C;
    return launch_pdl(k_scan_bwd_params, dim3((unsigned)((cols + 31) / 32)), dim3(kColumnThreads), 0, st, a);
}

}  // namespace gdr
