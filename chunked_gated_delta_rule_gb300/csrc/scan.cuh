// scan.cuh -- what the selective scan's kernels share: how channels and states
// lie over a block, how sequences are cut into pieces, pairs of FP32 values, and
// the time step.
//
// A thread holds some neighbouring states of one or two channels; LPC
// neighbouring lanes (a power of two) hold a channel's states.  States past S
// have A = B = C = 0, so they stay zero.
//
// Pieces: sequence n is cut into ceil(len / L) pieces of L tokens.  Piece j of
// it is slot floor(cu[n] / L) + n + j: since floor((a + len) / L) + 1 - floor(a /
// L) >= ceil(len / L), no two pieces share a slot, an empty sequence has one of
// its own, floor(T / L) + N slots hold all, and a block finds its piece from
// the slot without a table.
#pragma once

#include "layer.cuh"

namespace gdr {

constexpr int kNT = 128;  // threads of a block

// e^(d A) with A2 = A log2(e).  ex2.approx comes out too small by 1.4e-8 to 2.6e-8 of its value on
// average for exponents from -1 to 0 (measured), and a state multiplies the decays of as many tokens as
// it remembers: so the product's FMA adds what makes up for 2e-8.  (dA of 1023 tokens was off by
// 1.1e-6 of its size, now by 3.4e-7.)
constexpr float kEx2Lack = 2.9e-8f;
__device__ __forceinline__ F2 decay(F2 d, F2 A2) { return ex2(fma2(d, A2, f2(kEx2Lack))); }
__device__ __forceinline__ float decay(float d, float A2) { return ex2(fmaf(d, A2, kEx2Lack)); }

// A log2(e), finite where A = -inf: times the zero time step of a place past a sequence's end it has to
// give a decay of 1.
__device__ __forceinline__ float times_log2e(float A) {
    const float x = A * kLog2e;
    return x < -3e38f ? -3e38f : x;
}

// log(1 + e^x) = max(x, 0) + log(1 + u), u = e^-|x|, for two values.  u is 2^-t with what rounding
// t = |x| log2(e) lost put back.  log(1 + u) = 2 artanh(s) with 2 s = u / (1 + u / 2); artanh(s) / s
// is a polynomial in (2 s)^2 <= 4 / 9 (fitted here, off by 5e-9 at most).
__device__ __forceinline__ F2 softplus2(F2 x) {
    float a, b, ta, tb, va, vb;
    split(x, a, b);
    // from 100 on u counts for nothing; NaN stays
    const F2 m = f2(fabsf(a) > 100.f ? 100.f : fabsf(a), fabsf(b) > 100.f ? 100.f : fabsf(b));
    const F2 t = m * f2(kLog2e), lost = fma2(m, f2(-kLog2e), t);
    split(t, ta, tb);
    F2 u = f2(ex2(-ta), ex2(-tb));
    u = fma2(u, lost * f2(kLn2), u);
    split(fma2(u, f2(0.5f), f2(1.f)), va, vb);
    const F2 s = u * f2(rcp(va), rcp(vb)), w = s * s;
    F2 p = fma2(w, f2(0.00054710911f), f2(0.00218764110f));
    p = fma2(w, p, f2(0.01250672713f));
    p = fma2(w, p, f2(0.08333302289f));
    p = fma2(w, p, f2(1.f));
    return fma2(s, p, f2(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}

// Time steps of V channels from dt and its bias.
template <int V>
__device__ __forceinline__ void time_steps(const ScanArgs &a, const float (&raw)[V], const float (&bias)[V],
                                           float (&d)[V]) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
        F2 x = f2(raw[j], raw[j + 1]) + f2(bias[j], bias[j + 1]);
        if (a.softplus) x = softplus2(x);
        split(x, d[j], d[j + 1]);
    }
}

// A launch's blocks: `all` tiles of channels for each slot (or sequence), those of a group side by
// side, each of `per` channels.
struct Tiles {
    uint32_t all, group, per;
};
inline Tiles tiles_of(const ScanArgs &a, int channels) {
    const uint32_t per = (uint32_t)(a.C / a.G), group = (per + channels - 1) / channels;
    return Tiles{group * (uint32_t)a.G, group, per};
}

// The channels of tile `id`: a tile lies within one group of B and C.
struct Tile {
    int64_t c0;
    int valid, g;
};
template <int C>
__device__ __forceinline__ Tile tile_of(const Tiles &tiles, uint32_t id) {
    Tile t;
    t.g = tiles.group == tiles.all ? 0 : (int)(id / tiles.group);
    const int at = (int)(id - t.g * tiles.group) * C;
    t.c0 = (int64_t)t.g * tiles.per + at;
    t.valid = min(C, (int)tiles.per - at);
    return t;
}

// The piece in slot `slot` (found by each warp on its own): tokens [t0, t0 + len) of sequence n;
// n < 0: the slot is empty.
struct Piece {
    int64_t n, t0;
    int len, j;
    bool last;
};
__device__ __forceinline__ Piece piece_of(const ScanArgs &a, int64_t slot) {
    Piece p{};
    int64_t s, len;
    if (!a.piece) {
        p.n = slot;
        seq_span(a.r, slot, s, len);
        p.t0 = s;
        p.len = (int)len;
        p.last = true;
        return p;
    }
    const uint32_t L = (uint32_t)a.piece;
    auto first_slot = [&](int64_t n) { return (int64_t)((uint32_t)row_bound(a.r, n) / L) + n; };
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = a.r.N;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) >> 5, at = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < hi && first_slot(at) <= slot);
        const int last = m ? 31 - __clz(m) : 0;
        lo += last * step;
        if (lo + step < hi) hi = lo + step;
    }
    seq_span(a.r, lo, s, len);
    const int64_t j = slot - first_slot(lo), at = j * (int64_t)L;
    if (j < 0 || (at >= len && j > 0)) {
        p.n = -1;
        return p;
    }
    p.n = lo;
    p.j = (int)j;
    p.t0 = s + at;
    p.len = (int)min((int64_t)L, len - at);
    p.last = at + L >= len;
    return p;
}

// V neighbouring channels of token row t0 + tr of a tile, zeros past its ends.
template <typename T, int V>
__device__ __forceinline__ void load_row(Row<T, V> &r, const void *base, int64_t stride, int64_t t0,
                                         int tr, int len, const Tile &tile, int cv, int bytes) {
    const int valid = tr < len ? max(0, min(V, tile.valid - cv)) : 0;
    r.load((const T *)base + (t0 + tr) * stride + tile.c0 + cv, bytes, valid);
}

// K states of B or C of token row t0 + tr, zeros past the ends.
template <typename T, int K>
__device__ __forceinline__ void load_bc(Row<T, K> &r, const void *base, const int64_t (&st)[2], int g,
                                        int64_t t0, int tr, int len, int s0, int S, int bytes) {
    const int valid = tr < len ? max(0, min(K, S - s0)) : 0;
    r.load((const T *)base + (t0 + tr) * st[0] + g * st[1] + s0, bytes, valid);
}

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

// Calls f(LPC) for lanes of `states` states each.
template <typename F>
cudaError_t scan_lanes(int S, int states, F f) {
    if (S <= states) return f(std::integral_constant<int, 1>{});
    if (S <= 2 * states) return f(std::integral_constant<int, 2>{});
    if (S <= 4 * states) return f(std::integral_constant<int, 4>{});
    if (S <= 8 * states) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}
// Where a tile's channels lie in a row of shared memory.  A loading thread has V neighbouring ones,
// R threads a token's; its j-th value lies R behind its first, so that threads of a warp write side
// by side, and rows are kPad apart more than they hold, so that its four rows do not meet in the
// same banks.  (With channels in their order a store took 16 cycles for 2, which bound the scan.)
template <int V, int R>
struct Order {
    static constexpr int kPad = R < 16 ? R : 0;
    static __device__ __forceinline__ int channel(int place) { return place % R * V + place / R; }
    static __device__ __forceinline__ int place(int lane, int j) { return j * R + lane; }
};

template <typename F>
cudaError_t scan_type(int dtype, F f) {
    if (dtype == GDR_BF16) return f(__nv_bfloat16{});
    if (dtype == GDR_F16) return f(__half{});
    return f(float{});
}

}  // namespace gdr
