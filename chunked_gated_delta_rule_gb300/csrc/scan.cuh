// scan.cuh -- what the selective scan's kernels share: how channels and states
// lie over a block, how sequences are cut into pieces, and the staging of a
// tile of tokens.
//
// A thread holds four states of one channel; LPC neighbouring lanes (a power of
// two, S <= 4 LPC) hold a channel's states, a block kNT / LPC channels.  States
// past S have A = B = C = 0, so they stay zero.
//
// Pieces: sequence n is cut into ceil(len / L) pieces of L tokens.  Piece j of
// it is slot floor(cu[n] / L) + n + j: since floor((a + len) / L) + 1 - floor(a /
// L) >= ceil(len / L), no two pieces share a slot, an empty sequence has one of
// its own, floor(T / L) + N slots hold all, and a block finds its piece from
// the slot without a table.
#pragma once

#include "layer.cuh"

namespace gdr {

constexpr int kNT = 256;     // threads of a block
constexpr int kPS = 4;       // states of a thread
constexpr float kLog2e = 1.4426950408889634f;

template <int LPC>
struct Lay {
    static constexpr int kC = kNT / LPC;       // channels of a block
    static constexpr int kS = kPS * LPC;       // states, padded
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log(1 + e^x)
__device__ __forceinline__ float softplus_f(float x) {
    return fmaxf(x, 0.f) + log1pf(__expf(-fabsf(x)));
}
__device__ __forceinline__ float time_step(const ScanArgs &a, float raw) {
    return a.softplus ? softplus_f(raw) : raw;
}

// The channels of tile `tile`: a tile lies within one group of B and C.
struct Tile {
    int64_t c0;
    int valid, g;
};
template <int LPC>
__device__ __forceinline__ Tile tile_of(const ScanArgs &a, int tile) {
    const int per = (int)(a.C / a.G), tiles = (per + Lay<LPC>::kC - 1) / Lay<LPC>::kC;
    Tile t;
    t.g = tile / tiles;
    const int at = tile % tiles * Lay<LPC>::kC;
    t.c0 = (int64_t)t.g * per + at;
    t.valid = min(Lay<LPC>::kC, per - at);
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

// Four states of B or C of token row t0 + tr, zeros past the ends.
template <typename T>
__device__ __forceinline__ void load_bc(Row<T, 4> &r, const void *base, const int64_t (&st)[2], int g,
                                        int64_t t0, int tr, int len, int s0, int S, int bytes) {
    const int valid = tr < len ? max(0, min(4, S - s0)) : 0;
    r.load((const T *)base + (t0 + tr) * st[0] + g * st[1] + s0, bytes, valid);
}

template <typename F>
cudaError_t scan_lanes(int S, F f) {
    if (S <= 4) return f(std::integral_constant<int, 1>{});
    if (S <= 8) return f(std::integral_constant<int, 2>{});
    if (S <= 16) return f(std::integral_constant<int, 4>{});
    if (S <= 32) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}
template <typename F>
cudaError_t scan_type(int dtype, F f) {
    if (dtype == GDR_BF16) return f(__nv_bfloat16{});
    if (dtype == GDR_F16) return f(__half{});
    return f(float{});
}

}  // namespace gdr
