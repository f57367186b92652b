// attn_split.cuh -- how the tensor-core attention kernels share out a call.
//
// The work is cut into units, one for each (sequence, tile of M rows, key
// head), and a unit into steps of BN positions of the keys that its rows see
// (one step at least, so that rows that see nothing are written too).  All
// steps of the call form one line, sequence by sequence, and worker w of nw
// takes the steps [W w / nw, W (w + 1) / nw): equal shares whatever the
// lengths, known to every worker from the lengths alone, with no plan made on
// the host (the lengths are device data) and none passed between kernels.
//
// A unit also costs what comes before its first step and after its last; it
// stands for U0 steps more on the line, ahead of its own.  A share that holds
// only such steps of a unit does nothing of it.
//
// A worker's share meets at most two units that it does not do whole: its
// first (begun before it, slot 0) and its last (begun by it, slot 1).  Their
// unnormalised sums go to the worker's two scratch slots, and the worker that
// begins a split unit records how many pieces it has; a second kernel joins
// them in the order of the axis, so results do not depend on timing.
#pragma once

#include "attn.cuh"

namespace gdr {

// Scratch of a call: for `workers` workers, two slots each of M rows.
struct SplitScratch {
    float *o;      // [workers][2][M][V] sums of e^{s - m} v
    float *ml;     // [workers][2][M][2] m (base 2) and sum of e^{s - m}
    // [workers][2] the unit that the worker begins and others go on with:
    // {pieces (0: there is none), first token, new tokens, tile}, {key head}
    int4 *rec;
};

constexpr int kSplitSlots = 256;  // groups of sequences whose steps are summed up

struct Unit {
    int n, tile, head;
    int step, steps;       // next step, steps of the unit
    int lo, hi;            // positions that some row of it sees
    int in_lo, in_hi;      // positions that every row sees
    int t0, len, kv;       // the sequence: first token, new tokens, cached tokens
};

__device__ __forceinline__ void load_seq(const AttnProblem &p, int64_t n, int &t0, int &len,
                                         int &kv) {
    int64_t a, b;
    seq_span(p.r, n, a, b);
    t0 = (int)a;
    len = (int)b;
    kv = (int)cached_len(p.c, n, p.r.status);
}

template <int M>
__device__ __forceinline__ int tiles_of(const AttnProblem &p, int len) {
    return (len * p.G + (M - 1)) / M;  // the host sees to it that this fits
}

// Positions [u.lo, u.hi) that the rows of tile u.tile see, lo down to a
// multiple of p.align (a box of a page begins there), and the tile's steps.
template <int M, int BN>
__device__ __forceinline__ int tile_steps(const AttnProblem &p, Unit &u) {
    const int r0 = u.tile * M, i0 = p.by_G(r0);
    const int i1 = min(p.by_G(r0 + M - 1), u.len - 1);
    int a, d;
    visible(p, u.kv, u.kv - u.len + i0, a, u.in_hi);
    visible(p, u.kv, u.kv - u.len + i1, u.in_lo, d);
    u.hi = d > a ? d : a;
    u.lo = a & -p.align;
    const int s = (u.hi - u.lo + BN - 1) / BN;
    return s > 0 ? s : 1;
}
// Whether some row of the unit sees a part only of the BN positions at `base`.
template <int BN>
__device__ __forceinline__ bool step_masked(const Unit &u, int base) {
    return base < u.in_lo || base + BN > u.in_hi;
}
template <int M>
__device__ __forceinline__ int unit_rows(const AttnProblem &p, const Unit &u) {
    return min(M, u.len * p.G - u.tile * M);
}

// Length on the line of a sequence's tiles first, first + stride, ...
template <int M, int BN, int U0>
__device__ __forceinline__ int64_t seq_line(const AttnProblem &p, Unit &u, int first, int stride) {
    int64_t s = 0;
    const int tiles = tiles_of<M>(p, u.len);
    for (u.tile = first; u.tile < tiles; u.tile += stride) s += tile_steps<M, BN>(p, u) + U0;
    return s * p.c.H;
}

// Exclusive prefix sums, by the whole block, over kSplitSlots groups of `per`
// sequences (per = ceil(N / kSplitSlots)): lengths on the line in pre[0 ..
// kSplitSlots], and units in units[] where U0 > 0.  Each thread sums up a
// group's short sequences; those of many tiles are left to the block, which
// shares their tiles out.
template <int M, int BN, int U0, int NT>
__device__ void split_prefix(const AttnProblem &p, int64_t per, int64_t *pre, int64_t *units) {
    static_assert(NT % 32 == 0 && kSplitSlots % 32 == 0, "whole warps");
    constexpr int kFew = 4;
    __shared__ int64_t s_warp[2][kSplitSlots / 32];
    __shared__ int s_long[kSplitSlots], s_longs;  // groups with long sequences
    const int tid = threadIdx.x;
    if (tid == 0) s_longs = 0;
    __syncthreads();
    for (int e = tid; e < kSplitSlots; e += NT) {
        int64_t sum = 0, un = 0;
        bool any = false;
        for (int64_t n = e * per; n < (e + 1) * per && n < p.r.N; ++n) {
            Unit u;
            load_seq(p, n, u.t0, u.len, u.kv);
            const int tiles = tiles_of<M>(p, u.len);
            un += tiles;
            if (tiles <= kFew) sum += seq_line<M, BN, U0>(p, u, 0, 1);
            else any = true;
        }
        pre[e + 1] = sum;
        if (U0) units[e + 1] = un * p.c.H;
        if (any) s_long[atomicAdd(&s_longs, 1)] = e;
    }
    if (tid == 0) {
        pre[0] = 0;
        if (U0) units[0] = 0;
    }
    __syncthreads();
    const int longs = s_longs;
    for (int i = 0; i < longs; ++i) {
        const int e = s_long[i];
        int64_t sum = 0;
        for (int64_t n = e * per; n < (e + 1) * per && n < p.r.N; ++n) {
            Unit u;
            load_seq(p, n, u.t0, u.len, u.kv);
            if (tiles_of<M>(p, u.len) > kFew) sum += seq_line<M, BN, U0>(p, u, tid, NT);
        }
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if ((tid & 31) == 0 && sum)
            atomicAdd(reinterpret_cast<unsigned long long *>(&pre[e + 1]), (unsigned long long)sum);
    }
    if (longs) __syncthreads();
    for (int e = tid; e < kSplitSlots; e += NT) {  // whole warps: NT and the slots are multiples
        int64_t x = pre[e + 1], y = U0 ? units[e + 1] : 0;
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, x, d);
            const int64_t b = U0 ? __shfl_up_sync(0xffffffffu, y, d) : 0;
            if ((e & 31) >= d) {
                x += a;
                y += b;
            }
        }
        pre[e + 1] = x;
        if (U0) units[e + 1] = y;
        if ((e & 31) == 31) {
            s_warp[0][e >> 5] = x;
            s_warp[1][e >> 5] = y;
        }
    }
    __syncthreads();
    for (int e = tid; e < kSplitSlots; e += NT) {
        int64_t x = 0, y = 0;
        for (int w = 0; w < (e >> 5); ++w) {
            x += s_warp[0][w];
            y += s_warp[1][w];
        }
        pre[e + 1] += x;
        if (U0) units[e + 1] += y;
    }
    __syncthreads();
}

// The unit and the step of it that a worker begins with whose share begins at
// `at` on the line (0 <= at < pre[kSplitSlots]), and the steps of all units
// before that one in `real`; by a whole warp.
template <int M, int BN, int U0>
__device__ Unit split_locate(const AttnProblem &p, int64_t per, const int64_t *pre,
                             const int64_t *units, int64_t at, int64_t &real) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = kSplitSlots;  // the last e with pre[e] <= at
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, i = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, i < hi && pre[i] <= at);
        lo += (31 - __clz(m)) * step;
        if (lo + step < hi) hi = lo + step;
    }
    int64_t rem = at - pre[lo];
    real = pre[lo] - (U0 ? U0 * units[lo] : 0);
    Unit u{};
    for (int64_t n = lo * per;; ++n) {
        load_seq(p, n, u.t0, u.len, u.kv);
        const int tiles = tiles_of<M>(p, u.len);
        for (int t = 0; t < tiles; t += 32) {
            u.tile = t + lane;
            const int s = t + lane < tiles ? tile_steps<M, BN>(p, u) : -U0;
            int64_t x = (int64_t)(s + U0) * p.c.H;
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            const unsigned m = __ballot_sync(0xffffffffu, x > rem);
            if (m) {
                const int l = __ffs(m) - 1;
                u.n = (int)n;
                u.tile = t + l;
                u.steps = tile_steps<M, BN>(p, u);
                const int64_t before = __shfl_sync(0xffffffffu, x, l) - (int64_t)(u.steps + U0) * p.c.H;
                rem -= before;
                u.head = (int)(rem / (u.steps + U0));
                const int v = (int)(rem - (int64_t)u.head * (u.steps + U0)) - U0;
                u.step = v > 0 ? v : 0;
                real += before - (int64_t)U0 * p.c.H * l + (int64_t)u.head * u.steps;
                return u;
            }
            const int64_t all = __shfl_sync(0xffffffffu, x, 31);
            rem -= all;
            real += all - (int64_t)U0 * p.c.H * min(32, tiles - t);
        }
        if (n + 1 >= p.r.N) return u;  // not reached for a point of the line
    }
}

// On to the next unit of the line (there is one).
template <int M, int BN>
__device__ __forceinline__ void next_unit(const AttnProblem &p, Unit &u) {
    u.step = 0;
    if (++u.head < p.c.H) return;
    u.head = 0;
    ++u.tile;
    while (u.tile >= tiles_of<M>(p, u.len)) {
        u.tile = 0;
        if (++u.n >= p.r.N) return;
        load_seq(p, u.n, u.t0, u.len, u.kv);
    }
    u.steps = tile_steps<M, BN>(p, u);
}

// Where the share of worker w of nw begins.
__device__ __forceinline__ int64_t share_begin(int64_t total, int64_t w, int64_t nw) {
    return total / nw * w + total % nw * w / nw;
}
// Pieces of the unit that ends at `end` on the line, begun by worker w: the workers from w on whose shares begin before it.  Worker j's
// does iff floor(total j / nw) < end, that is iff total j < end nw.
__device__ __forceinline__ int pieces_from(int64_t total, int64_t w, int64_t nw, int64_t end) {
    const int64_t j = (end * nw + total - 1) / total;
    return (int)((j < nw ? j : nw) - w);
}

}  // namespace gdr
