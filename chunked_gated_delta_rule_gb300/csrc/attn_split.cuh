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
    // [workers] the unit that the worker begins and others go on with: key head
    // << 16 | pieces (0: there is none), first token, new tokens, tile
    int4 *rec;
};

struct Unit {
    int n, tile, head;
    int step, steps;       // next step, steps of the unit
    int lo, hi;            // positions that some row of it sees
    int in_lo, in_hi;      // positions that every row sees
    int t0, len, kv;       // the sequence: first token, new tokens, cached tokens
};

// The sequence's part of a unit.  Returns 0 or the code to report; nothing
// outside the call's tokens and the page table's row is addressed after it.  A
// packed table that does not begin at 0 or end at T is malformed, though each of
// its sequences may be well.
__device__ __forceinline__ int load_seq(const AttnProblem &p, int64_t n, Unit &u) {
    const int64_t t0 = row_bound(p.r, n), end = row_bound(p.r, n + 1);
    const int kv = p.c.kv_lens[n];
    const int cap = (int)(p.c.max_pages * p.c.page_size);
    int code = 0;
    u.t0 = (int)t0;
    u.len = (int)(end - t0);
    u.kv = kv;
    if (kv < 0 || kv > cap) {
        code = GDR_ERR_INDEX;
        u.kv = kv < 0 ? 0 : cap;
    }
    if (rows_packed(p.r)) {
        if (t0 < 0 || end < t0 || end > p.r.T) {
            code = GDR_ERR_SEQLENS;
            u.t0 = u.len = 0;
        } else if ((n == 0 && t0 != 0) || (n == p.r.N - 1 && end != p.r.T)) {
            code = GDR_ERR_SEQLENS;
        }
    }
    return code;
}

// The tokens that no sequence of a malformed table holds have o = 0 and lse = -inf.
// Warp w of nw takes every nw-th token; 16-bit o, rows on 16-byte boundaries.
__device__ __forceinline__ void clear_unheld(const AttnProblem &p, int64_t w, int64_t nw) {
    const int lane = threadIdx.x & 31, chunks = p.V / 8;
#pragma unroll 1
    for (int64_t t = w; t < p.r.T; t += nw) {
        bool held = false;
#pragma unroll 1
        for (int64_t n = lane; n < p.r.N; n += 32) {
            const int64_t t0 = row_bound(p.r, n), end = row_bound(p.r, n + 1);
            held |= t0 >= 0 && end <= p.r.T && t0 <= t && t < end;
        }
        if (__any_sync(0xffffffffu, held)) continue;
#pragma unroll 1
        for (int i = lane; i < p.Hq * chunks; i += 32) {
            const int h = i / chunks;
            uint16_t *o = reinterpret_cast<uint16_t *>(p.o) + tok_at(p.so, t, h);
            reinterpret_cast<uint4 *>(o)[i - h * chunks] = make_uint4(0, 0, 0, 0);
        }
        if (p.lse)
            for (int h = lane; h < p.Hq; h += 32) p.lse[t * p.Hq + h] = -INFINITY;
    }
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

// x / y, for 0 <= x and 0 < y: in 32 bits where both fit, as they do but for
// calls of many millions of steps.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    if (((uint64_t)(x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
    return x / y;
}
// Where the share of worker w of nw begins.
__device__ __forceinline__ int64_t share_begin(int64_t total, int64_t w, int64_t nw) {
    const int64_t q = quotient(total, nw);
    return q * w + quotient((total - q * nw) * w, nw);
}
// Length on the line of a sequence's tiles first, first + stride, ...
template <int M, int BN, int U0>
__device__ __forceinline__ int64_t seq_line(const AttnProblem &p, Unit &u, int first, int stride) {
    int64_t s = 0;
    const int tiles = tiles_of<M>(p, u.len);
    for (u.tile = first; u.tile < tiles; u.tile += stride) s += tile_steps<M, BN>(p, u) + U0;
    return s * p.c.H;
}

// Where a worker begins: the length of the whole line, and, once the caller
// has told where on the line its share begins, the unit and the step of it.
// A warp's work: lane l holds the sequences [l per, (l + 1) per), per =
// ceil(N / 32), sums them up, and the sums of the lanes are scanned.
template <int M, int BN, int U0>
struct SplitLine {
    int64_t total, units;      // length, units of the call
    int64_t line0, units0;     // those of the lanes before this one
    int64_t per;
    static constexpr int kFew = 16;  // more tiles of a sequence are shared out among the lanes

    // Whether the table of offsets is well formed.
    __device__ __forceinline__ bool measure(const AttnProblem &p) {
        const int lane = threadIdx.x & 31;
        per = (p.r.N + 31) >> 5;
        int64_t x = 0, y = 0;
        int code = 0;
        bool malformed = false;
#pragma unroll 4
        for (int64_t k = 0; k < per; ++k) {
            const int64_t n = lane * per + k;
            Unit u{};
            if (n < p.r.N) {
                const int c = load_seq(p, n, u);
                code = c ? c : code;
                malformed |= c == GDR_ERR_SEQLENS;
            }
            const int tiles = tiles_of<M>(p, u.len);
            y += tiles;
            if (tiles <= kFew) x += seq_line<M, BN, U0>(p, u, 0, 1);
            for (unsigned m = __ballot_sync(0xffffffffu, tiles > kFew); m; m &= m - 1) {
                const int l = __ffs(m) - 1;
                Unit v{};
                v.len = __shfl_sync(0xffffffffu, u.len, l);
                v.kv = __shfl_sync(0xffffffffu, u.kv, l);
                int64_t sum = seq_line<M, BN, U0>(p, v, lane, 32);
#pragma unroll
                for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (lane == l) x += sum;
            }
        }
        if (code) report(p.r.status, code);
        y *= p.c.H;
        line0 = x;
        units0 = y;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, x, d);
            const int64_t b = U0 ? __shfl_up_sync(0xffffffffu, y, d) : 0;
            if (lane >= d) {
                x += a;
                y += b;
            }
        }
        total = __shfl_sync(0xffffffffu, x, 31);
        units = U0 ? __shfl_sync(0xffffffffu, y, 31) : 0;
        line0 = x - line0;
        units0 = y - units0;
        return !__any_sync(0xffffffffu, malformed);
    }

    // The unit and step at `at` (0 <= at < total), and the steps of the call
    // before that unit in `real`.
    __device__ __forceinline__ Unit locate(const AttnProblem &p, int64_t at, int64_t &real) const {
        const int lane = threadIdx.x & 31;
        // the last lane that begins at or before it
        const int g = 31 - __clz(__ballot_sync(0xffffffffu, line0 <= at));
        int64_t rem = at - __shfl_sync(0xffffffffu, line0, g);
        real = __shfl_sync(0xffffffffu, line0, g) - (U0 ? U0 * __shfl_sync(0xffffffffu, units0, g) : 0);
        Unit u{};
        // of the lane's sequences, 32 at a time: a lane a sequence, down to the
        // one that holds it (if they are all short, as many sequences are)
        int64_t n = g * per;
        for (; per > 1 && n < (g + 1) * per; n += 32) {
            Unit v{};
            if (n + lane < (g + 1) * per && n + lane < p.r.N) load_seq(p, n + lane, v);
            const int tiles = tiles_of<M>(p, v.len);
            if (__any_sync(0xffffffffu, tiles > kFew)) break;
            const int64_t own = seq_line<M, BN, U0>(p, v, 0, 1);
            int64_t x = own;
            int un = tiles;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
                const int z = __shfl_up_sync(0xffffffffu, un, d);
                if (lane >= d) {
                    x += y;
                    un += z;
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, x > rem);
            const int l = m ? __ffs(m) - 1 : 31;  // none: all 32 lie before it
            const int64_t before = __shfl_sync(0xffffffffu, m ? x - own : x, l);
            rem -= before;
            real += before - (int64_t)U0 * p.c.H * __shfl_sync(0xffffffffu, m ? un - tiles : un, l);
            if (m) {
                n += l;
                break;
            }
        }
        for (;; ++n) {
            load_seq(p, n, u);
            const int tiles = tiles_of<M>(p, u.len);
            for (int t = 0; t < tiles; t += 32) {
                u.tile = t + lane;
                const int s = t + lane < tiles ? tile_steps<M, BN>(p, u) : -U0;
                int64_t x = (int64_t)(s + U0) * p.c.H;
#pragma unroll
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
                    const int64_t before =
                        __shfl_sync(0xffffffffu, x, l) - (int64_t)(u.steps + U0) * p.c.H;
                    rem -= before;
                    u.head = (int)quotient(rem, u.steps + U0);
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
};

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
        load_seq(p, u.n, u);
    }
    u.steps = tile_steps<M, BN>(p, u);
}

// Pieces of the unit that ends at `end` on the line, begun by worker w: the workers from w on whose shares begin before it.  Worker j's
// does iff floor(total j / nw) < end, that is iff total j < end nw.
__device__ __forceinline__ int pieces_from(int64_t total, int64_t w, int64_t nw, int64_t end) {
    const int64_t j = quotient(end * nw + total - 1, total);
    return (int)((j < nw ? j : nw) - w);
}

}  // namespace gdr
