// attn.cuh -- softmax attention of a call's new tokens over a paged cache:
// what every kernel of it shares.
//
//   s_ij = scale <q_i, k_j>,   o_i = sum_j e^{s_ij - lse_i} v_j,
//   lse_i = log sum_j e^{s_ij}
//
// over the positions j that token i (at position p_i = kv_len - L + i) sees:
// j < kv_len, j <= p_i when causal, j > p_i - window when there is a window.
// A row that sees nothing has o = 0 and lse = -inf.
//
// Query heads share a key head in groups of G; the kernels that work on tiles
// take the G heads of a token as G rows of one tile, so that a key is read
// once for all of them: row r of (sequence, key head) is token r / G, query
// head head * G + r % G.
#pragma once

#include "paged.cuh"

namespace gdr {

// Division by a number d that a call does not change, of x < 2^31: with l =
// ceil(log2 d) and m = ceil(2^(31 + l) / d), floor(x m / 2^(31 + l)) is
// floor(x / d), as m d - 2^(31 + l) < d <= 2^l.
struct Divisor {
    uint32_t m;
    int s;
    __device__ __forceinline__ int operator()(int x) const {
        return (int)(((uint64_t)(uint32_t)x * m) >> s);
    }
};
inline Divisor divisor(uint32_t d) {
    int l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    return Divisor{(uint32_t)(((uint64_t(1) << (31 + l)) + d - 1) / d), 31 + l};
}

struct AttnProblem {
    PagedCache c;
    TokenRows r;
    const void *q;        // [tokens, Hq, K] (strides sq)
    void *o;              // [tokens, Hq, V] (strides so)
    float *lse;           // [tokens, Hq] or nullptr
    TokStride sq, so;
    int Hq, G, K, V, dtype, causal;
    int window;           // 0: none
    float scale;
    int grid_limit;
    Divisor by_G, by_page;
    int align;            // tiles' first positions are multiples of it (a power of two)
};

// Positions [lo, hi) that the token at position pos (below 0: before the
// cache) of a sequence of kv cached tokens sees.  Positions fit 31 bits.
__device__ __forceinline__ void visible(const AttnProblem &p, int kv, int pos, int &lo, int &hi) {
    hi = p.causal && pos + 1 < kv ? pos + 1 : kv;
    lo = p.window && pos >= p.window ? pos - p.window + 1 : 0;
    if (hi < lo) hi = lo;
}

}  // namespace gdr
