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
