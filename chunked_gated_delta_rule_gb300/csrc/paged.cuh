// paged.cuh -- the paged cache of keys and values as the kernels see it, and
// the addressing that its writer, its reader and the attention share.
//
// Position p of sequence n is slot p % page_size of page page_table[n, p /
// page_size].  kv_lens[n] counts the tokens of sequence n including the L_n
// tokens of the call, so token i of the call sits at position
// kv_lens[n] - L_n + i.  All offsets into the pages are 64-bit: a cache of
// 2^31 elements is 4 GB, a small part of the device.
#pragma once

#include "gdr_internal.cuh"

namespace gdr {

struct PagedCache {
    void *k, *v;              // pages, elements of dtype (below)
    float *ks, *vs;           // [n_pages, H, page_size] scales (8-bit formats) or nullptr
    const int32_t *table;     // [N, max_pages]
    const int32_t *kv_lens;   // [N]
    int64_t kst[3], vst[3];   // element strides: page, slot, head
    int64_t max_pages;
    int32_t n_pages, page_size, H, dtype;
};

// The tokens of a call: N sequences packed along T (cu or cu64), or N rows of
// T tokens (both null).
struct TokenRows {
    const int32_t *cu;
    const int64_t *cu64;
    int64_t N, T;      // T: the total when packed, tokens of a row when dense
    int32_t *status;
};

__host__ __device__ __forceinline__ bool rows_packed(const TokenRows &r) {
    return r.cu != nullptr || r.cu64 != nullptr;
}
__device__ __forceinline__ int64_t row_bound(const TokenRows &r, int64_t n) {
    return r.cu64 ? r.cu64[n] : r.cu ? (int64_t)r.cu[n] : n * r.T;
}

__device__ __forceinline__ void report(int32_t *status, int code) {
    if (status) atomicCAS(status, 0, code);
}

// First token and token count of sequence n, {0, 0} where a packed table is
// malformed there (reported): nothing outside [0, T) is ever addressed.
__device__ __forceinline__ void seq_span(const TokenRows &r, int64_t n, int64_t &t0,
                                         int64_t &len) {
    t0 = row_bound(r, n);
    len = row_bound(r, n + 1) - t0;
    if (rows_packed(r) && (t0 < 0 || len < 0 || t0 > r.T || len > r.T - t0)) {
        report(r.status, GDR_ERR_SEQLENS);
        t0 = len = 0;
    }
}

// Reports a packed table that does not run from 0 to T without a step back.  A
// warp's work; the kernels whose warps each look at a few sequences have one do it.
__device__ __forceinline__ void check_offsets(const TokenRows &r) {
    if (!rows_packed(r)) return;
    bool bad = row_bound(r, 0) != 0 || row_bound(r, r.N) != r.T;
#pragma unroll 4
    for (int64_t n = threadIdx.x & 31; n < r.N; n += 32) bad |= row_bound(r, n + 1) < row_bound(r, n);
    if (bad) report(r.status, GDR_ERR_SEQLENS);
}

// Cached tokens of sequence n, cut to what its row of the page table holds.
__device__ __forceinline__ int64_t cached_len(const PagedCache &c, int64_t n, int32_t *status) {
    const int64_t cap = c.max_pages * c.page_size;
    const int64_t len = c.kv_lens[n];
    if (len < 0 || len > cap) {
        report(status, GDR_ERR_INDEX);
        return len < 0 ? 0 : cap;
    }
    return len;
}

// The sequence that holds token t, found by a whole warp: every round the
// lanes test 32 evenly spaced bounds, so 1024 sequences take two loads.  The
// result is the last n with cu[n] <= t, in [0, N).
__device__ __forceinline__ int64_t find_seq(const TokenRows &r, int64_t t) {
    if (!rows_packed(r)) return t / r.T;
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = r.N;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) >> 5, at = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < hi && row_bound(r, at) <= t);
        const int last = m ? 31 - __clz(m) : 0;
        lo += last * step;
        if (lo + step < hi) hi = lo + step;
    }
    return lo;
}

// Page of position `pos` (0 <= pos < max_pages * page_size) of sequence n, or
// -1 (reported) where the table's entry is outside the cache.
__device__ __forceinline__ int page_of(const PagedCache &c, int64_t n, int page_index,
                                       int32_t *status) {
    const int page = c.table[n * c.max_pages + page_index];
    if ((unsigned)page >= (unsigned)c.n_pages) {
        report(status, GDR_ERR_INDEX);
        return -1;
    }
    return page;
}

__device__ __forceinline__ int64_t page_at(const int64_t (&st)[3], int64_t page, int64_t slot,
                                           int64_t head) {
    return page * st[0] + slot * st[1] + head * st[2];
}
__device__ __forceinline__ int64_t scale_at(const PagedCache &c, int64_t page, int64_t slot,
                                            int64_t head) {
    return (page * c.H + head) * c.page_size + slot;
}

// 16-byte loads of a cache's rows: an aligned base and strides.
inline bool pages_aligned16(const void *p, const int64_t (&st)[3], int es) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(st[0] * es) | (uintptr_t)(st[1] * es) |
             (uintptr_t)(st[2] * es)) & 15u) == 0;
}

inline bool cache_quantised(int dtype) { return dtype == GDR_E4M3 || dtype == GDR_I8; }

}  // namespace gdr
