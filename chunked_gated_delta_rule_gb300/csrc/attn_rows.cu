// attn_rows.cu -- attention over a paged cache for few new tokens (decode
// steps, drafts): up to 16 rows of query heads and tokens a tile.
//
// Bound by memory: every cached key and value of the sequence is read once
// for G query heads (G L rows), 4 G flops a byte at 16 bits, far below the
// tensor rate.  So the products are the warp-level ones and the design goes to
// keeping loads in flight and to few instructions a byte:
//   * every warp is a worker of its own with an equal share of the call's
//     steps (attn_split.cuh), its own ring of tiles (keys or values of 32
//     positions) in shared memory and its own running maximum, sum and
//     accumulators in registers; warps never wait for each other;
//   * a tile comes by TMA as boxes of gcd(page size, 32) slots, each of one
//     page, a lane a box (16-byte asynchronous copies where pages are no
//     multiple of 8 slots); the pages of a step are looked up while the one
//     before it is at work, so a load never waits for the page table;
//   * the ring runs across the ends of units (sequences, heads);
//   * keys and values are the 16-row operand, S^T = K Q^T and O^T = V^T P^T, and
//     the rows of queries the 8-column one: the other way round, the products
//     of 4 or 8 rows are half empty (and twice as many).
// 8-bit caches stay 8-bit in shared memory.  The values q of a row times its
// FP32 scale s would not fit 16 bits, so scales are applied in FP32: keys'
// scales to the scores, values' scales to the weights, as
//   w_j s_j = 2^(t_j + log2 s_j - m),   sum_j w_j = sum_j (w_j s_j) / s_j,
// m the running maximum of t_j + log2 s_j, which keeps every weight at most 16
// and so within FP16; the values themselves are exact in FP16.
// Weights are split into hi + lo halves (two products) where they have the
// output's own type: the rounding of a single half would add as much error to
// o as o's own (FP16, one 64K context: 2.9e-4 against 2.0e-4), and the
// products cost nothing beside the loads.
#include "attn_map.cuh"
#include "attn_split.cuh"
#include "gdr_launch.cuh"
#include "tc_common.cuh"

namespace gdr {
namespace {

constexpr int kRowsMost = 16;  // rows of a tile: 8 or 16
constexpr int kRowsUnit = 2;   // what a unit costs beside its steps, in steps
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Sizes of one configuration.  FMT: 0 the call's own 16-bit type, 1 E4M3,
// 2 8-bit integers.
template <int FMT, int D>
struct RowsCfg {
    static constexpr int kES = FMT ? 1 : 2;
    static constexpr int kBN = 32;                   // positions a step
    static constexpr int kRow = D * kES;             // bytes of a row
    static constexpr int kLine = kRow < 128 ? kRow : 128;  // bytes of a row of a box
    static constexpr int kBlocks = kRow / kLine;     // boxes beside each other
    static constexpr int kRows = kBN * kRow;         // bytes of a tile
    static constexpr int kScale = FMT ? kBN * 4 : 0; // of a step's scales of keys, of values
    // 16 bits: three tiles (192 KB an SM), each loaded again as soon as it is
    // read.  8 bits: three or more pairs, keys and values of a step (the swizzle's
    // period apart) and both scales, loaded again together: there instructions
    // are what bounds the kernel, half of them waiting to be fetched, and the
    // loads then stand in the loop once.
    static constexpr bool kPairs = FMT != 0;
    static constexpr int kPair = (2 * kRows + 2 * kScale + 1023) / 1024 * 1024;
    static constexpr int kTiles = !kPairs ? (D == 64 ? 5 : 3) : D == 64 ? 8 : 6;
    static constexpr int kRing = kPairs ? kTiles / 2 * kPair : kTiles * kRows;
    static constexpr int kWarps = 8;
    static constexpr int kSmem = kWarps * kRing + 1024;
    static constexpr int kInfos = 4;                 // steps in the ring, at most
    static_assert(kPairs ? kTiles / 2 <= kInfos : kTiles / 2 + 2 <= kInfos, "steps in the ring");
    __host__ __device__ static constexpr int tile_at(int i) {
        return kPairs ? (i >> 1) * kPair + (i & 1) * kRows : i * kRows;
    }
    __host__ __device__ static constexpr int scale_at(int i) { return (i >> 1) * kPair + 2 * kRows; }
};

// What a step in the ring is.
struct StepInfo {
    int base, flags;               // first position; bits below
    int tile, head, t0, len, kv, hi;
    int steps_left;                // of the unit, after this step
};
constexpr int kFirst = 1, kLast = 2, kMask = 4;  // of the unit; some row sees a part

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    const int bytes = live ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, bool live) {
    const int bytes = live ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

// The transpose of an 8 x 8 matrix of 16-bit values.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
    if constexpr (std::is_same<T, __half>::value)
        return __half22float2(*reinterpret_cast<const __half2 *>(&x));
    else
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x));
}

// Shared-memory byte offset of 16-byte chunk `c` of token `t` in a tile: what
// TMA writes with the 128-byte swizzle (64-byte for rows of 64 bytes).  ldmatrix,
// which takes one chunk of eight tokens, meets no bank twice, nor do the reads
// of 8-bit rows below.
template <int FMT, int D>
__device__ __forceinline__ uint32_t kv_off(int t, int c) {
    using C = RowsCfg<FMT, D>;
    if constexpr (C::kLine == 128)
        return (c >> 3) * (C::kBN * 128) + t * 128 + (((c & 7) ^ (t & 7)) << 4);
    else
        return t * 64 + ((c ^ (t >> 1 & 3)) << 4);
}

// Token of row r of an 8-token part of a product.  8 bits: the keys' reads take
// chunks 0-3 or 4-7 of the tokens of rows r, r + 1 (r even), the values' reads
// one chunk or two of the tokens of rows r, r + 2, r + 4, r + 6; the order below
// puts either on different banks.
template <int FMT>
__device__ __forceinline__ int token_of(int r) {
    if constexpr (FMT == 0) return r;
    else return r & 1 ? ((r - 1) ^ 4) | 1 : r;
}

struct RowsArgs {
    AttnProblem p;
    SplitScratch ws;
    int min_steps;       // least steps a worker
    int box;             // slots of a TMA box (0: asynchronous copies)
    CUtensorMap tk, tv;  // [page][head][slot][column] of the caches
};

template <typename T, int FMT, int D, int NR>
__global__ void __launch_bounds__(32 * RowsCfg<FMT, D>::kWarps, 1)
    k_attn_rows(const __grid_constant__ RowsArgs a) {
    using C = RowsCfg<FMT, D>;
    using TP = typename std::conditional<FMT == 0, T, __half>::type;  // of the products
    constexpr int kM = 8 * NR;             // rows of a tile
    constexpr int kMT = C::kBN / 16;       // 16-token parts of a step
    constexpr int kKS = D / 16;            // products of a score
    constexpr int kDT = D / 16;            // 16-column parts of the output
    constexpr int kB = D / 8;              // 8 bits: value bytes a thread takes of a token
    // weights in two halves, where one rounding of them would be as large as
    // the output's own
    constexpr bool kSplitP = std::is_same<T, TP>::value;
    // whose o holds values of the least scales
    constexpr bool kBf = FMT != 0 && std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ uint8_t smem_raw[];
    __shared__ StepInfo s_info[C::kWarps][C::kInfos];
    __shared__ uint64_t s_bar[C::kWarps][C::kTiles];
    const AttnProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int qr = lane >> 2, qc = lane & 3;
    pdl_trigger();
    SplitLine<kM, C::kBN, kRowsUnit> line;
    const bool formed = line.measure(p);
    const int64_t total = line.total;
    const int64_t worker = (int64_t)blockIdx.x * C::kWarps + warp;
    int64_t nw = (int64_t)gridDim.x * C::kWarps;
    if (!formed) clear_unheld(p, worker, nw);
    if (nw * a.min_steps > total) nw = quotient(total + a.min_steps - 1, a.min_steps);
    if (lane == 0) a.ws.rec[worker] = make_int4(0, 0, 0, 0);
    if (worker >= nw) return;
    // where the share ends, then where it begins
    const int64_t end = share_begin(total, worker + 1, nw);
    Unit u{};
    int count = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int64_t at = i ? share_begin(total, worker, nw) : end;
        int64_t before = total - kRowsUnit * line.units;  // of the whole line
        if (at < total) {
            u = line.locate(p, at, before);
            before += u.step;
        }
        count = (int)(before - count);  // the second time the difference, negated
    }
    count = -count;
    if (count == 0) return;

    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023)) + warp * C::kRing;
    const uint32_t ring_u = tc::smem_u32(ring);
    StepInfo *info = s_info[warp];
    uint64_t *bars = s_bar[warp];
    if (lane == 0) {
        for (int i = 0; i < C::kTiles; ++i) tc::mbar_init(&bars[i], a.box ? 1 : 32);
        tc::mbar_init_fence();
    }
    __syncwarp();

    // what this lane asks of the step that is loaded next: the page-table entry
    // and slot of its box (boxes first, then columns) or of its token
    const int per = a.box ? a.box : 1, boxes = a.box ? C::kBN / a.box : 32;
    const int bx = lane & (boxes - 1), part = a.box ? lane / boxes : 0;
    int entry = -1, slot = 0;
    bool asked = false;
    auto look_up = [&]() {
        const int pos = u.lo + u.step * C::kBN + bx * per;
        asked = pos < u.hi;
        if (asked) {
            const int pi = p.by_page(pos);
            slot = pos - pi * p.c.page_size;
            entry = p.c.table[u.n * p.c.max_pages + pi];
        }
    };
    // tiles: keys of step 0, values of step 0, keys of step 1, ...
    int load_item = 0, load_tile = 0;
    auto load = [&]() {
        const int kv = load_item & 1;
        const uint32_t st = ring_u + C::tile_at(load_tile);
        uint64_t *bar = &bars[load_tile];
        const bool here = asked && (unsigned)entry < (unsigned)p.c.n_pages;
        if (a.box) {
            // a page past the cache reads as zeros
            const int page = here ? entry : p.c.n_pages, sl = here ? slot : 0;
            uint32_t bytes = C::kRows;
            if (FMT && !kv) bytes += __popc(__ballot_sync(0xffffffffu, here && part == 0)) * a.box * 8;
            if (lane == 0) tc::mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (part < C::kBlocks)
                tma_page(st + part * (C::kBN * 128) + bx * a.box * C::kLine, kv ? &a.tv : &a.tk, bar,
                         part * (C::kLine / C::kES), sl, u.head, page);
            if (FMT && !kv && here && part < 2)
                tc::bulk_load(ring + C::scale_at(load_tile) + part * C::kScale + bx * a.box * 4,
                              (part ? p.c.vs : p.c.ks) + gdr::scale_at(p.c, page, sl, u.head), a.box * 4, bar);
        } else {
            const uint8_t *base = reinterpret_cast<const uint8_t *>(kv ? p.c.v : p.c.k);
            const int64_t at = !here ? 0 : kv ? page_at(p.c.vst, entry, slot, u.head) * C::kES
                                              : page_at(p.c.kst, entry, slot, u.head) * C::kES;
            constexpr int kChunks = C::kRow / 16, kPer = 32 / kChunks;  // chunks a row, rows a load
#pragma unroll 2
            for (int i = 0; i < C::kBN / kPer; ++i) {
                const int t = i * kPer + lane / kChunks, c = lane % kChunks;
                const int64_t of = __shfl_sync(0xffffffffu, at, t);
                const bool live = __shfl_sync(0xffffffffu, here, t);
                cp16(st + kv_off<FMT, D>(t, c), base + of + (live ? c * 16 : 0), live);
            }
            if (FMT && !kv) {
                const int64_t so = here ? gdr::scale_at(p.c, entry, slot, u.head) : 0;
                const uint32_t sc = ring_u + C::scale_at(load_tile);
                cp4(sc + lane * 4, p.c.ks + so, here);
                cp4(sc + C::kScale + lane * 4, p.c.vs + so, here);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar))
                         : "memory");
        }
        if (!kv) {
            if (asked && !here) report(p.r.status, GDR_ERR_INDEX);
            if (lane == 0) {
                StepInfo &f = info[(load_item >> 1) % C::kInfos];
                f.base = u.lo + u.step * C::kBN;
                f.steps_left = u.steps - 1 - u.step;
                f.flags = (u.step == 0 ? kFirst : 0) | (f.steps_left == 0 ? kLast : 0) |
                          (step_masked<C::kBN>(u, f.base) ? kMask : 0);
                f.tile = u.tile;
                f.head = u.head;
                f.t0 = u.t0;
                f.len = u.len;
                f.kv = u.kv;
                f.hi = u.hi;
            }
        } else if ((load_item >> 1) + 1 < count) {
            if (++u.step == u.steps) next_unit<kM, C::kBN>(p, u);
            look_up();
        }
        ++load_item;
        if (++load_tile == C::kTiles) load_tile = 0;
    };

    look_up();
    if constexpr (!C::kPairs) {
#pragma unroll 1
        for (int i = 0; i < C::kTiles && i < 2 * count; ++i) load();
    }

    uint32_t qf[kKS][NR][2];
    float acc[kDT][NR][4];
    // of the thread's queries 2 qc, 2 qc + 1 (of every 8): maximum, sum, base-2
    // score of a unit of product, positions seen
    float m[NR][2], l[NR][2], f2[NR][2];
    int lo[NR][2], hi[NR][2];
    bool begun = false, several = false;
    int tile = 0;
    uint32_t phase = 0;
    auto arrived = [&]() {  // the next tile
        if (__all_sync(0xffffffffu, tc::mbar_wait(&bars[tile], phase, p.r.status))) return true;
        for (int i = 0; i < C::kTiles; ++i)  // its own copies first, for 10 ms
            tc::mbar_wait(&bars[i], i < tile ? phase ^ 1u : phase, nullptr, 10000000ull);
        return false;
    };
    auto next_tile = [&]() {
        if constexpr (!C::kPairs) {
            __syncwarp();  // the tile is free
            if (load_item < 2 * count) load();
        }
        if (++tile == C::kTiles) {
            tile = 0;
            phase ^= 1;
        }
    };

    // pairs: the first turns only load
#pragma unroll 1
    for (int it = C::kPairs ? 1 - C::kTiles / 2 : 0; it < count; ++it) {
        if constexpr (C::kPairs) {
            __syncwarp();  // the pair before is free
#pragma unroll 1
            for (int i = 0; i < 2 && load_item < 2 * count; ++i) load();
            if (it < 0) continue;
        }
        if (!arrived()) return;
        __syncwarp();
        const StepInfo *fi = &info[it % C::kInfos];
        const int base = fi->base, flags = fi->flags;

        if (it == 0 || (flags & kFirst)) {  // a piece begins: its queries, zero sums
            begun = flags & kFirst;
            const int r0 = fi->tile * kM, rows = min(kM, fi->len * p.G - r0);
            several = rows > p.G || p.by_G(r0 + rows - 1) != p.by_G(r0);
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const int ra = r0 + n * 8 + qr, ia = p.by_G(ra);
                const T *q = nullptr;
                if (n * 8 + qr < rows)
                    q = reinterpret_cast<const T *>(p.q) +
                        tok_at(p.sq, fi->t0 + ia, fi->head * p.G + ra - ia * p.G);
#pragma unroll
                for (int k = 0; k < kKS; ++k) {
                    // 8 bits: a thread's four key bytes of a product are consecutive
                    const int d0 = FMT ? (k >> 2) * 64 + qc * 16 + (k & 3) * 4 : k * 16 + qc * 2;
                    const int d1 = FMT ? d0 + 2 : d0 + 8;
                    qf[k][n][0] = q ? *reinterpret_cast<const uint32_t *>(q + d0) : 0u;
                    qf[k][n][1] = q ? *reinterpret_cast<const uint32_t *>(q + d1) : 0u;
                }
                float g = 1.f;
                if constexpr (FMT != 0 && std::is_same<T, __nv_bfloat16>::value) {
                    // BF16 queries as FP16 of the row's own power of two: 11 bits
                    // hold their 8 for every element within 2^-16 of the largest,
                    // the others to 2^-25 of it
                    float x = 0.f;
#pragma unroll
                    for (int k = 0; k < kKS; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 y = unpack2<T>(qf[k][n][e]);
                            x = fmaxf(x, fmaxf(fabsf(y.x), fabsf(y.y)));
                        }
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    const int ex = (__float_as_int(x) >> 23) & 255;  // 1 where x is no normal number
                    g = ex > 0 && ex < 254 ? __int_as_float((254 - ex) << 23) : 1.f;
#pragma unroll
                    for (int k = 0; k < kKS; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 y = unpack2<T>(qf[k][n][e]);
                            qf[k][n][e] = pack2<__half>(y.x * g, y.y * g);
                        }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = n * 8 + 2 * qc + e;
                    lo[n][e] = hi[n][e] = 0;
                    if (r < rows) visible(p, fi->kv, fi->kv - fi->len + p.by_G(r0 + r), lo[n][e], hi[n][e]);
                    f2[n][e] = p.scale * kLog2e / __shfl_sync(0xffffffffu, g, (2 * qc + e) * 4);
                    m[n][e] = -INFINITY;
                    l[n][e] = 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < kDT; ++i)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;
        }

        // scores: sc[t][n][.] of tokens 16 t + token_of(qr) (and + 8: 2, 3) and
        // queries 8 n + 2 qc (and + 1: 1, 3)
        const uint8_t *kt = ring + C::tile_at(tile);
        float sc[kMT][NR][4];
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[t][n][e] = 0.f;
        if constexpr (FMT == 0) {
            const uint32_t kt_u = ring_u + C::tile_at(tile);
#pragma unroll
            for (int k = 0; k < kKS; ++k)
#pragma unroll
                for (int t = 0; t < kMT; ++t) {
                    uint32_t x[4];
                    ldsm4(x, kt_u + kv_off<FMT, D>(t * 16 + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
                    for (int n = 0; n < NR; ++n) mma16<TP>(sc[t][n], x, qf[k][n][0], qf[k][n][1]);
                }
        } else {
#pragma unroll
            for (int g = 0; g < D / 64; ++g)
#pragma unroll
                for (int t = 0; t < kMT; ++t) {
                    const int ta = t * 16 + token_of<FMT>(qr);
                    const uint4 x = *reinterpret_cast<const uint4 *>(kt + kv_off<FMT, D>(ta, g * 4 + qc));
                    const uint4 y = *reinterpret_cast<const uint4 *>(kt + kv_off<FMT, D>(ta + 8, g * 4 + qc));
                    const uint32_t xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[4];
                        widen4<FMT>(xa[k], w[0], w[2]);
                        widen4<FMT>(ya[k], w[1], w[3]);
#pragma unroll
                        for (int n = 0; n < NR; ++n)
                            mma16<TP>(sc[t][n], w, qf[g * 4 + k][n][0], qf[g * 4 + k][n][1]);
                    }
                }
        }

        // base-2 scores; 8 bits: with the values' scales in them
        float inv_s[kMT][2];
        bool small = false;  // some value's scale is weighed as 2^-100
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float ks = 1.f, lg = 0.f;
                if constexpr (FMT) {
                    const float *s = reinterpret_cast<const float *>(ring + C::scale_at(tile)) + t * 16 + h * 8 +
                                     token_of<FMT>(qr);
                    ks = s[0];
                    const float vs = weighed_scale(s[C::kBN]);
                    if (kBf) small |= s[C::kBN] < kLeastScale && s[C::kBN] > 0.f;
                    lg = __log2f(vs);
                    inv_s[t][h] = __fdividef(1.f, vs);
                }
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = sc[t][n][2 * h + e];
                        x = FMT ? fmaf(x * ks, f2[n][e], lg) : x * f2[n][e];
                    }
            }
        next_tile();  // the keys are done with

        if (flags & kMask) {
#pragma unroll
            for (int t = 0; t < kMT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int pos = base + t * 16 + h * 8 + token_of<FMT>(qr);
                    bool any = false;
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const bool see = pos >= lo[n][e] && pos < hi[n][e];
                            if (!see) sc[t][n][2 * h + e] = -INFINITY;
                            any |= see;
                        }
                    // nobody's weight: its scale may be NaN
                    if (FMT && !any) inv_s[t][h] = 0.f;
                }
        }

        // running maximum; the sums are scaled down only when it has grown by
        // more than 2^4 for some query, so weights stay below 16
        float x[NR][2];
        bool grown = false;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                x[n][e] = fmaxf(sc[0][n][e], sc[0][n][2 + e]);
#pragma unroll
                for (int t = 1; t < kMT; ++t)
                    x[n][e] = fmaxf(x[n][e], fmaxf(sc[t][n][e], sc[t][n][2 + e]));
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    x[n][e] = fmaxf(x[n][e], __shfl_xor_sync(0xffffffffu, x[n][e], d));
                grown |= x[n][e] > m[n][e] + 4.f;
            }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // each row by its own scores alone
                    const float y = x[n][e] > m[n][e] + 4.f ? x[n][e] : m[n][e];
                    const float c = y == -INFINITY ? 1.f : ex2(m[n][e] - y);
                    m[n][e] = y;
                    l[n][e] *= c;
#pragma unroll
                    for (int i = 0; i < kDT; ++i) {
                        acc[i][n][e] *= c;
                        acc[i][n][2 + e] *= c;
                    }
                }
        }
        // weights, and their transposes as the second operand
        uint32_t ph[kMT][NR][2], pl[kMT][NR][2];
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &w = sc[t][n][2 * h + e];
                        w = ex2(w - (m[n][e] == -INFINITY ? 0.f : m[n][e]));
                        // a query that does not see the token has weight 0 there
                        // and takes nothing of its scale, NaN or not
                        l[n][e] += FMT ? (w == 0.f ? 0.f : w * inv_s[t][h]) : w;
                    }
                }
        if (kBf && __any_sync(0xffffffffu, small)) {
            // what 2^-100 leaves of their scales goes to their weights
#pragma unroll
            for (int t = 0; t < kMT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float s = reinterpret_cast<const float *>(ring + C::scale_at(tile))[
                        C::kBN + t * 16 + h * 8 + token_of<FMT>(qr)];
                    const float rest = s >= 0.f && s < kLeastScale ? s * (1.f / kLeastScale) : 1.f;
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) sc[t][n][2 * h + e] *= rest;
                }
        }
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w2 = pack2<TP>(sc[t][n][2 * h], sc[t][n][2 * h + 1]);
                    ph[t][n][h] = transpose8(w2);
                    if constexpr (kSplitP) {
                        const float2 r = unpack2<TP>(w2);
                        pl[t][n][h] = transpose8(pack2<TP>(sc[t][n][2 * h] - r.x, sc[t][n][2 * h + 1] - r.y));
                    }
                }

        if (!arrived()) return;
        uint8_t *vt = ring + C::tile_at(tile);
        // what lies past the last position, or before the first that the tile's
        // first row sees (steps begin where a box of a page does), is anything
        const int left = fi->hi - base, before = __shfl_sync(0xffffffffu, lo[0][0], 0) - base;
        if ((flags & kMask) && (left < C::kBN || before > 0)) {
            for (int i = lane; i < C::kBN * (C::kRow / 16); i += 32) {
                const int t = i / (C::kRow / 16);
                if (t >= left || t < before)
                    *reinterpret_cast<uint4 *>(vt + kv_off<FMT, D>(t, i % (C::kRow / 16))) =
                        make_uint4(0, 0, 0, 0);
            }
            tc::fence_async_smem();
            __syncwarp();
        }
        if constexpr (FMT == 0) {
            // a value that some rows see and others do not must not reach the
            // others as 0 * NaN: where one is not finite it is added by hand
            if ((flags & kMask) && several) {
                constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
                bool bad = false;
                for (int i = lane; i < C::kRows / 4; i += 32) {
                    const uint32_t y = *reinterpret_cast<uint32_t *>(vt + i * 4);
                    bad |= (y & kExp) == kExp || (y >> 16 & kExp) == kExp;
                }
                if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
                    for (int j = 0; j < C::kBN; ++j) {
                        const int src = (j & 7) * 4 + qc, pos = base + j;
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            float w[2] = {0.f, 0.f};
#pragma unroll
                            for (int t = 0; t < kMT; ++t)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const float y = __shfl_sync(0xffffffffu, sc[t][n][2 * h + e], src);
                                        if (j >> 3 == 2 * t + h) w[e] = y;
                                    }
#pragma unroll
                            for (int i = 0; i < kDT; ++i)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const T *v = reinterpret_cast<const T *>(vt + kv_off<FMT, D>(j, 2 * i + h));
                                    const float y = (float)v[qr];
                                    if (isfinite(y)) continue;
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        if (pos >= lo[n][e] && pos < hi[n][e])
                                            acc[i][n][2 * h + e] += w[e] * y;
                                }
                        }
                    }
                    __syncwarp();
                    for (int i = lane; i < C::kRows / 2; i += 32) {
                        T *e = reinterpret_cast<T *>(vt) + i;
                        if (!isfinite((float)*e)) *e = (T)0.f;
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                }
            }
            const uint32_t vt_u = ring_u + C::tile_at(tile);
#pragma unroll
            for (int t = 0; t < kMT; ++t)
#pragma unroll
                for (int i = 0; i < kDT; i += 2) {
                    uint32_t y[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        ldsm4t(y[h], vt_u + kv_off<FMT, D>(t * 16 + (lane & 7) + (lane >> 4) * 8,
                                                           2 * (i + h) + (lane >> 3 & 1)));
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) mma16<TP>(acc[i + h][n], y[h], ph[t][n][0], ph[t][n][1]);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) mma16<TP>(acc[i + h][n], y[h], pl[t][n][0], pl[t][n][1]);
                }
        } else {
#pragma unroll
            for (int t = 0; t < kMT; ++t) {
                uint32_t w[4][kB / 4];  // of tokens of rows 2 qc, 2 qc + 1, and + 8
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int tj = t * 16 + (j >> 1) * 8 + token_of<FMT>(2 * qc + (j & 1));
                    if constexpr (kB == 8) {
                        const uint2 y = *reinterpret_cast<const uint2 *>(
                            vt + kv_off<FMT, D>(tj, qr >> 1) + (qr & 1) * 8);
                        w[j][0] = y.x;
                        w[j][1] = y.y;
                    } else {
                        const uint4 y = *reinterpret_cast<const uint4 *>(vt + kv_off<FMT, D>(tj, qr));
                        w[j][0] = y.x;
                        w[j][1] = y.y;
                        w[j][2] = y.z;
                        w[j][3] = y.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < kB / 4; ++i) {
                    // pairs of tokens of columns 4 i, 4 i + 1 and 4 i + 2, 4 i + 3
                    const uint32_t p01 = __byte_perm(w[0][i], w[1][i], 0x5140);
                    const uint32_t p23 = __byte_perm(w[0][i], w[1][i], 0x7362);
                    const uint32_t q01 = __byte_perm(w[2][i], w[3][i], 0x5140);
                    const uint32_t q23 = __byte_perm(w[2][i], w[3][i], 0x7362);
                    uint32_t y[2][4];
                    widen4<FMT>(p01, y[0][0], y[0][1]);
                    widen4<FMT>(q01, y[0][2], y[0][3]);
                    widen4<FMT>(p23, y[1][0], y[1][1]);
                    widen4<FMT>(q23, y[1][2], y[1][3]);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            mma16<TP>(acc[2 * i + h][n], y[h], ph[t][n][0], ph[t][n][1]);
                            if constexpr (kSplitP)
                                mma16<TP>(acc[2 * i + h][n], y[h], pl[t][n][0], pl[t][n][1]);
                        }
                }
            }
        }

        if ((flags & kLast) || it + 1 == count) {  // the piece ends
            const int r0 = fi->tile * kM, rows = min(kM, fi->len * p.G - r0);
            const bool whole = begun && (flags & kLast);
            const int64_t part0 = (worker * 2 + (begun ? 1 : 0)) * kM;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                float inv[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &s = l[n][e];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                    inv[e] = s == 0.f ? 0.f : 1.f / s;
                }
                if (whole && FMT == 0) {
                    // transposed: query qr, columns 2 qc, 2 qc + 1 of every 8
                    const int row = r0 + n * 8 + qr, i0 = p.by_G(row);
                    T *o = reinterpret_cast<T *>(p.o) + tok_at(p.so, fi->t0 + i0, fi->head * p.G + row - i0 * p.G);
#pragma unroll
                    for (int i = 0; i < kDT; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t y = transpose8(
                                pack2<T>(acc[i][n][2 * h] * inv[0], acc[i][n][2 * h + 1] * inv[1]));
                            if (n * 8 + qr < rows)
                                *reinterpret_cast<uint32_t *>(o + i * 16 + h * 8 + 2 * qc) = y;
                        }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = n * 8 + 2 * qc + e;
                    if (r >= rows) continue;
                    const int row = r0 + r, i0 = p.by_G(row), hq = fi->head * p.G + row - i0 * p.G;
                    if (whole) {
                        if constexpr (FMT != 0) {  // columns kB qr ..
                            T *o = reinterpret_cast<T *>(p.o) + tok_at(p.so, fi->t0 + i0, hq) + qr * kB;
#pragma unroll
                            for (int i = 0; i < kDT; i += 4) {
                                uint4 y;
                                y.x = pack2<T>(acc[i][n][e] * inv[e], acc[i][n][2 + e] * inv[e]);
                                y.y = pack2<T>(acc[i + 1][n][e] * inv[e], acc[i + 1][n][2 + e] * inv[e]);
                                y.z = pack2<T>(acc[i + 2][n][e] * inv[e], acc[i + 2][n][2 + e] * inv[e]);
                                y.w = pack2<T>(acc[i + 3][n][e] * inv[e], acc[i + 3][n][2 + e] * inv[e]);
                                *reinterpret_cast<uint4 *>(o + 2 * i) = y;
                            }
                        }
                        if (p.lse && qr == 0)
                            p.lse[(int64_t)(fi->t0 + i0) * p.Hq + hq] =
                                l[n][e] == 0.f ? -INFINITY
                                               : ((m[n][e] == -INFINITY ? 0.f : m[n][e]) + log2f(l[n][e])) * kLn2;
                    } else {
                        float *po = a.ws.o + (part0 + r) * D;
#pragma unroll
                        for (int i = 0; i < kDT; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                po[FMT ? qr * kB + 2 * i + h : i * 16 + h * 8 + qr] = acc[i][n][2 * h + e];
                        if (qr == 0) {
                            a.ws.ml[(part0 + r) * 2] = m[n][e];
                            a.ws.ml[(part0 + r) * 2 + 1] = l[n][e];
                        }
                    }
                }
            }
            if (begun && !(flags & kLast) && lane == 0)
                a.ws.rec[worker] = make_int4(
                    fi->head << 16 | pieces_from(total, worker, nw, end + fi->steps_left), fi->t0,
                    fi->len, fi->tile);
        }
        next_tile();
    }
}

// ---- joining split units --------------------------------------------------
// The unit that worker w begins and others go on with, row by row:
//   m = max_j m_j,  o = sum_j 2^(m_j - m) O_j / sum_j 2^(m_j - m) l_j
// over its pieces j, in an order that only their number fixes: up to kBatch
// pieces by one warp a row; more by all warps of the CTA, each taking every
// kW-th piece of one row.  What a CTA waits for is loads, one behind the other
// (15 us a CTA when pieces came one by one), so a batch of pieces is asked for
// at once.
constexpr int kJoinThreads = 256;

// A lane's V = D / 32 consecutive columns.
template <int V>
__device__ __forceinline__ void load_cols(float (&o)[V], const float *p) {
    if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2 *>(p);
        o[0] = x.x; o[1] = x.y;
    }
}

constexpr int kBatch = 8;
template <int V>
struct Joined {
    float m = -INFINITY, l = 0.f, o[V] = {};
    // Pieces first, first + stride, ... below `pieces`, a batch of them; at(j)
    // gives piece j's row of the scratch.
    template <typename F>
    __device__ __forceinline__ void add(const SplitScratch &ws, int D, int lane, int first, int stride,
                                        int pieces, F at) {
        float oj[kBatch][V], mj[kBatch], lj[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int j = first + b * stride;
            mj[b] = -INFINITY;
            lj[b] = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) oj[b][i] = 0.f;
            if (j < pieces) {
                const int64_t r = at(j);
                const float2 ml = *reinterpret_cast<const float2 *>(ws.ml + r * 2);
                mj[b] = ml.x;
                lj[b] = ml.y;
                load_cols<V>(oj[b], ws.o + r * D + lane * V);
            }
        }
        float n = m;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) n = fmaxf(n, mj[b]);
        const float nu = n == -INFINITY ? 0.f : n, c = ex2(m - nu);
        m = n;
        l *= c;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] *= c;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const float cj = ex2(mj[b] - nu);
            l += lj[b] * cj;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] += oj[b][i] * cj;
        }
    }
};

template <typename T, int M, int D>
__global__ void __launch_bounds__(kJoinThreads, 4) k_attn_join(const __grid_constant__ AttnProblem p,
                                                               SplitScratch ws) {
    constexpr int kW = kJoinThreads / 32, kV = D / 32;
    __shared__ __align__(16) float s_o[kW][D];
    __shared__ __align__(8) float s_ml[kW][2];
    pdl_wait();
    const int64_t w = blockIdx.x;
    const int4 rec = ws.rec[w];
    const int pieces = rec.x & 0xffff, head = (int)((unsigned)rec.x >> 16);
    if (pieces == 0) return;
    const int t0 = rec.y, tile = rec.w, rows = min(M, rec.z * p.G - tile * M);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto write = [&](const Joined<kV> &a, int r) {
        const bool empty = a.l == 0.f;
        const float inv = empty ? 0.f : 1.f / a.l;
        const int row = tile * M + r, i = p.by_G(row), hq = head * p.G + row - i * p.G;
        T *o = reinterpret_cast<T *>(p.o) + tok_at(p.so, t0 + i, hq) + lane * kV;
#pragma unroll
        for (int e = 0; e < kV; e += 2)
            *reinterpret_cast<uint32_t *>(o + e) = pack2<T>(a.o[e] * inv, a.o[e + 1] * inv);
        if (p.lse && lane == 0)
            p.lse[(int64_t)(t0 + i) * p.Hq + hq] =
                empty ? -INFINITY : ((a.m == -INFINITY ? 0.f : a.m) + log2f(a.l)) * kLn2;
    };
    auto piece = [&](int r) {
        return [=](int j) { return ((w + j) * 2 + (j == 0 ? 1 : 0)) * M + r; };
    };
    if (pieces <= kBatch) {
        for (int r = blockIdx.y * kW + warp; r < rows; r += gridDim.y * kW) {
            Joined<kV> a;
            a.add(ws, D, lane, 0, 1, pieces, piece(r));
            write(a, r);
        }
        return;
    }
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        Joined<kV> a;
        for (int j = warp; j < pieces; j += kW * kBatch) a.add(ws, D, lane, j, kW, pieces, piece(r));
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kV; ++i) s_o[warp][lane * kV + i] = a.o[i];
        if (lane == 0) {
            s_ml[warp][0] = a.m;
            s_ml[warp][1] = a.l;
        }
        __syncthreads();
        if (warp) continue;
        Joined<kV> all;
        all.add(SplitScratch{&s_o[0][0], &s_ml[0][0], nullptr}, D, lane, 0, 1, kW,
                [](int j) { return (int64_t)j; });
        write(all, r);
    }
}

template <typename T, int FMT, int D, int NR>
cudaError_t launch_rows(const AttnProblem &p, const SplitScratch &ws, int ctas, cudaStream_t st) {
    using C = RowsCfg<FMT, D>;
    RowsArgs a{p, ws, 2};
    const int box = p.align < C::kBN ? p.align : C::kBN;
    if (box >= 8 && scales_aligned16(p.c) && page_map(&a.tk, p, p.c.k, p.c.kst, D, box, kPageSwizzled) &&
        page_map(&a.tv, p, p.c.v, p.c.vst, D, box, kPageSwizzled))
        a.box = box;
    auto k = k_attn_rows<T, FMT, D, NR>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_a_device(done, [&] {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess) return e;
    k<<<ctas, 32 * C::kWarps, C::kSmem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D, int NR>
cudaError_t launch_fmt(const AttnProblem &p, const SplitScratch &ws, int ctas, cudaStream_t st) {
    if (p.c.dtype == GDR_E4M3) return launch_rows<T, 1, D, NR>(p, ws, ctas, st);
    if (p.c.dtype == GDR_I8) return launch_rows<T, 2, D, NR>(p, ws, ctas, st);
    return launch_rows<T, 0, D, NR>(p, ws, ctas, st);
}

template <typename T>
cudaError_t launch_dim(const AttnProblem &p, const SplitScratch &ws, const SplitPlan &s, cudaStream_t st) {
    if (s.rows == 8)
        return p.K == 64 ? launch_fmt<T, 64, 1>(p, ws, s.ctas, st) : launch_fmt<T, 128, 1>(p, ws, s.ctas, st);
    return p.K == 64 ? launch_fmt<T, 64, 2>(p, ws, s.ctas, st) : launch_fmt<T, 128, 2>(p, ws, s.ctas, st);
}

template <typename T, int M>
cudaError_t join_dim(const AttnProblem &p, const SplitScratch &ws, int workers, cudaStream_t st) {
    // many pieces a unit (of which there are at least so many): a CTA for each
    // row of it; few: 8 rows share one, or 32 of a 256-row unit (4096 new tokens
    // over 16K in E4M3: 484 us the whole call, 486 with 8, 489 with 64 CTAs a
    // unit, half of them idle)
    const int64_t tokens = rows_packed(p.r) ? p.r.T : p.r.N * p.r.T, tiles = tokens * p.G / M;
    const bool many = workers > 8 * (p.r.N > tiles ? p.r.N : tiles) * p.c.H;
    const int y = !many ? (M > kRowsMost ? M / 32 : M / 8) : M <= kRowsMost ? (p.G < M ? p.G : M) : 64;
    const dim3 g((unsigned)workers, (unsigned)y);
    if (p.V == 64) return launch_pdl(k_attn_join<T, M, 64>, g, dim3(kJoinThreads), 0, st, p, ws);
    return launch_pdl(k_attn_join<T, M, 128>, g, dim3(kJoinThreads), 0, st, p, ws);
}

template <typename T>
cudaError_t join_rows(const AttnProblem &p, const SplitScratch &ws, const SplitPlan &s, cudaStream_t st) {
    if (s.rows == 8) return join_dim<T, 8>(p, ws, s.workers, st);
    if (s.rows == kRowsMost) return join_dim<T, kRowsMost>(p, ws, s.workers, st);
    return join_dim<T, 256>(p, ws, s.workers, st);
}

}  // namespace

SplitPlan attn_rows_plan(const AttnProblem &p, int64_t rows) {
    SplitPlan s{};
    const int g = device_sms();
    s.ctas = p.grid_limit > 0 && p.grid_limit < g ? p.grid_limit : g;
    s.workers = s.ctas * RowsCfg<0, 128>::kWarps;
    s.rows = rows <= 8 ? 8 : kRowsMost;
    return s;
}

bool attn_rows_supported(const AttnProblem &p) {
    const int ec = cache_quantised(p.c.dtype) ? 1 : 2;
    return (p.dtype == GDR_BF16 || p.dtype == GDR_F16) && p.K == p.V && (p.K == 64 || p.K == 128) &&
           p.r.T * p.G < INT32_MAX - 512 &&  // rows are counted in 32 bits
           rows_aligned16(p.q, p.sq, 2) && rows_aligned16(p.o, p.so, 2) &&
           pages_aligned16(p.c.k, p.c.kst, ec) && pages_aligned16(p.c.v, p.c.vst, ec);
}

cudaError_t attn_rows(const AttnProblem &p, const SplitScratch &ws, const SplitPlan &s,
                      cudaStream_t st) {
    return p.dtype == GDR_F16 ? launch_dim<__half>(p, ws, s, st) : launch_dim<__nv_bfloat16>(p, ws, s, st);
}
cudaError_t attn_join(const AttnProblem &p, const SplitScratch &ws, const SplitPlan &s,
                      cudaStream_t st) {
    return p.dtype == GDR_F16 ? join_rows<__half>(p, ws, s, st) : join_rows<__nv_bfloat16>(p, ws, s, st);
}

}  // namespace gdr
