// attn_rows.cu -- attention over a paged cache for few new tokens (decode
// steps, drafts): up to 16 rows of query heads and tokens a tile.
//
// Bound by memory: every cached key and value of the sequence is read once
// for G query heads (G L rows), 4 G flops a byte at 16 bits, far below the
// tensor rate.  So the tile is the smallest that the warp-level matrix
// instruction takes (16 rows; the 128-row tiles of tcgen05 would hold one
// part in eight of work), and the design goes to keeping loads in flight:
//   * every warp is a worker of its own with an equal share of the call's
//     steps (attn_split.cuh), its own ring of kStages steps in shared memory
//     and its own running maximum, sum and accumulators in registers; warps
//     never wait for each other;
//   * a step of 32 positions comes by TMA as boxes of gcd(page size, 32) slots,
//     each of one page, a lane a box (16-byte asynchronous copies where pages
//     are no multiple of 8 slots: 200 instructions a step more);
//   * the pages of the step after the next load are looked up one load ahead,
//     so a load never waits for the page table;
//   * the ring runs across the ends of units (sequences, heads).
// 8-bit caches stay 8-bit in shared memory.  The values q of a row times its
// FP32 scale s would not fit 16 bits, so scales are applied in FP32: keys'
// scales to the scores, values' scales to the weights, as
//   w_j s_j = 2^(t_j + log2 s_j - m),   sum_j w_j = sum_j (w_j s_j) / s_j,
// m the running maximum of t_j + log2 s_j, which keeps every weight at most 1
// and so within FP16; the values themselves are exact in FP16.
// Weights are split into hi + lo halves (two products) where they have the
// output's own type: the rounding of a single half would add as much error to
// o as o's own (FP16, one 64K context: 2.9e-4 against 2.0e-4), and the
// products cost nothing beside the loads.
#include <cuda_fp8.h>

#include "attn_map.cuh"
#include "attn_split.cuh"
#include "gdr_launch.cuh"
#include "tc_common.cuh"

namespace gdr {
namespace {

constexpr int kRowsM = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLeast = 7.888609052210118e-31f;  // 2^-100

// Sizes of one configuration.  FMT: 0 the call's own 16-bit type, 1 E4M3,
// 2 8-bit integers.
template <int FMT, int D>
struct RowsCfg {
    static constexpr int kES = FMT ? 1 : 2;
    static constexpr int kBN = 32;                   // positions a step
    static constexpr int kRow = D * kES;             // bytes of a row
    static constexpr int kLine = kRow < 128 ? kRow : 128;  // bytes of a row of a box
    static constexpr int kBlocks = kRow / kLine;     // boxes beside each other
    static constexpr int kKV = kBN * kRow;           // bytes of a step's keys
    static constexpr int kScale = FMT ? kBN * 4 : 0;
    // tiles start on the swizzle's period
    static constexpr int kStage = (2 * kKV + 2 * kScale + 1023) / 1024 * 1024;
    static constexpr int kStages = kStage > 12288 ? 2 : kStage > 6144 ? 3 : 4;
    static constexpr int kRing = kStages * kStage;
    // warps an SM: a ring each
    static constexpr int kWarps = kRing > 28672 ? 6 : 8;
    static constexpr int kSmem = kWarps * kRing + 1024;
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

// Two 8-bit values in the low half of x as FP16 (exact).
template <int FMT>
__device__ __forceinline__ uint32_t widen2(uint32_t x) {
    if constexpr (FMT == 1) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3);
        return (uint32_t)h.x | (uint32_t)h.y << 16;
    } else {
        // x + 128 as the low bits of 1024 + x + 128, less 1152
        const uint32_t u = __byte_perm(x ^ 0x8080u, 0x64646464u, 0x4140);
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u),
                                  __floats2half2_rn(1152.f, 1152.f));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Shared-memory byte offset of 16-byte chunk `c` of token `t` in a step's keys
// or values: what TMA writes with the 128-byte swizzle (64-byte for rows of 64
// bytes).  ldmatrix, which takes one chunk of eight tokens, meets no bank
// twice, nor do the reads of 8-bit rows below.
template <int FMT, int D>
__device__ __forceinline__ uint32_t kv_off(int t, int c) {
    using C = RowsCfg<FMT, D>;
    if constexpr (C::kLine == 128)
        return (c >> 3) * (C::kBN * 128) + t * 128 + (((c & 7) ^ (t & 7)) << 4);
    else
        return t * 64 + ((c ^ (t >> 1 & 3)) << 4);
}

// Token of column n of score tile nt.  8 bits: the keys' reads take chunks 0-3
// or 4-7 of the tokens of columns n, n + 1 (n even), the values' reads one
// chunk or two of the tokens of columns n, n + 2, n + 4, n + 6; the order below
// puts either on different banks.
template <int FMT>
__device__ __forceinline__ int token_of(int nt, int n) {
    if constexpr (FMT == 0) return nt * 8 + n;
    else return nt * 8 + (n & 1 ? ((n - 1) ^ 4) | 1 : n);
}

// Output column of column n of product tile nt.
template <int FMT, int D>
__device__ __forceinline__ int dim_of(int nt, int n) {
    return FMT == 0 ? nt * 8 + n : n * (D / 8) + nt;
}

struct RowsArgs {
    AttnProblem p;
    SplitScratch ws;
    int min_steps;       // least steps a worker
    int box;             // slots of a TMA box (0: asynchronous copies)
    CUtensorMap tk, tv;  // [page][head][slot][column] of the caches
};

template <typename T, int FMT, int D>
__global__ void __launch_bounds__(32 * RowsCfg<FMT, D>::kWarps, 1)
    k_attn_rows(const __grid_constant__ RowsArgs a) {
    using C = RowsCfg<FMT, D>;
    using TP = typename std::conditional<FMT == 0, T, __half>::type;  // of the products
    constexpr int kNT = C::kBN / 8;        // score tiles
    constexpr int kKS = D / 16;            // products of a score
    constexpr int kDT = D / 8;             // output tiles
    // weights in two halves, where one rounding of them would be as large as
    // the output's own
    constexpr bool kSplitP = std::is_same<T, TP>::value;
    extern __shared__ uint8_t smem_raw[];
    __shared__ StepInfo s_info[C::kWarps][C::kStages];
    __shared__ uint64_t s_bar[C::kWarps][C::kStages];
    const AttnProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int qr = lane >> 2, qc = lane & 3;
    pdl_trigger();
    SplitLine<kRowsM, C::kBN, 0> line;
    line.measure(p);
    const int64_t total = line.total;
    const int64_t worker = (int64_t)blockIdx.x * C::kWarps + warp;
    int64_t nw = (int64_t)gridDim.x * C::kWarps;
    if (nw * a.min_steps > total) nw = quotient(total + a.min_steps - 1, a.min_steps);
    if (lane == 0) a.ws.rec[worker * 2] = make_int4(0, 0, 0, 0);
    if (worker >= nw) return;
    const int64_t begin = share_begin(total, worker, nw);
    const int count = (int)(share_begin(total, worker + 1, nw) - begin);
    int64_t real;
    Unit u = line.locate(p, begin, real);

    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023)) + warp * C::kRing;
    const uint32_t ring_u = tc::smem_u32(ring);
    StepInfo *info = s_info[warp];
    uint64_t *bars = s_bar[warp];
    if (lane == 0) {
        for (int i = 0; i < C::kStages; ++i) tc::mbar_init(&bars[i], a.box ? 1 : 32);
        tc::mbar_init_fence();
    }
    __syncwarp();

    // what this lane asks of the step that is loaded next: the page-table entry
    // and slot of its box (boxes first, then keys and values, then columns) or
    // of its token, a step ahead
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
    auto load_step = [&](int s) {
        const uint32_t st = ring_u + s * C::kStage;
        const bool here = asked && (unsigned)entry < (unsigned)p.c.n_pages;
        if (asked && !here) report(p.r.status, GDR_ERR_INDEX);
        if (a.box) {
            // a page past the cache reads as zeros
            const int page = here ? entry : p.c.n_pages, sl = here ? slot : 0;
            uint32_t bytes = 2 * C::kKV;
            if constexpr (FMT) bytes += __popc(__ballot_sync(0xffffffffu, here && part == 0)) * a.box * 8;
            if (lane == 0) tc::mbar_arrive_expect_tx(&bars[s], bytes);
            __syncwarp();
            if (part < 2 * C::kBlocks) {
                const int kv = part & 1, c = part >> 1;
                const uint32_t dst = st + kv * C::kKV + c * (C::kBN * 128) + bx * a.box * C::kLine;
                tma_page(dst, kv ? &a.tv : &a.tk, &bars[s], c * (C::kLine / C::kES), sl, u.head, page);
                if constexpr (FMT) {
                    if (here)
                        tc::bulk_load(ring + s * C::kStage + 2 * C::kKV + kv * C::kScale + bx * a.box * 4,
                                      (kv ? p.c.vs : p.c.ks) + scale_at(p.c, page, sl, u.head),
                                      a.box * 4, &bars[s]);
                }
            }
        } else {
            const uint8_t *kc = reinterpret_cast<const uint8_t *>(p.c.k);
            const uint8_t *vc = reinterpret_cast<const uint8_t *>(p.c.v);
            const int64_t ko = here ? page_at(p.c.kst, entry, slot, u.head) * C::kES : 0;
            const int64_t vo = here ? page_at(p.c.vst, entry, slot, u.head) * C::kES : 0;
            constexpr int kChunks = C::kRow / 16, kPer = 32 / kChunks;  // chunks a row, rows a load
#pragma unroll 2
            for (int i = 0; i < C::kBN / kPer; ++i) {
                const int t = i * kPer + lane / kChunks, c = lane % kChunks;
                const int64_t kof = __shfl_sync(0xffffffffu, ko, t);
                const int64_t vof = __shfl_sync(0xffffffffu, vo, t);
                const bool live = __shfl_sync(0xffffffffu, here, t);
                cp16(st + kv_off<FMT, D>(t, c), kc + kof + (live ? c * 16 : 0), live);
                cp16(st + C::kKV + kv_off<FMT, D>(t, c), vc + vof + (live ? c * 16 : 0), live);
            }
            if constexpr (FMT) {
                const int64_t so = here ? scale_at(p.c, entry, slot, u.head) : 0;
                cp4(st + 2 * C::kKV + lane * 4, p.c.ks + so, here);
                cp4(st + 2 * C::kKV + C::kScale + lane * 4, p.c.vs + so, here);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                             tc::smem_u32(&bars[s]))
                         : "memory");
        }
        if (lane == 0) {
            StepInfo &f = info[s];
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
        if (++u.step == u.steps) next_unit<kRowsM, C::kBN>(p, u);
    };

    look_up();
#pragma unroll 1
    for (int s = 0; s < C::kStages && s < count; ++s) {
        load_step(s);
        if (s + 1 < count) look_up();
    }

    uint32_t qf[kKS][4];
    float acc[kDT][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float f0 = 0.f, f1 = 0.f;  // base-2 score of a unit of product, rows qr and qr + 8
    int lo0 = 0, hi0 = 0, lo1 = 0, hi1 = 0;
    bool begun = false, two = false, several = false;
    int stage = 0;
    uint32_t phase = 0;

#pragma unroll 1
    for (int it = 0; it < count; ++it) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait(&bars[stage], phase, p.r.status))) {
            for (int s = 0; s < C::kStages; ++s)  // its own copies first, for 10 ms
                tc::mbar_wait(&bars[s], s < stage ? phase ^ 1u : phase, nullptr, 10000000ull);
            return;
        }
        __syncwarp();
        const int base = info[stage].base, flags = info[stage].flags;
        const uint32_t ks_u = ring_u + stage * C::kStage, vs_u = ks_u + C::kKV;
        uint8_t *st = ring + stage * C::kStage;

        if (it == 0 || (flags & kFirst)) {  // a piece begins: its queries, zero sums
            const StepInfo f = info[stage];
            begun = flags & kFirst;
            const int rows = min(kRowsM, f.len * p.G - f.tile * kRowsM);
            two = rows > 8;
            const int ra = f.tile * kRowsM + qr, ia = p.by_G(ra), ib = p.by_G(ra + 8);
            several = __any_sync(0xffffffffu, rows > p.G || (qr == 0 && p.by_G(ra + rows - 1) != ia));
            lo0 = hi0 = lo1 = hi1 = 0;
            const T *qa = nullptr, *qb = nullptr;
            if (qr < rows) {
                visible(p, f.kv, f.kv - f.len + ia, lo0, hi0);
                qa = reinterpret_cast<const T *>(p.q) +
                     tok_at(p.sq, f.t0 + ia, f.head * p.G + ra - ia * p.G);
            }
            if (qr + 8 < rows) {
                visible(p, f.kv, f.kv - f.len + ib, lo1, hi1);
                qb = reinterpret_cast<const T *>(p.q) +
                     tok_at(p.sq, f.t0 + ib, f.head * p.G + ra + 8 - ib * p.G);
            }
#pragma unroll
            for (int k = 0; k < kKS; ++k) {
                // 8 bits: a thread's four key bytes of a product are consecutive
                const int d0 = FMT ? (k >> 2) * 64 + qc * 16 + (k & 3) * 4 : k * 16 + qc * 2;
                const int d1 = FMT ? d0 + 2 : d0 + 8;
                qf[k][0] = qa ? *reinterpret_cast<const uint32_t *>(qa + d0) : 0u;
                qf[k][1] = qb ? *reinterpret_cast<const uint32_t *>(qb + d0) : 0u;
                qf[k][2] = qa ? *reinterpret_cast<const uint32_t *>(qa + d1) : 0u;
                qf[k][3] = qb ? *reinterpret_cast<const uint32_t *>(qb + d1) : 0u;
            }
            f0 = f1 = p.scale * kLog2e;
            if constexpr (FMT != 0 && std::is_same<T, __nv_bfloat16>::value) {
                // BF16 queries as FP16 of the row's own power of two: 11 bits
                // hold their 8 for every element within 2^-16 of the largest,
                // the others to 2^-25 of it
                float x0 = 0.f, x1 = 0.f;
#pragma unroll
                for (int k = 0; k < kKS; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y2 = unpack2<T>(qf[k][e]);
                        float &xm = e & 1 ? x1 : x0;
                        xm = fmaxf(xm, fmaxf(fabsf(y2.x), fabsf(y2.y)));
                    }
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
                }
                auto power = [](float x) {  // 2^-floor(log2 x); 1 where x is no normal number
                    const int e = (__float_as_int(x) >> 23) & 255;
                    return e > 0 && e < 254 ? __int_as_float((254 - e) << 23) : 1.f;
                };
                const float g0 = power(x0), g1 = power(x1);
                f0 /= g0;
                f1 /= g1;
#pragma unroll
                for (int k = 0; k < kKS; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y2 = unpack2<T>(qf[k][e]);
                        const float gg = e & 1 ? g1 : g0;
                        qf[k][e] = pack2<__half>(y2.x * gg, y2.y * gg);
                    }
            }
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.f;
#pragma unroll
            for (int i = 0; i < kDT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
        }

        // scores: sc[nt] = rows x tokens token_of(nt, .)
        float sc[kNT][4];
#pragma unroll
        for (int i = 0; i < kNT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
        if constexpr (FMT == 0) {
#pragma unroll
            for (int k = 0; k < kKS; ++k) {
#pragma unroll
                for (int h = 0; h < kNT / 2; ++h) {
                    uint32_t b[4];  // tokens 0-7 and 8-15 of 16, both halves of the columns
                    const int t = h * 16 + (lane & 7) + ((lane >> 4) << 3), c = 2 * k + (lane >> 3 & 1);
                    ldsm4(b, ks_u + kv_off<FMT, D>(t, c));
                    mma16<TP>(sc[2 * h], qf[k], b[0], b[1]);
                    mma16<TP>(sc[2 * h + 1], qf[k], b[2], b[3]);
                }
            }
        } else {
#pragma unroll
            for (int g = 0; g < D / 64; ++g)
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    const int t = token_of<FMT>(nt, qr);
                    const uint4 w = *reinterpret_cast<const uint4 *>(st + kv_off<FMT, D>(t, g * 4 + qc));
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma16<TP>(sc[nt], qf[g * 4 + k], widen2<FMT>(x[k]), widen2<FMT>(x[k] >> 16));
                }
        }

        // base-2 scores; 8 bits: with the values' scales in them
        float inv_s[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            float ks2[2] = {1.f, 1.f}, lg[2] = {0.f, 0.f};
            if constexpr (FMT) {
                const float *sk = reinterpret_cast<const float *>(st + 2 * C::kKV), *sv = sk + C::kBN;
                const int ta = token_of<FMT>(nt, 2 * qc), tb = token_of<FMT>(nt, 2 * qc + 1);
                ks2[0] = sk[ta];
                ks2[1] = sk[tb];
                // no smaller than 2^-100, so that 1 / s is finite: a scale of
                // 0 stands for a row of zeros, for which any other will do
                const float v0 = sv[ta] < kLeast ? kLeast : sv[ta], v1 = sv[tb] < kLeast ? kLeast : sv[tb];
                lg[0] = __log2f(v0);
                lg[1] = __log2f(v1);
                inv_s[nt][0] = __fdividef(1.f, v0);
                inv_s[nt][1] = __fdividef(1.f, v1);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if constexpr (FMT) {
                    sc[nt][e] = fmaf(sc[nt][e] * ks2[e], f0, lg[e]);
                    sc[nt][2 + e] = fmaf(sc[nt][2 + e] * ks2[e], f1, lg[e]);
                } else {
                    sc[nt][e] *= f0;
                    sc[nt][2 + e] *= f1;
                }
            }
        }
        if (flags & kMask) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int pos = base + token_of<FMT>(nt, 2 * qc + e);
                    const bool see0 = pos >= lo0 && pos < hi0, see1 = pos >= lo1 && pos < hi1;
                    if (!see0) sc[nt][e] = -INFINITY;
                    if (!see1) sc[nt][2 + e] = -INFINITY;
                    // no row's weight: its scale may be NaN
                    if (FMT && !see0 && !see1) inv_s[nt][e] = 0.f;
                }
        }

        // running maximum; the sums are scaled down only when it has grown by
        // more than 2^4 in some row, so weights stay below 16
        float x0 = sc[0][0], x1 = sc[0][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            x0 = fmaxf(x0, fmaxf(sc[nt][0], sc[nt][1]));
            x1 = fmaxf(x1, fmaxf(sc[nt][2], sc[nt][3]));
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
        }
        if (__any_sync(0xffffffffu, x0 > m0 + 4.f || x1 > m1 + 4.f)) {
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
            const float c0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0);
            const float c1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= c0;
            l1 *= c1;
#pragma unroll
            for (int i = 0; i < kDT; ++i) {
                acc[i][0] *= c0;
                acc[i][1] *= c0;
                acc[i][2] *= c1;
                acc[i][3] *= c1;
            }
        }
        const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
        uint32_t ph[kNT][2], pl[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sc[nt][e] = ex2(sc[nt][e] - u0);
                sc[nt][2 + e] = two ? ex2(sc[nt][2 + e] - u1) : 0.f;
                if constexpr (FMT) {
                    // a row that does not see the token has weight 0 there
                    // and takes nothing of its scale, NaN or not
                    l0 += sc[nt][e] == 0.f ? 0.f : sc[nt][e] * inv_s[nt][e];
                    l1 += sc[nt][2 + e] == 0.f ? 0.f : sc[nt][2 + e] * inv_s[nt][e];
                } else {
                    l0 += sc[nt][e];
                    l1 += sc[nt][2 + e];
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ph[nt][h] = pack2<TP>(sc[nt][2 * h], sc[nt][2 * h + 1]);
                if constexpr (kSplitP) {
                    const float2 r = unpack2<TP>(ph[nt][h]);
                    pl[nt][h] = pack2<TP>(sc[nt][2 * h] - r.x, sc[nt][2 * h + 1] - r.y);
                }
            }
        }

        // what lies past the last position is anything
        if ((flags & kMask) && base + C::kBN > info[stage].hi) {
            const int left = info[stage].hi - base;
            for (int i = lane; i < C::kBN * (C::kRow / 16); i += 32) {
                const int t = i / (C::kRow / 16);
                if (t >= left)
                    *reinterpret_cast<uint4 *>(st + C::kKV + kv_off<FMT, D>(t, i % (C::kRow / 16))) =
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
                auto bad = [](uint32_t x) {
                    return (x & kExp) == kExp || (x >> 16 & kExp) == kExp;
                };
                bool any = false;
                for (int i = lane; i < C::kKV / 4; i += 32)
                    any |= bad(*reinterpret_cast<uint32_t *>(st + C::kKV + i * 4));
                if (__any_sync(0xffffffffu, any)) {
#pragma unroll 1
                    for (int t = 0; t < C::kBN; ++t) {
                        const int nt = t >> 3, src = (lane & ~3) + ((t & 7) >> 1);
                        float w0 = 0.f, w1 = 0.f;
#pragma unroll
                        for (int j = 0; j < kNT; ++j) {
                            const float a0 = __shfl_sync(0xffffffffu, t & 1 ? sc[j][1] : sc[j][0], src);
                            const float a1 = __shfl_sync(0xffffffffu, t & 1 ? sc[j][3] : sc[j][2], src);
                            if (j == nt) {
                                w0 = a0;
                                w1 = a1;
                            }
                        }
                        const int pos = base + t;
                        const bool see0 = pos >= lo0 && pos < hi0, see1 = pos >= lo1 && pos < hi1;
#pragma unroll
                        for (int i = 0; i < kDT; ++i) {
                            const uint32_t x = *reinterpret_cast<uint32_t *>(
                                st + C::kKV + kv_off<FMT, D>(t, i) + qc * 4);
                            const float2 v = unpack2<T>(x);
                            if (!isfinite(v.x)) {
                                if (see0) acc[i][0] += w0 * v.x;
                                if (see1) acc[i][2] += w1 * v.x;
                            }
                            if (!isfinite(v.y)) {
                                if (see0) acc[i][1] += w0 * v.y;
                                if (see1) acc[i][3] += w1 * v.y;
                            }
                        }
                    }
                    __syncwarp();
                    for (int i = lane; i < C::kKV / 2; i += 32) {
                        T *e = reinterpret_cast<T *>(st + C::kKV) + i;
                        if (!isfinite((float)*e)) *e = (T)0.f;
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                }
            }
#pragma unroll
            for (int h = 0; h < kNT / 2; ++h) {
                const uint32_t ah[4] = {ph[2 * h][0], ph[2 * h][1], ph[2 * h + 1][0], ph[2 * h + 1][1]};
                const uint32_t al[4] = {pl[2 * h][0], pl[2 * h][1], pl[2 * h + 1][0], pl[2 * h + 1][1]};
#pragma unroll
                for (int i = 0; i < kDT; i += 2) {
                    uint32_t b[4];  // columns 8 i .. and 8 (i + 1) .., tokens 0-7 and 8-15 of 16
                    const int t = h * 16 + (lane & 15), c = i + (lane >> 4);
                    ldsm4t(b, vs_u + kv_off<FMT, D>(t, c));
                    mma16<TP>(acc[i], ah, b[0], b[1]);
                    mma16<TP>(acc[i + 1], ah, b[2], b[3]);
                    mma16<TP>(acc[i], al, b[0], b[1]);
                    mma16<TP>(acc[i + 1], al, b[2], b[3]);
                }
            }
        } else {
            constexpr int kB = D / 8;  // value bytes a thread takes of a token
#pragma unroll
            for (int kk = 0; kk < C::kBN / 16; ++kk) {
                const uint32_t av[4] = {ph[2 * kk][0], ph[2 * kk][1], ph[2 * kk + 1][0],
                                        ph[2 * kk + 1][1]};
                const uint32_t al[4] = {pl[2 * kk][0], pl[2 * kk][1], pl[2 * kk + 1][0],
                                        pl[2 * kk + 1][1]};
                uint32_t w[4][kB / 4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = token_of<FMT>(2 * kk + (j >> 1), 2 * qc + (j & 1));
                    if constexpr (kB == 8) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(
                            st + C::kKV + kv_off<FMT, D>(t, qr >> 1) + (qr & 1) * 8);
                        w[j][0] = x.x;
                        w[j][1] = x.y;
                    } else {
#pragma unroll
                        for (int h = 0; h < kB / 16; ++h) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(
                                st + C::kKV + kv_off<FMT, D>(t, qr * (kB / 16) + h));
                            w[j][h * 4] = x.x;
                            w[j][h * 4 + 1] = x.y;
                            w[j][h * 4 + 2] = x.z;
                            w[j][h * 4 + 3] = x.w;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < kB / 4; ++i) {
                    const uint32_t a01 = __byte_perm(w[0][i], w[1][i], 0x5140);
                    const uint32_t a23 = __byte_perm(w[0][i], w[1][i], 0x7362);
                    const uint32_t b01 = __byte_perm(w[2][i], w[3][i], 0x5140);
                    const uint32_t b23 = __byte_perm(w[2][i], w[3][i], 0x7362);
                    const uint32_t ab[4] = {a01, a01 >> 16, a23, a23 >> 16};
                    const uint32_t bb[4] = {b01, b01 >> 16, b23, b23 >> 16};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t b0 = widen2<FMT>(ab[e]), b1 = widen2<FMT>(bb[e]);
                        mma16<TP>(acc[4 * i + e], av, b0, b1);
                        if constexpr (kSplitP) mma16<TP>(acc[4 * i + e], al, b0, b1);
                    }
                }
            }
        }

        if ((flags & kLast) || it + 1 == count) {  // the piece ends
            const StepInfo f = info[stage];
            float s0 = l0, s1 = l1;
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                s0 += __shfl_xor_sync(0xffffffffu, s0, d);
                s1 += __shfl_xor_sync(0xffffffffu, s1, d);
            }
            const int rows = min(kRowsM, f.len * p.G - f.tile * kRowsM);
            const bool whole = begun && (flags & kLast);
            float *po = a.ws.o + ((worker * 2 + (begun ? 1 : 0)) * kRowsM) * D;
            float *pm = a.ws.ml + ((worker * 2 + (begun ? 1 : 0)) * kRowsM) * 2;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = qr + 8 * h;
                if (r >= rows) continue;
                const float l = h ? s1 : s0, m = h ? m1 : m0;
                if (whole) {
                    const bool empty = l == 0.f;
                    const float inv = empty ? 0.f : 1.f / l;
                    const int row = f.tile * kRowsM + r, i = p.by_G(row);
                    const int hq = f.head * p.G + row - i * p.G;
                    T *o = reinterpret_cast<T *>(p.o) + tok_at(p.so, f.t0 + i, hq);
                    if constexpr (FMT == 0) {
#pragma unroll
                        for (int j = 0; j < kDT; ++j)
                            *reinterpret_cast<uint32_t *>(o + dim_of<FMT, D>(j, 2 * qc)) =
                                pack2<T>(acc[j][2 * h] * inv, acc[j][2 * h + 1] * inv);
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int j = 0; j < kDT; j += 8) {
                                uint4 x;
                                x.x = pack2<T>(acc[j][2 * h + e] * inv, acc[j + 1][2 * h + e] * inv);
                                x.y = pack2<T>(acc[j + 2][2 * h + e] * inv, acc[j + 3][2 * h + e] * inv);
                                x.z = pack2<T>(acc[j + 4][2 * h + e] * inv, acc[j + 5][2 * h + e] * inv);
                                x.w = pack2<T>(acc[j + 6][2 * h + e] * inv, acc[j + 7][2 * h + e] * inv);
                                *reinterpret_cast<uint4 *>(o + dim_of<FMT, D>(j, 2 * qc + e)) = x;
                            }
                    }
                    if (p.lse && qc == 0)
                        p.lse[(int64_t)(f.t0 + i) * p.Hq + hq] =
                            empty ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
                } else {
#pragma unroll
                    for (int j = 0; j < kDT; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            po[r * D + dim_of<FMT, D>(j, 2 * qc + e)] = acc[j][2 * h + e];
                    if (qc == 0) {
                        pm[r * 2] = m;
                        pm[r * 2 + 1] = l;
                    }
                }
            }
            if (begun && !(flags & kLast) && lane == 0) {
                a.ws.rec[worker * 2] = make_int4(
                    pieces_from(total, worker, nw, begin + it + 1 + f.steps_left), f.t0, f.len, f.tile);
                a.ws.rec[worker * 2 + 1].x = f.head;
            }
        }
        __syncwarp();  // the stage is free
        if (it + C::kStages < count) {
            load_step(stage);
            if (it + C::kStages + 1 < count) look_up();
        }
        if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
        }
    }
}

// ---- joining split units --------------------------------------------------
// The unit that worker w begins and others go on with, row by row:
//   m = max_j m_j,  o = sum_j 2^(m_j - m) O_j / sum_j 2^(m_j - m) l_j
// over its pieces j, in an order that only their number fixes: up to kW
// pieces by one warp, R rows at a time; more by all warps of the CTA, each
// taking every kW-th piece of one row.
constexpr int kJoinThreads = 256;

template <int V>
struct Joined {
    float m = -INFINITY, l = 0.f, o[V] = {};
    __device__ __forceinline__ void add(float mj, float lj, const float (&oj)[V]) {
        const float n = fmaxf(m, mj), nu = n == -INFINITY ? 0.f : n;
        const float c = exp2f(m - nu), cj = exp2f(mj - nu);
        m = n;
        l = l * c + lj * cj;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = o[i] * c + oj[i] * cj;
    }
};

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

template <typename T, int M, int D>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const __grid_constant__ AttnProblem p,
                                                            SplitScratch ws) {
    constexpr int kW = kJoinThreads / 32, kV = D / 32, kR = M > 16 ? 4 : 1;
    __shared__ __align__(16) float s_o[kW][D];
    __shared__ float s_ml[kW][2];
    pdl_wait();
    const int64_t w = blockIdx.x;
    const int4 rec = ws.rec[w * 2];
    const int pieces = rec.x;
    if (pieces == 0) return;
    const int head = ws.rec[w * 2 + 1].x, t0 = rec.y, tile = rec.w;
    const int rows = min(M, rec.z * p.G - tile * M);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto slot = [&](int j, int r) { return ((w + j) * 2 + (j == 0 ? 1 : 0)) * M + r; };
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
    if (pieces <= kW) {
        for (int r = (blockIdx.y * kW + warp) * kR; r < rows; r += gridDim.y * kW * kR) {
            Joined<kV> a[kR];
            for (int j = 0; j < pieces; ++j) {
                float oj[kR][kV], ml[kR][2];
#pragma unroll
                for (int e = 0; e < kR; ++e) {
                    const int64_t at = slot(j, min(r + e, rows - 1));
                    load_cols<kV>(oj[e], ws.o + at * D + lane * kV);
                    ml[e][0] = ws.ml[at * 2];
                    ml[e][1] = ws.ml[at * 2 + 1];
                }
#pragma unroll
                for (int e = 0; e < kR; ++e) a[e].add(ml[e][0], ml[e][1], oj[e]);
            }
#pragma unroll
            for (int e = 0; e < kR; ++e)
                if (r + e < rows) write(a[e], r + e);
        }
        return;
    }
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        Joined<kV> a;
#pragma unroll 4
        for (int j = warp; j < pieces; j += kW) {
            const int64_t at = slot(j, r);
            float oj[kV];
            load_cols<kV>(oj, ws.o + at * D + lane * kV);
            a.add(ws.ml[at * 2], ws.ml[at * 2 + 1], oj);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kV; ++i) s_o[warp][lane * kV + i] = a.o[i];
        if (lane == 0) {
            s_ml[warp][0] = a.m;
            s_ml[warp][1] = a.l;
        }
        __syncthreads();
        if (warp) continue;
        a = Joined<kV>();
        for (int j = 0; j < kW; ++j) {
            float oj[kV];
            load_cols<kV>(oj, &s_o[j][lane * kV]);
            a.add(s_ml[j][0], s_ml[j][1], oj);
        }
        write(a, r);
    }
}

template <typename T, int FMT, int D>
cudaError_t launch_rows(const AttnProblem &p, const SplitScratch &ws, int ctas, cudaStream_t st) {
    using C = RowsCfg<FMT, D>;
    RowsArgs a{p, ws, 2};
    const int box = p.align < C::kBN ? p.align : C::kBN;
    if (box >= 8 && scales_aligned16(p.c) && page_map(&a.tk, p, p.c.k, p.c.kst, D, box, kPageSwizzled) &&
        page_map(&a.tv, p, p.c.v, p.c.vst, D, box, kPageSwizzled))
        a.box = box;
    auto k = k_attn_rows<T, FMT, D>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    k<<<ctas, 32 * C::kWarps, C::kSmem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_fmt(const AttnProblem &p, const SplitScratch &ws, int ctas, cudaStream_t st) {
    if (p.c.dtype == GDR_E4M3) return launch_rows<T, 1, D>(p, ws, ctas, st);
    if (p.c.dtype == GDR_I8) return launch_rows<T, 2, D>(p, ws, ctas, st);
    return launch_rows<T, 0, D>(p, ws, ctas, st);
}

template <typename T>
cudaError_t launch_dim(const AttnProblem &p, const SplitScratch &ws, int ctas, cudaStream_t st) {
    return p.K == 64 ? launch_fmt<T, 64>(p, ws, ctas, st) : launch_fmt<T, 128>(p, ws, ctas, st);
}

template <typename T, int M>
cudaError_t join_dim(const AttnProblem &p, const SplitScratch &ws, int workers, cudaStream_t st) {
    // many pieces a unit: a CTA for each row of it; few: 8 rows (of 16-row
    // tiles) or 32 share one
    const bool many = workers > 8 * p.r.N * p.c.H;
    const int y = M == 16 ? (many ? (p.G < M ? p.G : M) : 1) : (many ? 64 : M / 32);
    const dim3 g((unsigned)workers, (unsigned)y);
    if (p.V == 64) return launch_pdl(k_attn_join<T, M, 64>, g, dim3(kJoinThreads), 0, st, p, ws);
    return launch_pdl(k_attn_join<T, M, 128>, g, dim3(kJoinThreads), 0, st, p, ws);
}

}  // namespace

// Warps a CTA of the configuration that a call takes.
static int rows_warps(const AttnProblem &p) {
    if (cache_quantised(p.c.dtype))
        return p.K == 64 ? RowsCfg<1, 64>::kWarps : RowsCfg<1, 128>::kWarps;
    return p.K == 64 ? RowsCfg<0, 64>::kWarps : RowsCfg<0, 128>::kWarps;
}

SplitPlan attn_rows_plan(const AttnProblem &p) {
    SplitPlan s{};
    const int g = device_sms();
    s.ctas = p.grid_limit > 0 && p.grid_limit < g ? p.grid_limit : g;
    s.workers = s.ctas * rows_warps(p);
    s.rows = kRowsM;
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
    return p.dtype == GDR_F16 ? launch_dim<__half>(p, ws, s.ctas, st)
                              : launch_dim<__nv_bfloat16>(p, ws, s.ctas, st);
}
cudaError_t attn_join(const AttnProblem &p, const SplitScratch &ws, const SplitPlan &s,
                      cudaStream_t st) {
    if (s.rows == kRowsM)
        return p.dtype == GDR_F16 ? join_dim<__half, kRowsM>(p, ws, s.workers, st)
                                  : join_dim<__nv_bfloat16, kRowsM>(p, ws, s.workers, st);
    return p.dtype == GDR_F16 ? join_dim<__half, 256>(p, ws, s.workers, st)
                              : join_dim<__nv_bfloat16, 256>(p, ws, s.workers, st);
}

}  // namespace gdr
