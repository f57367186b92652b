// attn_tiles.cu -- attention over a paged cache for many new tokens (chunks
// of a prompt) on tcgen05: tiles of 256 rows (query heads and tokens of one
// key head) against 128 positions a step.
//
// Per step and 128-row half, with the sums of the softmax taken in one pass:
//   S = Q K^T                        tcgen05, FP32 in TMEM
//   m' = max(m, max S),  P = e^(S - m')  (base 2, in registers; P back to TMEM
//                                    as 16-bit operand over S's own columns)
//   O <- O e^(m - m') + P V          tcgen05, A = P from TMEM
// O is scaled only when a row's maximum has grown by more than 2^8 since it
// was last scaled; the weights stay below 2^8 and the factor cancels in O / l.
//
// Weights go into the product as one 16-bit value each: two halves, as for few
// rows, would be half as many products again.  o against 64 bits, 4096 new tokens
// over 32K in BF16: 2.3e-3, of which 1.7e-3 are o's own rounding; 2.9e-4 and
// 2.1e-4 in FP16.  The sum takes them unrounded, so lse is FP32's.
// Two halves in turns, and sums rescaled only past a threshold, are published
// ideas.
//
// Bound by the tensor pipe while softmax keeps up: a step of a half is 2 x
// 512 cycles of products and 16384 exponentials (512 cycles of the special
// function units).  So the two halves run in turns: one half's exponentials
// beside the other's products.
//   warps 0-3, 4-7   softmax of rows 0-127, 128-255 (a thread a row)
//   warps 8-11       queries into shared memory; 8-bit rows widened to FP16;
//                    values of masked steps looked over (below)
//   warp 12          every tcgen05 product
//   warp 13          page look-up, keys and values by TMA
// A step's 128 positions come as boxes of gcd(page size, 128) slots, each of
// one page, into the 128-byte swizzled layout that the products read (page
// sizes that are no multiple of 8 go to the kernel of few rows).  A box
// without a page is filled with zeros.
// A position that some rows see and others do not must not reach the others
// as 0 * NaN, and what a page holds past the last position is anything: in
// masked steps (one to three a unit) warps 8-11 clear the values past the end
// and those that are not finite before the product, and the end of the piece
// adds the latter to the rows that see them.
// 8-bit caches: under FP16 queries the scales go where attn_rows.cu puts them,
// to scores and weights, which costs a thread three loads a column (393 KB of
// shared-memory traffic a step).  Under BF16 queries o is rounded to 8 bits, so
// that FP16's 11 are as good as exact for the values: there the products see q
// s / s' in FP16, s' a power of two for the step's 128 positions that brings the
// largest of them to [2^6, 2^7), and s' alone is left to the weights.  That is
// as exact for every position down to 2^-18 of the largest; a step of wider
// spread (a scale whose position a row does not see, or gives no weight, must
// not cost that row its own values) takes the way of FP16 queries.  The keys'
// scales stay with the scores: lse is FP32.
// E4M3 keys of 128 columns under BF16 queries are not widened at all: a row of
// queries, scaled by a power of two to have its largest magnitude in [2^14, 2^15),
// is split into three E5M2 parts, the upper three bits of what the ones before it
// leave.  They hold BF16's eight, so the split is exact for components down to
// 2^-23 of the row's largest (FP16 queries: 2^-17), however little the largest,
// an outlier channel say, has to do with the softmax.  Two E4M3 parts are exact
// down to 2^-9 only: with one channel of 2^10 where the keys do not vary, o was
// 4.9e-3 off.  S = (a + b + c) K^T takes three 8-bit products at twice the rate of
// one FP16 product, and the keys go from the cache into the products as they are:
// 507 us for 4096 new tokens over 16K (4 key heads), 691 with widened keys.  The
// third part's room is that of a second 8-bit tile of values (2 us).
// Measured (4 key heads of 128, 4 query heads each, BF16, replayed from a graph):
// 4096 new tokens over 32K: 615 us, 1678 TFLOP/s, 0.86 of a library product's
// rate; over 16K in E4M3: 507 us, bound by latency: the chain of a half's
// softmax, 3K cycles of which a third applies the step's 128 scales, and its
// products; 32 prompts of 128 to 512 tokens: 71 us, of which a unit costs 6 us
// beside 1.4 us a step.
//
// The steps of the call are shared out equally over one CTA an SM
// (attn_split.cuh).  Every wait is bounded: on expiry the CTA records
// GDR_ERR_TIMEOUT, its other roles leave too, and it exits once its loads in
// flight have landed.
#include "attn_map.cuh"
#include "attn_split.cuh"
#include "gdr_launch.cuh"

namespace gdr {
namespace {

using namespace tc;

constexpr int kTM = 256;       // rows of a unit
constexpr int kTN = 128;       // positions of a step
constexpr int kTThreads = 512;
// What a unit costs beside its steps, in steps: 6 us of 1.4 us (32 prompts: 71 us,
// with two 79).
constexpr int kTUnit = 4;
constexpr float kTLog2e = 1.4426950408889634f;
constexpr float kTLn2 = 0.6931471805599453f;
// Values' scales in FP16, less than 2^7 by choice: below this a step is wide.
// They keep 13 bits there (a part and what it leaves, both above 2^-25).
constexpr float kTNarrow = 0x1p-12f;
// log2 s' of a wide step: above any maximum, so that softmax comes to where it
// rescales its sums (a rare place) and finds the mark there.
constexpr float kTWide = 0x1p100f;

// Registers a thread of the softmax warps, the helpers and the rest: 128 each
// at launch, 2 x 192 + 72 + 56 = 4 x 128
// (184 / 88 / 56 spills more in the softmax, 200 / 64 / 48 in the helpers: 4096
// new tokens over 16K in E4M3 took 571 and 556 us beside 525).
constexpr int kRegSoftmax = 192, kRegHelp = 72, kRegRest = 56;
static_assert(2 * kRegSoftmax + kRegHelp + kRegRest <= 4 * 128, "the launch's registers");

template <typename T, int FMT, int D>
struct TilesCfg {
    // E4M3 keys as they are, the queries in three E5M2 parts (above)
    static constexpr bool kSplit = FMT == 1 && D == 128 && std::is_same<T, __nv_bfloat16>::value;
    static constexpr uint32_t kTile = kTN * D * 2;     // a 128-row tile of 16-bit values
    static constexpr uint32_t kQTile = kSplit ? kTN * D * 3 : kTile;  // a half's queries
    // tiles of keys and values, or of values alone beside kKeys of keys
    static constexpr int kRing = D == 64 ? 8 : kSplit ? 2 : FMT ? 3 : 4;
    static constexpr int kKeys = kSplit ? 2 : 0;
    // tiles given back in pairs, a step's keys and the values before them
    // (one commit a step instead of two); 0: one by one
    static constexpr int kPairs = FMT ? 0 : kRing / 2;
    static constexpr int kRaw = !FMT ? 0 : kSplit ? 1 : 2;  // 8-bit tiles on their way
    static constexpr uint32_t kRawTile = kTN * D, kRawSize = kRawTile + 2 * kTN * 4;
    // steps whose scales are kept: a step's keys are widened once the products
    // of the step kRing / 2 before it are done, so that softmax is at most
    // that far behind
    static constexpr int kScales = FMT ? (D == 64 ? 8 : 4) : 0;
    static constexpr uint32_t kOffRing = 2 * kQTile;   // after the queries
    static constexpr uint32_t kOffKeys = kOffRing + kRing * kTile;
    static constexpr uint32_t kOffRaw = kOffKeys + kKeys * kRawTile; // + scales of keys, values
    static constexpr uint32_t kOffScale = kOffRaw + kRaw * kRawSize; // [kScales][3][128]
    static constexpr uint32_t kOffQf = kOffScale + kScales * 3 * kTN * 4;  // [2 units][256]
    static constexpr uint32_t kOffBar = kOffQf + 2 * kTM * 4;
    static constexpr uint32_t kBytes = kOffBar + 512 + 1024;         // and to align
    static constexpr uint32_t kColS = 0, kColO = 256;  // TMEM: S / P of both halves, O
    // mbarriers
    static constexpr int kFull = 0, kEmpty = kRing;    // tiles
    static constexpr int kLand = 2 * kRing;            // FMT: raw tiles; else masked values, by tile
    static constexpr int kLands = FMT ? kRaw : kRing, kTaken = kLand + kLands;  // raw tiles read
    static constexpr int kKeyFull = kTaken + kRaw, kKeyEmpty = kKeyFull + kKeys;
    static constexpr int kQFull = kKeyEmpty + kKeys, kQEmpty = kQFull + 1, kS = kQFull + 2, kP = kS + 2,
                         kO = kP + 2, kDrain = kO + 2;
    static_assert((kDrain + 1) * 8 <= 512, "barriers");
    // Item 2 s is the keys of step s and 2 s + 1 its values: its tile, how often
    // the tile was used before, its barriers.
    __device__ static uint32_t turns(uint32_t item) {
        return !kSplit ? item / kRing : (item >> 1) / (item & 1 ? kRing : kKeys);
    }
    __device__ static uint32_t slot(uint32_t item) {
        return !kSplit ? item % kRing : (item >> 1) % (item & 1 ? kRing : kKeys);
    }
    __device__ static int full(uint32_t item) {
        return (kSplit && !(item & 1) ? kKeyFull : kFull) + slot(item);
    }
    __device__ static int empty(uint32_t item) {
        return (kSplit && !(item & 1) ? kKeyEmpty : kEmpty) + slot(item);
    }
    __device__ static uint32_t tile(uint32_t item) {
        return kSplit && !(item & 1) ? kOffKeys + slot(item) * kRawTile : kOffRing + slot(item) * kTile;
    }
};

struct TilesArgs {
    AttnProblem p;
    SplitScratch ws;
    int min_steps;       // least length of a share
    int box;             // slots of a TMA box
    int wide_o;          // rows of o lie on 32-byte boundaries
    int q_box;           // queries by TMA: tokens of a half (0: by the helpers)
    CUtensorMap tk, tv;  // [page][head][slot][column] of the caches
    CUtensorMap tq;      // [token][head][column]
};

template <int R>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <typename T>
__device__ __forceinline__ float2 wide16(uint32_t x) {
    if constexpr (std::is_same<T, __half>::value)
        return __half22float2(*reinterpret_cast<const __half2 *>(&x));
    else
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x));
}

__device__ __forceinline__ void cp16z(uint32_t dst, const void *src, bool live) {
    const int bytes = live ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
// Barrier of the helping warps: whether all of them are well.
__device__ __forceinline__ bool help_sync(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

// Two BF16 values of a row that holds an infinity or a NaN: an infinity becomes
// +-1, a NaN stays, anything finite is nothing beside them.
__device__ __forceinline__ uint32_t signs_of_infinities(uint32_t w) {
    uint32_t y = 0;
#pragma unroll
    for (int i = 0; i < 32; i += 16) {
        const uint32_t x = w >> i & 0x7fffu;
        if (x == 0x7f80u) y |= (0x3f80u | (w >> i & 0x8000u)) << i;
        else if (x > 0x7f80u) y |= 0x7fc0u << i;
    }
    return y;
}

// 32 bytes, a whole sector, by one lane (aligned).
__device__ __forceinline__ void store32(void *p, const uint32_t (&x)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]),
                 "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// Instruction descriptor: A and B of type T, A K-major, FP32 sums, M = 128.
// E4M3 operands have FP16's number, E5M2 ones BF16's.
template <typename T>
__host__ __device__ constexpr uint32_t tiles_idesc(int N, int b_mn) {
    const uint32_t f = std::is_same<T, __half>::value ? 0u : 1u;
    return (1u << 4) | (f << 7) | (f << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}

// tcgen05 products and commits for a warp that stays together: every lane goes
// through them and one issues (lead != 0).  The operands are then uniform, and
// the compiler keeps them so; issued from a branch of one lane, each product
// is a dozen instructions more, which beside eight busy warps take longer than
// the product (a product of 64 cycles every 68 cycles, against 290).
__device__ __forceinline__ uint32_t elect_lead() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
                 : "=r"(r));
    return r;
}
// E4M3 operands: 32 columns a product instead of 16.
__device__ __forceinline__ void lead_mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t add, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void lead_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t add, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void lead_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t add, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void lead_commit(uint64_t *bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(lead)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// A row's maximum m to that of a step's scores, its sum l and its output (at
// `to`, where there is one) with it.
template <int D>
__device__ __forceinline__ void rescale(uint32_t to, float mn, float &m, float &l, bool begun) {
    const float n = mn > m + 8.f ? mn : m;  // each row by its own scores alone
    const float c = n == -INFINITY ? 1.f : ex2(m - n);
    m = n;
    l *= c;
    if (!begun) return;
    // O holds the steps before: they are done, as this step's S is
#pragma unroll 1
    for (int q = 0; q < D / 16; ++q) {
        uint32_t o[16];
        tmem_ld16(to + 16 * q, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * c);
        tmem_st16(to + 16 * q, o);
    }
    tmem_wait_st();
}

// Softmax of a wide step, from its S at `ts`: t + log2 s over it, the sum of e^t
// by itself, then the weights, 32 columns at a time (they lie below the columns
// that they come from).  Columns [c0, c1) are seen; gives {m, l}.  Three times the
// other steps' time (1609 us for 4096 new tokens over 16K, all steps wide).  Not
// inlined, and with a tail of its own: in the middle of the softmax's loop it cost
// 4096 new tokens over 16K 30 us of 480 without being run once, so 16.
template <typename TP, int D>
__device__ __noinline__ float2 wide_step(uint32_t ts, uint32_t to, const float *scale, int c0, int c1, float f,
                                         float m, float l, bool begun) {
    const float *lg = scale + kTN + 1;
    float tm = -INFINITY, mn = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < kTN; j0 += 16) {
        uint32_t x[16];
        tmem_ld16(ts + j0, x);
        tmem_wait_ld(x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float t = __uint_as_float(x[e]) * scale[j0 + e] * f;
            const bool see = j0 + e >= c0 && j0 + e < c1;
            const float z = see ? t + lg[j0 + e] : -INFINITY;
            tm = fmaxf(tm, see ? t : -INFINITY);
            mn = fmaxf(mn, z);
            x[e] = __float_as_uint(z);
        }
        tmem_st16(ts + j0, x);
    }
    tmem_wait_st();
    rescale<D>(to, mn, m, l, begun);
    const float mu = m == -INFINITY ? 0.f : m, tu = tm == -INFINITY ? 0.f : tm;
#pragma unroll 1
    for (int j0 = 0; j0 < kTN; j0 += 32) {
        uint32_t ph[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t x[16];
            tmem_ld16(ts + j0 + 16 * h, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float z = __uint_as_float(x[e]);
                // what a row does not see may have no scale
                sum += z == -INFINITY ? 0.f : ex2(z - lg[j0 + 16 * h + e] - tu);
                x[e] = __float_as_uint(ex2(z - mu));
            }
#pragma unroll
            for (int e = 0; e < 16; e += 2)
                ph[8 * h + (e >> 1)] = pack16<TP>(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
        }
        tmem_st16(ts + j0 / 2, ph);
    }
    return make_float2(m, sum == 0.f ? l : l + sum * ex2(tu - mu));
}

template <typename T, int FMT, int D>
__global__ void __launch_bounds__(kTThreads, 1) k_attn_tiles(const __grid_constant__ TilesArgs a) {
    using C = TilesCfg<T, FMT, D>;
    using B = C;  // its barriers
    using TP = typename std::conditional<FMT == 0, T, __half>::type;
    constexpr bool kFold = FMT != 0 && std::is_same<T, __nv_bfloat16>::value;  // values' scales in them
    extern __shared__ uint8_t smem_raw[];
    __shared__ Unit s_unit;
    __shared__ int64_t s_share[3];  // length of the line, workers, where this one's share ends
    __shared__ int64_t s_real[2];   // steps of the call before this worker's, and with them
    __shared__ int s_poison[8];  // unit (count, modulo 8) + 1 whose masked values are not finite
    __shared__ int2 s_piece[8];  // steps and halves of the piece (count, modulo 8), for the products
    __shared__ uint2 s_span[4];          // largest and least scale of a step's values, by warp
    __shared__ uint2 s_ratio[kTN];       // scales in the values: FP16 hi and lo, each twice
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort_flag;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::kOffBar);
    volatile int *s_abort = &s_abort_flag;
    const AttnProblem &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_trigger();
    if (tid == 0) {
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(&bars[B::kFull + i], FMT ? 128 : 1);
            mbar_init(&bars[B::kEmpty + i], 1);
        }
        for (int i = 0; i < C::kLands; ++i) mbar_init(&bars[B::kLand + i], 1);
        for (int i = 0; i < C::kRaw; ++i) mbar_init(&bars[B::kTaken + i], 128);
        for (int i = 0; i < C::kKeys; ++i) {
            mbar_init(&bars[B::kKeyFull + i], 129);  // the keys, and the helpers with their scales
            mbar_init(&bars[B::kKeyEmpty + i], 1);
        }
        mbar_init(&bars[B::kQFull], a.q_box ? 1 : 128);
        mbar_init(&bars[B::kQEmpty], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[B::kS + i], 1);
            mbar_init(&bars[B::kP + i], 128);
            mbar_init(&bars[B::kO + i], 1);
        }
        mbar_init(&bars[B::kDrain], 1);
        mbar_init_fence();
        s_abort_flag = 0;
    }
    if (tid < 8) s_poison[tid] = 0;
    if (warp == 12) tmem_alloc(&s_tmem, 512);
    if (warp < 2) {  // where the share begins, and where it ends
        SplitLine<kTM, kTN, kTUnit> line;
        if (!line.measure(p)) clear_unheld(p, (int64_t)blockIdx.x * 2 + warp, (int64_t)gridDim.x * 2);
        const int64_t total = line.total, w = blockIdx.x;
        int64_t nw = gridDim.x;
        if (nw * a.min_steps > total) nw = quotient(total + a.min_steps - 1, a.min_steps);
        const int64_t at = w < nw ? share_begin(total, w + warp, nw) : total;
        int64_t real = total - kTUnit * line.units;  // of the whole line
        if (at < total) {
            const Unit u = line.locate(p, at, real);
            real += u.step;
            if (warp == 0 && lane == 0) s_unit = u;
        }
        if (lane == 0) {
            s_real[warp] = real;
            if (warp == 1) {
                s_share[0] = total;
                s_share[1] = nw;
                s_share[2] = at;
                a.ws.rec[w] = make_int4(0, 0, 0, 0);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto wait = [&](int b, uint32_t parity) {
        return mbar_wait_or_abort(&bars[b], parity & 1u, p.r.status, s_abort);
    };
    const int count = (int)(s_real[1] - s_real[0]);

    if (count == 0) {
        // no steps for this CTA
    } else if (warp < 8) {
        // ------------------------------------------------------- softmax
        regs_up<kRegSoftmax>();
        Unit u = s_unit;
        const int64_t worker = blockIdx.x;
        const int half = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 lanes a warp, lane << 16
        const uint32_t ts = tmem + lanes + C::kColS + half * 128;
        const uint32_t to = tmem + lanes + C::kColO + half * D;
        uint32_t k = 0, pieces = 0;  // steps and pieces that this half has done
        int left = count, seg = 0;
        for (int done = 0; left > 0; ++seg) {
            const int first = u.step, steps = min(left, u.steps - u.step);
            left -= steps;
            const int rows = unit_rows<kTM>(p, u);
            const bool begun = first == 0, ends = first + steps == u.steps;
            if (half == 0 || rows > 128) {
                const int r = half * 128 + row;
                const bool live = r < rows;
                const int ur = u.tile * kTM + r, tok = p.by_G(ur), hq = u.head * p.G + ur - tok * p.G;
                int lo = 0, hi = 0;
                if (live) visible(p, u.kv, u.kv - u.len + tok, lo, hi);
                float m = -INFINITY, l = 0.f;
                float f = p.scale * kTLog2e;
                bool ok = true;
                for (int s = 0; s < steps; ++s, ++k) {
                    ok = __all_sync(0xffffffffu, wait(B::kS + half, k));
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t sr[4][32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, sr[q]);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 4; ++q) reg_fence(sr[q]);
                    const int base = u.lo + (first + s) * kTN;
                    const float *scale = nullptr;
                    float fs = f, lgs = 0.f, invs = 1.f;  // of the step
                    if constexpr (FMT != 0) {
                        if (s == 0 && kFold)
                            fs = f *= reinterpret_cast<const float *>(sm + C::kOffQf)[(seg & 1) * kTM + r];
                        scale = reinterpret_cast<const float *>(sm + C::kOffScale) + ((done + s) % C::kScales) * 3 * kTN;
                        if constexpr (kFold) {
                            lgs = scale[kTN];
                            invs = scale[2 * kTN + 1];
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 ks = *reinterpret_cast<const float4 *>(scale + q * 32 + e);
                                const float4 lg = kFold ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                        : *reinterpret_cast<const float4 *>(scale + kTN + q * 32 + e);
                                const float2 ff = make_float2(f, f);
                                float2 x = make_float2(__uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1]));
                                float2 y = make_float2(__uint_as_float(sr[q][e + 2]), __uint_as_float(sr[q][e + 3]));
                                x = mul2(x, make_float2(ks.x, ks.y));
                                y = mul2(y, make_float2(ks.z, ks.w));
                                if constexpr (!kFold) {
                                    x = fma2(x, ff, make_float2(lg.x, lg.y));
                                    y = fma2(y, ff, make_float2(lg.z, lg.w));
                                }
                                sr[q][e] = __float_as_uint(x.x);
                                sr[q][e + 1] = __float_as_uint(x.y);
                                sr[q][e + 2] = __float_as_uint(y.x);
                                sr[q][e + 3] = __float_as_uint(y.y);
                                // no more than eight columns' loads ahead: the
                                // registers are full of scores
                                if (e & 4) asm volatile("" ::: "memory");
                            }
                    }
                    const bool masked = __any_sync(0xffffffffu, base < lo || base + kTN > hi);
                    if (masked) {
                        const int c0 = lo - base, c1 = hi - base;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (q * 32 + e < c0 || q * 32 + e >= c1) sr[q][e] = 0xff800000u;
                    }
                    float mx[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        mx[q] = max3(__uint_as_float(sr[q][0]), __uint_as_float(sr[q][1]),
                                     __uint_as_float(sr[q][2]));
#pragma unroll
                        for (int e = 3; e + 1 < 32; e += 2)
                            mx[q] = max3(mx[q], __uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1]));
                        mx[q] = fmaxf(mx[q], __uint_as_float(sr[q][31]));
                    }
                    float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if constexpr (FMT == 0 || kFold) mn = mn == -INFINITY ? mn : fmaf(mn, fs, lgs);
                    if (__any_sync(0xffffffffu, mn > m + 8.f)) {
                        if (kFold && lgs == kTWide) {
                            const float2 ml = wide_step<TP, D>(ts, to, scale, lo - base, hi - base, f, m, l, s > 0);
                            m = ml.x;
                            l = ml.y;
                            tmem_wait_st();
                            tc_fence_before();
                            mbar_arrive(&bars[B::kP + half]);
                            continue;
                        }
                        rescale<D>(to, mn, m, l, s > 0);
                    }
                    const float mu = m == -INFINITY ? 0.f : m;
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    const float2 ff = make_float2(fs, fs), nm = make_float2(lgs - mu, lgs - mu);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t ph[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 x = make_float2(__uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1]));
                            if constexpr (FMT == 0 || kFold) x = fma2(x, ff, nm);
                            else x = add2(x, nm);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            if constexpr (FMT == 0 || kFold) {
                                sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], x);
                            } else {
                                float2 iv = *reinterpret_cast<const float2 *>(scale + 2 * kTN + q * 32 + e);
                                if (masked) {  // what a row does not see may have no scale
                                    if (x.x == 0.f) iv.x = 0.f;
                                    if (x.y == 0.f) iv.y = 0.f;
                                }
                                sum[(e >> 1) & 1] = fma2(x, iv, sum[(e >> 1) & 1]);
                            }
                            ph[e >> 1] = pack16<TP>(x.x, x.y);
                        }
                        tmem_st16(ts + 16 * q, ph);
                    }
                    sum[0] = add2(sum[0], sum[1]);
                    l = fmaf(sum[0].x + sum[0].y, invs, l);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&bars[B::kP + half]);
                }
                if (!ok) break;
                // ------------------------------------------- the piece ends
                ok = __all_sync(0xffffffffu, wait(B::kO + half, pieces++));
                if (!ok) break;
                tc_fence_after();
                if ((FMT == 0 || kFold) && s_poison[seg & 7] == seg + 1) {
                    // values that are not finite at masked positions went in
                    // as zeros: add them to the rows that see them
#pragma unroll 1
                    for (int q = 0; q < D / 16; ++q) {
                        uint32_t o[16];
                        tmem_ld16(to + 16 * q, o);
                        tmem_wait_ld(o);
#pragma unroll 1
                        for (int s = first; s < first + steps; ++s) {
                            const int base = u.lo + s * kTN;
                            if (!step_masked<kTN>(u, base)) continue;
#pragma unroll 1
                            for (int j = max(base, lo); j < min(base + kTN, hi); ++j) {
                                const int page = page_of(p.c, u.n, p.by_page(j), p.r.status);
                                if (page < 0) continue;
                                const int at = j - p.by_page(j) * p.c.page_size;
                                if constexpr (FMT == 0) {
                                    const T *v = reinterpret_cast<const T *>(p.c.v) +
                                                 page_at(p.c.vst, page, at, u.head) + 16 * q;
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const float x = (float)v[e];
                                        if (!isfinite(x)) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
                                    }
                                } else if (!isfinite(p.c.vs[scale_at(p.c, page, at, u.head)])) {
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = 0x7fc00000u;
                                }
                            }
                        }
                        __syncwarp();
                        tmem_st16(to + 16 * q, o);
                    }
                    tmem_wait_st();
                }
                const bool whole = begun && ends;
                const bool empty = l == 0.f;
                const float inv = whole ? (empty ? 0.f : 1.f / l) : 1.f;
                T *o16 = reinterpret_cast<T *>(p.o) + (live ? tok_at(p.so, u.t0 + tok, hq) : 0);
                const int64_t slot = (worker * 2 + (begun ? 1 : 0)) * kTM + r;
                // not unrolled: this runs once a unit, and code that is not in the
                // instruction cache costs as much as what it does
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {
                    uint32_t o[16];
                    tmem_ld16(to + 16 * q, o);
                    tmem_wait_ld(o);
                    if (live && whole) {
                        uint32_t x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            x[e] = pack16<T>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                        if (a.wide_o) {
                            store32(o16 + 16 * q, x);
                        } else {
                            reinterpret_cast<uint4 *>(o16 + 16 * q)[0] = make_uint4(x[0], x[1], x[2], x[3]);
                            reinterpret_cast<uint4 *>(o16 + 16 * q)[1] = make_uint4(x[4], x[5], x[6], x[7]);
                        }
                    } else if (live) {
                        store32(a.ws.o + slot * D + 16 * q, *reinterpret_cast<const uint32_t(*)[8]>(&o[0]));
                        store32(a.ws.o + slot * D + 16 * q + 8, *reinterpret_cast<const uint32_t(*)[8]>(&o[8]));
                    }
                }
                tc_fence_before();  // O is read before the next unit's first product is let go
                if (live && whole && p.lse)
                    p.lse[(int64_t)(u.t0 + tok) * p.Hq + hq] =
                        empty ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kTLn2;
                if (live && !whole) {
                    a.ws.ml[slot * 2] = m;
                    a.ws.ml[slot * 2 + 1] = l;
                }
            }
            done += steps;
            if (begun && !ends && tid == 0) {
                const int pieces = pieces_from(s_share[0], worker, s_share[1],
                                               s_share[2] + (u.steps - first - steps));
                a.ws.rec[worker] = make_int4(u.head << 16 | pieces, u.t0, u.len, u.tile);
            }
            if (left) next_unit<kTM, kTN>(p, u);
        }
    } else if (warp < 12) {
        // ------------------------------------------------------- helpers
        regs_down<kRegHelp>();
        Unit u = s_unit;
        const int t = tid - 256;
        bool ok = true;
        int seg = 0;
        uint32_t item = 0, landed = 0;
        auto queries = [&]() {
            ok = __all_sync(0xffffffffu, wait(B::kQEmpty, (uint32_t)seg + 1));
            if (!ok) return;
            const int rows = unit_rows<kTM>(p, u);
            constexpr int kQC = D / 8, kQP = 128 / kQC;  // chunks a row, rows a pass
            const int qc = t % kQC, halves = rows > 128 ? 2 : 1;
            float *qf = reinterpret_cast<float *>(sm + C::kOffQf) + (seg & 1) * kTM;
            constexpr bool kConvert = FMT != 0 && std::is_same<T, __nv_bfloat16>::value;
            // rows in steps of kQP from this thread's first: token and head move
            // by the same amounts
            const int dt = p.by_G(kQP), dh = kQP - dt * p.G;
            int tok = p.by_G(u.tile * kTM + t / kQC), hq = u.tile * kTM + t / kQC - tok * p.G;
            auto place = [&](int r, const T *&src) {  // whether the unit has the row, and where
                const bool live = r < rows;
                src = reinterpret_cast<const T *>(p.q) +
                      (live ? tok_at(p.sq, u.t0 + tok, u.head * p.G + hq) + qc * 8 : 0);
                tok += dt;
                hq += dh;
                if (hq >= p.G) {
                    hq -= p.G;
                    ++tok;
                }
                return live;
            };
            auto dst = [&](int r) { return (r >> 7) * C::kQTile + sw128_chunk(r & 127, qc, 128); };
            if constexpr (kConvert) {
                // FP16 of the row's own power of two (see attn_rows.cu), or the
                // parts of it, two rows at a time (4096 tokens over 16K in E4M3:
                // 507 us; four rows 513, eight 542)
                const uint32_t first8 = sw128_chunk(t / kQC, qc >> 1, 128) + (qc & 1) * 8;
#pragma unroll 1
                for (int r0 = t / kQC; r0 < 128 * halves; r0 += 2 * kQP) {
                    uint4 x[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const T *src;
                        const bool live = place(r0 + i * kQP, src);
                        x[i] = live ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                        // the largest magnitude's bits: they are in its order
                        uint32_t big = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                                __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
#pragma unroll
                        for (int d = 1; d < kQC; d <<= 1)
                            big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, d));
                        big = max(big & 0xffffu, big >> 16);
                        const int ex = (int)(big >> 7), r = r0 + i * kQP;
                        float back;
                        if constexpr (C::kSplit) {
                            // the largest magnitude into [2^14, 2^15); a row with an
                            // infinity is its infinities' signs, times infinity
                            const int at = max(ex, 15);
                            float g = __int_as_float((268 - at) << 23);
                            back = __int_as_float((at - 14) << 23);
                            if (__any_sync(0xffffffffu, ex == 255)) {
                                g = ex == 255 ? 1.f : g;
                                back = ex == 255 ? INFINITY : back;
#pragma unroll
                                for (int e = 0; e < 4; ++e) w[e] = ex == 255 ? signs_of_infinities(w[e]) : w[e];
                            }
                            // FP16 holds what the parts do, and E5M2 is its upper byte
                            uint32_t h[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                h[e] = pack16<__half>(__uint_as_float(w[e] << 16) * g,
                                                      __uint_as_float(w[e] & 0xffff0000u) * g);
                            // first the 128 columns of the first part, then the next's;
                            // the swizzle is that of the thread's first row
                            uint8_t *to = sm + first8 + (r >> 7) * C::kQTile + (r & 127) / 8 * 1024;
#pragma unroll
                            for (int i = 0; i < 3; ++i) {
                                *reinterpret_cast<uint2 *>(to + i * 16384) =
                                    make_uint2(__byte_perm(h[0], h[1], 0x7531), __byte_perm(h[2], h[3], 0x7531));
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t top = h[e] & 0xff00ff00u;
                                    const __half2 left = __hsub2(*reinterpret_cast<const __half2 *>(&h[e]),
                                                                 *reinterpret_cast<const __half2 *>(&top));
                                    h[e] = *reinterpret_cast<const uint32_t *>(&left);
                                }
                            }
                        } else {
                            const bool normal = ex > 0 && ex < 254;
                            const float g = normal ? __int_as_float((254 - ex) << 23) : 1.f;
                            back = normal ? __int_as_float(ex << 23) : 1.f;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack16<__half>(__uint_as_float(w[e] << 16) * g,
                                                      __uint_as_float(w[e] & 0xffff0000u) * g);
                            *reinterpret_cast<uint4 *>(sm + dst(r)) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        if (qc == 0) qf[r] = back;
                    }
                }
            } else {
#pragma unroll 8
                for (int r = t / kQC; r < 128 * halves; r += kQP) {
                    const T *src;
                    const bool live = place(r, src);
                    cp16z(sb + dst(r), src, live);
                }
            }
            if constexpr (!kConvert) asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            mbar_arrive(&bars[B::kQFull]);
        };
        // a warp that gives up says so at the next barrier of the others, the
        // last of which is at the end; one that has heard it comes to none
        bool heard = false;
        auto together = [&]() {
            ok = help_sync(ok);
            heard = !ok;
            return ok;
        };
        for (int it = 0; it < count && ok; ++it) {
            if (!together()) break;
            if (it > 0 && u.step == 0) ++seg;
            if (!a.q_box && (it == 0 || u.step == 0)) queries();
            const int base = u.lo + u.step * kTN, left = u.hi - base;  // positions of the step
            if constexpr (FMT == 0) {
                const int b = (item + 1) % C::kRing;
                item += 2;
                if (ok && step_masked<kTN>(u, base)) {
                    ok = __all_sync(0xffffffffu, wait(B::kLand + b, landed >> b));
                    landed ^= 1u << b;
                    if (ok) {
                        constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
                        uint8_t *tile = sm + C::kOffRing + b * C::kTile;
                        bool bad = false;
#pragma unroll 4
                        for (int i = t; i < kTN * D / 8; i += 128) {
                            const int r = i / (D / 8);
                            uint4 *w4 = reinterpret_cast<uint4 *>(tile + sw128_chunk(r, i % (D / 8), kTN));
                            if (r >= left) {
                                *w4 = make_uint4(0, 0, 0, 0);
                                continue;
                            }
                            uint4 x = *w4;
                            // a half word whose exponent is all ones, less
                            // the ones below: its top bit is set by the borrow
                            auto odd = [](uint32_t y) {
                                y = (y & (kExp | kExp << 16)) ^ (kExp | kExp << 16);
                                return (y - 0x00010001u) & ~y & 0x80008000u;
                            };
                            if (!(odd(x.x) | odd(x.y) | odd(x.z) | odd(x.w))) continue;
                            uint32_t *w = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t y = w[e];
                                const bool b0 = (y & kExp) == kExp, b1 = (y >> 16 & kExp) == kExp;
                                w[e] = (b0 ? 0u : y & 0xffffu) | (b1 ? 0u : y & 0xffff0000u);
                                bad |= b0 || b1;
                            }
                            *w4 = x;
                        }
                        if (bad) s_poison[seg & 7] = seg + 1;
                        fence_async_smem();
                    }
                    if (!ok || !together()) break;
                    if (t == 0) mbar_arrive(&bars[B::kFull + b]);
                }
            } else {
                constexpr int kChunks = D / 16, kPass = 128 / kChunks, kPasses = kTN / kPass;
                const int ch = t % kChunks, r0 = t / kChunks;
                const bool masked = step_masked<kTN>(u, base);
                for (int kv = C::kSplit ? 1 : 0; kv < 2 && ok; ++kv, ++item) {
                    // scales come with the first 8-bit tile of a step
                    const bool scales = C::kSplit || kv == 0;
                    const uint32_t tile_item = C::kSplit ? 2 * item + 1 : item;
                    const int w = item % C::kRaw;
                    const uint8_t *raw = sm + C::kOffRaw + w * C::kRawSize;
                    ok = __all_sync(0xffffffffu, wait(B::kLand + w, item / C::kRaw));
                    if (!ok) break;
                    float ks = 0.f, vs = kFold ? 0.f : 1.f;
                    if (scales && t < left) {
                        ks = reinterpret_cast<const float *>(raw + C::kRawTile)[t];
                        vs = reinterpret_cast<const float *>(raw + C::kRawTile)[kTN + t];
                    }
                    if (!C::kSplit) {
                        ok = __all_sync(0xffffffffu, wait(C::empty(tile_item), C::turns(tile_item) + 1));
                        if (!ok) break;
                    }
                    if (kFold && scales) {
                        // the span of the values' scales, and every row's part of
                        // the largest (rows of zeros and rows without a scale aside)
                        const bool some = vs > 0.f && isfinite(vs);
                        const uint32_t bits = __float_as_uint(vs);  // in their values' order
                        const uint32_t most = __reduce_max_sync(0xffffffffu, some ? bits : 0u);
                        const uint32_t least = __reduce_min_sync(0xffffffffu, some ? bits : 0x7f800000u);
                        if (lane == 0) s_span[warp - 8] = make_uint2(most, least);
                        float *sc = reinterpret_cast<float *>(sm + C::kOffScale) + (it % C::kScales) * 3 * kTN;
                        sc[t] = ks;
                        if (!together()) break;
                        const uint2 s0 = s_span[0], s1 = s_span[1], s2 = s_span[2], s3 = s_span[3];
                        const uint32_t vm = max(max(s0.x, s1.x), max(s2.x, s3.x));
                        const float vl = __uint_as_float(min(min(s0.y, s1.y), min(s2.y, s3.y)));
                        // s' = 2^(at - 127): the largest, rounded up to a power of
                        // two, over 2^7; 2^-100 at least, so that 1 / s' leaves room
                        const int at = max((int)(vm >> 23) - 6, 27);
                        const float inv = __int_as_float((254 - at) << 23);
                        float part = vs * inv, lgs = (float)(at - 127), invs = inv;
                        if (__builtin_expect(vl * inv < kTNarrow, 0)) {  // wide
                            sc[kTN + 1 + t] = __log2f(weighed_scale(vs));
                            part = fminf(vs * 0x1p100f, 1.f);  // what 2^-100 leaves of smaller ones
                            lgs = kTWide;
                            invs = 0.f;
                        }
                        if (t == 0) {
                            sc[kTN] = lgs;
                            sc[2 * kTN + 1] = invs;
                        }
                        const __half2 hi = __float2half2_rn(part);
                        const __half2 lo = __float2half2_rn(part - __low2float(hi));
                        s_ratio[t] = make_uint2(*reinterpret_cast<const uint32_t *>(&hi),
                                                *reinterpret_cast<const uint32_t *>(&lo));
                        if (C::kSplit) mbar_arrive(&bars[C::full(2 * item)]);
                        if (!together()) break;
                    }
                    if (C::kSplit) {
                        ok = __all_sync(0xffffffffu, wait(C::empty(tile_item), C::turns(tile_item) + 1));
                        if (!ok) break;
                    }
                    if (!kFold && scales) {
                        float *sc = reinterpret_cast<float *>(sm + C::kOffScale) + (it % C::kScales) * 3 * kTN;
                        const float v = weighed_scale(vs);
                        sc[t] = ks;
                        sc[kTN + t] = __log2f(v);
                        sc[2 * kTN + t] = __fdividef(1.f, v);
                    }
                    uint8_t *tile = sm + C::tile(tile_item);
#pragma unroll 4
                    for (int i = 0; i < kPasses; ++i) {
                        const int r = r0 + i * kPass;
                        uint4 x = *reinterpret_cast<const uint4 *>(raw + r * D + ch * 16), e0, e1;
                        if (r >= left) x = make_uint4(0, 0, 0, 0);  // past the end: anything
                        widen4<FMT>(x.x, e0.x, e0.y);
                        widen4<FMT>(x.y, e0.z, e0.w);
                        widen4<FMT>(x.z, e1.x, e1.y);
                        widen4<FMT>(x.w, e1.z, e1.w);
                        if (kFold && kv) {  // times hi + lo, rounded once
                            const uint2 ra = s_ratio[r];
                            const __half2 hi = *reinterpret_cast<const __half2 *>(&ra.x);
                            const __half2 lo = *reinterpret_cast<const __half2 *>(&ra.y);
                            // a value row without a scale, in a step that some
                            // rows see a part of: added at the end
                            const bool out = masked && __hisnan(__low2half(hi));
                            if (out) s_poison[seg & 7] = seg + 1;
                            uint32_t *w[8] = {&e0.x, &e0.y, &e0.z, &e0.w, &e1.x, &e1.y, &e1.z, &e1.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const __half2 y = *reinterpret_cast<const __half2 *>(w[e]);
                                const __half2 z = __hfma2(y, hi, __hmul2(y, lo));
                                *w[e] = out ? 0u : *reinterpret_cast<const uint32_t *>(&z);
                            }
                        }
                        // odd chunks first in the upper columns: the two
                        // column blocks lie on the same banks
                        const bool odd = ch >= kChunks / 2 && D == 128;
                        *reinterpret_cast<uint4 *>(tile + sw128_chunk(r, 2 * ch + (odd ? 1 : 0), kTN)) = odd ? e1 : e0;
                        *reinterpret_cast<uint4 *>(tile + sw128_chunk(r, 2 * ch + (odd ? 0 : 1), kTN)) = odd ? e0 : e1;
                    }
                    mbar_arrive(&bars[B::kTaken + w]);
                    fence_async_smem();
                    mbar_arrive(&bars[C::full(tile_item)]);
                }
            }
            if (it + 1 < count && ++u.step == u.steps) next_unit<kTM, kTN>(p, u);
        }
        if (!heard) help_sync(ok);
    } else {
        regs_down<kRegRest>();
        if (warp == 12) {
            // -------------------------------------------------- products
            // loops and conditions go by votes, so that they are uniform
            constexpr uint32_t kIdS = tiles_idesc<TP>(128, 0) | (C::kSplit ? 1u << 7 : 0u);  // E5M2 times E4M3
            constexpr uint32_t kIdO = tiles_idesc<TP>(D, 1);
            const uint32_t lead = elect_lead();
            auto all_wait = [&](int b, uint32_t parity) {
                return (bool)__all_sync(0xffffffffu, wait(b, parity));
            };
            // descriptors as a base plus a constant for each product: the
            // address is their low 14 bits, in units of 16 bytes
            const uint64_t dk0 = sdesc_sw128(sb, 16, 1024), dv0 = sdesc_sw128(sb, 16384, 1024);
            auto score = [&](int half, uint32_t i) {
                const uint64_t q = dk0 + half * (C::kQTile >> 4);
                const uint64_t kt = dk0 + (C::tile(i) >> 4);
                if constexpr (C::kSplit) {  // the parts one by one, with the same keys
#pragma unroll
                    for (int d = 0; d < 12; ++d)
                        lead_mma8(tmem + C::kColS + half * 128, q + (((d >> 2) * 16384 + (d & 3) * 32) >> 4),
                                  kt + (((d & 3) * 32) >> 4), kIdS, d > 0, lead);
                } else {
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        const uint64_t o = ((d >> 2) * 16384 + (d & 3) * 32) >> 4;
                        lead_mma(tmem + C::kColS + half * 128, q + o, kt + o, kIdS, d > 0, lead);
                    }
                }
                lead_commit(&bars[B::kS + half], lead);
            };
            auto gather = [&](int half, uint32_t i, uint32_t add) {
                const uint64_t vt = dv0 + (C::tile(i) >> 4);
#pragma unroll
                for (int j = 0; j < kTN / 16; ++j)
                    lead_mma_ts(tmem + C::kColO + half * D, tmem + C::kColS + half * 128 + 8 * j,
                                vt + ((j * 2048) >> 4), kIdO, j ? 1u : add, lead);
            };
            // the keys of item 2 k, and with them the values before, are done
            auto release_k = [&](uint32_t i) {
                if constexpr (C::kPairs > 0) lead_commit(&bars[B::kEmpty + (i >> 1) % C::kPairs], lead);
                else lead_commit(&bars[C::empty(i)], lead);
            };
            uint32_t item = 0, kp0 = 0, kp1 = 0, seg = 0;
            int left = count;
            bool ok = true;
            while (ok && __any_sync(0xffffffffu, left > 0)) {
                ok = all_wait(C::full(item), C::turns(item)) && all_wait(B::kQFull, seg);
                if (!ok) break;
                tc_fence_after();
                const int steps = s_piece[seg & 7].x;
                const bool two = __any_sync(0xffffffffu, s_piece[seg & 7].y == 2);
                ++seg;
                left -= steps;
                score(0, item);
                if (two) score(1, item);
                release_k(item);
                uint32_t add = 0;
                for (int s = 1;; ++s) {
                    const bool more = __any_sync(0xffffffffu, s < steps);
                    if (!more) lead_commit(&bars[B::kQEmpty], lead);
                    const uint32_t iv = item + 1, ik = item + 2;
                    ok = all_wait(C::full(iv), C::turns(iv));
                    if (ok && more) ok = all_wait(C::full(ik), C::turns(ik));
                    ok = ok && all_wait(B::kP, kp0++);
                    if (!ok) break;
                    tc_fence_after();
                    gather(0, iv, add);
                    if (more) score(0, ik);
                    else lead_commit(&bars[B::kO], lead);
                    if (two) {
                        ok = all_wait(B::kP + 1, kp1++);
                        if (!ok) break;
                        tc_fence_after();
                        gather(1, iv, add);
                        if (C::kPairs == 0) lead_commit(&bars[C::empty(iv)], lead);
                        if (more) score(1, ik);
                        else lead_commit(&bars[B::kO + 1], lead);
                    } else if (C::kPairs == 0) {
                        lead_commit(&bars[C::empty(iv)], lead);
                    }
                    if (more) release_k(item + 2);
                    item += 2;
                    add = 1;
                    if (!more) break;
                }
            }
        }
        __syncwarp();
        if (warp == 13) {
            // ----------------------------------------------------- loads
            Unit u = s_unit;
            const int box = a.box, boxes = kTN / box;
            // the page-table entry and slot of this lane's box of the step that
            // is loaded next, asked for a step ahead
            int entry = -1, slot = 0;
            bool asked = false;
            auto look_up = [&]() {
                const int pos = u.lo + u.step * kTN + lane * box;
                asked = lane < boxes && pos < u.hi;
                if (asked) {
                    const int pi = p.by_page(pos);
                    slot = pos - pi * p.c.page_size;
                    entry = p.c.table[u.n * p.c.max_pages + pi];
                }
            };
            uint32_t item = 0, seg = 0, landed = 0;  // landed: by tile, whether kLand has had an odd number
            bool ok = true;
            look_up();
            for (int it = 0; it < count && ok; ++it) {
                const bool first = it == 0 || u.step == 0;
                if (first && lane == 0)
                    s_piece[seg & 7] = make_int2(min(count - it, u.steps - u.step),
                                                 unit_rows<kTM>(p, u) > 128 ? 2 : 1);
                // a page past the cache reads as zeros
                const bool here = asked && (unsigned)entry < (unsigned)p.c.n_pages;
                if (asked && !here) report(p.r.status, GDR_ERR_INDEX);
                const int pg = here ? entry : p.c.n_pages, sl = here ? slot : 0, head = u.head;
                const bool masked = FMT == 0 && step_masked<kTN>(u, u.lo + u.step * kTN);
                constexpr int kScaled = C::kSplit ? 1 : 0;  // the scales come with the keys or the values
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++item) {
                    const CUtensorMap *map = kv ? &a.tv : &a.tk;
                    int bar;
                    uint32_t dst, bytes;
                    if constexpr (FMT == 0) {
                        const int b = item % C::kRing;
                        // values s and keys s + 1 go into the tiles of values
                        // s - kPairs and keys s + 1 - kPairs
                        const int e = (int)((item + 1) >> 1) - C::kPairs;
                        if (e >= 0) ok = __all_sync(0xffffffffu, wait(B::kEmpty + e % C::kPairs, e / C::kPairs));
                        bar = kv && masked ? B::kLand + b : B::kFull + b;
                        landed ^= (uint32_t)(kv && masked) << b;
                        dst = C::kOffRing + b * C::kTile;
                        bytes = C::kTile;
                    } else if (C::kSplit && kv == 0) {
                        ok = __all_sync(0xffffffffu, wait(C::empty(item), C::turns(item) + 1));
                        bar = C::full(item);
                        dst = C::tile(item);
                        bytes = C::kRawTile;
                    } else {
                        const uint32_t i = C::kSplit ? item >> 1 : item;
                        const int w = i % C::kRaw;
                        ok = __all_sync(0xffffffffu, wait(B::kTaken + w, i / C::kRaw + 1));
                        bar = B::kLand + w;
                        dst = C::kOffRaw + w * C::kRawSize;
                        bytes = C::kRawTile;
                        if (kv == kScaled) bytes += __popc(__ballot_sync(0xffffffffu, here)) * box * 8;
                    }
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&bars[bar], bytes);
                    __syncwarp();
                    if (lane < boxes) {
                        if constexpr (FMT == 0) {
#pragma unroll
                            for (int c = 0; c < D / 64; ++c)
                                tma_page(sb + dst + c * 16384 + lane * box * 128, map, &bars[bar],
                                            c * 64, sl, head, pg);
                        } else {
                            tma_page(sb + dst + lane * box * D, map, &bars[bar], 0, sl, head, pg);
                            if (kv == kScaled && here) {
                                const int64_t so = scale_at(p.c, pg, sl, head);
                                uint8_t *sc = sm + dst + C::kRawTile + lane * box * 4;
                                bulk_load(sc, p.c.ks + so, box * 4, &bars[bar]);
                                bulk_load(sc + kTN * 4, p.c.vs + so, box * 4, &bars[bar]);
                            }
                        }
                    }
                    if (first && kv == 0 && a.q_box) {
                        // rows past the unit's are those of other tokens, or
                        // zeros; they see nothing
                        ok = __all_sync(0xffffffffu, wait(B::kQEmpty, seg + 1));
                        if (!ok) {
                            ++item;  // it is on its way
                            break;
                        }
                        const int halves = unit_rows<kTM>(p, u) > 128 ? 2 : 1;
                        if (lane == 0) mbar_arrive_expect_tx(&bars[B::kQFull], halves * C::kQTile);
                        __syncwarp();
                        if (lane < halves * (D / 64)) {
                            const int h = lane / (D / 64), c = lane % (D / 64);
                            tma_load_3d(sm + h * C::kQTile + c * 16384, &a.tq, &bars[B::kQFull], c * 64,
                                        u.head * p.G, u.t0 + (u.tile * 2 + h) * a.q_box);
                        }
                    }
                }
                seg += first;
                if (it + 1 < count) {
                    if (++u.step == u.steps) next_unit<kTM, kTN>(p, u);
                    look_up();
                }
            }
            // Whether or not anybody still waits for them, the loads land before the
            // memory goes back: the last turn of every barrier (turn -1, of one not
            // used, is over).  10 ms, as a turn may need others who gave up.
            auto land = [&](int bar, uint32_t turns) { mbar_wait(&bars[bar], (turns - 1) & 1u, nullptr, 10000000ull); };
            auto used = [](uint32_t n, uint32_t i, uint32_t of) { return (n + of - 1 - i) / of; };  // i < of
            if (FMT == 0 && lane < C::kRing) {
                land(B::kFull + lane, used(item, lane, C::kRing));
                land(B::kLand + lane, landed >> lane);
            }
            if (FMT != 0 && lane < C::kRaw)
                land(B::kLand + lane, used(C::kSplit ? item >> 1 : item, lane, C::kRaw));
            if (C::kSplit && lane < C::kKeys) land(B::kKeyFull + lane, used((item + 1) >> 1, lane, C::kKeys));
            if (a.q_box && lane == 0) land(B::kQFull, seg);
        }
        if (warp == 12 && lane == 0) {  // nothing is in flight when the memory goes back
            umma_commit(&bars[B::kDrain]);
            mbar_wait(&bars[B::kDrain], 0, p.r.status);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) {
        tmem_relinquish();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int FMT, int D>
cudaError_t launch_tiles(const AttnProblem &p, const SplitScratch &ws, int ctas, cudaStream_t st) {
    using C = TilesCfg<T, FMT, D>;
    TilesArgs a{p, ws, 1, p.align};
    a.wide_o = ((reinterpret_cast<uintptr_t>(p.o) | (uintptr_t)(p.so.t * 2) | (uintptr_t)(p.so.h * 2)) & 31u) == 0;
    if (!page_map(&a.tk, p, p.c.k, p.c.kst, D, a.box, C::kSplit ? kPageSwizzled : kPagePlain) ||
        !page_map(&a.tv, p, p.c.v, p.c.vst, D, a.box, kPagePlain))
        return cudaErrorInvalidValue;
    // a half's rows are whole tokens: its queries are one box of 128 / G
    // tokens by G heads
    constexpr bool kConvert = FMT != 0 && std::is_same<T, __nv_bfloat16>::value;
    if (!kConvert && p.G <= 128 && 128 % p.G == 0) {
        auto enc = tensor_map_encoder();
        const uint64_t tokens = rows_packed(p.r) ? p.r.T : p.r.N * p.r.T;
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)tokens};
        const cuuint64_t strides[2] = {(cuuint64_t)p.sq.h * 2, (cuuint64_t)p.sq.t * 2};
        const cuuint32_t bx[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(128 / p.G)}, one[3] = {1, 1, 1};
        if (enc(&a.tq, p.dtype == GDR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                3, const_cast<void *>(p.q), dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
            a.q_box = 128 / p.G;
    }
    auto k = k_attn_tiles<T, FMT, D>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_a_device(done, [&] {
        cudaFuncAttributes at;
        const cudaError_t x = cudaFuncGetAttributes(&at, k);
        if (x != cudaSuccess) return x;
        // the split of the registers draws on what the launch holds
        if (at.numRegs * 4 < 2 * kRegSoftmax + kRegHelp + kRegRest) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
    });
    if (e != cudaSuccess) return e;
    k<<<ctas, kTThreads, C::kBytes, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_fmt(const AttnProblem &p, const SplitScratch &ws, int ctas, cudaStream_t st) {
    if (p.c.dtype == GDR_E4M3) return launch_tiles<T, 1, D>(p, ws, ctas, st);
    if (p.c.dtype == GDR_I8) return launch_tiles<T, 2, D>(p, ws, ctas, st);
    return launch_tiles<T, 0, D>(p, ws, ctas, st);
}

template <typename T>
cudaError_t launch_dim(const AttnProblem &p, const SplitScratch &ws, int ctas, cudaStream_t st) {
    return p.K == 64 ? launch_fmt<T, 64>(p, ws, ctas, st) : launch_fmt<T, 128>(p, ws, ctas, st);
}

}  // namespace

SplitPlan attn_tiles_plan(const AttnProblem &p) {
    SplitPlan s{};
    const int g = device_sms();
    s.ctas = p.grid_limit > 0 && p.grid_limit < g ? p.grid_limit : g;
    s.workers = s.ctas;
    s.rows = kTM;
    return s;
}

// Boxes of 8 slots and more, and scales on 16-byte boundaries.
bool attn_tiles_supported(const AttnProblem &p) {
    return attn_rows_supported(p) && p.c.page_size % 8 == 0 && scales_aligned16(p.c);
}

cudaError_t attn_tiles(const AttnProblem &p, const SplitScratch &ws, const SplitPlan &s,
                       cudaStream_t st) {
    return p.dtype == GDR_F16 ? launch_dim<__half>(p, ws, s.ctas, st)
                              : launch_dim<__nv_bfloat16>(p, ws, s.ctas, st);
}

}  // namespace gdr
