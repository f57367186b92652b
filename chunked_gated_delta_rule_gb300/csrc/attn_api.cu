// attn_api.cu -- host side of the paged cache and of the attention over it:
// argument checks, choice of kernel, scratch, launches.
#include <cmath>

#include "attn_split.cuh"
#include "gdr_launch.cuh"

namespace gdr {
namespace {

constexpr int64_t kMaxPagedV = 256;

// The cache against the call's sizes.  `heads` is what the call's k and v
// have (the cache's own), or its query heads, a multiple of the cache's.
int check_cache(const gdr_dims &d, const gdr_paged_cache *c, bool attention) {
    if (!c || !c->k || !c->v || !c->page_table || !c->kv_lens) return GDR_ERR_INVALID;
    if (c->n_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->H < 1) return GDR_ERR_INVALID;
    const bool quant = cache_quantised(c->dtype);
    if (!quant && c->dtype != d.dtype) return GDR_ERR_INVALID;
    if (quant && (!c->k_scale || !c->v_scale)) return GDR_ERR_INVALID;
    if (attention ? d.H % c->H != 0 : d.H != c->H) return GDR_ERR_INVALID;
    for (const int64_t *s : {c->k_stride, c->v_stride}) {
        const int zeros = (s[0] == 0) + (s[1] == 0) + (s[2] == 0);
        if ((zeros != 0 && zeros != 3) || s[0] < 0 || s[1] < 0 || s[2] < 0) return GDR_ERR_INVALID;
    }
    if (d.V > kMaxPagedV) return GDR_ERR_UNSUPPORTED;
    if (c->n_pages > INT32_MAX || c->page_size > INT32_MAX || c->H > 65535 ||
        c->max_pages > INT32_MAX / c->page_size)
        return GDR_ERR_UNSUPPORTED;  // positions fit 31 bits
    // those of the attention's steps as well, which pass the last by up to 127
    if (attention && c->max_pages > (INT32_MAX - 1023) / c->page_size) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

int64_t seqs_of(const gdr_dims &d) { return d.N > 0 ? d.N : d.B; }

PagedCache device_cache(const gdr_dims &d, const gdr_paged_cache &c) {
    PagedCache p{};
    p.k = c.k; p.v = c.v; p.ks = c.k_scale; p.vs = c.v_scale;
    p.table = c.page_table; p.kv_lens = c.kv_lens;
    p.max_pages = c.max_pages;
    p.n_pages = (int32_t)c.n_pages; p.page_size = (int32_t)c.page_size;
    p.H = (int32_t)c.H; p.dtype = c.dtype;
    for (int i = 0; i < 3; ++i) {
        const int64_t dk[3] = {c.page_size * c.H * d.K, c.H * d.K, d.K};
        const int64_t dv[3] = {c.page_size * c.H * d.V, c.H * d.V, d.V};
        p.kst[i] = c.k_stride[0] ? c.k_stride[i] : dk[i];
        p.vst[i] = c.v_stride[0] ? c.v_stride[i] : dv[i];
    }
    return p;
}

TokenRows token_rows(const gdr_dims &d, const int32_t *cu, int32_t *status) {
    TokenRows r{};
    if (cu && (d.flags & GDR_SEQLENS_I64)) r.cu64 = reinterpret_cast<const int64_t *>(cu);
    else r.cu = cu;
    r.N = seqs_of(d);
    r.T = d.T;
    r.status = status;
    return r;
}

int cache_call(bool write, const gdr_dims *dims, const gdr_paged_cache *cache, const void *k,
               const void *v, const int32_t *cu, int32_t *status, gdr_stream_t stream) {
    int rc = check_dims(dims);
    if (rc != GDR_OK) return rc;
    // tensors without elements may have no address
    if (((!k || !v) && dims->T > 0) || (cu != nullptr) != (dims->N > 0)) return GDR_ERR_INVALID;
    rc = check_cache(*dims, cache, false);
    if (rc != GDR_OK) return rc;
    if (!write) {  // outputs: two rows must not share an address
        gdr_dims o = *dims;
        for (int i = 0; i < 2; ++i) o.o_stride[i] = dims->v_stride[i];
        if (check_dims(&o) != GDR_OK) return GDR_ERR_INVALID;
        for (int i = 0; i < 2; ++i) o.o_stride[i] = dims->k_stride[i];
        o.V = dims->K;
        if (check_dims(&o) != GDR_OK) return GDR_ERR_INVALID;
    }
    return cache_rows(write, device_cache(*dims, *cache), token_rows(*dims, cu, status),
                      dims->dtype, k, v, dims_stride(dims->k_stride, dims->H, dims->K),
                      dims_stride(dims->v_stride, dims->H, dims->V), (int)dims->K, (int)dims->V,
                      reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GDR_OK
               : GDR_ERR_CUDA;
}

// New tokens of a sequence, as far as the host knows: the longest (dense, or
// the caller's hint), else the mean.
int64_t tile_rows(const gdr_dims &d) {
    if (d.N == 0) return d.T;
    return d.max_len > 0 ? d.max_len : (d.T + d.N - 1) / d.N;
}
// Rows of a key head (new tokens x G) up to which the kernel of small tiles is
// taken, which reads every key for each 16 of them, against that of 256-row
// tiles.  Measured, small against large, head width 128, 4 key heads:
//   32 sequences of 4K tokens, BF16:  16 rows 55 / 60 us, 32: 65 / 60, 64: 100 / 60
//   128 of 512 tokens, BF16:          32 rows 47 / 53 us, 64: 69 / 56
//   32 of 4K, E4M3:                   32 rows 65 / 100 us, 64: 107 / 106
//   one of 32K, BF16:                  8 rows 27 / 29 us, 16: 40 / 29
//   one of 32K, E4M3:                  8 rows 31 / 44 us, 16: 50 / 44
// so with few (sequence, key head) pairs, where each is shared by many workers,
// the limit is lower.
int64_t few_rows(const gdr_dims &d, const gdr_paged_cache &c) {
    if (seqs_of(d) * c.H < 32) return 8;
    return cache_quantised(c.dtype) ? 64 : 32;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t split_bytes(const SplitPlan &s, int64_t V) {
    const size_t rows = (size_t)s.workers * 2 * s.rows;
    return align256(rows * V * sizeof(float)) + align256(rows * 2 * sizeof(float)) +
           align256((size_t)s.workers * sizeof(int4));
}

SplitScratch carve_split(void *base, const SplitPlan &s, int64_t V) {
    const size_t rows = (size_t)s.workers * 2 * s.rows;
    char *c = static_cast<char *>(base);
    SplitScratch ws{};
    ws.o = reinterpret_cast<float *>(c);
    c += align256(rows * V * sizeof(float));
    ws.ml = reinterpret_cast<float *>(c);
    c += align256(rows * 2 * sizeof(float));
    ws.rec = reinterpret_cast<int4 *>(c);
    return ws;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_cache_write(const gdr_dims *dims, const gdr_paged_cache *cache, const void *k,
                    const void *v, const int32_t *cu_seqlens, int32_t *status,
                    gdr_stream_t stream) {
    return cache_call(true, dims, cache, k, v, cu_seqlens, status, stream);
}

int gdr_cache_read(const gdr_dims *dims, const gdr_paged_cache *cache, void *k, void *v,
                   const int32_t *cu_seqlens, int32_t *status, gdr_stream_t stream) {
    return cache_call(false, dims, cache, k, v, cu_seqlens, status, stream);
}

size_t gdr_attn_workspace_size(const gdr_dims *dims, const gdr_paged_cache *cache) {
    if (check_dims(dims) != GDR_OK || check_cache(*dims, cache, true) != GDR_OK) return 0;
    AttnProblem p{};
    const size_t a = split_bytes(attn_rows_plan(p, 16), dims->V);
    const size_t b = split_bytes(attn_tiles_plan(p), dims->V);
    return a > b ? a : b;
}

int gdr_paged_attn(const gdr_dims *dims, const gdr_paged_cache *cache, const void *q,
                   const int32_t *cu_seqlens, void *o, float *lse, int causal, int64_t window,
                   const gdr_options *opt, gdr_stream_t stream) {
    int rc = check_dims(dims);
    if (rc != GDR_OK) return rc;
    if (((!q || !o) && dims->T > 0) || window < 0 || (cu_seqlens != nullptr) != (dims->N > 0))
        return GDR_ERR_INVALID;
    rc = check_cache(*dims, cache, true);
    if (rc != GDR_OK) return rc;
    if (opt && (!(opt->scale >= 0.f) || opt->grid_limit < 0 || opt->force_bv ||
                opt->force_path < 0 || opt->force_path > 3))
        return GDR_ERR_INVALID;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    AttnProblem p{};
    p.c = device_cache(*dims, *cache);
    p.r = token_rows(*dims, cu_seqlens, opt ? opt->status : nullptr);
    p.q = q; p.o = o; p.lse = lse;
    p.sq = dims_stride(dims->q_stride, dims->H, dims->K);
    p.so = dims_stride(dims->o_stride, dims->H, dims->V);
    p.Hq = (int)dims->H; p.G = (int)(dims->H / cache->H);
    p.K = (int)dims->K; p.V = (int)dims->V;
    p.dtype = dims->dtype;
    p.causal = causal != 0;
    p.window = window < INT32_MAX ? (int)window : INT32_MAX;
    p.scale = opt && opt->scale > 0.f ? opt->scale : 1.0f / std::sqrt((float)dims->K);
    p.grid_limit = opt ? opt->grid_limit : 0;
    LaunchRecorder rec;
    rec.st = st;
    if (opt) {
        rec.events = reinterpret_cast<cudaEvent_t *>(opt->events);
        rec.ids = opt->launch_ids;
        rec.max_launches = opt->events || opt->launch_ids ? opt->max_launches : 0;
        if (opt->n_launches) *opt->n_launches = 0;
    }
    if (seqs_of(*dims) == 0 || dims->T == 0) return GDR_OK;
    const int force = opt ? opt->force_path : 0;
    const bool tensor = force != 1 && attn_rows_supported(p);
    if (force > 1 && !tensor) return GDR_ERR_UNSUPPORTED;
    if (!tensor) {
        if (rec.begin(kKAttnSimt) != cudaSuccess || attn_simt(p, st) != cudaSuccess ||
            rec.end() != cudaSuccess)
            return GDR_ERR_CUDA;
        if (opt && opt->n_launches) *opt->n_launches = rec.count;
        return GDR_OK;
    }
    const bool can = attn_tiles_supported(p);
    if (force == 2 && !can) return GDR_ERR_UNSUPPORTED;
    const bool tiles = force == 2 || (force == 0 && can && tile_rows(*dims) * p.G > few_rows(*dims, *cache));
    p.by_G = divisor((uint32_t)p.G);
    p.by_page = divisor((uint32_t)p.c.page_size);
    for (p.align = 1; p.align < 128 && p.c.page_size % (2 * p.align) == 0;) p.align *= 2;
    const SplitPlan plan = tiles ? attn_tiles_plan(p) : attn_rows_plan(p, tile_rows(*dims) * p.G);
    const size_t need = split_bytes(plan, p.V);
    void *base = opt ? opt->workspace : nullptr;
    if (base) {
        if (opt->workspace_bytes < need) return GDR_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(base) % 256) return GDR_ERR_INVALID;
    } else if (scratch_alloc(&base, need, st) != cudaSuccess) {
        return GDR_ERR_CUDA;
    }
    const SplitScratch ws = carve_split(base, plan, p.V);
    rc = rec.begin(tiles ? kKAttnTiles : kKAttnRows) == cudaSuccess &&
                 (tiles ? attn_tiles(p, ws, plan, st) : attn_rows(p, ws, plan, st)) == cudaSuccess &&
                 rec.end() == cudaSuccess && rec.begin(kKAttnJoin) == cudaSuccess &&
                 attn_join(p, ws, plan, st) == cudaSuccess && rec.end() == cudaSuccess
             ? GDR_OK
             : GDR_ERR_CUDA;
    if (!(opt && opt->workspace) && cudaFreeAsync(base, st) != cudaSuccess && rc == GDR_OK)
        rc = GDR_ERR_CUDA;
    if (opt && opt->n_launches) *opt->n_launches = rec.count;
    return rc;
}

}  // extern "C"
