// layer_api.cu -- host side of the short convolution, the selective scan and
// the norm: argument checks, plans, scratch, launches.
#include "layer.cuh"

namespace gdr {
namespace {

constexpr int64_t kMaxTokens = INT32_MAX;  // of a call; the kernels' offsets are 64-bit

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
bool known(int dtype) { return dtype == GDR_F32 || dtype == GDR_BF16 || dtype == GDR_F16; }
int64_t size_of(int dtype) { return dtype == GDR_F32 ? 4 : 2; }
// A stride: the caller's, or `dense` where that is 0.
int64_t stride_or(int64_t s, int64_t dense) { return s ? s : dense; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int check_rows(int64_t B, int64_t T, int64_t N, int32_t dtype, int32_t flags, int64_t max_len) {
    if (!known(dtype) || (flags & ~GDR_SEQLENS_I64) || B < 1 || T < 0 || N < 0 || max_len < 0)
        return GDR_ERR_INVALID;
    if (N > 0 && B != 1) return GDR_ERR_INVALID;
    if (T > kMaxTokens / B || N > kMaxTokens) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// What the options may hold here: scratch, a status word, the launch events.
int check_options(const gdr_options *opt) {
    if (opt && (opt->scale != 0.f || opt->force_path || opt->force_bv || opt->grid_limit))
        return GDR_ERR_INVALID;
    return GDR_OK;
}

template <typename D>
TokenRows rows_of(const D &d, const int32_t *cu, const gdr_options *opt) {
    TokenRows r{};
    if (cu && (d.flags & GDR_SEQLENS_I64)) r.cu64 = reinterpret_cast<const int64_t *>(cu);
    else r.cu = cu;
    r.N = d.N > 0 ? d.N : d.B;
    r.T = d.T;
    r.status = opt ? opt->status : nullptr;
    return r;
}
template <typename D>
int64_t tokens_of(const D &d) { return d.N > 0 ? d.T : d.B * d.T; }
// Tokens of the longest sequence as far as the host knows, else of the mean one.
template <typename D>
int64_t longest_of(const D &d) {
    if (d.N == 0) return d.T;
    const int64_t len = d.max_len > 0 ? d.max_len : ceil_div(d.T, d.N);
    return len < d.T ? len : d.T;
}
// A sequence of so many is one thread's (of the scan: one warp's) work.  256 sequences of 1 / 4 / 8 / 16
// tokens x 2048 channels: convolution 13 / 15 / 19 / 24 us so, 41 / 24 / 22 / 26 in runs; scan 27 / 38 / 53 / 83
// against 94 / 89 / 89 / 92; 16 sequences of 8 / 16: 16 / 20 against 20 / 20, and 17 / 22 against 17 / 18.
constexpr int64_t kFewTokens = 8;

// An output in the place of one of these inputs, which other threads still read.
bool over(const void *out, std::initializer_list<const void *> in) {
    for (const void *p : in)
        if (out && out == p) return true;
    return false;
}
// ... one of these outputs, or two of them in one place.
bool clash(std::initializer_list<const void *> out, std::initializer_list<const void *> in) {
    for (const void *const *p = out.begin(); p != out.end(); ++p) {
        if (over(*p, in)) return true;
        for (const void *const *q = out.begin(); q != p; ++q)
            if (*p && *p == *q) return true;
    }
    return false;
}

// A call's launches, timed where the caller wants them, and its scratch.
struct Call {
    LaunchRecorder rec;
    cudaStream_t st;
    const gdr_options *opt;
    char *base = nullptr;
    bool own = false, failed = false;

    Call(const gdr_options *o, gdr_stream_t s) : st(reinterpret_cast<cudaStream_t>(s)), opt(o) {
        rec.st = st;
        if (o) {
            rec.events = reinterpret_cast<cudaEvent_t *>(o->events);
            rec.ids = o->launch_ids;
            rec.max_launches = o->events || o->launch_ids ? o->max_launches : 0;
            if (o->n_launches) *o->n_launches = 0;
        }
    }
    int scratch(size_t bytes) {
        if (!bytes) return GDR_OK;
        if (opt && opt->workspace) {
            if (opt->workspace_bytes < bytes) return GDR_ERR_WORKSPACE;
            if (reinterpret_cast<uintptr_t>(opt->workspace) % 256) return GDR_ERR_INVALID;
            base = static_cast<char *>(opt->workspace);
            return GDR_OK;
        }
        void *p = nullptr;
        if (scratch_alloc(&p, bytes, st) != cudaSuccess) return GDR_ERR_CUDA;
        base = static_cast<char *>(p);
        own = true;
        return GDR_OK;
    }
    template <typename F>
    void run(int id, F f) {
        if (!failed) failed = rec.begin(id) != cudaSuccess || f() != cudaSuccess || rec.end() != cudaSuccess;
    }
    int done() {
        if (own && cudaFreeAsync(base, st) != cudaSuccess) failed = true;
        if (opt && opt->n_launches) *opt->n_launches = rec.count;
        return failed ? GDR_ERR_CUDA : GDR_OK;
    }
};

// ---- short convolution ----------------------------------------------------
int check_conv(const gdr_conv_dims *d) {
    if (!d) return GDR_ERR_INVALID;
    const int rc = check_rows(d->B, d->T, d->N, d->dtype, d->flags, d->max_len);
    if (rc != GDR_OK) return rc;
    if (d->C < 1 || d->W < 2 || (d->activation != 0 && d->activation != 1) ||
        (d->weight_dtype != d->dtype && d->weight_dtype != GDR_F32) || d->x_stride < 0 ||
        (d->y_stride != 0 && d->y_stride < d->C))
        return GDR_ERR_INVALID;
    if (d->W > 4 || d->C > INT32_MAX / 8) return GDR_ERR_UNSUPPORTED;
    // blocks of a launch: a thread for each channel of each sequence or run of 8 tokens
    const int64_t seqs = (d->N > 0 ? d->N : d->B) + 1;
    if (tokens_of(*d) / 8 + seqs > INT32_MAX * (int64_t)128 / d->C) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// Tokens of a run, at most about `most`: long ones read few rows twice and leave few sums, and the
// threads (one for each vector of channels of a run) fill the device a whole number of times.  64K
// tokens x 2048 channels, by events around each launch, cold: forward at most 32 / 64 / 128 / 256: 101 /
// 102 / 110 / 113 us; backward with its sums 64 / 128 / 256 / 512: 218 / 196 / 182 / 175 us (the kernels
// alone, as they are: 92 and 167).
int run_of(int64_t tokens, int64_t vectors, int most) {
    const int64_t fill = (int64_t)device_sms() * kConvThreads, all = tokens * vectors;
    const int64_t waves = ceil_div(all, fill * most);
    const int64_t run = waves ? ceil_div(ceil_div(all, fill * waves), 4) * 4 : 0;
    return run < 8 ? 8 : (int)run;
}
int conv_bwd_run(const gdr_conv_dims &d) { return run_of(tokens_of(d), ceil_div(d.C, 4), 512); }

ConvArgs conv_args(const gdr_conv_dims &d, const void *x, const void *weight, const void *bias,
                   const int32_t *cu, const gdr_options *opt) {
    ConvArgs a{};
    a.r = rows_of(d, cu, opt);
    a.x = x;
    a.w = Param{weight, d.weight_dtype == GDR_F32};
    a.b = Param{bias, d.weight_dtype == GDR_F32};
    a.xs = stride_or(d.x_stride, d.C);
    a.ys = stride_or(d.y_stride, d.C);
    a.C = d.C;
    a.silu = d.activation == 1;
    a.w_bytes = common_bytes({addr(weight)});
    return a;
}

size_t conv_bwd_bytes(const gdr_conv_dims &d) {
    return (size_t)ceil_div(tokens_of(d), conv_bwd_run(d)) * (d.W + 1) * d.C * sizeof(float);
}

// ---- selective scan -------------------------------------------------------
int check_scan(const gdr_scan_dims *d) {
    if (!d) return GDR_ERR_INVALID;
    const int rc = check_rows(d->B, d->T, d->N, d->dtype, d->flags, d->max_len);
    if (rc != GDR_OK) return rc;
    if (d->C < 1 || d->S < 1 || d->G < 1 || d->C % d->G || (d->softplus != 0 && d->softplus != 1))
        return GDR_ERR_INVALID;
    for (int64_t s : {d->x_stride, d->dt_stride, d->z_stride, d->b_stride[0], d->b_stride[1],
                      d->c_stride[0], d->c_stride[1]})
        if (s < 0) return GDR_ERR_INVALID;
    if ((d->b_stride[0] != 0) != (d->b_stride[1] != 0) || (d->c_stride[0] != 0) != (d->c_stride[1] != 0) ||
        (d->y_stride != 0 && d->y_stride < d->C))
        return GDR_ERR_INVALID;
    if (d->S > 64 || d->C > INT32_MAX / 64) return GDR_ERR_UNSUPPORTED;
    // blocks of a launch: every piece (of 32 tokens at least) of every tile of channels; 128 states of
    // the join
    const int64_t seqs = d->N > 0 ? d->N : d->B, tiles = scan_tiles(d->C, scan_bwd_channels((int)d->S), (int)d->G);
    if (tokens_of(*d) / 32 + seqs + 1 > INT32_MAX / tiles ||
        seqs > INT32_MAX * (int64_t)128 / (d->C * d->S) - 1)
        return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

constexpr int64_t kPieceUnit = 32;  // tokens: whole tiles

// Tokens of a piece of the forward scan, 0 for whole sequences.
int64_t scan_piece(const gdr_scan_dims &d, int n_segments) {
    const int64_t longest = longest_of(d);
    int64_t piece = 0;
    if (n_segments > 1) {
        piece = ceil_div(longest, n_segments);
    } else if (n_segments == 0) {
        const int64_t tiles = scan_tiles(d.C, scan_channels((int)d.S), (int)d.G), sms = device_sms();
        const int64_t tokens = tokens_of(d), seqs = d.N > 0 ? d.N : d.B;
        const bool equal = tokens == seqs * longest;
        // Cycles of an SM.  Whole sequences: a token of the longest takes 187 where an SM has one block,
        // 50 more for each other until they fill it, then 100 a block.
        const int64_t mine = ceil_div(seqs * tiles, sms), slow = 187 + 50 * (mine - 1);
        int64_t least = longest * (slow > 100 * mine ? slow : 100 * mine);
        // Pieces that fill four blocks an SM a whole number of times: 163 a token of a block in both
        // passes, less where a last round leaves blocks out; beginnings and ends; the join.
        // (2048 channels in BF16, whole / in pieces; FP32 goes by the same.  16 states: one sequence of 16384
        // tokens 1530 / 278 us, 4 of 4096 389 / 287, 5 of 2048 245 / 191, 8 of 2048 245 / 287, 32 of 320 112 /
        // 197.  8 states, 8 of 2048: 291 us, in 5 pieces each, 640 blocks where 608 fit, 282, in 10 225.  64
        // states, one of 16384: 2850 us; in pieces of 4096 tokens 1688, 3277 2174, 1171 1355, 863 1367.)
        for (int64_t rounds = 1; rounds <= 4; ++rounds) {
            const int64_t blocks = rounds * 4 * sms, fit = blocks / tiles;  // pieces
            const int64_t each = equal ? fit / seqs : fit;
            if (each < 1) continue;
            const int64_t cut = ceil_div(ceil_div(equal ? longest : tokens, each), kPieceUnit) * kPieceUnit;
            if (cut >= longest) continue;
            const int64_t pieces = equal ? seqs * ceil_div(longest, cut) : ceil_div(tokens, cut);
            const int64_t full = pieces * tiles / (4 * sms), left = ceil_div(pieces * tiles - full * 4 * sms, sms);
            const int64_t last = left == 0 ? 0 : left * 163 > 305 + 82 * (left - 1) ? left * 163 : 305 + 82 * (left - 1);
            const int64_t cycles = (full * 652 + last) * cut + (full + (left > 0)) * 12000 +
                                   longest / cut * 300 + 25000;
            if (cycles < least) {
                least = cycles;
                piece = cut;
            }
        }
    }
    if (piece == 0) return 0;
    piece = ceil_div(piece, kPieceUnit) * kPieceUnit;
    return piece < longest ? piece : 0;
}
int64_t slots_of(const gdr_scan_dims &d, int64_t piece) {
    return (piece ? tokens_of(d) / piece : 0) + (d.N > 0 ? d.N : d.B);
}

struct ScanScratch {
    size_t E, R, sd, pd, part, keep, keep_d, total;
};
ScanScratch scan_scratch(const gdr_scan_dims &d, int64_t piece, bool backward) {
    const size_t slots = (size_t)slots_of(d, piece), C = (size_t)d.C, S = (size_t)d.S;
    ScanScratch s{};
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t here = at;
        at += align256(floats * sizeof(float));
        return here;
    };
    s.E = take(slots * C * S);
    s.sd = take(slots * C);
    if (backward) {
        s.R = take(slots * C * S);
        s.pd = take(slots * 2 * C);
        s.keep = take(slots * (kScanBwdPiece / kScanBwdKeep) * C * S);
        s.keep_d = take(slots * (kScanBwdPiece / kScanBwdKeep) * C);
        s.part = take((size_t)scan_tiles(d.C, scan_bwd_channels((int)d.S), (int)d.G) * (size_t)tokens_of(d) * 2 * S);
    }
    s.total = at;
    return s;
}

ScanArgs scan_args(const gdr_scan_dims &d, const gdr_scan_tensors &t, const int32_t *cu,
                   const gdr_options *opt) {
    ScanArgs a{};
    a.r = rows_of(d, cu, opt);
    a.x = t.x; a.dt = t.dt; a.z = t.z; a.Bm = t.B; a.Cm = t.C;
    a.A = t.A; a.D = t.D; a.dt_bias = t.dt_bias;
    a.xs = stride_or(d.x_stride, d.C);
    a.dts = stride_or(d.dt_stride, d.C);
    a.zs = stride_or(d.z_stride, d.C);
    a.ys = stride_or(d.y_stride, d.C);
    a.bs[0] = stride_or(d.b_stride[0], d.G * d.S);
    a.bs[1] = stride_or(d.b_stride[1], d.S);
    a.cs[0] = stride_or(d.c_stride[0], d.G * d.S);
    a.cs[1] = stride_or(d.c_stride[1], d.S);
    a.C = d.C;
    a.S = (int)d.S; a.G = (int)d.G;
    a.softplus = d.softplus;
    const uint64_t es = (uint64_t)size_of(d.dtype), group = (uint64_t)(d.C / d.G) * es;
    a.bytes = common_bytes({addr(t.x), addr(t.dt), addr(t.z), a.xs * es, a.dts * es,
                            t.z ? a.zs * es : 0, a.ys * es, d.G > 1 ? group : 0});
    a.bc_bytes = common_bytes({addr(t.B), addr(t.C), a.bs[0] * es, a.cs[0] * es,
                               d.G > 1 ? a.bs[1] * es : 0, d.G > 1 ? a.cs[1] * es : 0});
    return a;
}
bool scan_inputs(const gdr_scan_dims &d, const gdr_scan_tensors *t) {
    return t && t->A && (tokens_of(d) == 0 || (t->x && t->dt && t->B && t->C));
}

// ---- norm -----------------------------------------------------------------
int check_norm(const gdr_norm_dims *d) {
    if (!d || !known(d->dtype) || d->rows < 0 || d->D < 1 || !(d->eps >= 0.f) ||
        (d->weight_dtype != d->dtype && d->weight_dtype != GDR_F32))
        return GDR_ERR_INVALID;
    const bool quant = d->out_dtype == GDR_E4M3 || d->out_dtype == GDR_I8;
    if ((!quant && d->out_dtype != d->dtype) || (d->group != 0 && (d->group != 128 || !quant)))
        return GDR_ERR_INVALID;
    for (int64_t s : {d->x_stride, d->residual_stride, d->sum_stride, d->y_stride})
        if (s != 0 && s < d->D) return GDR_ERR_INVALID;
    if (d->D > 16384 || d->rows > INT32_MAX) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// Values that a thread of the norm takes at once: 16 bytes, 4 bytes or one value, as addresses
// and strides of the call's type (in bytes) allow, and others (bytes, size of a value) too.
int norm_vec(uint64_t es, std::initializer_list<uint64_t> rows,
             std::initializer_list<std::pair<uint64_t, uint64_t>> others) {
    const int bytes = common_bytes(rows);
    for (uint64_t vec : {16 / es, 4 / es}) {
        bool fits = (uint64_t)bytes >= vec * es;
        for (const auto &o : others)  // at most 16 bytes are loaded at once
            fits = fits && o.first % (vec * o.second < 16 ? vec * o.second : 16) == 0;
        if (fits) return (int)vec;
    }
    return 1;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_short_conv_fwd(const gdr_conv_dims *dims, const void *x, const void *weight, const void *bias,
                       const int32_t *cu_seqlens, const void *h0, void *ht, int64_t n_states,
                       const int32_t *state_indices, void *y, const gdr_options *opt,
                       gdr_stream_t stream) {
    int rc = check_conv(dims);
    if (rc == GDR_OK) rc = check_options(opt);
    if (rc != GDR_OK) return rc;
    const gdr_conv_dims &d = *dims;
    const int64_t tokens = tokens_of(d), seqs = d.N > 0 ? d.N : d.B;
    if (!weight || (tokens > 0 && (!x || !y)) || (cu_seqlens != nullptr) != (d.N > 0)) return GDR_ERR_INVALID;
    if ((h0 || ht) ? n_states < (state_indices ? 1 : seqs) : state_indices != nullptr) return GDR_ERR_INVALID;
    if (over(y, {h0}) || clash({y, ht}, {x, weight, bias, cu_seqlens, state_indices}))
        return GDR_ERR_INVALID;
    ConvArgs a = conv_args(d, x, weight, bias, cu_seqlens, opt);
    a.h0 = h0; a.ht = ht; a.y = y;
    a.n_states = n_states;
    a.idx = state_indices;
    const uint64_t es = (uint64_t)size_of(d.dtype);
    a.wide = common_bytes({addr(x), addr(y), addr(h0), addr(ht), a.xs * es, a.ys * es, d.C * es}) == 16;
    const bool step = longest_of(d) <= kFewTokens;
    a.run = run_of(tokens, ceil_div(d.C, 16 / (int)es), 64);
    a.runs = ceil_div(tokens, a.run);
    Call call(opt, stream);
    if (step) {
        call.run(kKConvStep, [&] { return conv_fwd(a, (int)d.W, d.dtype, true, call.st); });
        return call.done();
    }
    if (a.runs) call.run(kKConv, [&] { return conv_fwd(a, (int)d.W, d.dtype, false, call.st); });
    if (ht) call.run(kKConvState, [&] { return conv_state(a, (int)d.W, d.dtype, call.st); });
    return call.done();
}

int gdr_short_conv_bwd(const gdr_conv_dims *dims, const void *x, const void *weight, const void *bias,
                       const int32_t *cu_seqlens, const void *h0, const void *dy, const void *dht,
                       void *dx, float *dweight, float *dbias, void *dh0, const gdr_options *opt,
                       gdr_stream_t stream) {
    int rc = check_conv(dims);
    if (rc == GDR_OK) rc = check_options(opt);
    if (rc != GDR_OK) return rc;
    const gdr_conv_dims &d = *dims;
    const int64_t tokens = tokens_of(d);
    if (!weight || !dweight || (tokens > 0 && (!x || !dy || !dx)) || (dbias && !bias) ||
        (cu_seqlens != nullptr) != (d.N > 0) ||
        clash({dx, dweight, dbias, dh0}, {x, weight, bias, cu_seqlens, h0, dy, dht}))
        return GDR_ERR_INVALID;
    ConvArgs a = conv_args(d, x, weight, bias, cu_seqlens, opt);
    a.h0 = h0; a.dy = dy; a.dht = dht; a.dx = dx; a.dh0 = dh0;
    a.dw = dweight; a.db = dbias;
    const uint64_t es = (uint64_t)size_of(d.dtype);
    a.wide = common_bytes({addr(x), addr(dy), addr(h0), addr(dht), addr(dx), addr(dh0), a.xs * es,
                           a.ys * es, d.C * es}) == 16;
    a.run = conv_bwd_run(d);
    a.runs = ceil_div(tokens, a.run);
    Call call(opt, stream);
    rc = call.scratch(conv_bwd_bytes(d));
    if (rc != GDR_OK) return rc;
    a.part = reinterpret_cast<float *>(call.base);
    if (a.runs) call.run(kKConvBwd, [&] { return conv_bwd(a, (int)d.W, d.dtype, call.st); });
    call.run(kKConvParams, [&] { return conv_params(a, (int)d.W, call.st); });
    if (dh0) call.run(kKConvDh0, [&] { return conv_dh0(a, (int)d.W, d.dtype, call.st); });
    return call.done();
}

size_t gdr_short_conv_bwd_workspace_size(const gdr_conv_dims *dims) {
    return check_conv(dims) == GDR_OK ? conv_bwd_bytes(*dims) : 0;
}

int gdr_selective_scan_fwd(const gdr_scan_dims *dims, const gdr_scan_tensors *in,
                           const int32_t *cu_seqlens, const float *h0, float *ht, int64_t n_states,
                           const int32_t *state_indices, void *y, int n_segments,
                           const gdr_options *opt, gdr_stream_t stream) {
    int rc = check_scan(dims);
    if (rc == GDR_OK) rc = check_options(opt);
    if (rc != GDR_OK) return rc;
    const gdr_scan_dims &d = *dims;
    const int64_t tokens = tokens_of(d), seqs = d.N > 0 ? d.N : d.B;
    if (!scan_inputs(d, in) || (tokens > 0 && !y) || (cu_seqlens != nullptr) != (d.N > 0) || n_segments < 0)
        return GDR_ERR_INVALID;
    if ((h0 || ht) ? n_states < (state_indices ? 1 : seqs) : state_indices != nullptr) return GDR_ERR_INVALID;
    if (over(y, {h0}) ||
        clash({y, ht}, {in->x, in->dt, in->A, in->B, in->C, in->D, in->z, in->dt_bias, cu_seqlens, state_indices}))
        return GDR_ERR_INVALID;
    ScanArgs a = scan_args(d, *in, cu_seqlens, opt);
    a.h0 = h0; a.ht = ht; a.y = y;
    a.n_states = n_states;
    a.idx = state_indices;
    a.bytes = (int)common_bytes({(uint64_t)a.bytes, addr(y)});
    a.st_bytes = common_bytes({addr(h0), addr(ht), addr(in->A)});
    Call call(opt, stream);
    // its kernel counts warps, of 32 channels of a sequence each, in 32 bits
    const bool step = longest_of(d) <= kFewTokens && (seqs + 1) * scan_tiles(d.C, 32, (int)d.G) <= UINT32_MAX;
    if (n_segments == 0 && step) {
        call.run(kKScanStep, [&] { return scan_step(a, d.dtype, call.st); });
        return call.done();
    }
    const int64_t piece = scan_piece(d, n_segments);
    a.piece = (int)piece;
    a.slots = slots_of(d, piece);
    if (piece) {
        const ScanScratch s = scan_scratch(d, piece, false);
        rc = call.scratch(s.total);
        if (rc != GDR_OK) return rc;
        a.E = reinterpret_cast<float *>(call.base + s.E);
        a.sd = reinterpret_cast<float *>(call.base + s.sd);
        call.run(kKScanEnds, [&] { return scan_pieces(a, d.dtype, true, call.st); });
        call.run(kKScanJoin, [&] { return scan_join(a, false, call.st); });
    }
    call.run(kKScan, [&] { return scan_pieces(a, d.dtype, false, call.st); });
    return call.done();
}

size_t gdr_selective_scan_workspace_size(const gdr_scan_dims *dims, int n_segments) {
    if (check_scan(dims) != GDR_OK || n_segments < 0) return 0;
    const int64_t piece = scan_piece(*dims, n_segments);
    return piece ? scan_scratch(*dims, piece, false).total : 0;
}

int gdr_selective_scan_bwd(const gdr_scan_dims *dims, const gdr_scan_tensors *in,
                           const int32_t *cu_seqlens, const float *h0, const void *dy,
                           const float *dht, const gdr_scan_grads *out, const gdr_options *opt,
                           gdr_stream_t stream) {
    int rc = check_scan(dims);
    if (rc == GDR_OK) rc = check_options(opt);
    if (rc != GDR_OK) return rc;
    const gdr_scan_dims &d = *dims;
    const int64_t tokens = tokens_of(d), seqs = d.N > 0 ? d.N : d.B;
    if (!scan_inputs(d, in) || !out || !out->dA || (cu_seqlens != nullptr) != (d.N > 0) ||
        (tokens > 0 && (!dy || !out->dx || !out->ddt || !out->dB || !out->dC || (in->z && !out->dz))) ||
        (out->dD && !in->D) || (out->ddt_bias && !in->dt_bias) || (out->dz && !in->z))
        return GDR_ERR_INVALID;
    if (clash({out->dx, out->ddt, out->dA, out->dB, out->dC, out->dD, out->dz, out->ddt_bias, out->dh0},
              {in->x, in->dt, in->A, in->B, in->C, in->D, in->z, in->dt_bias, cu_seqlens, h0, dy, dht}))
        return GDR_ERR_INVALID;
    if (tokens > INT32_MAX * (int64_t)128 / (d.G * d.S)) return GDR_ERR_UNSUPPORTED;  // blocks of dB, dC
    ScanArgs a = scan_args(d, *in, cu_seqlens, opt);
    a.h0 = h0; a.dy = dy; a.dht = dht;
    a.n_states = seqs;
    a.dx = out->dx; a.ddt = out->ddt; a.dz = out->dz; a.dBm = out->dB; a.dCm = out->dC;
    a.dA = out->dA; a.dD = out->dD; a.dbias = out->ddt_bias; a.dh0 = out->dh0;
    const uint64_t es = (uint64_t)size_of(d.dtype), group = (uint64_t)(d.C / d.G) * es;
    a.bytes = (int)common_bytes({(uint64_t)a.bytes, addr(dy)});
    a.st_bytes = common_bytes({addr(in->A), addr(h0), addr(dht), addr(out->dh0)});
    a.out_bytes = common_bytes({addr(out->dx), addr(out->ddt), addr(out->dz), d.C * es, d.G > 1 ? group : 0});
    a.piece = kScanBwdPiece;
    a.slots = slots_of(d, kScanBwdPiece);
    const ScanScratch s = scan_scratch(d, kScanBwdPiece, true);
    Call call(opt, stream);
    rc = call.scratch(s.total);
    if (rc != GDR_OK) return rc;
    a.E = reinterpret_cast<float *>(call.base + s.E);
    a.R = reinterpret_cast<float *>(call.base + s.R);
    a.sd = reinterpret_cast<float *>(call.base + s.sd);
    a.pd = reinterpret_cast<float *>(call.base + s.pd);
    a.keep = reinterpret_cast<float *>(call.base + s.keep);
    a.keep_d = reinterpret_cast<float *>(call.base + s.keep_d);
    a.part = reinterpret_cast<float *>(call.base + s.part);
    call.run(kKScanBwdEnds, [&] { return scan_bwd_ends(a, d.dtype, call.st); });
    call.run(kKScanJoin, [&] { return scan_join(a, true, call.st); });
    call.run(kKScanBwd, [&] { return scan_bwd(a, d.dtype, call.st); });
    if (tokens) call.run(kKScanBwdBC, [&] { return scan_bwd_bc(a, d.dtype, call.st); });
    call.run(kKScanBwdParams, [&] { return scan_bwd_params(a, call.st); });
    return call.done();
}

size_t gdr_selective_scan_bwd_workspace_size(const gdr_scan_dims *dims) {
    return check_scan(dims) == GDR_OK ? scan_scratch(*dims, kScanBwdPiece, true).total : 0;
}

int gdr_rms_norm_fwd(const gdr_norm_dims *dims, const void *x, const void *residual, const void *weight,
                     void *sum, void *y, float *scale, const gdr_options *opt, gdr_stream_t stream) {
    int rc = check_norm(dims);
    if (rc == GDR_OK) rc = check_options(opt);
    if (rc != GDR_OK) return rc;
    const gdr_norm_dims &d = *dims;
    const bool quant = d.out_dtype != d.dtype;
    if ((residual != nullptr) != (sum != nullptr) ||
        (d.rows > 0 && (!x || !y || (quant && !scale))) || (!quant && scale))
        return GDR_ERR_INVALID;
    // two outputs in one place; values of other sizes over rows that are still to be read
    if (clash({sum, y, scale}, {weight}) || over(scale, {x, residual}) || (quant && over(y, {x, residual})))
        return GDR_ERR_INVALID;
    NormArgs a{};
    a.x = x; a.res = residual; a.r = sum; a.y = y; a.scale = scale;
    a.w = Param{weight, d.weight_dtype == GDR_F32};
    a.rows = d.rows; a.D = d.D;
    a.xs = stride_or(d.x_stride, d.D);
    a.ress = stride_or(d.residual_stride, d.D);
    a.rs = stride_or(d.sum_stride, d.D);
    a.ys = stride_or(d.y_stride, d.D);
    // rows in place, but not those of other rows
    if ((over(sum, {x}) && a.rs != a.xs) || (over(sum, {residual}) && a.rs != a.ress) ||
        (over(y, {x}) && a.ys != a.xs) || (over(y, {residual}) && a.ys != a.ress))
        return GDR_ERR_INVALID;
    a.eps = d.eps;
    a.group = d.group;
    const uint64_t es = (uint64_t)size_of(d.dtype);
    const uint64_t ws = d.weight_dtype == GDR_F32 ? 4 : es, os = quant ? 1 : es;
    a.vec = norm_vec(es, {addr(x), a.xs * es, addr(residual), residual ? a.ress * es : 0, addr(sum),
                          sum ? a.rs * es : 0, d.D * es},
                     {{addr(y), os}, {a.ys * os, os}, {addr(weight), ws}});
    Call call(opt, stream);
    if (d.rows) call.run(kKNorm, [&] { return norm_fwd(a, d.dtype, d.out_dtype, call.st); });
    return call.done();
}

int gdr_rms_norm_bwd(const gdr_norm_dims *dims, const void *r, const void *weight, const void *dy,
                     const void *dsum, void *dx, float *dweight, const gdr_options *opt,
                     gdr_stream_t stream) {
    int rc = check_norm(dims);
    if (rc == GDR_OK) rc = check_options(opt);
    if (rc != GDR_OK) return rc;
    const gdr_norm_dims &d = *dims;
    if (d.out_dtype != d.dtype || (d.rows > 0 && (!r || !dy || !dx)) || (dweight && !weight) ||
        clash({dx, dweight}, {r, weight, dy, dsum}))
        return GDR_ERR_INVALID;
    NormArgs a{};
    a.r = const_cast<void *>(r); a.dy = dy; a.dres = dsum; a.dx = dx; a.dw = dweight;
    a.w = Param{weight, d.weight_dtype == GDR_F32};
    a.rows = d.rows; a.D = d.D;
    a.rs = stride_or(d.x_stride, d.D);
    a.dys = stride_or(d.y_stride, d.D);
    a.dress = stride_or(d.residual_stride, d.D);
    a.eps = d.eps;
    const uint64_t es = (uint64_t)size_of(d.dtype);
    const uint64_t ws = d.weight_dtype == GDR_F32 ? 4 : es;
    a.vec = norm_vec(es, {addr(r), a.rs * es, addr(dy), a.dys * es, addr(dsum), dsum ? a.dress * es : 0,
                          addr(dx), d.D * es}, {{addr(weight), ws}});
    Call call(opt, stream);
    const int64_t blocks = norm_bwd_blocks(d.rows, d.D, a.vec, d.dtype);
    rc = call.scratch(dweight ? (size_t)(blocks * d.D) * sizeof(float) : 0);
    if (rc != GDR_OK) return rc;
    a.part = reinterpret_cast<float *>(call.base);
    if (d.rows) call.run(kKNormBwd, [&] { return norm_bwd(a, d.dtype, blocks, call.st); });
    if (dweight) call.run(kKNormWeight, [&] { return norm_weight_grad(a, blocks, call.st); });
    return call.done();
}

size_t gdr_rms_norm_bwd_workspace_size(const gdr_norm_dims *dims) {
    if (check_norm(dims) != GDR_OK) return 0;
    const int es = (int)size_of(dims->dtype);
    size_t most = 0;  // whatever the tensors' alignment
    for (int vec : {1, 4 / es, 16 / es}) {
        const size_t n = (size_t)(norm_bwd_blocks(dims->rows, dims->D, vec, dims->dtype) * dims->D) * sizeof(float);
        if (n > most) most = n;
    }
    return most;
}

}  // extern "C"
