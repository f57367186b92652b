// layer.cuh -- the arguments and launch functions of the operators of a
// state-space layer: short convolution (conv.cu), selective scan (scan.cu,
// scan_bwd.cu) and root-mean-square norm (norm.cu).
#pragma once

#include "gdr_launch.cuh"
#include "rowvec.cuh"

namespace gdr {

struct ConvArgs {
    TokenRows r;
    const void *x, *dy;
    Param w, b;              // [C, W]; [C] or no address
    const void *h0, *dht;    // [.., W - 1, C] or nullptr
    void *y, *ht, *dx, *dh0;
    float *dw, *db, *part;   // part: [runs][(W + 1) C]
    int64_t xs, ys;          // token strides of x, and of y (backward: dy)
    int64_t C, n_states, runs;
    const int32_t *idx;
    int run;                 // tokens of a run
    int silu;
    bool wide;               // 16 bytes of channels a thread
    int w_bytes;             // alignment of the weights
};
constexpr int kConvThreads = 512;  // of k_conv and k_conv_bwd on an SM: so many registers they take
// step: a thread a sequence, from h0 and into ht; else runs of tokens, and conv_state after it.
cudaError_t conv_fwd(const ConvArgs &a, int W, int dtype, bool step, cudaStream_t st);
cudaError_t conv_state(const ConvArgs &a, int W, int dtype, cudaStream_t st);
cudaError_t conv_bwd(const ConvArgs &a, int W, int dtype, cudaStream_t st);
cudaError_t conv_dh0(const ConvArgs &a, int W, int dtype, cudaStream_t st);
cudaError_t conv_params(const ConvArgs &a, int W, cudaStream_t st);

struct NormArgs {
    const void *x, *res, *dy, *dres;
    Param w;
    void *r, *y, *dx;
    float *scale, *dw, *part;          // part: [blocks][D]
    int64_t rows, D;
    int64_t xs, ress, rs, ys, dys, dress;  // row strides
    float eps;
    int group;                         // values of a scale; 0: the row
    int vec;                           // values that a thread loads at once
};
cudaError_t norm_fwd(const NormArgs &a, int dtype, int out_dtype, cudaStream_t st);
int64_t norm_bwd_blocks(int64_t rows, int64_t D, int vec, int dtype);
cudaError_t norm_bwd(const NormArgs &a, int dtype, int64_t blocks, cudaStream_t st);
cudaError_t norm_weight_grad(const NormArgs &a, int64_t blocks, cudaStream_t st);

struct ScanArgs {
    TokenRows r;
    const void *x, *dt, *z, *Bm, *Cm, *dy;
    const float *A, *D, *dt_bias, *h0, *dht;
    void *y, *dx, *ddt, *dz, *dBm, *dCm;
    float *ht, *dh0, *dA, *dD, *dbias;
    int64_t xs, dts, zs, ys, bs[2], cs[2];  // token strides; of B and C token and group
    int64_t C, n_states;
    int S, G, softplus;
    const int32_t *idx;
    int piece;                // tokens of a piece; 0: sequences are whole
    int64_t slots;            // of pieces
    float *E, *sd;            // [slots][C][S] states, [slots][C] sums of the time steps
    float *R, *part;          // backward: [slots][C][S]; [tiles][tokens][2 S]
    float *pd;                // backward: [slots][2 C] of D and dt_bias
    float *keep, *keep_d;     // backward: [slots][kScanBwdPiece / kScanBwdKeep][C][S] and [..][C]
    int bytes, bc_bytes;      // alignment: x, dt, z, y, dy; B and C
    int st_bytes, out_bytes;  // A, h0, ht, dht, dh0; dx, ddt, dz
};
cudaError_t scan_step(const ScanArgs &a, int dtype, cudaStream_t st);
cudaError_t scan_pieces(const ScanArgs &a, int dtype, bool summary, cudaStream_t st);
cudaError_t scan_join(const ScanArgs &a, bool backward, cudaStream_t st);
cudaError_t scan_bwd_ends(const ScanArgs &a, int dtype, cudaStream_t st);
cudaError_t scan_bwd(const ScanArgs &a, int dtype, cudaStream_t st);
cudaError_t scan_bwd_bc(const ScanArgs &a, int dtype, cudaStream_t st);
cudaError_t scan_bwd_params(const ScanArgs &a, cudaStream_t st);
// Channels that a block of the forward and of the backward scan takes, and the blocks (each within
// a group) that all channels take.
int scan_channels(int S);
int scan_bwd_channels(int S);
inline int64_t scan_tiles(int64_t C, int channels, int G) { return G * ((C / G + channels - 1) / channels); }
// The backward's pieces, and the tokens between the states that its first pass leaves for the main
// one.
constexpr int kScanBwdPiece = 64, kScanBwdKeep = 8;

}  // namespace gdr
