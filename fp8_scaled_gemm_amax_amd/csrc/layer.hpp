// layer.hpp - host-side launchers of the layer kernels around the products
// (norm, SwiGLU with checkpoints, the MoE layer for a few tokens), internal to
// the library as kernels.hpp; arguments were validated by the C ABI layer.
#pragma once

#include "kernels.hpp"

namespace fp8amax {

// Layer norm / RMS norm with the rowwise cast, and its backward pass. gamma and
// beta (NULL: 1 and 0) are bf16, or fp32 with w_f32. xq / xs: the MX
// checkpoint of the normalised rows (NULL: none; vector layout only).
constexpr int64_t kNormMaxVecCols = 16384;          // columns of the register kernels
constexpr int64_t kNormMaxBands = 512;              // bands of rows of the weights' gradients

struct NormFwd {
    const uint16_t* x;
    int64_t rows, cols, ldx;
    const uint16_t* res;                            // NULL: the norm of x, else of sum = bf16(x + res)
    int64_t ldres;
    uint16_t* sum;
    int64_t ldsum;
    const void *gamma, *beta;
    int w_f32, rms, margin, ckpt_e5m2;
    float eps;
    uint8_t* q;
    int64_t ldq;
    float* scale_inv;
    uint16_t* y;
    int64_t ldy;
    float *mean, *rstd;
    uint8_t* xq;
    int64_t ldxq;
    uint8_t* xs;
    int64_t ldxs;
};

// x (with mean and rstd) or xq / xs (with rstd): where the normalised rows come
// from. ds (NULL: none): what is added to dx. partial: kNormMaxBands * 2 * cols floats at most; band, longer and bands
// are the launcher's.
struct NormBwd {
    const uint16_t* dy;
    int64_t rows, cols, lddy;
    const uint16_t* ds;
    int64_t ldds;
    const uint16_t* x;
    int64_t ldx;
    const uint8_t* xq;
    int64_t ldxq;
    const uint8_t* xs;
    int64_t ldxs;
    int ckpt_e5m2, w_f32, rms;
    const void *gamma, *beta;
    const float *mean, *rstd;
    uint16_t* dx;
    int64_t lddx;
    uint16_t* y;
    int64_t ldy;
    float *dgamma, *dbeta, *partial;
    int64_t band, longer, bands;
};

// Rows of one launch of the row kernels: longer calls are cut, so that a grid's
// threads stay below 2^32 whatever the rows.
constexpr int64_t kLaunchRows = (int64_t)1 << 20;

// Whether the register kernels take these operands (16-byte chunks everywhere).
inline bool chunked(const void* p, int64_t ld, unsigned align) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0 && ld % 8 == 0);
}
inline bool norm_vector_layout(const NormFwd& p) {
    return p.cols % 8 == 0 && p.cols <= kNormMaxVecCols && chunked(p.x, p.ldx, 16) && chunked(p.gamma, 0, 16) &&
           chunked(p.beta, 0, 16) && chunked(p.q, p.ldq, 8) && chunked(p.y, p.ldy, 16) &&
           chunked(p.res, p.ldres, 16) && chunked(p.sum, p.ldsum, 16);
}
inline bool norm_vector_layout(const NormBwd& p) {
    return p.cols % 8 == 0 && p.cols <= kNormMaxVecCols && chunked(p.dy, p.lddy, 16) && chunked(p.dx, p.lddx, 16) &&
           chunked(p.gamma, 0, 16) && chunked(p.beta, 0, 16) && chunked(p.x, p.ldx, 16) && chunked(p.y, p.ldy, 16) &&
           chunked(p.ds, p.ldds, 16);
}
// Columns and slices of the rows of a workgroup of the weights' gradients in any
// layout, and its grid over the columns: at most 2^21 workgroups side by side,
// since a grid's threads (32 a column here) stay below 2^32 in each direction.
constexpr int kAnyCols = 32, kAnySlices = 32;
struct ColsGrid {
    unsigned x, z;
};
inline ColsGrid any_cols_grid(int64_t cols) {
    const int64_t blocks = (cols + kAnyCols - 1) / kAnyCols, most = (int64_t)1 << 21;
    const int64_t x = blocks < most ? blocks : most;
    return {(unsigned)x, (unsigned)((blocks + x - 1) / x)};
}
hipError_t launch_norm_quant_row(const NormFwd& p, int fmt, hipStream_t st);
hipError_t launch_norm_backward(const NormBwd& p, hipStream_t st);

// SwiGLU with the rowwise cast and the MX checkpoint of h, and its backward
// pass from h or from the checkpoint (hq != NULL).
constexpr int64_t kSwigluMxMaxInter = 16384;

struct SwigluFwd {
    const uint16_t* h;
    int64_t rows, inter, ldh;
    int margin, ckpt_e5m2;
    uint8_t* q;
    int64_t ldq;
    float* scale_inv;
    uint8_t* hq;
    int64_t ldhq;
    uint8_t* hs;
    int64_t ldhs;
};

struct SwigluBwd {
    const uint16_t* da;
    int64_t rows, inter, ldda;
    const uint16_t* h;
    int64_t ldh;
    const uint8_t* hq;
    int64_t ldhq;
    const uint8_t* hs;
    int64_t ldhs;
    int ckpt_e5m2;
    uint16_t* dh;
    int64_t lddh;
    uint16_t* a;
    int64_t lda;
};

hipError_t launch_swiglu_quant_row_mx(const SwigluFwd& p, int fmt, hipStream_t st);
hipError_t launch_swiglu_backward(const SwigluBwd& p, hipStream_t st);

// The MoE layer for a few tokens (kMoeFewTokens at most), two launches. ws
// holds for every entry 2 * inter bf16 values: the activation's high and low
// parts, in the order of the down product's loads.
constexpr int kMoeFewTokens = 64;

struct MoeFew {
    const uint16_t* x;
    int64_t ldx;
    const int32_t* idx;
    const float* weights;
    int tokens, topk, experts;
    const uint8_t* w1;
    int64_t ld1, gs1;
    const float* s1;
    const uint8_t* w2;
    int64_t ld2, gs2;
    const float* s2;
    int hidden, inter;
    uint16_t* ws;
    uint16_t* out;
    int64_t ldo;
};

hipError_t launch_moe_few_tokens(const MoeFew& p, int f1, int f2, hipStream_t st);

}  // namespace fp8amax
