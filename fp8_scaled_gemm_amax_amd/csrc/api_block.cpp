// api_block.cpp - the C ABI of a feed-forward block's operators (include/fp8amax.h):
// the residual's addition with the norm and the cast, the gated products with
// SwiGLU, adapters. Argument validation before any launch, then dispatch.
#include "block.hpp"
#include "layer_checks.hpp"

#include <cmath>

namespace fp8amax {
namespace {

// One output in an input's place: the same rows, or the caller's promise that
// the two do not overlap.
fp8_status_t check_same_rows(const char* fn, const char* names, const void* p, int64_t ldp, const void* q, int64_t ldq,
                             int64_t rows) {
    if (p && p == q && rows > 1 && ldp != ldq)
        return fail(FP8_ERR_INVALID_ARG, "%s: %s at one address with leading dimensions %lld and %lld", fn, names,
                    (long long)ldp, (long long)ldq);
    return FP8_OK;
}

fp8_status_t check_wide(const char* fn, int64_t ld) {
    if (ld >= (1 << 25))
        return fail(FP8_ERR_UNSUPPORTED, "%s: leading dimension %lld: those of act, h and dh must be < 2^25", fn, (long long)ld);
    return FP8_OK;
}

// Operands and factors of the gated products.
fp8_status_t check_product(const char* fn, const uint8_t* a, int fa, int64_t lda, const uint8_t* b, int fb, int64_t ldb,
                           int64_t m, int64_t inter, int64_t k, const float* sa, int a_mode, const float* sb,
                           int b_mode) {
    if (m < 0 || inter < 0 || k < 0)
        return fail(FP8_ERR_INVALID_ARG, "%s: negative size m=%lld inter=%lld k=%lld", fn, (long long)m,
                    (long long)inter, (long long)k);
    if (!valid_fmt(fa) || !valid_fmt(fb)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown format (%d, %d)", fn, fa, fb);
    if (k % 16 != 0) return fail(FP8_ERR_INVALID_ARG, "%s: k = %lld is not a multiple of 16", fn, (long long)k);
    if (lda < k || ldb < k) return fail(FP8_ERR_INVALID_ARG, "%s: leading dimension smaller than the row", fn);
    if ((a_mode != FP8_SCALE_TENSOR && a_mode != FP8_SCALE_VECTOR) ||
        (b_mode != FP8_SCALE_TENSOR && b_mode != FP8_SCALE_VECTOR))
        return fail(FP8_ERR_INVALID_ARG, "%s: unknown scale mode", fn);
    if (m > 0 && inter > 0) {
        if (k > 0 && (!a || !b)) return fail(FP8_ERR_INVALID_ARG, "%s: a or b is NULL", fn);
        if (!sa || !sb) return fail(FP8_ERR_INVALID_ARG, "%s: scale is NULL", fn);
    }
    if (k > 0 && (!aligned(a, 16) || !aligned(b, 16) || lda % 16 != 0 || ldb % 16 != 0))
        return fail(FP8_ERR_ALIGNMENT, "%s: a, b must be 16-byte aligned with lda, ldb multiples of 16", fn);
    if (!aligned(sa, 4) || !aligned(sb, 4)) return fail(FP8_ERR_ALIGNMENT, "%s: misaligned scale pointer", fn);
    if (!ocp_fmt(fa) || !ocp_fmt(fb))
        return fail(FP8_ERR_UNSUPPORTED, "%s: fnuz operands (%d, %d): OCP e4m3 / e5m2 only", fn, fa, fb);
    if (lda >= (1 << 24) || ldb >= (1 << 24) || inter >= (1 << 24))
        return fail(FP8_ERR_UNSUPPORTED, "%s: lda, ldb and inter must be < 2^24 (tiles use 32-bit offsets)", fn);
    // (a grid's threads stay below 2^32: tiles of 128 x 64 outputs, 256 threads each)
    if (m >= ((int64_t)1 << 30) || (m + 127) / 128 * ((inter + 63) / 64) >= (1 << 24))
        return fail(FP8_ERR_UNSUPPORTED, "%s: %lld x %lld outputs", fn, (long long)m, (long long)inter);
    return FP8_OK;
}

}  // namespace
}  // namespace fp8amax

using namespace fp8amax;

extern "C" {

fp8_status_t fp8_add_norm_quantize_row(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, const uint16_t* res,
                                       int64_t ldres, uint16_t* sum, int64_t ldsum, const void* gamma,
                                       const void* beta, fp8_out_t w_type, float eps, fp8_norm_t kind,
                                       fp8_format_t fmt, int32_t margin, uint8_t* q, int64_t ldq,
                                       float* scale_inv_out, uint16_t* y, int64_t ldy, float* mean_out,
                                       float* rstd_out, uint8_t* xhat_q, fp8_format_t xhat_fmt, int64_t ldxq,
                                       uint8_t* xhat_scale, int64_t ld_scale, void* stream) {
    const char* fn = "fp8_add_norm_quantize_row";
    FP8_TRY(check_common_quant(fn, x, rows, cols, ldx, (int)fmt, margin));
    if (cols < 1) return fail(FP8_ERR_INVALID_ARG, "%s: no columns", fn);
    FP8_TRY(check_matrix(fn, "res", res, rows, cols, ldres));
    FP8_TRY(check_matrix(fn, "sum", sum, rows, cols, ldsum));
    FP8_TRY(check_kind(fn, (int)kind));
    FP8_TRY(check_weights(fn, gamma, beta, (int)w_type));
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(FP8_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
    if (rows > 0 && !q && !y) return fail(FP8_ERR_INVALID_ARG, "%s: neither q nor y is asked for", fn);
    if (rows > 0 && (q != nullptr) != (scale_inv_out != nullptr))
        return fail(FP8_ERR_INVALID_ARG, "%s: q and scale_inv_out go together", fn);
    if (q) FP8_TRY(check_matrix(fn, "q", q, rows, cols, ldq));
    if (y) FP8_TRY(check_matrix(fn, "y", y, rows, cols, ldy));
    FP8_TRY(check_same_rows(fn, "x and sum", x, ldx, sum, ldsum, rows));
    FP8_TRY(check_same_rows(fn, "res and sum", res, ldres, sum, ldsum, rows));
    if (!aligned(res, 2) || !aligned(sum, 2)) return fail(FP8_ERR_ALIGNMENT, "%s: res or sum is not 2-byte aligned", fn);
    if (!aligned(y, 2) || !aligned(scale_inv_out, 4) || !aligned(mean_out, 4) || !aligned(rstd_out, 4))
        return fail(FP8_ERR_ALIGNMENT, "%s: misaligned output", fn);
    const bool save = xhat_q || xhat_scale;
    if (save) {
        FP8_TRY(check_checkpoint(fn, "xhat_q", xhat_q, (int)xhat_fmt, ldxq, xhat_scale, ld_scale, rows, cols));
        if (cols > kNormMaxVecCols)
            return fail(FP8_ERR_UNSUPPORTED, "%s: a checkpoint of more than %lld columns", fn, (long long)kNormMaxVecCols);
    }
    FP8_TRY(check_rows(fn, rows, kMaxRows));
    if (rows == 0) return ok();
    NormFwd p{};
    p.x = x;
    p.rows = rows;
    p.cols = cols;
    p.ldx = ldx;
    p.res = res;
    p.ldres = ldres;
    p.sum = sum;
    p.ldsum = ldsum;
    p.gamma = gamma;
    p.beta = beta;
    p.w_f32 = w_type == FP8_OUT_F32;
    p.rms = kind == FP8_NORM_RMS;
    p.margin = margin;
    p.ckpt_e5m2 = xhat_fmt == FP8_E5M2;
    p.eps = eps;
    p.q = q;
    p.ldq = ldq;
    p.scale_inv = scale_inv_out;
    p.y = y;
    p.ldy = ldy;
    p.mean = mean_out;
    p.rstd = rstd_out;
    p.xq = xhat_q;
    p.ldxq = ldxq;
    p.xs = xhat_scale;
    p.ldxs = ld_scale;
    if (save && !norm_vector_layout(p))
        return fail(FP8_ERR_ALIGNMENT, "%s: a checkpoint needs x, res, sum, y, gamma, beta 16-byte and q 8-byte aligned, "
                    "with row strides that are multiples of 8", fn);
    FP8_TRY(check_device());
    return launched(launch_norm_quant_row(p, (int)fmt, (hipStream_t)stream), fn);
}

fp8_status_t fp8_add_norm_backward(const uint16_t* dsum, int64_t lddsum, const uint16_t* dy, int64_t rows, int64_t cols,
                                   int64_t lddy, const uint16_t* sum, int64_t ldsum, const void* gamma,
                                   fp8_out_t w_type, const float* mean, const float* rstd, fp8_norm_t kind,
                                   uint16_t* dx, int64_t lddx, float* dgamma, float* dbeta, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
    const char* fn = "fp8_add_norm_backward";
    FP8_TRY(check_norm_backward(fn, dy, rows, cols, lddy, gamma, nullptr, (int)w_type, rstd, (int)kind, dx, lddx, dgamma,
                                dbeta, workspace, workspace_bytes));
    FP8_TRY(check_matrix(fn, "sum", sum, rows, cols, ldsum));
    FP8_TRY(check_matrix(fn, "dsum", dsum, rows, cols, lddsum));
    FP8_TRY(check_same_rows(fn, "dsum and dx", dsum, lddsum, dx, lddx, rows));
    if (rows > 0 && kind == FP8_NORM_LAYER && !mean) return fail(FP8_ERR_INVALID_ARG, "%s: mean is NULL", fn);
    if (!aligned(sum, 2) || !aligned(dsum, 2) || !aligned(mean, 4))
        return fail(FP8_ERR_ALIGNMENT, "%s: misaligned pointer", fn);
    FP8_TRY(check_device());
    NormBwd p{};
    p.dy = dy;
    p.rows = rows;
    p.cols = cols;
    p.lddy = lddy;
    p.ds = dsum;
    p.ldds = lddsum;
    p.x = sum;
    p.ldx = ldsum;
    p.w_f32 = w_type == FP8_OUT_F32;
    p.rms = kind == FP8_NORM_RMS;
    p.gamma = gamma;
    p.mean = p.rms ? nullptr : mean;
    p.rstd = rstd;
    p.dx = dx;
    p.lddx = lddx;
    p.dgamma = dgamma;
    p.dbeta = dbeta;
    p.partial = static_cast<float*>(workspace);
    return launched(launch_norm_backward(p, (hipStream_t)stream), fn);
}

fp8_status_t fp8_mx_add_norm_backward(const uint16_t* dsum, int64_t lddsum, const uint16_t* dy, int64_t rows,
                                      int64_t cols, int64_t lddy, const uint8_t* xhat_q, fp8_format_t xhat_fmt,
                                      int64_t ldxq, const uint8_t* xhat_scale, int64_t ld_scale, const void* gamma,
                                      const void* beta, fp8_out_t w_type, const float* rstd, fp8_norm_t kind,
                                      uint16_t* dx, int64_t lddx, float* dgamma, float* dbeta, uint16_t* y,
                                      int64_t ldy, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "fp8_mx_add_norm_backward";
    FP8_TRY(check_norm_backward(fn, dy, rows, cols, lddy, gamma, beta, (int)w_type, rstd, (int)kind, dx, lddx, dgamma,
                                dbeta, workspace, workspace_bytes));
    FP8_TRY(check_matrix(fn, "dsum", dsum, rows, cols, lddsum));
    FP8_TRY(check_same_rows(fn, "dsum and dx", dsum, lddsum, dx, lddx, rows));
    FP8_TRY(check_checkpoint(fn, "xhat_q", xhat_q, (int)xhat_fmt, ldxq, xhat_scale, ld_scale, rows, cols));
    if (y) FP8_TRY(check_matrix(fn, "y", y, rows, cols, ldy));
    if (cols > kNormMaxVecCols)
        return fail(FP8_ERR_UNSUPPORTED, "%s: a checkpoint of more than %lld columns", fn, (long long)kNormMaxVecCols);
    NormBwd p{};
    p.dy = dy;
    p.rows = rows;
    p.cols = cols;
    p.lddy = lddy;
    p.ds = dsum;
    p.ldds = lddsum;
    p.xq = xhat_q;
    p.ldxq = ldxq;
    p.xs = xhat_scale;
    p.ldxs = ld_scale;
    p.ckpt_e5m2 = xhat_fmt == FP8_E5M2;
    p.w_f32 = w_type == FP8_OUT_F32;
    p.rms = kind == FP8_NORM_RMS;
    p.gamma = gamma;
    p.beta = beta;
    p.rstd = rstd;
    p.dx = dx;
    p.lddx = lddx;
    p.y = y;
    p.ldy = ldy;
    p.dgamma = dgamma;
    p.dbeta = dbeta;
    p.partial = static_cast<float*>(workspace);
    if (rows > 0 && !norm_vector_layout(p))
        return fail(FP8_ERR_ALIGNMENT, "%s: dsum, dy, dx, y, gamma and beta must be 16-byte aligned with row strides that "
                    "are multiples of 8", fn);
    FP8_TRY(check_device());
    return launched(launch_norm_backward(p, (hipStream_t)stream), fn);
}

fp8_status_t fp8_gemm_swiglu(const uint8_t* a, fp8_format_t fa, int64_t lda, const uint8_t* b, fp8_format_t fb,
                             int64_t ldb, int64_t m, int64_t inter, int64_t k, const float* a_scale_inv,
                             fp8_scale_mode_t a_mode, const float* b_scale_inv, fp8_scale_mode_t b_mode, uint16_t* act,
                             int64_t ldact, uint16_t* h, int64_t ldh, void* stream) {
    const char* fn = "fp8_gemm_swiglu";
    FP8_TRY(check_product(fn, a, (int)fa, lda, b, (int)fb, ldb, m, inter, k, a_scale_inv, (int)a_mode, b_scale_inv,
                          (int)b_mode));
    FP8_TRY(check_matrix(fn, "act", act, m, inter, ldact));
    if (h) FP8_TRY(check_matrix(fn, "h", h, m, 2 * inter, ldh));
    if (!aligned(act, 2) || !aligned(h, 2)) return fail(FP8_ERR_ALIGNMENT, "%s: misaligned output", fn);
    FP8_TRY(check_wide(fn, ldact));
    if (h) FP8_TRY(check_wide(fn, ldh));
    FP8_TRY(check_device());
    GluFwd p{};
    p.a = a;
    p.lda = lda;
    p.b = b;
    p.ldb = ldb;
    p.m = m;
    p.inter = inter;
    p.k = k;
    p.sa = a_scale_inv;
    p.sa_vec = a_mode == FP8_SCALE_VECTOR;
    p.sb = b_scale_inv;
    p.sb_vec = b_mode == FP8_SCALE_VECTOR;
    p.act = act;
    p.ldact = ldact;
    p.h = h;
    p.ldh = ldh;
    return launched(launch_gemm_swiglu(p, (int)fa, (int)fb, (hipStream_t)stream), fn);
}

fp8_status_t fp8_gemm_swiglu_backward(const uint8_t* a, fp8_format_t fa, int64_t lda, const uint8_t* b,
                                      fp8_format_t fb, int64_t ldb, int64_t m, int64_t inter, int64_t k,
                                      const float* a_scale_inv, fp8_scale_mode_t a_mode, const float* b_scale_inv,
                                      fp8_scale_mode_t b_mode, const uint16_t* h, int64_t ldh, uint16_t* dh,
                                      int64_t lddh, uint16_t* act, int64_t ldact, void* stream) {
    const char* fn = "fp8_gemm_swiglu_backward";
    FP8_TRY(check_product(fn, a, (int)fa, lda, b, (int)fb, ldb, m, inter, k, a_scale_inv, (int)a_mode, b_scale_inv,
                          (int)b_mode));
    FP8_TRY(check_matrix(fn, "h", h, m, 2 * inter, ldh));
    FP8_TRY(check_matrix(fn, "dh", dh, m, 2 * inter, lddh));
    if (act) FP8_TRY(check_matrix(fn, "act", act, m, inter, ldact));
    if (!aligned(h, 2) || !aligned(dh, 2) || !aligned(act, 2))
        return fail(FP8_ERR_ALIGNMENT, "%s: misaligned h, dh or act", fn);
    FP8_TRY(check_wide(fn, ldh));
    FP8_TRY(check_wide(fn, lddh));
    if (act) FP8_TRY(check_wide(fn, ldact));
    FP8_TRY(check_device());
    GluBwd p{};
    p.a = a;
    p.lda = lda;
    p.b = b;
    p.ldb = ldb;
    p.m = m;
    p.inter = inter;
    p.k = k;
    p.sa = a_scale_inv;
    p.sa_vec = a_mode == FP8_SCALE_VECTOR;
    p.sb = b_scale_inv;
    p.sb_vec = b_mode == FP8_SCALE_VECTOR;
    p.h = h;
    p.ldh = ldh;
    p.dh = dh;
    p.lddh = lddh;
    p.act = act;
    p.ldact = ldact;
    return launched(launch_gemm_swiglu_backward(p, (int)fa, (int)fb, (hipStream_t)stream), fn);
}

int64_t fp8_lora_workspace(int64_t tokens, int32_t rank) {
    if (tokens < 1 || tokens >= kMaxRows || rank < 8 || rank > kLoraMaxRank || rank % 8 != 0) return 0;
    return lora_part_rows(tokens) * rank * (int64_t)sizeof(float);
}

fp8_status_t fp8_lora_add(const uint16_t* x, int64_t tokens, int64_t k, int64_t ldx, const int32_t* adapter_idx,
                          const uint16_t* a, int64_t ld_a, int64_t a_stride, const uint16_t* b, int64_t ld_b,
                          int64_t b_stride, const float* scaling, int32_t adapters, int32_t rank, int64_t n,
                          const uint16_t* base, int64_t ldbase, uint16_t* out, int64_t ldout, void* workspace,
                          int64_t workspace_bytes, void* stream) {
    const char* fn = "fp8_lora_add";
    static_assert(kLoraMaxRank == FP8_LORA_MAX_RANK, "one limit");
    if (rank < 8 || rank > kLoraMaxRank || rank % 8 != 0)
        return fail(FP8_ERR_INVALID_ARG, "%s: rank %d is not a multiple of 8 from 8 to %d", fn, rank, kLoraMaxRank);
    if (k < 8 || k % 8 != 0) return fail(FP8_ERR_INVALID_ARG, "%s: k = %lld is not a multiple of 8, 8 or more", fn, (long long)k);
    FP8_TRY(check_matrix(fn, "x", x, tokens, k, ldx));
    FP8_TRY(check_matrix(fn, "out", out, tokens, n, ldout));
    if (base) FP8_TRY(check_matrix(fn, "base", base, tokens, n, ldbase));
    FP8_TRY(check_same_rows(fn, "base and out", base, ldbase, out, ldout, tokens));
    if (adapters < 1) return fail(FP8_ERR_INVALID_ARG, "%s: %d adapters", fn, adapters);
    if (ld_a < k || ld_b < rank || a_stride < 0 || b_stride < 0)
        return fail(FP8_ERR_INVALID_ARG, "%s: leading dimension smaller than the row, or negative adapter stride", fn);
    if (tokens > 0 && n > 0 && (!adapter_idx || !a || !b || !scaling))
        return fail(FP8_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || ldx % 8 != 0 || ld_a % 8 != 0 || ld_b % 8 != 0 ||
        a_stride % 8 != 0 || b_stride % 8 != 0)
        return fail(FP8_ERR_ALIGNMENT, "%s: x, a, b must be 16-byte aligned with leading dimensions and adapter strides "
                    "that are multiples of 8", fn);
    if (!aligned(base, 2) || !aligned(out, 2) || !aligned(adapter_idx, 4) || !aligned(scaling, 4) ||
        !aligned(workspace, 16))
        return fail(FP8_ERR_ALIGNMENT, "%s: misaligned pointer", fn);
    // (grids: 64 tokens a workgroup in the first direction, at most one for 256 columns in the second)
    if (tokens >= ((int64_t)1 << 25) || n >= ((int64_t)1 << 24))
        return fail(FP8_ERR_UNSUPPORTED, "%s: %lld x %lld outputs", fn, (long long)tokens, (long long)n);
    if (ldx >= (1 << 24) || ld_a >= (1 << 24) || ld_b >= (1 << 24) || (base && ldbase >= (1 << 24)) || ldout >= (1 << 24))
        return fail(FP8_ERR_UNSUPPORTED, "%s: leading dimensions must be < 2^24 (rows use 32-bit offsets)", fn);
    if (tokens > 0 && n > 0 && (!workspace || workspace_bytes < fp8_lora_workspace(tokens, rank)))
        return fail(FP8_ERR_INVALID_ARG, "%s: a workspace of %lld bytes is needed", fn,
                    (long long)fp8_lora_workspace(tokens, rank));
    FP8_TRY(check_device());
    Lora p{};
    p.x = x;
    p.tokens = tokens;
    p.k = k;
    p.ldx = ldx;
    p.adapter = adapter_idx;
    p.adapters = adapters;
    p.rank = rank;
    p.a = a;
    p.lda = ld_a;
    p.gsa = a_stride;
    p.b = b;
    p.ldb = ld_b;
    p.gsb = b_stride;
    p.scaling = scaling;
    p.n = n;
    p.base = base;
    p.ldbase = ldbase;
    p.out = out;
    p.ldout = ldout;
    p.ws = static_cast<float*>(workspace);
    return launched(launch_lora_add(p, (hipStream_t)stream), fn);
}

}  // extern "C"
