// api_layer.cpp - the C ABI of the layer around the products (include/fp8amax.h):
// norm and its gradient, SwiGLU with checkpoints and its gradient, the MoE
// layer for a few tokens. Argument validation before any launch, then dispatch.
#include "layer_checks.hpp"

#include <cmath>

namespace fp8amax {
namespace {

fp8_status_t check_swiglu_backward(const char* fn, const uint16_t* da, int64_t rows, int64_t inter, int64_t ldda,
                                   const uint16_t* dh, int64_t lddh, const uint16_t* a, int64_t lda) {
    if (inter < 0 || inter >= ((int64_t)1 << 30))
        return fail(FP8_ERR_INVALID_ARG, "%s: intermediate size %lld", fn, (long long)inter);
    FP8_TRY(check_matrix(fn, "da", da, rows, inter, ldda));
    FP8_TRY(check_matrix(fn, "dh", dh, rows, 2 * inter, lddh));
    if (a) FP8_TRY(check_matrix(fn, "a", a, rows, inter, lda));
    if (!aligned(da, 16) || ldda % 8 != 0 || !aligned(dh, 16) || lddh % 8 != 0 || inter % 8 != 0 ||
        (a && (!aligned(a, 16) || lda % 8 != 0)))
        return fail(FP8_ERR_ALIGNMENT, "%s: da, dh and a must be 16-byte aligned with row strides and inter multiples "
                    "of 8", fn);
    return check_rows(fn, rows, kMaxRows);
}

}  // namespace
}  // namespace fp8amax

using namespace fp8amax;

extern "C" {

fp8_status_t fp8_norm_quantize_row(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, const void* gamma,
                                   const void* beta, fp8_out_t w_type, float eps, fp8_norm_t kind, fp8_format_t fmt,
                                   int32_t margin, uint8_t* q, int64_t ldq, float* scale_inv_out, uint16_t* y,
                                   int64_t ldy, float* mean_out, float* rstd_out, uint8_t* xhat_q,
                                   fp8_format_t xhat_fmt, int64_t ldxq, uint8_t* xhat_scale, int64_t ld_scale,
                                   void* stream) {
    const char* fn = "fp8_norm_quantize_row";
    FP8_TRY(check_common_quant(fn, x, rows, cols, ldx, (int)fmt, margin));
    if (cols < 1) return fail(FP8_ERR_INVALID_ARG, "%s: no columns", fn);
    FP8_TRY(check_kind(fn, (int)kind));
    FP8_TRY(check_weights(fn, gamma, beta, (int)w_type));
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(FP8_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
    if (rows > 0 && !q && !y) return fail(FP8_ERR_INVALID_ARG, "%s: neither q nor y is asked for", fn);
    if (rows > 0 && (q != nullptr) != (scale_inv_out != nullptr))
        return fail(FP8_ERR_INVALID_ARG, "%s: q and scale_inv_out go together", fn);
    if (q) FP8_TRY(check_matrix(fn, "q", q, rows, cols, ldq));
    if (y) FP8_TRY(check_matrix(fn, "y", y, rows, cols, ldy));
    if (!aligned(y, 2) || !aligned(scale_inv_out, 4) || !aligned(mean_out, 4) || !aligned(rstd_out, 4))
        return fail(FP8_ERR_ALIGNMENT, "%s: misaligned output", fn);
    const bool save = xhat_q || xhat_scale;
    if (save) {
        FP8_TRY(check_checkpoint(fn, "xhat_q", xhat_q, (int)xhat_fmt, ldxq, xhat_scale, ld_scale, rows, cols));
        if (cols > kNormMaxVecCols)
            return fail(FP8_ERR_UNSUPPORTED, "%s: a checkpoint of more than %lld columns", fn, (long long)kNormMaxVecCols);
    }
    FP8_TRY(check_rows(fn, rows, kMaxRows));
    NormFwd p{};
    p.x = x;
    p.rows = rows;
    p.cols = cols;
    p.ldx = ldx;
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
    if (save && rows > 0 && !norm_vector_layout(p))
        return fail(FP8_ERR_ALIGNMENT, "%s: a checkpoint needs x, y, gamma, beta 16-byte and q 8-byte aligned, with row "
                    "strides that are multiples of 8", fn);
    FP8_TRY(check_device());
    return launched(launch_norm_quant_row(p, (int)fmt, (hipStream_t)stream), fn);
}

int64_t fp8_norm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1 || rows >= kMaxRows || cols >= kMaxCols) return 0;
    return (rows < kNormMaxBands ? rows : kNormMaxBands) * 2 * cols * (int64_t)sizeof(float);
}

fp8_status_t fp8_norm_backward(const uint16_t* dy, int64_t rows, int64_t cols, int64_t lddy, const uint16_t* x,
                               int64_t ldx, const void* gamma, fp8_out_t w_type, const float* mean, const float* rstd,
                               fp8_norm_t kind, uint16_t* dx, int64_t lddx, float* dgamma, float* dbeta,
                               void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "fp8_norm_backward";
    FP8_TRY(check_norm_backward(fn, dy, rows, cols, lddy, gamma, nullptr, (int)w_type, rstd, (int)kind, dx, lddx, dgamma,
                                dbeta, workspace, workspace_bytes));
    FP8_TRY(check_matrix(fn, "x", x, rows, cols, ldx));
    if (rows > 0 && kind == FP8_NORM_LAYER && !mean) return fail(FP8_ERR_INVALID_ARG, "%s: mean is NULL", fn);
    if (!aligned(x, 2) || !aligned(mean, 4)) return fail(FP8_ERR_ALIGNMENT, "%s: misaligned pointer", fn);
    FP8_TRY(check_device());
    NormBwd p{};
    p.dy = dy;
    p.rows = rows;
    p.cols = cols;
    p.lddy = lddy;
    p.x = x;
    p.ldx = ldx;
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

fp8_status_t fp8_mx_norm_backward(const uint16_t* dy, int64_t rows, int64_t cols, int64_t lddy, const uint8_t* xhat_q,
                                  fp8_format_t xhat_fmt, int64_t ldxq, const uint8_t* xhat_scale, int64_t ld_scale,
                                  const void* gamma, const void* beta, fp8_out_t w_type, const float* rstd,
                                  fp8_norm_t kind, uint16_t* dx, int64_t lddx, float* dgamma, float* dbeta,
                                  uint16_t* y, int64_t ldy, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "fp8_mx_norm_backward";
    FP8_TRY(check_norm_backward(fn, dy, rows, cols, lddy, gamma, beta, (int)w_type, rstd, (int)kind, dx, lddx, dgamma,
                                dbeta, workspace, workspace_bytes));
    FP8_TRY(check_checkpoint(fn, "xhat_q", xhat_q, (int)xhat_fmt, ldxq, xhat_scale, ld_scale, rows, cols));
    if (y) FP8_TRY(check_matrix(fn, "y", y, rows, cols, ldy));
    if (cols > kNormMaxVecCols)
        return fail(FP8_ERR_UNSUPPORTED, "%s: a checkpoint of more than %lld columns", fn, (long long)kNormMaxVecCols);
    NormBwd p{};
    p.dy = dy;
    p.rows = rows;
    p.cols = cols;
    p.lddy = lddy;
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
        return fail(FP8_ERR_ALIGNMENT, "%s: dy, dx, y, gamma and beta must be 16-byte aligned with row strides that are "
                    "multiples of 8", fn);
    FP8_TRY(check_device());
    return launched(launch_norm_backward(p, (hipStream_t)stream), fn);
}

fp8_status_t fp8_swiglu_quantize_row_mx(const uint16_t* h, int64_t rows, int64_t inter, int64_t ldh, fp8_format_t fmt,
                                        int32_t margin, uint8_t* q, int64_t ldq, float* scale_inv_out, uint8_t* hq,
                                        fp8_format_t h_fmt, int64_t ldhq, uint8_t* h_scale, int64_t ld_scale,
                                        void* stream) {
    const char* fn = "fp8_swiglu_quantize_row_mx";
    if (inter < 0 || inter >= ((int64_t)1 << 30))
        return fail(FP8_ERR_INVALID_ARG, "%s: intermediate size %lld", fn, (long long)inter);
    FP8_TRY(check_common_quant(fn, h, rows, 2 * inter, ldh, (int)fmt, margin));
    FP8_TRY(check_matrix(fn, "q", q, rows, inter, ldq));
    if (rows > 0 && inter > 0 && !scale_inv_out) return fail(FP8_ERR_INVALID_ARG, "%s: scale_inv_out is NULL", fn);
    if (inter % FP8_MX_BLOCK != 0)
        return fail(FP8_ERR_INVALID_ARG, "%s: inter = %lld is not a multiple of %d", fn, (long long)inter, FP8_MX_BLOCK);
    FP8_TRY(check_checkpoint(fn, "hq", hq, (int)h_fmt, ldhq, h_scale, ld_scale, rows, 2 * inter));
    if (!aligned(h, 16) || ldh % 8 != 0 || !aligned(q, 8) || ldq % 8 != 0 || !aligned(scale_inv_out, 4))
        return fail(FP8_ERR_ALIGNMENT, "%s: h must be 16-byte aligned with ldh a multiple of 8, q 8-byte aligned with "
                    "ldq a multiple of 8", fn);
    if (inter > kSwigluMxMaxInter)
        return fail(FP8_ERR_UNSUPPORTED, "%s: intermediate size above %lld", fn, (long long)kSwigluMxMaxInter);
    FP8_TRY(check_rows(fn, rows, (int64_t)1 << 26));
    FP8_TRY(check_device());
    SwigluFwd p{};
    p.h = h;
    p.rows = rows;
    p.inter = inter;
    p.ldh = ldh;
    p.margin = margin;
    p.ckpt_e5m2 = h_fmt == FP8_E5M2;
    p.q = q;
    p.ldq = ldq;
    p.scale_inv = scale_inv_out;
    p.hq = hq;
    p.ldhq = ldhq;
    p.hs = h_scale;
    p.ldhs = ld_scale;
    return launched(launch_swiglu_quant_row_mx(p, (int)fmt, (hipStream_t)stream), fn);
}

fp8_status_t fp8_swiglu_backward(const uint16_t* da, int64_t rows, int64_t inter, int64_t ldda, const uint16_t* h,
                                 int64_t ldh, uint16_t* dh, int64_t lddh, uint16_t* a, int64_t lda, void* stream) {
    const char* fn = "fp8_swiglu_backward";
    FP8_TRY(check_swiglu_backward(fn, da, rows, inter, ldda, dh, lddh, a, lda));
    FP8_TRY(check_matrix(fn, "h", h, rows, 2 * inter, ldh));
    if (!aligned(h, 16) || ldh % 8 != 0)
        return fail(FP8_ERR_ALIGNMENT, "%s: h must be 16-byte aligned with ldh a multiple of 8", fn);
    FP8_TRY(check_device());
    SwigluBwd p{};
    p.da = da;
    p.rows = rows;
    p.inter = inter;
    p.ldda = ldda;
    p.h = h;
    p.ldh = ldh;
    p.dh = dh;
    p.lddh = lddh;
    p.a = a;
    p.lda = lda;
    return launched(launch_swiglu_backward(p, (hipStream_t)stream), fn);
}

fp8_status_t fp8_mx_swiglu_backward(const uint16_t* da, int64_t rows, int64_t inter, int64_t ldda, const uint8_t* hq,
                                    fp8_format_t h_fmt, int64_t ldhq, const uint8_t* h_scale, int64_t ld_scale,
                                    uint16_t* dh, int64_t lddh, uint16_t* a, int64_t lda, void* stream) {
    const char* fn = "fp8_mx_swiglu_backward";
    FP8_TRY(check_swiglu_backward(fn, da, rows, inter, ldda, dh, lddh, a, lda));
    if (inter % FP8_MX_BLOCK != 0)
        return fail(FP8_ERR_INVALID_ARG, "%s: inter = %lld is not a multiple of %d", fn, (long long)inter, FP8_MX_BLOCK);
    FP8_TRY(check_checkpoint(fn, "hq", hq, (int)h_fmt, ldhq, h_scale, ld_scale, rows, 2 * inter));
    FP8_TRY(check_device());
    SwigluBwd p{};
    p.da = da;
    p.rows = rows;
    p.inter = inter;
    p.ldda = ldda;
    p.hq = hq;
    p.ldhq = ldhq;
    p.hs = h_scale;
    p.ldhs = ld_scale;
    p.ckpt_e5m2 = h_fmt == FP8_E5M2;
    p.dh = dh;
    p.lddh = lddh;
    p.a = a;
    p.lda = lda;
    return launched(launch_swiglu_backward(p, (hipStream_t)stream), fn);
}

fp8_status_t fp8_moe_few_tokens(const uint16_t* x, int64_t tokens, int64_t hidden, int64_t ldx,
                                const int32_t* expert_idx, const float* weights, int32_t topk, int32_t num_experts,
                                const uint8_t* w1, fp8_format_t f1, int64_t ld1, int64_t w1_expert_stride,
                                const float* w1_scale_inv, const uint8_t* w2, fp8_format_t f2, int64_t ld2,
                                int64_t w2_expert_stride, const float* w2_scale_inv, int64_t inter, uint16_t* out,
                                int64_t ldo, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "fp8_moe_few_tokens";
    static_assert(kMoeFewTokens == FP8_MOE_FEW_TOKENS, "one limit");
    if (hidden < 16 || inter < 16 || hidden % 16 != 0 || inter % 16 != 0 || hidden >= (1 << 20) || inter >= (1 << 20))
        return fail(FP8_ERR_INVALID_ARG, "%s: hidden = %lld and inter = %lld must be multiples of 16, 16 .. 2^20 - 16",
                    fn, (long long)hidden, (long long)inter);
    FP8_TRY(check_matrix(fn, "x", x, tokens, hidden, ldx));
    FP8_TRY(check_matrix(fn, "out", out, tokens, hidden, ldo));
    if (topk < 1 || topk > kMoeMaxTopk) return fail(FP8_ERR_INVALID_ARG, "%s: topk %d outside 1..%d", fn, topk, kMoeMaxTopk);
    if (num_experts < 1 || num_experts > kMoeMaxExperts)
        return fail(FP8_ERR_INVALID_ARG, "%s: expert count %d outside 1..%d", fn, num_experts, kMoeMaxExperts);
    if (!valid_fmt((int)f1) || !valid_fmt((int)f2))
        return fail(FP8_ERR_INVALID_ARG, "%s: unknown format (%d, %d)", fn, (int)f1, (int)f2);
    if (ld1 < hidden || ld2 < inter || w1_expert_stride < 0 || w2_expert_stride < 0)
        return fail(FP8_ERR_INVALID_ARG, "%s: leading dimension smaller than the row, or negative expert stride", fn);
    if (tokens > 0 && (!expert_idx || !weights || !w1 || !w1_scale_inv || !w2 || !w2_scale_inv || !workspace))
        return fail(FP8_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(w1, 16) || !aligned(w2, 16) || ld1 % 16 != 0 || ld2 % 16 != 0 ||
        w1_expert_stride % 16 != 0 || w2_expert_stride % 16 != 0)
        return fail(FP8_ERR_ALIGNMENT, "%s: x, w1, w2 must be 16-byte aligned with ldx a multiple of 8, ld1, ld2 and the "
                    "expert strides multiples of 16", fn);
    if (!aligned(expert_idx, 4) || !aligned(weights, 4) || !aligned(w1_scale_inv, 4) || !aligned(w2_scale_inv, 4) ||
        !aligned(out, 2) || !aligned(workspace, 16))
        return fail(FP8_ERR_ALIGNMENT, "%s: misaligned pointer", fn);
    if (!ocp_fmt((int)f1) || !ocp_fmt((int)f2))
        return fail(FP8_ERR_UNSUPPORTED, "%s: fnuz weights (%d, %d): OCP e4m3 / e5m2 only", fn, (int)f1, (int)f2);
    if (tokens > kMoeFewTokens)
        return fail(FP8_ERR_UNSUPPORTED, "%s: %lld tokens, at most %d", fn, (long long)tokens, kMoeFewTokens);
    if (tokens > 0 && workspace_bytes < tokens * topk * inter * 4)
        return fail(FP8_ERR_INVALID_ARG, "%s: a workspace of %lld bytes is needed", fn,
                    (long long)(tokens * topk * inter * 4));
    FP8_TRY(check_device());
    MoeFew p{};
    p.x = x;
    p.ldx = ldx;
    p.idx = expert_idx;
    p.weights = weights;
    p.tokens = (int)tokens;
    p.topk = topk;
    p.experts = num_experts;
    p.w1 = w1;
    p.ld1 = ld1;
    p.gs1 = w1_expert_stride;
    p.s1 = w1_scale_inv;
    p.w2 = w2;
    p.ld2 = ld2;
    p.gs2 = w2_expert_stride;
    p.s2 = w2_scale_inv;
    p.hidden = (int)hidden;
    p.inter = (int)inter;
    p.ws = static_cast<uint16_t*>(workspace);
    p.out = out;
    p.ldo = ldo;
    return launched(launch_moe_few_tokens(p, (int)f1, (int)f2, (hipStream_t)stream), fn);
}

}  // extern "C"
