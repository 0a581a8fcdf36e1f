// layer_checks.hpp - argument checks that the entry points of the layer around the
// products share (api_layer.cpp, api_block.cpp).
#pragma once

#include "checks.hpp"
#include "layer.hpp"

namespace fp8amax {

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxCols = (int64_t)1 << 27;      // of a norm's gradient: 16 threads a column add the bands, in one grid

inline fp8_status_t check_rows(const char* fn, int64_t rows, int64_t limit) {
    if (rows >= limit) return fail(FP8_ERR_UNSUPPORTED, "%s: %lld rows or more", fn, (long long)limit);
    return FP8_OK;
}

inline fp8_status_t check_weights(const char* fn, const void* gamma, const void* beta, int w_type) {
    if (w_type != FP8_OUT_BF16 && w_type != FP8_OUT_F32)
        return fail(FP8_ERR_INVALID_ARG, "%s: unknown weight type %d", fn, w_type);
    const unsigned a = w_type == FP8_OUT_F32 ? 4 : 2;
    if (!aligned(gamma, a) || !aligned(beta, a))
        return fail(FP8_ERR_ALIGNMENT, "%s: gamma and beta must be aligned to their type", fn);
    return FP8_OK;
}

inline fp8_status_t check_kind(const char* fn, int kind) {
    if (kind != FP8_NORM_LAYER && kind != FP8_NORM_RMS)
        return fail(FP8_ERR_INVALID_ARG, "%s: unknown norm %d", fn, kind);
    return FP8_OK;
}

// An MX checkpoint [rows x cols]: codes q (ldq) and scale records (ld_scale).
inline fp8_status_t check_checkpoint(const char* fn, const char* name, const uint8_t* q, int fmt, int64_t ldq,
                              const uint8_t* scale, int64_t ld_scale, int64_t rows, int64_t cols) {
    FP8_TRY(check_matrix(fn, name, q, rows, cols, ldq));
    if (!ocp_fmt(fmt)) return fail(FP8_ERR_INVALID_ARG, "%s: the checkpoint's codes are OCP e4m3 or e5m2 (format %d)", fn, fmt);
    if (cols % FP8_MX_BLOCK != 0)
        return fail(FP8_ERR_INVALID_ARG, "%s: the checkpoint's %lld columns are not a multiple of %d", fn,
                    (long long)cols, FP8_MX_BLOCK);
    if (rows > 0 && !scale) return fail(FP8_ERR_INVALID_ARG, "%s: the checkpoint's scale records are NULL", fn);
    if (ld_scale < rows || ld_scale < 1)
        return fail(FP8_ERR_INVALID_ARG, "%s: scale record stride %lld < rows", fn, (long long)ld_scale);
    if (!aligned(q, 8) || ldq % 8 != 0 || !aligned(scale, 4))
        return fail(FP8_ERR_ALIGNMENT, "%s: the checkpoint's codes must be 8-byte aligned with a row stride that is a "
                    "multiple of 8, its scale records 4-byte aligned", fn);
    return FP8_OK;
}

inline fp8_status_t check_norm_backward(const char* fn, const uint16_t* dy, int64_t rows, int64_t cols, int64_t lddy,
                                 const void* gamma, const void* beta, int w_type, const float* rstd, int kind,
                                 const uint16_t* dx, int64_t lddx, const float* dgamma, const float* dbeta,
                                 const void* workspace, int64_t workspace_bytes) {
    FP8_TRY(check_matrix(fn, "dy", dy, rows, cols, lddy));
    FP8_TRY(check_matrix(fn, "dx", dx, rows, cols, lddx));
    if (cols < 1) return fail(FP8_ERR_INVALID_ARG, "%s: no columns", fn);
    FP8_TRY(check_kind(fn, kind));
    FP8_TRY(check_weights(fn, gamma, beta, w_type));
    if (rows > 0 && !rstd) return fail(FP8_ERR_INVALID_ARG, "%s: rstd is NULL", fn);
    if (!aligned(dy, 2) || !aligned(dx, 2) || !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4))
        return fail(FP8_ERR_ALIGNMENT, "%s: misaligned pointer", fn);
    FP8_TRY(check_rows(fn, rows, kMaxRows));
    if (cols >= kMaxCols) return fail(FP8_ERR_UNSUPPORTED, "%s: %lld columns or more", fn, (long long)kMaxCols);
    if (dgamma || dbeta) {
        const int64_t need = fp8_norm_backward_workspace(rows, cols);
        if (need > 0 && (!workspace || workspace_bytes < need))
            return fail(FP8_ERR_INVALID_ARG, "%s: a workspace of %lld bytes is needed", fn, (long long)need);
        if (!aligned(workspace, 16)) return fail(FP8_ERR_ALIGNMENT, "%s: the workspace must be 16-byte aligned", fn);
    }
    return FP8_OK;
}

}  // namespace fp8amax
