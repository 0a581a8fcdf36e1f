// api_layer_sanitize_driver.cpp - the host code of the layer's entry points
// (csrc/api_layer.cpp: argument validation and dispatch) under the address and
// undefined-behaviour sanitizers, without a GPU. The kernel launchers and the
// HIP runtime calls are stubs (one gfx950 device); each launcher checks that
// what reaches it is what the call said, and the extreme sizes that the
// documentation allows and refuses go through the arithmetic of the checks.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>

#include "../fp8_scaled_gemm_amax_amd/csrc/checks.hpp"
#include "../fp8_scaled_gemm_amax_amd/csrc/layer.hpp"

static int g_fail = 0, g_launched = 0;
#define CHECK(cond)                                                         \
    do {                                                                    \
        if (!(cond)) {                                                      \
            std::fprintf(stderr, "FAILED line %d: %s (%s)\n", __LINE__, #cond, fp8amax::g_err); \
            ++g_fail;                                                       \
        }                                                                   \
    } while (0)

extern "C" {
hipError_t hipGetDevice(int* d) {
    *d = 0;
    return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
    std::memset(p, 0, sizeof *p);
    std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
    p->multiProcessorCount = 256;
    return hipSuccess;
}
const char* hipGetErrorString(hipError_t) { return "stub"; }
}

namespace fp8amax {
hipError_t launch_norm_quant_row(const NormFwd& p, int fmt, hipStream_t) {
    ++g_launched;
    CHECK(p.cols >= 1 && p.rows >= 0 && fmt >= 0 && fmt <= 3);
    CHECK(!p.xq || norm_vector_layout(p) || p.rows == 0);
    return hipSuccess;
}
hipError_t launch_norm_backward(const NormBwd& p, hipStream_t) {
    ++g_launched;
    CHECK(!p.xq || norm_vector_layout(p) || p.rows == 0);
    CHECK(!(p.dgamma || p.dbeta) || p.partial || p.rows == 0);
    return hipSuccess;
}
hipError_t launch_swiglu_quant_row_mx(const SwigluFwd& p, int, hipStream_t) {
    ++g_launched;
    CHECK(p.inter % 32 == 0 && p.inter <= kSwigluMxMaxInter);
    return hipSuccess;
}
hipError_t launch_swiglu_backward(const SwigluBwd& p, hipStream_t) {
    ++g_launched;
    CHECK(p.inter % 8 == 0 && (p.h != nullptr) != (p.hq != nullptr));
    return hipSuccess;
}
hipError_t launch_moe_few_tokens(const MoeFew& p, int f1, int f2, hipStream_t) {
    ++g_launched;
    CHECK(p.tokens <= kMoeFewTokens && f1 <= 1 && f2 <= 1 && p.hidden % 16 == 0 && p.inter % 16 == 0);
    return hipSuccess;
}
}  // namespace fp8amax

static void* dev(uintptr_t i) { return reinterpret_cast<void*>((uintptr_t)0x7f0000000000ull + i * 0x100000ull); }
#define U16(i) static_cast<uint16_t*>(dev(i))
#define U8(i) static_cast<uint8_t*>(dev(i))
#define F32(i) static_cast<float*>(dev(i))
#define RUN(call, want)                     \
    do {                                    \
        const int before = g_launched;      \
        CHECK((call) == (want));            \
        CHECK(g_launched == before + ((want) == FP8_OK)); \
    } while (0)

int main() {
    const int64_t big = INT64_MAX;
    const auto LN = FP8_NORM_LAYER;
    const auto BF = FP8_OUT_BF16;
    auto norm = [&](int64_t rows, int64_t cols, int64_t ld, bool save) {
        return fp8_norm_quantize_row(U16(1), rows, cols, ld, dev(2), dev(3), BF, 1e-5f, LN, FP8_E4M3, 0, U8(4), ld,
                                     F32(5), U16(6), ld, F32(7), F32(8), save ? U8(9) : nullptr, FP8_E4M3, ld,
                                     save ? U8(10) : nullptr, rows > 1 ? rows : 1, nullptr);
    };
    RUN(norm(4, 64, 64, true), FP8_OK);
    RUN(norm(4, 63, 63, false), FP8_OK);
    RUN(norm(0, 64, 64, true), FP8_OK);
    RUN(norm((1 << 30) - 1, 16384, 16384, true), FP8_OK);
    RUN(norm(big, 64, 64, false), FP8_ERR_UNSUPPORTED);
    RUN(norm(4, big, big, false), FP8_OK);
    RUN(norm(4, big, 64, false), FP8_ERR_INVALID_ARG);
    RUN(norm(-big, 64, 64, false), FP8_ERR_INVALID_ARG);
    auto grad = [&](int64_t rows, int64_t cols, int64_t ld, int64_t bytes) {
        return fp8_norm_backward(U16(1), rows, cols, ld, U16(2), ld, dev(3), BF, F32(4), F32(5), LN, U16(6), ld, F32(7),
                                 F32(8), dev(9), bytes, nullptr);
    };
    RUN(grad(4, 64, 64, 2048), FP8_OK);
    RUN(grad(4, 64, 64, 2047), FP8_ERR_INVALID_ARG);
    RUN(grad(0, 64, 64, 0), FP8_OK);
    RUN(grad((1 << 30) - 1, 64, 64, 512 * 2 * 64 * 4), FP8_OK);
    RUN(grad(big, 64, 64, big), FP8_ERR_UNSUPPORTED);
    CHECK(fp8_norm_backward_workspace(big, big) == 0 && fp8_norm_backward_workspace(1000, ((int64_t)1 << 27) - 1) > 0);
    auto mx = [&](int64_t rows, int64_t cols, int64_t ld) {
        return fp8_mx_norm_backward(U16(1), rows, cols, ld, U8(2), FP8_E5M2, ld, U8(3), rows > 1 ? rows : 1, dev(4),
                                    dev(5), FP8_OUT_F32, F32(6), FP8_NORM_RMS, U16(7), ld, nullptr, nullptr, U16(8), ld,
                                    nullptr, 0, nullptr);
    };
    RUN(mx(4, 64, 64), FP8_OK);
    RUN(mx(4, 16384, 16384), FP8_OK);
    RUN(mx(4, 16416, 16416), FP8_ERR_UNSUPPORTED);
    RUN(mx(4, 64, big), FP8_ERR_ALIGNMENT);
    auto save = [&](int64_t rows, int64_t inter) {
        const int64_t w = inter > 0 && inter < (1 << 20) ? inter : 64;
        return fp8_swiglu_quantize_row_mx(U16(1), rows, inter, 2 * w, FP8_E4M3, 0, U8(2), w, F32(3), U8(4), FP8_E4M3,
                                          2 * w, U8(5), rows > 1 ? rows : 1, nullptr);
    };
    RUN(save(4, 64), FP8_OK);
    RUN(save(0, 64), FP8_OK);
    RUN(save(4, 16384), FP8_OK);
    RUN(save(4, 16416), FP8_ERR_UNSUPPORTED);
    RUN(save(4, big), FP8_ERR_INVALID_ARG);
    RUN(save(4, -32), FP8_ERR_INVALID_ARG);
    RUN(save(big, 64), FP8_ERR_UNSUPPORTED);
    auto back = [&](int64_t rows, int64_t inter) {
        const int64_t w = inter > 0 && inter < (1 << 20) ? inter : 64;
        return fp8_swiglu_backward(U16(1), rows, inter, w, U16(2), 2 * w, U16(3), 2 * w, U16(4), w, nullptr);
    };
    RUN(back(4, 40), FP8_OK);
    RUN(back((1 << 30) - 1, 64), FP8_OK);
    RUN(back(big, 64), FP8_ERR_UNSUPPORTED);
    RUN(back(4, big), FP8_ERR_INVALID_ARG);
    RUN(fp8_mx_swiglu_backward(U16(1), 4, 64, 64, U8(2), FP8_E4M3, 128, U8(3), 4, U16(4), 128, nullptr, 0, nullptr), FP8_OK);
    auto moe = [&](int64_t tokens, int32_t topk, int64_t hidden, int64_t inter, int64_t bytes) {
        const int64_t H = hidden > 0 && hidden < (1 << 20) ? hidden : 16, I = inter > 0 && inter < (1 << 20) ? inter : 16;
        return fp8_moe_few_tokens(U16(1), tokens, hidden, H, static_cast<int32_t*>(dev(2)), F32(3), topk, 8, U8(4),
                                  FP8_E4M3, H, 0, F32(5), U8(6), FP8_E5M2, I, big / 16 * 16, F32(7), inter, U16(8), H,
                                  dev(9), bytes, nullptr);
    };
    RUN(moe(64, 64, (1 << 20) - 16, (1 << 20) - 16, (int64_t)64 * 64 * ((1 << 20) - 16) * 4), FP8_OK);
    RUN(moe(64, 64, (1 << 20) - 16, (1 << 20) - 16, (int64_t)64 * 64 * ((1 << 20) - 16) * 4 - 1), FP8_ERR_INVALID_ARG);
    RUN(moe(0, 2, 64, 64, 0), FP8_OK);
    RUN(moe(65, 2, 64, 64, big), FP8_ERR_UNSUPPORTED);
    RUN(moe(big, 2, 64, 64, big), FP8_ERR_UNSUPPORTED);
    RUN(moe(1, 2, big, 64, big), FP8_ERR_INVALID_ARG);
    RUN(moe(1, 2, 64, -big, big), FP8_ERR_INVALID_ARG);
    if (g_fail) return 1;
    std::printf("layer api host code: every check passed under the sanitizers\n");
    return 0;
}
