// api_block_sanitize_driver.cpp - the host code of a block's entry points
// (csrc/api_block.cpp: argument validation and dispatch) under the address and
// undefined-behaviour sanitizers, without a GPU. The kernel launchers and the HIP
// runtime calls are stubs (one gfx950 device); each launcher checks what its kernels
// assume, and the extreme sizes that the documentation allows and refuses go through
// the arithmetic of the checks.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>

#include "../fp8_scaled_gemm_amax_amd/csrc/block.hpp"
#include "../fp8_scaled_gemm_amax_amd/csrc/layer_checks.hpp"

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
// (the norm's own workspace size is api_layer.cpp's)
int64_t fp8_norm_backward_workspace(int64_t rows, int64_t cols) {
    return (rows < 512 ? rows : 512) * 2 * cols * 4;
}
}

namespace fp8amax {
hipError_t launch_norm_quant_row(const NormFwd& p, int fmt, hipStream_t) {
    ++g_launched;
    CHECK(p.cols >= 1 && p.rows >= 1 && p.res && p.sum && fmt >= 0 && fmt <= 3);
    CHECK(!p.xq || norm_vector_layout(p));
    return hipSuccess;
}
hipError_t launch_norm_backward(const NormBwd& p, hipStream_t) {
    ++g_launched;
    CHECK(p.ds || p.rows == 0);
    CHECK(!p.xq || norm_vector_layout(p) || p.rows == 0);
    CHECK(!(p.dgamma || p.dbeta) || p.partial || p.rows == 0);
    return hipSuccess;
}
hipError_t launch_gemm_swiglu(const GluFwd& p, int fa, int fb, hipStream_t) {
    ++g_launched;
    CHECK(fa <= 1 && fb <= 1 && p.k % 16 == 0 && p.lda < (1 << 24) && p.ldb < (1 << 24) && p.inter < (1 << 24));
    CHECK((p.m + 127) / 128 * ((p.inter + 63) / 64) < (1 << 24) && p.ldact < (1 << 25) && (!p.h || p.ldh < (1 << 25)));
    return hipSuccess;
}
hipError_t launch_gemm_swiglu_backward(const GluBwd& p, int fa, int fb, hipStream_t) {
    ++g_launched;
    CHECK(fa <= 1 && fb <= 1 && p.k % 16 == 0 && p.lda < (1 << 24) && p.ldb < (1 << 24) && p.inter < (1 << 24));
    CHECK(p.ldh < (1 << 25) && p.lddh < (1 << 25) && (!p.act || p.ldact < (1 << 25)));
    return hipSuccess;
}
hipError_t launch_lora_add(const Lora& p, hipStream_t) {
    ++g_launched;
    CHECK(p.rank % 8 == 0 && p.rank >= 8 && p.rank <= kLoraMaxRank && p.k % 8 == 0 && p.k >= 8 && p.adapters >= 1);
    CHECK(p.tokens < (1 << 25) && p.n < (1 << 24) && p.ldx < (1 << 24) && p.ldout < (1 << 24));
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
    const auto BF = FP8_OUT_BF16;
    auto norm = [&](int64_t rows, int64_t cols, int64_t ld, bool save, int sum) {
        return fp8_add_norm_quantize_row(U16(1), rows, cols, ld, U16(2), ld, U16(sum), ld, dev(4), dev(5), BF, 1e-5f,
                                         FP8_NORM_LAYER, FP8_E4M3, 0, U8(6), ld, F32(7), U16(8), ld, F32(9), F32(10),
                                         save ? U8(11) : nullptr, FP8_E4M3, ld, save ? U8(12) : nullptr,
                                         rows > 1 ? rows : 1, nullptr);
    };
    RUN(norm(4, 64, 64, true, 3), FP8_OK);
    RUN(norm(4, 64, 64, true, 2), FP8_OK);
    RUN(norm(4, 63, 63, false, 1), FP8_OK);
    CHECK(norm(0, 64, 64, true, 3) == FP8_OK);
    RUN(norm((1 << 30) - 1, 16384, 16384, true, 3), FP8_OK);
    RUN(norm(big, 64, 64, false, 3), FP8_ERR_UNSUPPORTED);
    RUN(norm(4, big, big, false, 3), FP8_OK);
    RUN(norm(4, big, 64, false, 3), FP8_ERR_INVALID_ARG);
    RUN(norm(-big, 64, 64, false, 3), FP8_ERR_INVALID_ARG);
    auto grad = [&](int64_t rows, int64_t cols, int64_t ld, int64_t bytes) {
        return fp8_add_norm_backward(U16(10), ld, U16(1), rows, cols, ld, U16(2), ld, dev(3), BF, F32(4), F32(5),
                                     FP8_NORM_LAYER, U16(6), ld, F32(7), F32(8), dev(9), bytes, nullptr);
    };
    RUN(grad(4, 64, 64, 2048), FP8_OK);
    RUN(grad(4, 64, 64, 2047), FP8_ERR_INVALID_ARG);
    RUN(grad(0, 64, 64, 0), FP8_OK);
    RUN(grad((1 << 30) - 1, 64, 64, 512 * 2 * 64 * 4), FP8_OK);
    RUN(grad(big, 64, 64, big), FP8_ERR_UNSUPPORTED);
    auto mx = [&](int64_t rows, int64_t cols, int64_t ld) {
        return fp8_mx_add_norm_backward(U16(10), ld, U16(1), rows, cols, ld, U8(2), FP8_E5M2, ld, U8(3),
                                        rows > 1 ? rows : 1, dev(4), dev(5), FP8_OUT_F32, F32(6), FP8_NORM_RMS, U16(7), ld,
                                        nullptr, nullptr, U16(8), ld, nullptr, 0, nullptr);
    };
    RUN(mx(4, 64, 64), FP8_OK);
    RUN(mx(4, 16384, 16384), FP8_OK);
    RUN(mx(4, 16416, 16416), FP8_ERR_UNSUPPORTED);
    RUN(mx(4, 64, big), FP8_ERR_ALIGNMENT);
    auto glu = [&](int64_t m, int64_t inter, int64_t k, int64_t ldk, int64_t ldh) {
        return fp8_gemm_swiglu(U8(1), FP8_E4M3, ldk, U8(2), FP8_E5M2, ldk, m, inter, k, F32(3), FP8_SCALE_VECTOR, F32(4),
                               FP8_SCALE_TENSOR, U16(5), ldh, U16(6), ldh, nullptr);
    };
    auto glu_back = [&](int64_t m, int64_t inter, int64_t k, int64_t ldk, int64_t ldh) {
        return fp8_gemm_swiglu_backward(U8(1), FP8_E5M2, ldk, U8(2), FP8_E4M3, ldk, m, inter, k, F32(3), FP8_SCALE_VECTOR,
                                        F32(4), FP8_SCALE_VECTOR, U16(5), ldh, U16(6), ldh, U16(7), ldh, nullptr);
    };
    const int64_t wide = (1 << 25) - 1;
    for (int which = 0; which < 2; ++which) {
        auto run = [&](int64_t m, int64_t inter, int64_t k, int64_t ldk, int64_t ldh) {
            return which ? glu_back(m, inter, k, ldk, ldh) : glu(m, inter, k, ldk, ldh);
        };
        RUN(run(4, 64, 64, 64, 128), FP8_OK);
        RUN(run(0, 64, 64, 64, 128), FP8_OK);
        RUN(run(4, 0, 64, 64, 1), FP8_OK);
        RUN(run(4, 64, 0, 16, 128), FP8_OK);
        RUN(run(4, 64, (1 << 24) - 16, (1 << 24) - 16, 128), FP8_OK);
        RUN(run(128 * 64 - 1, (1 << 24) - 128, 64, 64, wide), FP8_OK);
        RUN(run(128 * 64 + 1, (1 << 24) - 64, 64, 64, wide), FP8_ERR_UNSUPPORTED);
        RUN(run(4, 1 << 24, 64, 64, big), FP8_ERR_UNSUPPORTED);
        RUN(run(4, 64, 64, 1 << 24, 128), FP8_ERR_UNSUPPORTED);
        RUN(run(4, 64, 64, 64, wide + 1), FP8_ERR_UNSUPPORTED);
        RUN(run(big, 64, 64, 64, 128), FP8_ERR_UNSUPPORTED);
        RUN(run(4, big, 64, 64, 128), FP8_ERR_UNSUPPORTED);
        RUN(run(4, 64, big / 16 * 16, 64, 128), FP8_ERR_INVALID_ARG);
        RUN(run(4, 64, big / 16 * 16, big / 16 * 16, 128), FP8_ERR_UNSUPPORTED);
        RUN(run(-big, 64, 64, 64, 128), FP8_ERR_INVALID_ARG);
    }
    auto lora = [&](int64_t tokens, int64_t k, int32_t rank, int64_t n, int64_t ld, int64_t bytes) {
        return fp8_lora_add(U16(1), tokens, k, ld, static_cast<int32_t*>(dev(2)), U16(3), ld, 0, U16(4), 128, 0, F32(5),
                            INT32_MAX, rank, n, U16(6), ld, U16(6), ld, dev(7), bytes, nullptr);
    };
    RUN(lora(4, 64, 16, 64, 64, 4 * 16 * 16 * 4), FP8_OK);
    RUN(lora(4, 64, 16, 64, 64, 4 * 16 * 16 * 4 - 1), FP8_ERR_INVALID_ARG);
    RUN(lora(0, 64, 16, 64, 64, 0), FP8_OK);
    RUN(lora(4, 64, 16, 0, 64, 0), FP8_OK);
    RUN(lora((1 << 25) - 1, (1 << 24) - 8, 128, (1 << 24) - 8, (1 << 24) - 8, big), FP8_OK);
    RUN(lora(1 << 25, 64, 16, 64, 64, big), FP8_ERR_UNSUPPORTED);
    RUN(lora(4, 64, 16, 1 << 24, 1 << 24, big), FP8_ERR_UNSUPPORTED);
    RUN(lora(4, 64, 16, 64, 1 << 24, big), FP8_ERR_UNSUPPORTED);
    RUN(lora(big, 64, 16, 64, 64, big), FP8_ERR_UNSUPPORTED);
    RUN(lora(4, big, 16, 64, 64, big), FP8_ERR_INVALID_ARG);
    RUN(lora(4, 64, 16, big, 64, big), FP8_ERR_INVALID_ARG);
    RUN(lora(-big, 64, 16, 64, 64, big), FP8_ERR_INVALID_ARG);
    CHECK(fp8_lora_workspace(big, 16) == 0 && fp8_lora_workspace(-big, 16) == 0 && fp8_lora_workspace(1 << 29, 128) > 0);
    using namespace fp8amax;
    for (int64_t t = 1; t < 20000; ++t) {       // parts * tokens fit
        const int64_t rows = lora_part_rows(t), parts = kLoraPartRows / t < kLoraMaxParts ? kLoraPartRows / t : kLoraMaxParts;
        CHECK((parts < 1 ? 1 : parts) * t <= rows);
    }
    if (g_fail) return 1;
    std::printf("block api host code: every check passed under the sanitizers\n");
    return 0;
}
