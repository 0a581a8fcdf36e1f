// checks.hpp - what the files of the C ABI share: the thread's error message,
// the per-device properties cache, and the argument checks that run before any
// launch.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/fp8amax.h"
#include "kernels.hpp"

namespace fp8amax {

inline thread_local char g_err[512] = "";

inline fp8_status_t fail(fp8_status_t st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return st;
}

inline fp8_status_t ok() {
    g_err[0] = '\0';
    return FP8_OK;
}

constexpr int kMaxDevices = 64;
struct PropsSlot {
    std::once_flag once;
    DeviceProps props{};
    bool gfx950 = false;
    hipError_t err = hipSuccess;
};
inline PropsSlot g_props[kMaxDevices];

inline PropsSlot* slot_for_current(int* dev_out) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    PropsSlot& s = g_props[dev];
    std::call_once(s.once, [&s, dev]() {
        hipDeviceProp_t p;
        s.err = hipGetDeviceProperties(&p, dev);
        if (s.err == hipSuccess) {
            s.props.cus = p.multiProcessorCount;
            s.gfx950 = std::strncmp(p.gcnArchName, "gfx950", 6) == 0;
        }
    });
    if (dev_out) *dev_out = dev;
    return &s;
}

inline bool valid_fmt(int f) { return f >= FP8_E4M3 && f <= FP8_E5M2_FNUZ; }
inline bool ocp_fmt(int f) { return f == FP8_E4M3 || f == FP8_E5M2; }
inline bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Device check shared by every compute entry point (after argument checks).
inline fp8_status_t check_device() {
    int dev = 0;
    PropsSlot* s = slot_for_current(&dev);
    if (!s) return fail(FP8_ERR_HIP, "cannot query the current HIP device");
    if (s->err != hipSuccess) return fail(FP8_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(s->err));
    if (!s->gfx950) return fail(FP8_ERR_UNSUPPORTED, "device %d is not gfx950 (MI355X); this library is built for gfx950 only", dev);
    return FP8_OK;
}

inline fp8_status_t launched(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(FP8_ERR_HIP, "%s: launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

inline fp8_status_t check_matrix(const char* fn, const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (rows < 0 || cols < 0) return fail(FP8_ERR_INVALID_ARG, "%s: %s has negative size %lld x %lld", fn, name,
                                          (long long)rows, (long long)cols);
    if (ld < cols || ld < 1) return fail(FP8_ERR_INVALID_ARG, "%s: leading dimension of %s (%lld) < max(cols, 1) (%lld)",
                                        fn, name, (long long)ld, (long long)cols);
    if (!p && rows > 0 && cols > 0) return fail(FP8_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    return FP8_OK;
}

#define FP8_TRY(expr)                          \
    do {                                       \
        fp8_status_t _s = (expr);              \
        if (_s != FP8_OK) return _s;           \
    } while (0)

inline fp8_status_t check_common_quant(const char* fn, const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, int fmt,
                                       int margin) {
    FP8_TRY(check_matrix(fn, "x", x, rows, cols, ldx));
    if (!valid_fmt(fmt)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown format %d", fn, fmt);
    if (margin < 0 || margin > 32) return fail(FP8_ERR_INVALID_ARG, "%s: margin %d outside 0..32", fn, margin);
    if (!aligned(x, 2)) return fail(FP8_ERR_ALIGNMENT, "%s: x is not 2-byte aligned", fn);
    return FP8_OK;
}

}  // namespace fp8amax
