// norm_grid_driver.cpp - the grid of the weights' gradients of a norm in any layout
// (any_cols_grid of csrc/layer.hpp) up to the largest number of columns that the
// entry point accepts: every column has its thread, a direction's threads stay
// below 2^32, and no more than one row of workgroups is partly past the columns.
#include <cstdint>
#include <cstdio>

#include "../fp8_scaled_gemm_amax_amd/csrc/layer.hpp"

using namespace fp8amax;

int main() {
    const int64_t limit = (int64_t)1 << 27, threads = (int64_t)kAnyCols * kAnySlices;
    int bad = 0;
    auto check = [&](int64_t cols) {
        if (cols < 1 || cols >= limit) return;
        const ColsGrid g = any_cols_grid(cols);
        const bool fits = g.x >= 1 && g.z >= 1 && g.z < 65536 && g.x * threads < ((int64_t)1 << 32);
        const bool covers = (int64_t)g.x * g.z * kAnyCols >= cols && (int64_t)g.x * (g.z - 1) * kAnyCols < cols;
        if (!fits || !covers) {
            ++bad;
            std::fprintf(stderr, "%lld columns: grid %u x %u\n", (long long)cols, g.x, g.z);
        }
    };
    for (int64_t cols = 1; cols < 4096; ++cols) check(cols);
    for (int64_t p = 4096; p <= limit; p *= 2)
        for (int64_t d = -65; d <= 65; ++d) check(p + d);
    for (int64_t cols = 1000003; cols < limit; cols += 1000003) check(cols);
    if (bad) return 1;
    std::printf("every grid fits and covers its columns\n");
    return 0;
}
