// block_rules_driver.cpp - the rules of csrc/block.hpp that choose a kernel of the gated
// product, on the host: the choices of the sizes that they were measured at, on 256 CUs,
// and the same ones on a device with a quarter of them for a quarter of the columns.
#include <cstdint>
#include <cstdio>

#include "../fp8_scaled_gemm_amax_amd/csrc/block.hpp"

using namespace fp8amax;

static int bad = 0;

static void few(int64_t m, int64_t inter, bool want) {
    for (int64_t cus : {256, 64}) {
        const bool got = glu_few_rows(m, inter * cus / 256, cus);
        if (got == want) continue;
        ++bad;
        std::fprintf(stderr, "%lld rows x %lld columns on %lld CUs: few rows' kernel %d\n", (long long)m,
                     (long long)(inter * cus / 256), (long long)cus, got);
    }
}

static void tiles(const char* rule, bool (*choose)(int64_t, int64_t), int64_t count, bool want) {
    for (int64_t cus : {256, 64}) {
        if (choose(count * cus / 256, cus) == want) continue;
        ++bad;
        std::fprintf(stderr, "%s, %lld tiles on %lld CUs: not %d\n", rule, (long long)(count * cus / 256), (long long)cus, want);
    }
}

int main() {
    const auto rows64 = [](int64_t t, int64_t cus) { return glu_tiles_of_64_rows(65, t, cus); };
    for (int64_t t : {0, 4, 64}) tiles("large tiles", glu_large_tiles, t, false);
    for (int64_t t : {68, 112, 128, 100000}) tiles("large tiles", glu_large_tiles, t, true);
    for (int64_t t : {4, 66, 88, 128}) tiles("tiles of 64 rows", rows64, t, true);
    for (int64_t t : {132, 154, 224, 100000}) tiles("tiles of 64 rows", rows64, t, false);
    for (int64_t t : {1, 256, 100000})
        if (!glu_tiles_of_64_rows(64, t, 256)) ++bad;
    for (int64_t inter : {4, 1408, 4096, 6144, 11008, 14336, 28672, 100000}) {
        for (int64_t m : {1, 2, 16}) few(m, inter, true);
        for (int64_t m : {33, 64, 1000}) few(m, inter, false);
    }
    for (int64_t m : {17, 24, 32}) {
        for (int64_t inter : {4, 1408, 2048, 4096, 28672}) few(m, inter, true);
        for (int64_t inter : {6144, 8192, 11008, 14336}) few(m, inter, false);
    }
    if (bad) return 1;
    std::printf("every rule chooses what was measured\n");
    return 0;
}
