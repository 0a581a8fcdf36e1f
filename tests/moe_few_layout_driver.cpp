// moe_few_layout_driver.cpp - every place of the workspace that the MoE layer for
// a few tokens writes and loads, replayed on the host with the kernels' own
// arithmetic (csrc/moe_few_layout.hpp): for every number of an expert's tokens
// and lengths of K that end at every group of a step, no write and no load
// leaves the rows of the entries up to the expert's last one (the smallest
// workspace that the call may be given), writes do not meet, and the columns
// that are used load the token, part and K that they are multiplied as.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "../fp8_scaled_gemm_amax_amd/csrc/moe_few_layout.hpp"

using namespace fp8amax;

static int g_fail = 0;
static void fail(const char* what, int count, int base, int inter, int64_t at, int64_t rows) {
    if (++g_fail <= 20)
        std::fprintf(stderr, "%s: %d tokens after %d entries, inter %d: value %lld of %lld\n", what, count, base, inter,
                     (long long)at, (long long)rows * 2 * inter);
}

// The value that stands at a place: token, part and K of the activation.
static int32_t tag(int token, int part, int k) { return ((token * 2 + part) << 16 | k) + 1; }

static void replay(int count, int base, int inter) {
    const int64_t rows = base + count, values = rows * 2 * inter;
    std::vector<int32_t> ws((size_t)values, 0);
    // gate and up: 16 columns from c0 on, token c of the expert, row 0 .. 15
    for (int c = 0; c < count; ++c) {
        ActTile t;
        t.set(base, count, inter, c / kActTile);
        for (int k = 0; k < inter; ++k)
            for (int part = 0; part < 2; ++part) {
                const int64_t at = t.first + t.offset(k >> 6, (k >> 3) & 1, (k >> 4) & 3, part, c % kActTile) + (k & 7);
                if (at < (int64_t)base * 2 * inter || at >= values) fail("a write out of range", count, base, inter, at, rows);
                else if (ws[(size_t)at]) fail("two writes of one value", count, base, inter, at, rows);
                else ws[(size_t)at] = tag(c, part, k);
            }
    }
    // down: whole blocks, then what is left of K
    const DownShape shape = down_shape(count);
    for (int n = 0; n < shape.tiles; ++n) {
        ActTile t;
        t.set(base, count, inter, n);
        for (int lane = 0; lane < 64; ++lane) {
            const int c = n * kActTile + (lane & 7), part = (lane >> 3) & 1, group = lane >> 4;
            auto load = [&](int64_t at, int k) {
                if (at < 0 || at + 8 > values) return fail("a load out of range", count, base, inter, at, rows);
                if (at % 8) return fail("a load off 16 bytes", count, base, inter, at, rows);
                if (c >= count) return;                     // (the column is used nowhere)
                for (int i = 0; i < 8; ++i)
                    if (ws[(size_t)at + i] != tag(c, part, k + i)) return fail("a load of another value", count, base, inter, at, rows);
            };
            const int col = t.lane(lane), bytes = 64 * shape.steps, whole = inter / bytes;
            for (int step = 0; step < whole * shape.steps; ++step)
                for (int h = 0; h < 2; ++h) load(t.first + t.whole(step, h, col), step * 64 + group * 16 + h * 8);
            for (int k0 = whole * bytes; k0 < inter; k0 += 64) {
                const int k = k0 + group * 16;
                for (int h = 0; k < inter && h < 2; ++h) load(t.first + t.last(k, h, lane), k + h * 8);
            }
        }
    }
}

int main() {
    std::vector<int> lengths;
    for (int inter = 16; inter <= 1040; inter += inter < 336 ? 16 : 176) lengths.push_back(inter);
    for (int count = 1; count <= 64; ++count) {
        if (down_shape(count).tiles * kActTile < count) fail("tokens without a tile", count, 0, 0, 0, 0);
        for (int inter : lengths)
            for (int base : {0, 1, 5, 64}) replay(count, base, inter);
        replay(count, 64 * 64 - count, 80);                 // the last expert of the largest call
    }
    // 32-bit offsets within a tile at the largest inter
    const int64_t most = (int64_t)2 * kActTile * ((1 << 20) - 16);
    if (most > INT32_MAX) fail("a tile past 32 bits", 64, 0, 1 << 20, most, 0);
    if (g_fail) {
        std::fprintf(stderr, "%d failures\n", g_fail);
        return 1;
    }
    std::printf("every write and load of the workspace is in place\n");
    return 0;
}
