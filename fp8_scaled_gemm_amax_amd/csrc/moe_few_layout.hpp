// moe_few_layout.hpp - the workspace between the two launches of the MoE layer
// for a few tokens: where an entry's activation is written and where the down
// product loads it. Plain arithmetic, which the kernels and a host test share.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define FP8_LAYOUT __host__ __device__ __forceinline__
#else
#define FP8_LAYOUT inline
#endif

namespace fp8amax {

// An expert's activations as the down product loads them. Tile n of an expert
// (8 of its tokens, w of them there) has 2 * inter * w values from (base + 8 n) *
// 2 * inter on, base being the entries of the experts before it; its step kb of
// 64 values of K has w * 128 of them, as [half h][group j][high | low][token][8]
// for K = 64 kb + 16 j + 8 h + 0..7. A load of a wavefront (lane: token, part and
// group) is 128 w consecutive bytes and holds both parts: the high ones are
// columns 0..7 of the product, the low ones columns 8..15. (Rows of K per token
// made every load 16 lines: 32 tokens, 32 experts of 7168 x 2048, the down
// product 150 us, without its loads of activations 86; tiles of 16 tokens with
// one load for either part 108, these 105; one token 30 and 25; all of them with
// the weights loaded as the cores want them.) The last step of K has K / 16 % 4
// groups. The tiles that hold tokens add up to at most tokens * topk rows of 2 *
// inter values over all experts.
//
// The product's instances are made for 1, 2, 4 or 8 tiles, so an expert of 17 to
// 24 or of 33 to 56 tokens leaves some of them without tokens. Such a tile is
// tile 0 once more: its loads are as wide as the others', the last expert's
// included, and its columns are used nowhere.
constexpr int kActTile = 8;

struct ActTile {
    int64_t first;      // its first value in the workspace
    int w, inter;
    FP8_LAYOUT void set(int base, int count, int inter_, int n) {
        const int r = n * kActTile < count ? n * kActTile : 0;
        w = count - r < kActTile ? count - r : kActTile;
        inter = inter_;
        first = (int64_t)(base + r) * 2 * inter_;
    }
    // values from the start to step kb, half h, group j, part (0 high, 1 low), token c
    FP8_LAYOUT int offset(int kb, int h, int j, int part, int c) const {
        const int left = inter / 16 - kb * 4, groups = left < 4 ? left : 4;
        return kb * 128 * w + (((h * groups + j) * 2 + part) * w + c) * 8;
    }
    // this lane's token, and where its loads of a whole step start
    FP8_LAYOUT int token(int lane) const { return (lane & 7) < w ? lane & 7 : 0; }
    FP8_LAYOUT int lane(int lane) const { return (((lane >> 4) * 2 + ((lane >> 3) & 1)) * w + token(lane)) * 8; }
    // 16 bytes of a whole step (four groups), half h; `at` is what lane() gave
    FP8_LAYOUT int whole(int step, int h, int at) const { return step * 128 * w + h * 64 * w + at; }
    // the same in the last step, K from 16 j on (K < inter)
    FP8_LAYOUT int last(int k, int h, int lane) const {
        return offset(k >> 6, h, lane >> 4, (lane >> 3) & 1, token(lane));
    }
};

// Tiles, and steps in a block of loads, of the down product's instance for an
// expert of `count` tokens.
struct DownShape {
    int tiles, steps;
};
FP8_LAYOUT constexpr DownShape down_shape(int count) {
    return count > 32 ? DownShape{8, 1} : count > 16 ? DownShape{4, 2} : count > 8 ? DownShape{2, 4} : DownShape{1, 4};
}

}  // namespace fp8amax
