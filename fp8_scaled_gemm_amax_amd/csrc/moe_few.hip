// moe_few.hip - a whole MoE layer for a few tokens (decoding): two launches
// that read the FP8 weights of each expert in use once.
//
//   h = x_t W1_e^T (gate | up), a = silu(g) u, out[t] = sum_j w_tj a_j W2_e^T,
//   e = expert_idx[t, j]; factors of the weight rows applied to the fp32 sums
//
// With a few tokens per expert every weight byte is used by at most a few
// dozen products, so the time is that of reading the weights once. The matrix
// cores still do the products (bf16 16x16x32: 16 weight rows against 16 token
// columns): a product with one token in use costs no more than with sixteen,
// and the cores have room for it: a 64-lane 16-byte load of weights feeds two
// of them. The weights are decoded to bf16 in registers (exact). x is bf16 as
// given. The activation w_tj a is kept as the sum of two bf16 numbers (16
// significant bits) and multiplied in two products, so the only rounding that
// counts is the output's: rounding it to one bf16 would add as large an error
// as the output's own.
//
// K runs in lane order, not memory order: lane l of a 64-byte step of a row
// holds its bytes 16 (l / 16) .. + 15, and the token's values are read in the
// same order, so that a lane's 16 bytes are one access.
#include "layer.hpp"
#include "layer_device.hpp"
#include "moe_few_layout.hpp"

namespace fp8amax {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// Eight OCP codes -> bf16 (exact; the scale operand is 1).
template <int F>
__device__ __forceinline__ v8bf decode_bf16(uint32_t w0, uint32_t w1) {
    v2bf p[4];
    if constexpr (F == kE4M3) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w0, 1.0f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w0, 1.0f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w1, 1.0f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w1, 1.0f, true);
    }
    const v4u w = {__builtin_bit_cast(uint32_t, p[0]), __builtin_bit_cast(uint32_t, p[1]),
                   __builtin_bit_cast(uint32_t, p[2]), __builtin_bit_cast(uint32_t, p[3])};
    return __builtin_bit_cast(v8bf, w);
}

__device__ __forceinline__ v4f mfma(v8bf a, v8bf b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

constexpr int kStep = 64;                   // bytes of a weight row per load of a wavefront
constexpr int kMaxWords = kMoeMaxExperts / 32;

__device__ __forceinline__ uint4 load_weights(const uint8_t* p) {
    return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ uint4 load_weights_once(const uint8_t* p) {
    const v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ v8bf load_acts(const uint16_t* p) {
    return __builtin_bit_cast(v8bf, *reinterpret_cast<const v4u*>(p));
}
// The same where `in`, zeros elsewhere (nothing is read there).
__device__ __forceinline__ uint4 load_weights_if(bool in, const uint8_t* p) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (in) v = load_weights(p);
    return v;
}
__device__ __forceinline__ v8bf load_acts_if(bool in, const uint16_t* p) {
    v4u v = {0u, 0u, 0u, 0u};
    if (in) v = *reinterpret_cast<const v4u*>(p);
    return __builtin_bit_cast(v8bf, v);
}

// A tile of 16 weight rows by a block of kStep * U bytes of each, on its way from
// memory to the matrix cores. Loads take a row's bytes in order (16 U lanes a
// row); the cores want lane l to hold bytes 16 (l / 16) .. + 15 of a 64-byte step of
// row l % 16. The wavefront turns the one into the other through LDS of its own
// (no barrier: a wavefront's LDS accesses happen in order), the chunks of a row
// exchanged such that neither side meets a bank twice. Loading them as the cores
// want them (16 rows a load, 64 bytes of each) took, of 32 experts of 7168 x 2048,
// one token 69.7 us instead of 67.2 and 64 tokens 332 instead of 303.
// Loads of whole lines (U >= 2) leave no copy in the caches: a layer's weights are
// used once a call, and the tokens' values stay (one token 67.1 -> 62.0 us, 32
// tokens 264 -> 247; where all weights of a few small experts could have stayed
// from the call before, 3 tokens of 8 experts of 2048 x 1408, 17.4 -> 19.0).
// Half lines go through the caches, since the other half follows.
template <int U>
struct RowTile {
    static constexpr int kChunks = 4 * U, kRowsPerLoad = 16 / U, kWords = 64 * U;     // kWords: 16-byte words of LDS
    static __device__ __forceinline__ int place(int row, int chunk) {
        return row * kChunks + (chunk ^ ((row * U) >> 2));
    }
    // this lane's first address in the tile whose first row is at `rows`
    static __device__ __forceinline__ const uint8_t* lane(const uint8_t* rows, int64_t ld) {
        const int l = threadIdx.x & 63;
        return rows + (l / kChunks) * ld + (l % kChunks) * 16;
    }
    static __device__ __forceinline__ void load(const uint8_t* lane, int64_t ld, int k, uint4* w) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint8_t* p = lane + i * kRowsPerLoad * ld + k;
            w[i] = U >= 2 ? load_weights_once(p) : load_weights(p);
        }
    }
    static __device__ __forceinline__ void put(uint4* lds, const uint4* w) {
        const int l = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < U; ++i) lds[place(i * kRowsPerLoad + l / kChunks, l % kChunks)] = w[i];
    }
    static __device__ __forceinline__ uint4 get(const uint4* lds, int s) {
        const int l = threadIdx.x & 63;
        return lds[place(l & 15, s * 4 + (l >> 4))];
    }
};
// Orders this wavefront's LDS accesses on either side for the compiler (the
// hardware keeps their order).
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Copies the entries' experts to LDS (-1 for one out of range) and sets the bits
// of those named (all threads; ends with a barrier).
__device__ __forceinline__ void read_entries(const MoeFew& p, int16_t* idx, uint32_t* bits) {
    for (int i = threadIdx.x; i < kMaxWords; i += blockDim.x) bits[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < p.tokens * p.topk; i += blockDim.x) {
        const int e = p.idx[i];
        const bool valid = e >= 0 && e < p.experts;
        idx[i] = (int16_t)(valid ? e : -1);
        if (valid) atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
}

// Experts set in the words below this lane's word (lanes 0 .. 31), and their
// total in *total.
__device__ __forceinline__ int words_below(uint32_t word, int* total) {
    const int lane = threadIdx.x & 63;
    const int pc = lane < kMaxWords ? __popc(word) : 0;
    int incl = pc;
#pragma unroll
    for (int o = 1; o < kMaxWords; o <<= 1) {
        const int y = __shfl_up(incl, o, 64);
        if (lane >= o) incl += y;
    }
    *total = __shfl(incl, kMaxWords - 1, 64);
    return incl - pc;
}

// The tokens of one expert, in token order, lane r holding the r-th: token |
// (its first slot that names the expert) << 8; lanes past count hold other
// tokens' numbers. base: the entries of the experts before it.
struct Entries {
    int item, count, base;
    __device__ __forceinline__ int token(int r) const { return __shfl(item, r, 64) & 0xff; }
    __device__ __forceinline__ int slot(int r) const { return __shfl(item, r, 64) >> 8; }
};
__device__ __forceinline__ Entries find_entries(const MoeFew& p, const int16_t* idx, int e) {
    const int t = threadIdx.x & 63;
    int first = -1, before = 0;
    if (t < p.tokens)
        for (int j = p.topk - 1; j >= 0; --j) {
            const int i = idx[t * p.topk + j];
            first = i == e ? j : first;
            before += (unsigned)i < (unsigned)e ? 1 : 0;    // (-1 is above every expert)
        }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) before += __shfl_xor(before, o, 64);
    const uint64_t has = __ballot(first >= 0), below = (1ull << t) - 1ull;
    Entries en;
    en.base = __builtin_amdgcn_readfirstlane(before);
    en.count = __popcll(has);
    const int to = first >= 0 ? __popcll(has & below) : en.count + __popcll(~has & below);
    en.item = __builtin_amdgcn_ds_permute(4 * to, t | ((first < 0 ? 0 : first) << 8));
    return en;
}

// A tile of activations (its layout: moe_few_layout.hpp) in the workspace.
struct ActRows : ActTile {
    uint16_t* base;
    __device__ __forceinline__ void set(const MoeFew& p, const Entries& en, int n) {
        ActTile::set(en.base, en.count, p.inter, n);
        base = p.ws + first;
    }
};

// ------------------------------------------------------------- gate and up --
// Workgroup (tile, a): RT * 16 columns of the a-th expert in use. Its
// wavefronts split K in blocks of kStep * U bytes, and their sums meet in LDS.
// The next block's weights are on their way while a block is multiplied; the
// tokens' values (from L2) are asked for before them, since loads return in
// order. A load of the tokens' values (16 rows, 64 bytes of each) costs the
// caches as much as one of weights: with two row tiles it serves four of them.
constexpr int kUpWaves = 4;

// Sums of 2 RT tiles of weight rows (gate and up) against the tokens of tiles
// 0 .. NT-1 (NT * 16 entries) over this wavefront's share of K.
// wp: first row of each tile; stage: this wavefront's LDS, 2 RT tiles.
template <int F, int RT, int NT, int U>
__device__ __forceinline__ void up_sums(const uint8_t* const* wp, int64_t ld, const uint16_t* const* xp, int K, int wave,
                                        uint4* stage, v4f (*acc)[NT]) {
    using Tile = RowTile<U>;
    const int j16 = ((threadIdx.x & 63) >> 4) * 16;
    const int whole = K / (kStep * U);
    const uint8_t* lp[2 * RT];
    uint4 w[2 * RT][U];
#pragma unroll
    for (int r = 0; r < 2 * RT; ++r) {
        lp[r] = Tile::lane(wp[r], ld);
        if (wave < whole) Tile::load(lp[r], ld, wave * (kStep * U), w[r]);
    }
    for (int b = wave; b < whole; b += kUpWaves) {
        const int k0 = b * (kStep * U) + j16;
        v8bf x[NT][U][2];
        uint4 wn[2 * RT][U];
#pragma unroll
        for (int s = 0; s < U; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                x[n][s][0] = load_acts(xp[n] + k0 + s * kStep);
                x[n][s][1] = load_acts(xp[n] + k0 + s * kStep + 8);
            }
        __builtin_amdgcn_sched_barrier(0);
        if (b + kUpWaves < whole) {
#pragma unroll
            for (int r = 0; r < 2 * RT; ++r) Tile::load(lp[r], ld, (b + kUpWaves) * (kStep * U), wn[r]);
        }
        __builtin_amdgcn_sched_barrier(0);
        wave_lds_fence();
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) Tile::put(stage + r * Tile::kWords, w[r]);
        wave_lds_fence();
#pragma unroll
        for (int s = 0; s < U; ++s)
#pragma unroll
            for (int r = 0; r < 2 * RT; ++r) {
                const uint4 v = Tile::get(stage + r * Tile::kWords, s);
                const v8bf w0 = decode_bf16<F>(v.x, v.y), w1 = decode_bf16<F>(v.z, v.w);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[r][n] = mfma(w0, x[n][s][0], acc[r][n]);
                    acc[r][n] = mfma(w1, x[n][s][1], acc[r][n]);
                }
            }
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r)
#pragma unroll
            for (int i = 0; i < U; ++i) w[r][i] = wn[r][i];
    }
    wave_lds_fence();
    // what is left of K, 64 bytes a step, the last step's lanes past K zero on both sides
    const int left0 = whole * U, steps = (K + kStep - 1) / kStep;
    for (int st = left0 + (wave + kUpWaves - whole % kUpWaves) % kUpWaves; st < steps; st += kUpWaves) {
        const int k = st * kStep + j16;
        const bool in = k < K;
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
            const uint4 wl = load_weights_if(in, wp[r] + (threadIdx.x & 15) * ld + k);
            const v8bf w0 = decode_bf16<F>(wl.x, wl.y), w1 = decode_bf16<F>(wl.z, wl.w);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[r][n] = mfma(w0, load_acts_if(in, xp[n] + k), acc[r][n]);
                acc[r][n] = mfma(w1, load_acts_if(in, xp[n] + k + 8), acc[r][n]);
            }
        }
    }
}

// Floats of LDS of a wavefront: 2 RT tiles of U KB of weights, or of NT KB of sums.
template <int RT, int NT, int U>
constexpr int up_part() {
    return 2 * RT * 256 * (NT > U ? NT : U);
}

// One workgroup's columns for NT tiles of entries.
template <int F, int RT, int NT, int U>
__device__ __forceinline__ void up_tile(const MoeFew& p, const int16_t* idx, int e, int c0, const Entries& ent,
                                        float* red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint8_t* we = p.w1 + (int64_t)e * p.gs1;
    const uint8_t* wp[2 * RT];                              // gate tile, up tile, gate tile, ..
#pragma unroll
    for (int r = 0; r < 2 * RT; ++r)
        wp[r] = we + (int64_t)((r & 1) * p.inter + c0 + (r >> 1) * 16) * p.ld1;
    const uint16_t* xp[NT];
    v4f acc[2 * RT][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int c = n * 16 + (lane & 15);
        xp[n] = p.x + (int64_t)ent.token(c < ent.count ? c : 0) * p.ldx;     // (columns past the entries are not used)
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) acc[r][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // for the end: factors of the rows, and the weights of the columns' tokens
    // (the sum over all slots of the token that name the expert)
    const int row = threadIdx.x & 15;
    float factor[2 * RT], share[NT];
#pragma unroll
    for (int r = 0; r < 2 * RT; ++r) factor[r] = p.s1[((int64_t)2 * e + (r & 1)) * p.inter + c0 + (r >> 1) * 16 + row];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int c = n * 16 + (threadIdx.x >> 4);
        const int token = ent.token(c), slot = ent.slot(c);
        share[n] = 0.0f;
        if (c >= ent.count) continue;
        share[n] = p.weights[token * p.topk + slot];
        for (int j = slot + 1; j < p.topk; ++j)
            if (idx[token * p.topk + j] == e) share[n] += p.weights[token * p.topk + j];
    }
    // A wavefront's part of red holds its tiles of weights, then its sums: [tile of
    // entries][row tile][column * 16 + row], row = 4 (lane / 16) + i.
    constexpr int kPart = up_part<RT, NT, U>();
    float* mine = red + wave * kPart;
    up_sums<F, RT, NT, U>(wp, p.ld1, xp, p.hidden, wave, reinterpret_cast<uint4*>(mine), acc);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r)
            *reinterpret_cast<v4f*>(mine + (n * 2 * RT + r) * 256 + (lane & 15) * 16 + (lane >> 4) * 4) = acc[r][n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int col = threadIdx.x >> 4;
        if (n * 16 + col >= ent.count) continue;
        const int c = n * 16 + col;
        ActRows tile;
        tile.set(p, ent, c / kActTile);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < kUpWaves; ++w) {
                g += red[w * kPart + (n * 2 * RT + 2 * r) * 256 + threadIdx.x];
                u += red[w * kPart + (n * 2 * RT + 2 * r + 1) * 256 + threadIdx.x];
            }
            const float a = silu_fast(g * factor[2 * r]) * (u * factor[2 * r + 1]) * share[n];
            // (an Inf or NaN is carried by the high part alone; a finite value that
            // bf16 would round to Inf is bf16's largest and the rest)
            const bool finite = __builtin_isfinite(a);
            uint32_t hi = f32_to_bf16(a);
            hi -= finite && (hi & 0x7fffu) == 0x7f80u ? 1u : 0u;
            const uint32_t lo = finite ? f32_to_bf16(a - __uint_as_float(hi << 16)) : 0u;
            const int k = c0 + r * 16, kb = k >> 6, j = (k >> 4) & 3, half = row >> 3;
            tile.base[tile.offset(kb, half, j, 0, c % kActTile) + (row & 7)] = (uint16_t)hi;
            tile.base[tile.offset(kb, half, j, 1, c % kActTile) + (row & 7)] = (uint16_t)lo;
        }
    }
}

template <int F, int RT, int NTMAX>
__global__ __launch_bounds__(kUpWaves * 64) void k_moe_few_up(MoeFew p) {
    __shared__ uint32_t bits[kMaxWords];
    __shared__ int16_t idx[NTMAX * 16 * kMoeMaxTopk];
    // 256 bytes of a row at a time; 128 with two row tiles of up to 64 tokens (32
    // experts of 7168 x 2048: 32 tokens 252 us with 128, 245 with 256; 64 tokens 296
    // and 310)
    constexpr int U1 = RT == 1 || NTMAX < 4 ? 4 : 2;
    constexpr int kPart = NTMAX >= 4 ? up_part<RT, 4, U1>() : up_part<RT, NTMAX, U1>();
    __shared__ __attribute__((aligned(16))) float red[kUpWaves * kPart];
    const int lane = threadIdx.x & 63;
    read_entries(p, idx, bits);
    const uint32_t word = lane < kMaxWords ? bits[lane] : 0u;
    int total;
    const int below = words_below(word, &total);
    const int a = blockIdx.y;
    if (a >= total) return;                                 // (uniform: every wavefront has the same bitmap)
    const bool mine = lane < kMaxWords && a >= below && a < below + __popc(word);
    uint32_t w = word;
    for (int i = below; mine && i < a; ++i) w &= w - 1u;    // drop the experts before it
    const int owner = __ffsll((unsigned long long)__ballot(mine)) - 1;
    const int e = __builtin_amdgcn_readfirstlane(__shfl(lane * 32 + __ffs((int)w) - 1, owner, 64));
    const Entries ent = find_entries(p, idx, e);
    const int c0 = blockIdx.x * (RT * 16);
    if constexpr (NTMAX >= 4) {
        if (ent.count > 32) {
            up_tile<F, RT, 4, 1>(p, idx, e, c0, ent, red);
            return;
        }
    }
    if constexpr (NTMAX >= 2) {
        if (ent.count > 16) {
            up_tile<F, RT, 2, 2>(p, idx, e, c0, ent, red);
            return;
        }
    }
    up_tile<F, RT, 1, U1>(p, idx, e, c0, ent, red);
}

// -------------------------------------------------------------------- down --
// Workgroup: RT * 16 output columns of every token. The units of work are
// pieces of K of the experts in use, dealt to the wavefronts in order. A
// wavefront multiplies the expert's rows with the expert's tokens, 8 at a
// time, and adds the sums, times the rows' factors, to its own sums of those
// tokens in LDS; at the end the wavefronts' sums are added in order. A token's
// sums are never touched by an expert that it does not use.
constexpr int kDownWaves = 8;

// Products of RT * 16 weight rows with the entries of tiles 0 .. NT-1 over the
// blocks b0, b0 + db, .. of K.
// wp: first row of each tile; stage: this wavefront's LDS, RT tiles.
template <int F, int RT, int NT, int U>
__device__ __forceinline__ void down_sums(const uint8_t* const* wp, int64_t ld, const ActRows* tile, const int* col, int K,
                                          int b0, int db, uint4* stage, v4f (*acc)[NT]) {
    using Tile = RowTile<U>;
    const int lane = threadIdx.x & 63, j16 = (lane >> 4) * 16;
    const int whole = K / (kStep * U);
    const uint8_t* lp[RT];
    uint4 w[RT][U];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        lp[r] = Tile::lane(wp[r], ld);
        if (b0 < whole) Tile::load(lp[r], ld, b0 * (kStep * U), w[r]);
    }
    constexpr int G = NT > 4 ? 4 : NT;                      // tiles at a time (eight's activations do not fit)
    v8bf a[G][U][2];
    auto load_tiles = [&](int b, int n0) {
#pragma unroll
        for (int s = 0; s < U; ++s)
#pragma unroll
            for (int n = 0; n < G; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {               // (a whole step: 4 groups)
                    const ActRows& t = tile[n0 + n];
                    a[n][s][h] = load_acts(t.base + t.whole(b * U + s, h, col[n0 + n]));
                }
    };
    int b = b0;
    for (; b < whole; b += db) {
        uint4 wn[RT][U];
        load_tiles(b, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (b + db < whole) {
#pragma unroll
            for (int r = 0; r < RT; ++r) Tile::load(lp[r], ld, (b + db) * (kStep * U), wn[r]);
        }
        __builtin_amdgcn_sched_barrier(0);
        wave_lds_fence();
#pragma unroll
        for (int r = 0; r < RT; ++r) Tile::put(stage + r * Tile::kWords, w[r]);
        wave_lds_fence();
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += G) {
            if (n0 > 0) load_tiles(b, n0);
#pragma unroll
            for (int s = 0; s < U; ++s)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint4 v = Tile::get(stage + r * Tile::kWords, s);
                    const v8bf w0 = decode_bf16<F>(v.x, v.y), w1 = decode_bf16<F>(v.z, v.w);
#pragma unroll
                    for (int n = 0; n < G; ++n) {
                        acc[r][n0 + n] = mfma(w0, a[n][s][0], acc[r][n0 + n]);
                        acc[r][n0 + n] = mfma(w1, a[n][s][1], acc[r][n0 + n]);
                    }
                }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < U; ++i) w[r][i] = wn[r][i];
    }
    wave_lds_fence();
    if (b * (kStep * U) >= K) return;                       // (the last, partial block is this wavefront's or another's)
    for (int k = b * (kStep * U) + j16; k - j16 < K; k += kStep) {
        const bool in = k < K;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            v8bf a[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) a[h] = load_acts_if(in, tile[n].base + tile[n].last(k, h, lane));
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint4 wl = load_weights_if(in, wp[r] + (threadIdx.x & 15) * ld + k);
                const v8bf w0 = decode_bf16<F>(wl.x, wl.y), w1 = decode_bf16<F>(wl.z, wl.w);
                acc[r][n] = mfma(w0, a[0], acc[r][n]);
                acc[r][n] = mfma(w1, a[1], acc[r][n]);
            }
        }
    }
}

// One unit for NT tiles of entries; sums: this wavefront's [token][RT * 16].
template <int F, int RT, int NT, int U>
__device__ __forceinline__ void down_unit(const MoeFew& p, int e, int row0, const Entries& ent, int b0, int db,
                                          uint4* stage, float* sums) {
    const int lane = threadIdx.x & 63;
    const uint8_t* we = p.w2 + (int64_t)e * p.gs2;
    const uint8_t* wp[RT];
    v4f acc[RT][NT], sc[RT];
    auto load_factors = [&]() {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[r][i] = p.s2[(int64_t)e * p.hidden + row0 + r * 16 + (lane >> 4) * 4 + i];
    };
    if (NT <= 4) load_factors();                            // (eight tiles leave no registers for them)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        wp[r] = we + (int64_t)(row0 + r * 16) * p.ld2;
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    ActRows tile[NT];
    int col[NT];                                            // this lane's place in a whole step
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        tile[n].set(p, ent, n);
        col[n] = tile[n].lane(lane);
    }
    down_sums<F, RT, NT, U>(wp, p.ld2, tile, col, p.inter, b0, db, stage, acc);
    if (NT > 4) load_factors();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int c = n * kActTile + (lane & 7);
        const int t = ent.token(c);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {                   // the high column's sum and the low one's
                const float hi = acc[r][n][i], lo = __shfl_xor(hi, 8, 64);
                // (an infinite weight: the low parts, of either sign or 0, would make NaN of Inf)
                acc[r][n][i] = __builtin_isfinite(hi) ? hi + lo : hi;
            }
        if (c >= ent.count || (lane & 8)) continue;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            v4f* d = reinterpret_cast<v4f*>(sums + t * (RT * 16) + r * 16 + (lane >> 4) * 4);
            v4f v = *d;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fmaf(acc[r][n][i], sc[r][i], v[i]);
            *d = v;
        }
    }
}

// TT: the tokens, rounded up to 16, 32 or 64.
template <int F, int RT, int TT>
__global__ __launch_bounds__(kDownWaves * 64) void k_moe_few_down(MoeFew p) {
    constexpr int W = TT * RT * 16;                          // a wavefront's sums
    __shared__ uint32_t bits[kMaxWords];
    __shared__ int16_t idx[TT * kMoeMaxTopk];
    __shared__ uint16_t list[kMoeMaxExperts];
    __shared__ __attribute__((aligned(16))) float red[kDownWaves * W];
    __shared__ uint4 tiles[kDownWaves * RT * RowTile<4>::kWords];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kDownWaves * W; i += kDownWaves * 64) red[i] = 0.0f;
    read_entries(p, idx, bits);
    uint32_t word = lane < kMaxWords ? bits[lane] : 0u;
    int total;
    int at = words_below(word, &total);
    if (wave == 0)
        for (; word; word &= word - 1u) list[at++] = (uint16_t)(lane * 32 + __ffs((int)word) - 1);
    __syncthreads();
    const int row0 = blockIdx.x * (RT * 16);
    const int blocks = (p.inter + 4 * kStep - 1) / (4 * kStep);
    int pieces = total > 0 ? kDownWaves / total : 1;
    pieces = pieces < 1 ? 1 : (pieces > blocks ? blocks : pieces);
    float* sums = red + wave * W;
    uint4* stage = tiles + wave * (RT * RowTile<4>::kWords);
    for (int unit = wave; unit < total * pieces; unit += kDownWaves) {
        const int e = __builtin_amdgcn_readfirstlane(list[unit / pieces]);
        const Entries ent = find_entries(p, idx, e);
        const int b0 = unit % pieces;
        const int tiles = down_shape(ent.count).tiles;
#define FP8_DOWN(N) down_unit<F, RT, N, down_shape(N * kActTile).steps>(p, e, row0, ent, b0, pieces, stage, sums)
        if (TT > 32 && tiles == 8) FP8_DOWN(8);
        else if (TT > 16 && tiles == 4) FP8_DOWN(4);
        else if (tiles == 2) FP8_DOWN(2);
        else FP8_DOWN(1);
#undef FP8_DOWN
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.tokens * (RT * 16); i += kDownWaves * 64) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) s += red[w * W + i];
        p.out[(int64_t)(i / (RT * 16)) * p.ldo + row0 + i % (RT * 16)] = (uint16_t)f32_to_bf16(s);
    }
}

}  // namespace

template <int F>
hipError_t moe_few_up(const MoeFew& p, hipStream_t st) {
    const int entries = p.tokens * p.topk;
    const unsigned experts = (unsigned)(entries < p.experts ? entries : p.experts);
    // Two row tiles where that leaves four workgroups per CU and an expert has
    // four tokens or more on average (32 experts of 7168 x 2048: 64 tokens 344 us
    // for both launches with one tile, 303 with two; 4096 x 1536, 8 tokens, 108 and
    // 114 us).
    const bool two = p.inter % 32 == 0 && (int64_t)(p.inter / 32) * experts >= 1024 && entries >= 4 * (int)experts;
    const dim3 grid((unsigned)(p.inter / (two ? 32 : 16)), experts), block(kUpWaves * 64);
#define FP8_UP(R, N) hipLaunchKernelGGL((k_moe_few_up<F, R, N>), grid, block, 0, st, p)
    if (p.tokens <= 16) {
        if (two) FP8_UP(2, 1); else FP8_UP(1, 1);
    } else if (p.tokens <= 32) {
        if (two) FP8_UP(2, 2); else FP8_UP(1, 2);
    } else {
        if (two) FP8_UP(2, 4); else FP8_UP(1, 4);
    }
#undef FP8_UP
    return hipGetLastError();
}

template <int F, int RT>
hipError_t moe_few_down(const MoeFew& p, hipStream_t st) {
    const dim3 grid((unsigned)(p.hidden / (RT * 16))), block(kDownWaves * 64);
    if (p.tokens <= 16) hipLaunchKernelGGL((k_moe_few_down<F, RT, 16>), grid, block, 0, st, p);
    else if (p.tokens <= 32) hipLaunchKernelGGL((k_moe_few_down<F, RT, 32>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_moe_few_down<F, RT, 64>), grid, block, 0, st, p);
    return hipGetLastError();
}

hipError_t launch_moe_few_tokens(const MoeFew& p, int f1, int f2, hipStream_t st) {
    if (p.tokens == 0) return hipSuccess;
    const hipError_t e = f1 == kE4M3 ? moe_few_up<kE4M3>(p, st) : moe_few_up<kE5M2>(p, st);
    if (e != hipSuccess) return e;
    // 32 rows a workgroup where that leaves most CUs one: an activation load serves
    // two of weights (64 tokens, 32 experts of 7168 x 2048: 303 us for both
    // launches, 363 with 16 rows); below, twice the workgroups count for more (4096 x
    // 1536, 8 tokens: 120 us with 32 rows, 108 with 16).
    const bool wide = p.hidden % 32 == 0 && p.hidden >= 32 * 160;
    if (f2 == kE4M3) return wide ? moe_few_down<kE4M3, 2>(p, st) : moe_few_down<kE4M3, 1>(p, st);
    return wide ? moe_few_down<kE5M2, 2>(p, st) : moe_few_down<kE5M2, 1>(p, st);
}

}  // namespace fp8amax
