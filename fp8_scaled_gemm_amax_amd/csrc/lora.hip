// lora.hip - low-rank adapters of many requests at once, beside a projection that
// they share: out[t] = base[t] + c_e (x_t A_e^T) B_e^T, e = adapter[t].
//
// Two launches: the first forms v = x A^T in fp32, the second multiplies v c_e with B
// and adds the base. Each product takes 16 tokens on the matrix cores and is kept
// for the tokens of its own adapter alone: what another token or another adapter
// holds never enters a token's result.
//
// Up to kFewTokens (decoding: most tokens have an adapter of their own) a workgroup
// takes up to 16 tokens of one adapter out of 64, wherever they stand, so that the
// adapter's weights are read once for them; the sums of v are split over parts of k, for there
// are few of them. More tokens (prompts: neighbours share an adapter) are taken 16 or
// 32 neighbours at a time, through the adapters that they name.
//
// v c_e is kept as the sum of two bf16 numbers and multiplied in two products, so
// that the only rounding that counts is the output's.
#include "block.hpp"
#include "layer_device.hpp"

namespace fp8amax {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;                       // tokens of a product
constexpr int kStepK = 64;                      // columns of x of one step of a wavefront

__device__ __forceinline__ v4f mfma(u32x4 a, u32x4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}
// Eight columns of base or out, at any alignment: a pointer that is uniform over the
// wavefront and the lane's offset in bytes. Nontemporal: each is met once, and the
// adapters' weights keep their place in the caches.
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
__device__ __forceinline__ u32x4 load8(const uint16_t* base, uint32_t bytes) {
    return __builtin_nontemporal_load(at<u32x4_a2>(base, bytes));
}
__device__ __forceinline__ void store8(uint16_t* base, uint32_t bytes, u32x4 v) {
    __builtin_nontemporal_store(v, at<u32x4_a2>(base, bytes));
}

// v = sum of its parts times the factor, as a high and a low bf16 number. (An Inf or
// NaN is carried by the high part alone; a finite value that bf16 would round to Inf
// is bf16's largest and the rest.)
__device__ __forceinline__ void put_value(const Lora& p, int64_t t, int j, float c, uint16_t* hi, uint16_t* lo) {
    const float* src = p.ws + t * p.rank + j;
    const int64_t step = p.tokens * p.rank;
    float v = 0.0f;
    int part = 0;
    for (; part + 8 <= p.parts; part += 8) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = src[(part + i) * step];
#pragma unroll
        for (int i = 0; i < 8; ++i) v += f[i];
    }
    for (; part < p.parts; ++part) v += src[part * step];
    v *= c;
    const bool finite = __builtin_isfinite(v);
    uint32_t h = f32_to_bf16(v);
    h -= finite && (h & 0x7fffu) == 0x7f80u ? 1u : 0u;
    *hi = (uint16_t)h;
    *lo = (uint16_t)(finite ? f32_to_bf16(v - __uint_as_float(h << 16)) : 0u);
}

// Orders this wavefront's LDS accesses on either side for the compiler (the
// hardware keeps their order).
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The first product: 16 NT tokens (NT * 16 rows of x) against 16 RT rows of A, a
// wavefront the steps s, s + W, .. of 64 columns. Loads take 8 lanes a row of 128
// bytes; the matrix cores want lane l to hold a chunk of row l % 16: each wavefront
// turns the one into the other through LDS of its own (16 rows x 128 bytes, chunk c
// of row r at c ^ (r / 2 % 8): neither side meets a bank twice). The next step's loads
// are on their way while a step is multiplied. The sums take the tiles' place in the end.
template <int NT, int RT, int W>
struct DownLds {
    static constexpr int kTiles = (NT + RT) * 2048, kSums = NT * RT * 1024;
    __attribute__((aligned(16))) uint8_t own[W][kTiles > kSums ? kTiles : kSums];
};

// xo, ao: offsets in bytes of this lane's two rows of each tile, from x0 and a0 (uniform).
template <int NT, int RT, int W>
__device__ __forceinline__ void down_sums(const Lora& p, DownLds<NT, RT, W>& lds, const uint16_t* x0,
                                          const uint32_t (&xo)[NT][2], const uint16_t* a0, const uint32_t (&ao)[RT][2],
                                          int64_t s, int64_t s1, v4f (&acc)[NT][RT]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, m = lane & 15;
    uint8_t* own = lds.own[wave];
    struct Step {
        u32x4 x[NT][2], a[RT][2];
    };
    auto load = [&](int64_t at_s, Step& k) {
        // lanes behind k's end (in its last step) load the row's last chunk, for zeros
        const int64_t rest = p.k - at_s * kStepK;
        const int last = rest < kStepK ? (int)rest / 8 - 1 : 7, c = lane & 7;
        const uint32_t in = c <= last ? ~0u : 0u, back = c <= last ? 0u : (uint32_t)(c - last) * 16;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) k.x[n][i] = *at<u32x4>(x0 + at_s * kStepK, xo[n][i] - back) & in;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) k.a[r][i] = *at<u32x4>(a0 + at_s * kStepK, ao[r][i] - back) & in;
    };
    auto put = [&](int tile, const u32x4(&v)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = 8 * i + (lane >> 3);
            *reinterpret_cast<u32x4*>(own + tile * 2048 + row * 128 + (((lane & 7) ^ ((row >> 1) & 7)) << 4)) = v[i];
        }
    };
    auto get = [&](int tile, int h) {           // K in the order of the chunks 4 h + q, on both sides
        return *reinterpret_cast<const u32x4*>(own + tile * 2048 + m * 128 + (((4 * h + q) ^ ((m >> 1) & 7)) << 4));
    };
    auto work = [&](const Step& k) {
        wave_lds_fence();
#pragma unroll
        for (int n = 0; n < NT; ++n) put(n, k.x[n]);
#pragma unroll
        for (int r = 0; r < RT; ++r) put(NT + r, k.a[r]);
        wave_lds_fence();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 x[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n] = get(n, h);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const u32x4 a = get(NT + r, h);
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][r] = mfma(a, x[n], acc[n][r]);
            }
        }
    };
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[n][r] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    s += wave;
    if (s >= s1) return;
    Step a;
    if constexpr (RT == 8) {                    // (two steps' rows: spills)
        for (; s < s1; s += W) {
            load(s, a);
            work(a);
        }
        return;
    }
    Step b;
    load(s, a);
    for (;;) {
        if (s + W < s1) load(s + W, b);
        work(a);
        if (s + W >= s1) return;
        if (s + 2 * W < s1) load(s + 2 * W, a);
        work(b);
        s += 2 * W;
        if (s >= s1) return;
    }
}
template <int RT>
__device__ __forceinline__ void a_offsets(const Lora& p, uint32_t (&ao)[RT][2]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = r * 16 + i * 8 + (lane >> 3);
            ao[r][i] = (uint32_t)(row < p.rank ? row : p.rank - 1) * (uint32_t)p.lda * 2 + (lane & 7) * 16;
        }
}
// The wavefronts' sums added, in order: store(tile, column (token), row, sum).
template <int NT, int RT, int W, typename Store>
__device__ __forceinline__ void add_waves(const Lora& p, DownLds<NT, RT, W>& lds, const v4f (&acc)[NT][RT], Store store) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    wave_lds_fence();
    float* mine = reinterpret_cast<float*>(lds.own[wave]);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < RT; ++r)            // column (token) lane % 16, rows 4 (lane / 16) ..
            *reinterpret_cast<v4f*>(mine + (n * RT + r) * 256 + (lane & 15) * 16 + (lane >> 4) * 4) = acc[n][r];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * RT * 256; i += W * 64) {
        const int col = (i & 255) >> 4, row = (i >> 8) % RT * 16 + (i & 15);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += reinterpret_cast<const float*>(lds.own[w])[i];
        if (row < p.rank) store((i >> 8) / RT, col, row, v);
    }
    __syncthreads();                            // (the tiles' place is free again)
}

// LDS of the second product. vs: 16 NT tokens' values of v, high and low parts, zeros
// behind the rank. A wavefront's own 16-byte aligned part: its 64 rows of B (padded
// to RS steps of 32), then, in their place, its sums (fp32, 16 NT tokens x 64
// columns). Both pitches put 16 neighbouring rows on 16 different groups of banks.
template <int NT, int RS>
struct UpLds {
    static constexpr int kPitch = RS * 32 + 8, kSums = 68;          // bf16 values, fp32 values
    static constexpr int kB = 64 * kPitch * 2, kS = NT * kTile * kSums * 4;
    uint16_t vs[2][NT * kTile * kPitch];
    __attribute__((aligned(16))) uint8_t own[4][kB > kS ? kB : kS];

    template <typename Token>           // token(i, &e): the i-th token and its adapter (-1: none, zeros)
    __device__ __forceinline__ void fill(const Lora& p, Token token) {
        for (int i = threadIdx.x; i < NT * kTile * (RS * 32); i += 256) {
            const int tok = i / (RS * 32), j = i % (RS * 32);
            int e;
            const int64_t t = token(tok, &e);
            uint16_t hi = 0, lo = 0;
            if (e >= 0 && j < p.rank) put_value(p, t, j, p.scaling[e], &hi, &lo);
            vs[0][tok * kPitch + j] = hi;
            vs[1][tok * kPitch + j] = lo;
        }
    }
};

// base + v B^T (or the base's own bits, `add` false) for 16 NT tokens of one adapter
// and the blocks nb, nb + step, .. of 256 columns, a wavefront 64 of them. Memory is
// met 8 lanes a row of 128 bytes (B: as its rows lie): lane l has the tokens t0 + t[i],
// rows 8 i + l / 8 of the 16 NT, where live, and 8 columns of each. (In the
// product's own order, 16 rows of 16 bytes a quarter of a load, 5003 tokens of rank 64
// took 131 us, in this one 97.) With two tiles of tokens the next block's weights and
// base are on their way while a block is multiplied.
template <int NT, int RS>
__device__ __forceinline__ void up_blocks(const Lora& p, int e, int64_t t0, const int (&t)[2 * NT],
                                          const bool (&live)[2 * NT], const bool (&add)[2 * NT], UpLds<NT, RS>& lds,
                                          int64_t nb, int64_t step, int64_t blocks_n) {
    using L = UpLds<NT, RS>;
    constexpr int CH = RS * 4;                  // 16-byte chunks of a padded row of B
    struct Block {
        u32x4 w[CH], base[2 * NT];
    };
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, m = lane & 15;
    uint16_t* bl = reinterpret_cast<uint16_t*>(lds.own[wave]);
    float* sums = reinterpret_cast<float*>(lds.own[wave]);
    const uint16_t* be = p.b + e * p.gsb;
    uint32_t from[2 * NT], to[2 * NT];          // (leading dimensions below 2^24: 64 rows in 32 bits)
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
        from[i] = (uint32_t)t[i] * (uint32_t)p.ldbase * 2 + (lane & 7) * 16;
        to[i] = (uint32_t)t[i] * (uint32_t)p.ldout * 2 + (lane & 7) * 16;
    }
    auto load = [&](int64_t b, Block& k) {
        const int64_t n0 = b * 256 + wave * 64;
        const int left = p.n - n0 < 64 ? (int)(p.n - n0) : 64;
        if (left <= 0) return;                  // (uniform over the wavefront)
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int row = i * (64 / CH) + lane / CH, ch = lane % CH;
            const uint32_t off = (uint32_t)(row < left ? row : left - 1) * (uint32_t)p.ldb * 2 + ch * 16;
            k.w[i] = u32x4{0u, 0u, 0u, 0u};
            if (ch * 8 < p.rank) k.w[i] = *at<u32x4>(be + n0 * p.ldb, off);
        }
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
            k.base[i] = u32x4{0u, 0u, 0u, 0u};
            if (p.base && live[i] && (lane & 7) * 8 + 8 <= left) k.base[i] = load8(p.base + t0 * p.ldbase + n0, from[i]);
        }
    };
    auto work = [&](int64_t b, const Block& k) {
        const int64_t n0 = b * 256 + wave * 64;
        const int left = p.n - n0 < 64 ? (int)(p.n - n0) : 64;
        if (left <= 0) return;
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < CH; ++i)
            *reinterpret_cast<u32x4*>(bl + (i * (64 / CH) + lane / CH) * L::kPitch + (lane % CH) * 8) = k.w[i];
        wave_lds_fence();
        v4f acc[NT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u32x4 w[RS];
#pragma unroll
            for (int s = 0; s < RS; ++s)
                w[s] = *reinterpret_cast<const u32x4*>(bl + (i * 16 + m) * L::kPitch + s * 32 + q * 8);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int at = (n * kTile + m) * L::kPitch + q * 8;
                v4f hi = {0.0f, 0.0f, 0.0f, 0.0f}, lo = hi;
#pragma unroll
                for (int s = 0; s < RS; ++s) {
                    hi = mfma(w[s], *reinterpret_cast<const u32x4*>(&lds.vs[0][at + s * 32]), hi);
                    lo = mfma(w[s], *reinterpret_cast<const u32x4*>(&lds.vs[1][at + s * 32]), lo);
                }
                // (an infinite weight: the low parts, of either sign or 0, would make NaN of Inf)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[n][i][c] = __builtin_isfinite(hi[c]) ? hi[c] + lo[c] : hi[c];
            }
        }
        wave_lds_fence();
#pragma unroll
        for (int n = 0; n < NT; ++n)            // token m of tile n, columns 16 i + 4 q ..
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<v4f*>(sums + (n * kTile + m) * L::kSums + i * 16 + q * 4) = acc[n][i];
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
            const float* f = sums + (i * 8 + (lane >> 3)) * L::kSums + (lane & 7) * 8;
            const int rest = left - (lane & 7) * 8;
            if (live[i] && rest >= 8) {
                const v4f f0 = *reinterpret_cast<const v4f*>(f), f1 = *reinterpret_cast<const v4f*>(f + 4);
                const u32x4 o = k.base[i];
                float g[8];
                unpack8(make_uint4(o[0], o[1], o[2], o[3]), g);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    g[c] += f0[c];
                    g[4 + c] += f1[c];
                }
                const uint4 s = pack8(g);       // (no adapter: the base's own bits)
                store8(p.out + t0 * p.ldout + n0, to[i], add[i] ? u32x4{s.x, s.y, s.z, s.w} : o);
            } else if (live[i] && rest > 0) {   // a chunk that the columns end in
#pragma unroll 1
                for (int c = 0; c < rest; ++c) {
                    const uint32_t o = p.base ? *at<uint16_t>(p.base + t0 * p.ldbase + n0, from[i] + 2 * c) : 0u;
                    *at<uint16_t>(p.out + t0 * p.ldout + n0, to[i] + 2 * c) =
                        (uint16_t)(add[i] ? f32_to_bf16(__uint_as_float(o << 16) + f[c]) : o);
                }
            }
        }
    };
    Block a;
    // A workgroup of few tokens has few blocks, and more of them fit without a second
    // block in registers (128 tokens, rank 16, 4096 x 14336: 22 -> 19 us); of rank 128 two
    // blocks do not fit.
    if constexpr (NT == 1) {
        for (; nb < blocks_n; nb += step) {
            load(nb, a);
            work(nb, a);
        }
        return;
    }
    Block b;                                    // in turn, so that no load waits to be copied
    load(nb, a);
    for (;;) {
        const int64_t n1 = nb + step, n2 = n1 + step;
        if (n1 < blocks_n) load(n1, b);
        work(nb, a);
        if (n1 >= blocks_n) return;
        if (n2 < blocks_n) load(n2, a);
        work(n1, b);
        if (n2 >= blocks_n) return;
        nb = n2;
    }
}

// -------------------------------------------------------------- few tokens --
constexpr int kFewTokens = 512, kGroup = 64;

// Up to 16 tokens of one adapter out of a group of 64: the slot-th such unit (by its
// first token), an adapter of more tokens has several. Lane r holds the place in the
// group of the adapter's r-th token; the unit's are c0 .. c0 + count - 1.
struct Unit {
    int e, c0, count, token;
    uint64_t without;                           // tokens without an adapter
    __device__ __forceinline__ bool find(const Lora& p, int64_t t0, int slot) {
        const int lane = threadIdx.x & 63;
        const int n = p.tokens - t0 < kGroup ? (int)(p.tokens - t0) : kGroup;
        int mine = lane < n ? p.adapter[t0 + lane] : -1;
        mine = mine >= 0 && mine < p.adapters ? mine : -1;
        const uint64_t some = __ballot(mine >= 0);
        without = ~some & (n < 64 ? (1ull << n) - 1ull : ~0ull);
        // the tokens that name this lane's adapter, bit by bit of its number
        uint64_t same = some;
        for (int bit = 0; bit < 31 && (p.adapters - 1) >> bit; ++bit) {
            const uint64_t set = __ballot((mine >> bit) & 1);
            same &= (mine >> bit) & 1 ? set : ~set;
        }
        const uint64_t below = (1ull << lane) - 1ull;
        const int rank = __popcll(same & below);
        const uint64_t heads = __ballot(mine >= 0 && rank % kTile == 0);
        if (slot >= __popcll(heads)) return false;
        const uint64_t one = __ballot(((heads >> lane) & 1u) && __popcll(heads & below) == slot);
        const int head = __ffsll((unsigned long long)one) - 1;
        e = __builtin_amdgcn_readlane(mine, head);
        c0 = __builtin_amdgcn_readlane(rank, head);
        const uint64_t tokens = __ballot(mine == e);
        const int all = __popcll(tokens), to = mine == e ? __popcll(tokens & below) : all + __popcll(~tokens & below);
        token = __builtin_amdgcn_ds_permute(4 * to, lane);
        count = all - c0 < kTile ? all - c0 : kTile;
        return true;
    }
    // the c-th token of the unit (the first one past the last: loads of it are not used)
    __device__ __forceinline__ int at(int c) const { return __shfl(token, c0 + (c < count ? c : 0), 64); }
};

template <int RT>
__global__ __launch_bounds__(256) void k_lora_down_few(Lora p) {
    __shared__ DownLds<1, RT, 4> lds;
    const int lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)blockIdx.x * kGroup;
    Unit unit;
    if (!unit.find(p, t0, blockIdx.z)) return;
    const int64_t steps = (p.k + kStepK - 1) / kStepK;
    const int64_t s0 = steps * blockIdx.y / p.parts, s1 = steps * (blockIdx.y + 1) / p.parts;
    uint32_t ao[RT][2], xo[1][2];
    a_offsets<RT>(p, ao);
#pragma unroll
    for (int i = 0; i < 2; ++i) xo[0][i] = (uint32_t)unit.at(i * 8 + (lane >> 3)) * (uint32_t)p.ldx * 2 + (lane & 7) * 16;
    v4f acc[1][RT];
    down_sums<1, RT, 4>(p, lds, p.x + t0 * p.ldx, xo, p.a + unit.e * p.gsa, ao, s0, s1, acc);
    const int c = threadIdx.x >> 4, token = unit.at(c);         // (256 threads: 16 columns a pass)
    add_waves<1, RT, 4>(p, lds, acc, [&](int, int, int row, float v) {
        if (c < unit.count) p.ws[((int64_t)blockIdx.y * p.tokens + t0 + token) * p.rank + row] = v;
    });
}

// Workgroup: a unit, blocks y, y + gridDim.y, .. of columns.
// Slot 0 also copies the base of the tokens without an adapter.
template <int RS>
__global__ __launch_bounds__(256, RS == 1 ? 4 : RS == 2 ? 3 : 2) void k_lora_up_few(Lora p, int64_t blocks_n) {
    __shared__ UpLds<1, RS> lds;
    const int lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)blockIdx.x * kGroup;
    Unit unit;
    const bool any = unit.find(p, t0, blockIdx.z);
    if (blockIdx.z == 0 && p.base != p.out) {
        for (uint64_t left = unit.without; left; left &= left - 1) {
            const int64_t t = t0 + __ffsll((unsigned long long)left) - 1;
            for (int64_t nb = blockIdx.y; nb < blocks_n; nb += gridDim.y) {
                const int64_t n = nb * 256 + threadIdx.x;
                if (n < p.n) p.out[t * p.ldout + n] = p.base ? p.base[t * p.ldbase + n] : (uint16_t)0;
            }
        }
    }
    if (!any) return;
    lds.fill(p, [&](int tok, int* e) {
        const int token = unit.at(tok);
        *e = tok < unit.count ? unit.e : -1;
        return t0 + token;
    });
    __syncthreads();
    int t[2];
    bool live[2], add[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = i * 8 + (lane >> 3);
        t[i] = unit.at(c);
        live[i] = c < unit.count;
        add[i] = true;
    }
    up_blocks<1, RS>(p, unit.e, t0, t, live, add, lds, blockIdx.y, gridDim.y, blocks_n);
}

// ------------------------------------------------------------- many tokens --
// The adapters of the tokens t0 .. t0 + n - 1 (n at most 64), in the order of their
// first tokens; every wavefront goes through the same ones.
struct Adapters {
    int mine;                                   // of token lane: -1 for none
    uint64_t left;                              // tokens whose adapter is still to come
    __device__ __forceinline__ Adapters(const Lora& p, int64_t t0, int n) {
        const int lane = threadIdx.x & 63;
        const int e = lane < n && t0 + lane < p.tokens ? p.adapter[t0 + lane] : -1;
        mine = e >= 0 && e < p.adapters ? e : -1;
        left = __ballot(mine >= 0);
    }
    // the next adapter, and a bit for each of its tokens
    __device__ __forceinline__ int next(uint64_t* tokens) {
        const int e = __builtin_amdgcn_readlane(mine, __ffsll((unsigned long long)left) - 1);
        *tokens = __ballot(mine == e);
        left &= ~*tokens;
        return e;
    }
};

// Workgroup (tile, part): 16 NT neighbours; its W wavefronts share the part's steps.
template <int NT, int RT, int W>
__global__ __launch_bounds__(W * 64) void k_lora_down(Lora p) {
    __shared__ DownLds<NT, RT, W> lds;
    const int lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)blockIdx.x * (NT * kTile);
    Adapters todo(p, t0, NT * kTile);
    const int64_t steps = (p.k + kStepK - 1) / kStepK;
    const int64_t s0 = steps * blockIdx.y / p.parts, s1 = steps * (blockIdx.y + 1) / p.parts;
    uint32_t ao[RT][2], xo[NT][2];
    a_offsets<RT>(p, ao);
    const int last = p.tokens - t0 < NT * kTile ? (int)(p.tokens - t0) - 1 : NT * kTile - 1;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = n * kTile + i * 8 + (lane >> 3);
            xo[n][i] = (uint32_t)(row < last ? row : last) * (uint32_t)p.ldx * 2 + (lane & 7) * 16;
        }
    while (todo.left) {
        uint64_t tokens;
        const int e = todo.next(&tokens);
        v4f acc[NT][RT];
        down_sums<NT, RT, W>(p, lds, p.x + t0 * p.ldx, xo, p.a + e * p.gsa, ao, s0, s1, acc);
        add_waves<NT, RT, W>(p, lds, acc, [&](int n, int col, int row, float v) {
            const int c = n * kTile + col;
            if ((tokens >> c) & 1u) p.ws[((int64_t)blockIdx.y * p.tokens + t0 + c) * p.rank + row] = v;
        });
    }
}

// Workgroup: 16 NT neighbours, blocks y, y + gridDim.y, .. of columns. v is added up
// once; tokens of one adapter (the usual case) are taken together, others one adapter
// after the other, a token stored with its own.
template <int NT, int RS>
__global__ __launch_bounds__(256, 2) void k_lora_up(Lora p, int64_t blocks_n) {
    __shared__ UpLds<NT, RS> lds;
    const int lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)blockIdx.x * (NT * kTile);
    Adapters todo(p, t0, NT * kTile);
    const uint64_t some = todo.left;
    lds.fill(p, [&](int tok, int* e) {
        *e = __shfl(todo.mine, tok, 64);
        return t0 + tok;
    });
    __syncthreads();
    int t[2 * NT];
    bool add[2 * NT];
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
        t[i] = i * 8 + (lane >> 3);
        add[i] = (some >> (i * 8 + (lane >> 3))) & 1u;
    }
    uint64_t without = ~some;                   // stored with the first adapter's tokens
    do {
        uint64_t tokens = 0;
        const int e = todo.left ? todo.next(&tokens) : 0;           // (none at all: e's products are not used)
        bool live[2 * NT];
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i)
            live[i] = (((tokens | without) >> (i * 8 + (lane >> 3))) & 1u) && t0 + t[i] < p.tokens;
        without = 0;
        up_blocks<NT, RS>(p, e, t0, t, live, add, lds, blockIdx.y, gridDim.y, blocks_n);
    } while (todo.left);
}

// 16-row tiles of the rank of the first launch.
#define FP8_LORA_BY_RANK(CALL)          \
    do {                                \
        if (p.rank <= 16) CALL(1);      \
        else if (p.rank <= 32) CALL(2); \
        else if (p.rank <= 64) CALL(4); \
        else CALL(8);                   \
    } while (0)

// Steps of 32 of the rank of the second launch.
#define FP8_LORA_BY_STEPS(CALL)         \
    do {                                \
        if (p.rank <= 32) CALL(1);      \
        else if (p.rank <= 64) CALL(2); \
        else CALL(4);                   \
    } while (0)

int64_t at_most(int64_t a, int64_t b) { return a < b ? a : b; }

hipError_t few_tokens(Lora p, hipStream_t st) {
    const int64_t groups = (p.tokens + kGroup - 1) / kGroup, steps = (p.k + kStepK - 1) / kStepK;
    // units of a group: one a token at most, and one an adapter and one for 16 tokens
    const int64_t most = at_most(p.tokens, kGroup), slots = at_most(most, p.adapters + most / kTile), active = groups * slots;
    // Short workgroups, many of them: one spends its time on a chain of dependent loads.
    // (128 tokens of as many requests, rank 16, 4096 x 14336: 4 blocks of columns a
    // workgroup 20 us, 14 of them 34; one 26, for the values of v added up again.)
    p.parts = (int)at_most(at_most((2048 + active - 1) / active, 16), (steps + 3) / 4);        // (16 * kFewTokens = kLoraPartRows)
#define CALL(RT)                                                                                              \
    hipLaunchKernelGGL((k_lora_down_few<RT>), dim3((unsigned)groups, (unsigned)p.parts, (unsigned)slots), dim3(256), 0, \
                       st, p)
    FP8_LORA_BY_RANK(CALL);
#undef CALL
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks_n = (p.n + 255) / 256;
    const dim3 grid((unsigned)groups, (unsigned)at_most((4096 + active - 1) / active, blocks_n), (unsigned)slots);
#define CALL(RS) hipLaunchKernelGGL((k_lora_up_few<RS>), grid, dim3(256), 0, st, p, blocks_n)
    FP8_LORA_BY_STEPS(CALL);
#undef CALL
    return hipGetLastError();
}

hipError_t many_tokens(Lora p, hipStream_t st) {
    constexpr int W = 8;
    // 32 tokens a workgroup, 16 where LDS and registers hold no more
    const int nt = p.rank <= 64 ? 2 : 1;
    const int64_t tiles = (p.tokens + nt * kTile - 1) / (nt * kTile), steps = (p.k + kStepK - 1) / kStepK;
    const int64_t parts = at_most(kLoraPartRows / p.tokens, (steps + W - 1) / W);
    p.parts = (int)(parts < 1 ? 1 : parts);
#define CALL(RT) \
    hipLaunchKernelGGL((k_lora_down<RT <= 4 ? 2 : 1, RT, W>), dim3((unsigned)tiles, (unsigned)p.parts), dim3(W * 64), 0, st, p)
    FP8_LORA_BY_RANK(CALL);
#undef CALL
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks_n = (p.n + 255) / 256;
    const int64_t y = 1024 / tiles;             // about four workgroups a CU
    const dim3 grid((unsigned)tiles, (unsigned)at_most(y < 1 ? 1 : y, blocks_n));
#define CALL(RS) hipLaunchKernelGGL((k_lora_up<RS <= 2 ? 2 : 1, RS>), grid, dim3(256), 0, st, p, blocks_n)
    FP8_LORA_BY_STEPS(CALL);
#undef CALL
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_add(const Lora& p, hipStream_t st) {
    if (p.tokens == 0 || p.n == 0) return hipSuccess;
    return p.tokens <= kFewTokens ? few_tokens(p, st) : many_tokens(p, st);
}

}  // namespace fp8amax
