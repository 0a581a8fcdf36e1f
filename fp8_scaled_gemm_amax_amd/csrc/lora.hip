// lora.hip - low-rank adapters of many requests at once, beside a projection that
// they share: out[t] = base[t] + c_e (x_t A_e^T) B_e^T, e = adapter[t].
//
// Two launches: the first forms v = x A^T in fp32, the second multiplies v c_e with B
// and adds the base. Each product takes 16 tokens of one adapter on the matrix cores:
// what another token or another adapter holds never enters a token's result.
//
// A workgroup takes up to 16 tokens of one adapter out of 64, wherever they stand, so
// that the adapter's weights are read once for them, in whatever order the requests'
// tokens come: 5003 tokens of 9 requests, rank 16, 4096 x 14336, take 16 + 70 us, and
// 23 + 114 if each is another request's of 16 adapters. (16 or 32 neighbours a workgroup, one
// adapter after the other: 20 + 86 and 145 + 532.) What bounds many tokens is base and
// out, read and written once, and few ones the latency of two short launches (one
// token 4 + 5 us). For few tokens the sums of v are split over parts of k.
//
// v c_e, fp32, is multiplied as the sum of three bf16 numbers of 8 bits each in three
// products: no bit of it is lost.
#include "block.hpp"
#include "layer_device.hpp"

namespace fp8amax {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;                       // tokens of a product
constexpr int kStepK = 64;                      // columns of x of one step of a wavefront
constexpr int kWaves = 4, kGroup = 64;          // wavefronts of a workgroup, tokens that it looks at

__device__ __forceinline__ v4f mfma(u32x4 a, u32x4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}
// Up to 16 tokens of one adapter out of a group of 64: the slot-th such unit (by its
// first token), an adapter of more tokens has several. Tokens without an adapter are
// units too, those of e = p.adapters. Lane r holds the place in the group of the
// adapter's r-th token; the unit's are c0 .. c0 + count - 1. pick(number of units): the
// workgroup's, no unit past the last.
struct Unit {
    int e, c0, count, token;
    template <typename Pick>
    __device__ __forceinline__ bool find(const Lora& p, int64_t t0, Pick pick) {
        const int lane = threadIdx.x & 63;
        const int n = p.tokens - t0 < kGroup ? (int)(p.tokens - t0) : kGroup;
        int mine = lane < n ? p.adapter[t0 + lane] : p.adapters;
        mine = mine >= 0 && mine < p.adapters ? mine : p.adapters;
        const uint64_t some = n < 64 ? (1ull << n) - 1ull : ~0ull;
        // the tokens that name this lane's adapter, bit by bit of its number
        uint64_t same = some;
        for (int bit = 0; bit < 31 && p.adapters >> bit; ++bit) {
            const uint64_t set = __ballot((mine >> bit) & 1);
            same &= (mine >> bit) & 1 ? set : ~set;
        }
        const uint64_t below = (1ull << lane) - 1ull;
        const int rank = __popcll(same & below);
        const uint64_t heads = __ballot(lane < n && rank % kTile == 0);
        const int units = __popcll(heads), slot = pick(units);
        if (slot >= units) return false;
        const uint64_t one = __ballot(((heads >> lane) & 1u) && __popcll(heads & below) == slot);
        const int head = __ffsll((unsigned long long)one) - 1;
        e = __builtin_amdgcn_readlane(mine, head);
        c0 = __builtin_amdgcn_readlane(rank, head);
        const uint64_t tokens = __ballot(lane < n && mine == e);
        const int all = __popcll(tokens), to = (tokens >> lane) & 1u ? __popcll(tokens & below) : all + __popcll(~tokens & below);
        token = __builtin_amdgcn_ds_permute(4 * to, lane);
        count = all - c0 < kTile ? all - c0 : kTile;
        return true;
    }
    // the c-th token of the unit (the first one past the last: loads of it are not used)
    __device__ __forceinline__ int at(int c) const { return __shfl(token, c0 + (c < count ? c : 0), 64); }
};

// v = sum of its parts times the factor, as a high, a middle and a low bf16 number, whose
// sum it is. (An Inf or NaN is carried by the high part alone; a finite value that bf16
// would round to Inf is bf16's largest and the rest.)
__device__ __forceinline__ void put_value(const Lora& p, int64_t t, int j, float c, uint16_t (&out)[3]) {
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
    const float rest = finite ? v - __uint_as_float(h << 16) : 0.0f;
    const uint32_t mid = f32_to_bf16(rest);
    out[0] = (uint16_t)h;
    out[1] = (uint16_t)mid;
    out[2] = (uint16_t)f32_to_bf16(rest - __uint_as_float(mid << 16));
}

// Orders this wavefront's LDS accesses on either side for the compiler (the
// hardware keeps their order).
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The first product: 16 tokens (rows of x) against 16 RT rows of A, a wavefront the
// steps s, s + 4, .. of 64 columns. Loads take 8 lanes a row of 128
// bytes; the matrix cores want lane l to hold a chunk of row l % 16: each wavefront
// turns the one into the other through LDS of its own (16 rows x 128 bytes, chunk c
// of row r at c ^ (r / 2 % 8): neither side meets a bank twice). The next step's loads
// are on their way while a step is multiplied. The sums take the tiles' place in the end.
template <int RT>
struct DownLds {
    static constexpr int kTiles = (1 + RT) * 2048, kSums = RT * 1024;
    __attribute__((aligned(16))) uint8_t own[kWaves][kTiles > kSums ? kTiles : kSums];
};

// xo, ao: offsets in bytes of this lane's two rows of each tile, from x0 and a0 (uniform).
template <int RT>
__device__ __forceinline__ void down_sums(const Lora& p, DownLds<RT>& lds, const uint16_t* x0, const uint32_t (&xo)[2],
                                          const uint16_t* a0, const uint32_t (&ao)[RT][2], int64_t s, int64_t s1,
                                          v4f (&acc)[RT]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, m = lane & 15;
    uint8_t* own = lds.own[wave];
    struct Step {
        u32x4 x[2], a[RT][2];
    };
    auto load = [&](int64_t at_s, Step& k) {
        // lanes behind k's end (in its last step) load the row's last chunk, for zeros
        const int64_t rest = p.k - at_s * kStepK;
        const int last = rest < kStepK ? (int)rest / 8 - 1 : 7, c = lane & 7;
        const uint32_t in = c <= last ? ~0u : 0u, back = c <= last ? 0u : (uint32_t)(c - last) * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) k.x[i] = *at<u32x4>(x0 + at_s * kStepK, xo[i] - back) & in;
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
        put(0, k.x);
#pragma unroll
        for (int r = 0; r < RT; ++r) put(1 + r, k.a[r]);
        wave_lds_fence();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 x = get(0, h);
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[r] = mfma(get(1 + r, h), x, acc[r]);
        }
    };
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    s += wave;
    if (s >= s1) return;
    Step a;
    if constexpr (RT == 8) {                    // (two steps' rows: spills)
        for (; s < s1; s += kWaves) {
            load(s, a);
            work(a);
        }
        return;
    }
    Step b;                                     // in turn, so that no load waits to be copied
    load(s, a);
    for (;;) {
        if (s + kWaves < s1) load(s + kWaves, b);
        work(a);
        if (s + kWaves >= s1) return;
        if (s + 2 * kWaves < s1) load(s + 2 * kWaves, a);
        work(b);
        s += 2 * kWaves;
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
// The wavefronts' sums added, in order: store(token, row, sum).
template <int RT, typename Store>
__device__ __forceinline__ void add_waves(const Lora& p, DownLds<RT>& lds, const v4f (&acc)[RT], Store store) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    wave_lds_fence();
    float* mine = reinterpret_cast<float*>(lds.own[wave]);
#pragma unroll
    for (int r = 0; r < RT; ++r)                // token lane % 16, rows 4 (lane / 16) ..
        *reinterpret_cast<v4f*>(mine + r * 256 + (lane & 15) * 16 + (lane >> 4) * 4) = acc[r];
    __syncthreads();
    for (int i = threadIdx.x; i < RT * 256; i += kWaves * 64) {
        const int token = (i & 255) >> 4, row = (i >> 8) * 16 + (i & 15);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += reinterpret_cast<const float*>(lds.own[w])[i];
        if (row < p.rank) store(token, row, v);
    }
}

template <int RT>
__global__ __launch_bounds__(kWaves * 64) void k_lora_down(Lora p) {
    __shared__ DownLds<RT> lds;
    const int lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)blockIdx.x * kGroup;
    Unit unit;
    if (!unit.find(p, t0, [](int) { return (int)blockIdx.z; }) || unit.e == p.adapters) return;
    const int64_t steps = (p.k + kStepK - 1) / kStepK;
    const int64_t s0 = steps * blockIdx.y / p.parts, s1 = steps * (blockIdx.y + 1) / p.parts;
    uint32_t ao[RT][2], xo[2];
    a_offsets<RT>(p, ao);
#pragma unroll
    for (int i = 0; i < 2; ++i) xo[i] = (uint32_t)unit.at(i * 8 + (lane >> 3)) * (uint32_t)p.ldx * 2 + (lane & 7) * 16;
    v4f acc[RT];
    down_sums<RT>(p, lds, p.x + t0 * p.ldx, xo, p.a + unit.e * p.gsa, ao, s0, s1, acc);
    const int token = unit.at(threadIdx.x >> 4);                // (256 threads: 16 tokens a pass)
    add_waves<RT>(p, lds, acc, [&](int c, int row, float v) {
        if (c < unit.count) p.ws[((int64_t)blockIdx.y * p.tokens + t0 + token) * p.rank + row] = v;
    });
}

// LDS of the second product. A wavefront's own 16-byte aligned part: its 64 rows of B
// (padded to RS steps of 32), then, in their place, its sums (fp32, 16 tokens x 64
// columns). Both pitches put 16 neighbouring rows on 16 different groups of banks. In the
// beginning 16 tokens' values of v stand there, three parts each, zeros behind the rank,
// until every wavefront has its share of them in registers.
template <int RS>
struct UpLds {
    static constexpr int kPitch = RS * 32 + 8, kSums = 68;          // bf16 values, fp32 values
    static constexpr int kB = 64 * kPitch * 2, kS = kTile * kSums * 4;
    __attribute__((aligned(16))) uint8_t own[kWaves][kB > kS ? kB : kS];

    __device__ __forceinline__ void values(const Lora& p, const Unit& unit, int64_t t0, u32x4 (&v)[3][RS]) {
        constexpr int kPart = kTile * kPitch;
        static_assert(3 * kPart * 2 <= (int)sizeof(own), "the values of v stand in the wavefronts' parts");
        uint16_t* vs = reinterpret_cast<uint16_t*>(own);
        const float c = p.scaling[unit.e];
        for (int i = threadIdx.x; i < kTile * (RS * 32); i += 256) {
            const int tok = i / (RS * 32), j = i % (RS * 32), token = unit.at(tok);
            uint16_t part[3] = {0, 0, 0};
            if (tok < unit.count && j < p.rank) put_value(p, t0 + token, j, c, part);
#pragma unroll
            for (int k = 0; k < 3; ++k) vs[k * kPart + tok * kPitch + j] = part[k];
        }
        __syncthreads();
        const int q = (threadIdx.x & 63) >> 4, m = threadIdx.x & 15;
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int s = 0; s < RS; ++s) v[k][s] = *reinterpret_cast<const u32x4*>(&vs[k * kPart + m * kPitch + s * 32 + q * 8]);
        __syncthreads();
    }
};

// base + v B^T for a unit and the blocks nb, nb + step, .. of 256 columns, a wavefront
// 64 of them. Memory is met 8 lanes a row of 128 bytes (B: as its rows lie): lane l
// has the tokens t0 + t[i], rows 8 i + l / 8 of the 16, where live, and 8 columns of
// each. (In the product's own order, 16 rows of 16 bytes a quarter of a load, 5003
// tokens of rank 64 took a third longer.) A workgroup has few blocks, and more of
// them fit a CU without a second block in registers (128 tokens, rank 16,
// 4096 x 14336: 22 -> 19 us).
template <int RS>
__device__ __forceinline__ void up_blocks(const Lora& p, int e, int64_t t0, const int (&t)[2], const bool (&live)[2],
                                          UpLds<RS>& lds, const u32x4 (&v)[3][RS], int64_t nb, int64_t step,
                                          int64_t blocks_n) {
    using L = UpLds<RS>;
    constexpr int CH = RS * 4;                  // 16-byte chunks of a padded row of B
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, m = lane & 15;
    uint16_t* bl = reinterpret_cast<uint16_t*>(lds.own[wave]);
    float* sums = reinterpret_cast<float*>(lds.own[wave]);
    const uint16_t* be = p.b + e * p.gsb;
    uint32_t from[2], to[2];          // (leading dimensions below 2^24: 64 rows in 32 bits)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        from[i] = (uint32_t)t[i] * (uint32_t)p.ldbase * 2 + (lane & 7) * 16;
        to[i] = (uint32_t)t[i] * (uint32_t)p.ldout * 2 + (lane & 7) * 16;
    }
    for (; nb < blocks_n; nb += step) {
        const int64_t n0 = nb * 256 + wave * 64;
        const int left = p.n - n0 < 64 ? (int)(p.n - n0) : 64;
        if (left <= 0) return;                  // (uniform over the wavefront)
        u32x4 wide[CH], base[2];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int row = i * (64 / CH) + lane / CH, ch = lane % CH;
            const uint32_t off = (uint32_t)(row < left ? row : left - 1) * (uint32_t)p.ldb * 2 + ch * 16;
            wide[i] = u32x4{0u, 0u, 0u, 0u};
            if (ch * 8 < p.rank) wide[i] = *at<u32x4>(be + n0 * p.ldb, off);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            base[i] = u32x4{0u, 0u, 0u, 0u};
            if (p.base && live[i] && (lane & 7) * 8 + 8 <= left) base[i] = load8(p.base + t0 * p.ldbase + n0, from[i]);
        }
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < CH; ++i)
            *reinterpret_cast<u32x4*>(bl + (i * (64 / CH) + lane / CH) * L::kPitch + (lane % CH) * 8) = wide[i];
        wave_lds_fence();
        v4f acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v4f hi = {0.0f, 0.0f, 0.0f, 0.0f}, lo = hi;
#pragma unroll
            for (int s = 0; s < RS; ++s) {
                const u32x4 w = *reinterpret_cast<const u32x4*>(bl + (i * 16 + m) * L::kPitch + s * 32 + q * 8);
                hi = mfma(w, v[0][s], hi);
                lo = mfma(w, v[1][s], lo);
                lo = mfma(w, v[2][s], lo);
            }
            // (an infinite weight: the low parts, of either sign or 0, would make NaN of Inf)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] = __builtin_isfinite(hi[c]) ? hi[c] + lo[c] : hi[c];
        }
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < 4; ++i)             // token m, columns 16 i + 4 q ..
            *reinterpret_cast<v4f*>(sums + m * L::kSums + i * 16 + q * 4) = acc[i];
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float* f = sums + (i * 8 + (lane >> 3)) * L::kSums + (lane & 7) * 8;
            const int rest = left - (lane & 7) * 8;
            if (live[i] && rest >= 8) {
                const v4f f0 = *reinterpret_cast<const v4f*>(f), f1 = *reinterpret_cast<const v4f*>(f + 4);
                const u32x4 o = base[i];
                float g[8];
                unpack8(make_uint4(o[0], o[1], o[2], o[3]), g);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    g[c] += f0[c];
                    g[4 + c] += f1[c];
                }
                const uint4 s = pack8(g);
                store8(p.out + t0 * p.ldout + n0, to[i], u32x4{s.x, s.y, s.z, s.w});
            } else if (live[i] && rest > 0) {   // a chunk that the columns end in
#pragma unroll 1
                for (int c = 0; c < rest; ++c) {
                    const uint32_t o = p.base ? *at<uint16_t>(p.base + t0 * p.ldbase + n0, from[i] + 2 * c) : 0u;
                    *at<uint16_t>(p.out + t0 * p.ldout + n0, to[i] + 2 * c) =
                        (uint16_t)f32_to_bf16(__uint_as_float(o << 16) + f[c]);
                }
            }
        }
    }
}

// The base's own bits for a unit without an adapter (blocks as up_blocks).
__device__ __forceinline__ void copy_blocks(const Lora& p, int64_t t0, const int (&t)[2], const bool (&live)[2], int64_t nb,
                                            int64_t step, int64_t blocks_n) {
    const int lane = threadIdx.x & 63;
    const int64_t c = (threadIdx.x >> 6) * 64 + (lane & 7) * 8;
    for (; nb < blocks_n; nb += step) {
        const int64_t col = nb * 256 + c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!live[i] || col >= p.n) continue;
            const uint16_t* src = p.base ? p.base + (t0 + t[i]) * p.ldbase + col : nullptr;
            uint16_t* dst = p.out + (t0 + t[i]) * p.ldout + col;
            if (col + 8 <= p.n) {
                u32x4 v = {0u, 0u, 0u, 0u};
                if (src) v = load8(src, 0);
                store8(dst, 0, v);
            } else {
#pragma unroll 1
                for (int k = 0; k < p.n - col; ++k) dst[k] = src ? src[k] : (uint16_t)0;
            }
        }
    }
}

// a / b, a below 4096 (the reciprocal's error, 2^-10 of 1 / b, is far from the quotient's
// distance to a whole number, half of 1 / b).
__device__ __forceinline__ int small_quotient(int a, int b) {
    return (int)(((float)a + 0.5f) * __builtin_amdgcn_rcpf((float)b));
}

// Workgroup: a unit, blocks share, share + shares, .. of columns. The group's `workgroups`
// are shared out among the units that it has, not the adapters loaded, up to most_shares
// of them a unit (and each unit has one: the grid has workgroups + the most units - 1).
template <int RS>
__global__ __launch_bounds__(256, RS == 1 ? 4 : RS == 2 ? 3 : 2) void k_lora_up(Lora p, int64_t blocks_n, int workgroups,
                                                                                         int most_shares) {
    __shared__ UpLds<RS> lds;
    const int lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)blockIdx.x * kGroup;
    Unit unit;
    int share, shares;
    const bool found = unit.find(p, t0, [&](int units) {
        const int even = small_quotient(workgroups + units - 1, units);
        shares = even < most_shares ? even : most_shares;
        const int slot = small_quotient(blockIdx.y, shares);
        share = (int)blockIdx.y - slot * shares;
        return slot;
    });
    if (!found) return;
    int t[2];
    bool live[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = i * 8 + (lane >> 3);
        t[i] = unit.at(c);
        live[i] = c < unit.count;
    }
    if (unit.e == p.adapters) {
        if (p.base != p.out) copy_blocks(p, t0, t, live, share, shares, blocks_n);
        return;
    }
    u32x4 v[3][RS];
    lds.values(p, unit, t0, v);
    up_blocks<RS>(p, unit.e, t0, t, live, lds, v, share, shares, blocks_n);
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
int64_t at_least(int64_t a, int64_t b) { return a > b ? a : b; }

}  // namespace

hipError_t launch_lora_add(const Lora& call, hipStream_t st) {
    Lora p = call;
    if (p.tokens == 0 || p.n == 0) return hipSuccess;
    const int64_t groups = (p.tokens + kGroup - 1) / kGroup, steps = (p.k + kStepK - 1) / kStepK;
    // units of a group: at most one a token, and one an adapter (or none) and one for 16 tokens
    const int64_t most = at_most(p.tokens, kGroup), slots = at_most(most, (int64_t)p.adapters + 1 + most / kTile);
    // Parts of k for few tokens, as short workgroups, many of them: one spends its time on a
    // chain of dependent loads. (One token, k = 14336: 16 parts 4.7 + 4.5 us, 8 of them 6.0 + 4.3,
    // 56 of them 3.6 + 6.4. 1500 tokens of 9 requests, rank 16, 4096 x 4096: 5 parts 6.7 + 12.1,
    // 2 of them 9.4 + 10.5; 512 of as many requests: 8 parts 10.8 + 15.7, 16 of them 14 + 16.) By
    // the sizes alone: the order of a token's sums must not change with the adapters that are
    // loaded beside its own.
    const int64_t by_tokens = at_least(at_most(kLoraMaxParts, 4096 / p.tokens), at_most(8, kLoraPartRows / p.tokens));
    p.parts = (int)at_least(at_most(by_tokens, (steps + 3) / 4), 1);
#define CALL(RT)                                                                                              \
    hipLaunchKernelGGL((k_lora_down<RT>), dim3((unsigned)groups, (unsigned)p.parts, (unsigned)slots), dim3(256), 0, \
                       st, p)
    FP8_LORA_BY_RANK(CALL);
#undef CALL
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // About eleven workgroups a CU, those of a group of tokens shared out among the units that
    // it has, whatever is loaded. (128 tokens of as many requests, rank 16, 4096 x 14336, 64
    // adapters: 16 a CU 18 us, 11 of them 16. 5003 of as many of 16 adapters, rank 128: 10 a CU
    // 567, 11 of them 533. 5003 of one request, rank 64: 97 with 8 or with 64 adapters loaded;
    // shared out among those, 95 and 122.) A unit has at most what it would have of 16 a CU
    // in a group of 12 units: with more of them the values of v are added up too often (20000
    // tokens of 9 requests, rank 64, 4096 x 4096: 148 us without this limit, 101 with it).
    const int64_t blocks_n = (p.n + 255) / 256, cus = current_device_props().cus;
    const int64_t shares = at_most((16 * cus + 12 * groups - 1) / (12 * groups), blocks_n);
    const int64_t workgroups = at_most((11 * cus + groups - 1) / groups, slots * shares);
    const dim3 grid((unsigned)groups, (unsigned)(workgroups + slots - 1));
#define CALL(RS) hipLaunchKernelGGL((k_lora_up<RS>), grid, dim3(256), 0, st, p, blocks_n, (int)workgroups, (int)shares)
    FP8_LORA_BY_STEPS(CALL);
#undef CALL
    return hipGetLastError();
}

}  // namespace fp8amax
