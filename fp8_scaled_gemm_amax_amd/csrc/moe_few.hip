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
// same order, so that a lane's 16 bytes are one load.
#include "kernels.hpp"
#include "layer_device.hpp"

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

// Bitmap of the experts that some entry names, in LDS (all threads).
__device__ __forceinline__ void mark_experts(const MoeFew& p, uint32_t* bits) {
    for (int i = threadIdx.x; i < kMaxWords; i += blockDim.x) bits[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < p.tokens * p.topk; i += blockDim.x) {
        const int e = p.idx[i];
        if (e >= 0 && e < p.experts) atomicOr(&bits[e >> 5], 1u << (e & 31));
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
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(incl, o, 64);
        if (lane >= o) incl += y;
    }
    *total = __shfl(incl, 63, 64);
    return incl - pc;
}

// Token `lane`'s first slot that names expert e, -1 if none; the sum of the
// weights of all its slots that do in *share.
__device__ __forceinline__ int token_slot(const MoeFew& p, int e, float* share) {
    const int t = threadIdx.x & 63;
    int first = -1;
    float s = 0.0f;
    if (t < p.tokens)
        for (int j = 0; j < p.topk; ++j) {
            const int i = t * p.topk + j;
            if (p.idx[i] != e) continue;
            if (share) s += p.weights[i];
            if (first < 0) first = j;
        }
    if (share) *share = s;
    return first;
}

__device__ __forceinline__ uint4 load_weights(const uint8_t* p) {
    return load_stream(reinterpret_cast<const uint4*>(p));
}
// The same where `in`, zeros elsewhere (nothing is read there).
__device__ __forceinline__ uint4 load_weights_if(bool in, const uint8_t* p) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (in) v = load_weights(p);
    return v;
}
__device__ __forceinline__ v8bf load_bf16x8_if(bool in, const uint16_t* p) {
    v4u v = {0u, 0u, 0u, 0u};
    if (in) v = *reinterpret_cast<const v4u*>(p);
    return __builtin_bit_cast(v8bf, v);
}

// ------------------------------------------------------------- gate and up --
// Workgroup (tile, a): 16 columns of the a-th expert in use. Its wavefronts
// split K in blocks of kStep * U bytes, and their sums meet in LDS.
constexpr int kUpWaves = 4;

// Sums of 16 gate rows and 16 up rows against the tokens of tiles 0 .. NT-1
// (NT * 16 entries) over this wavefront's share of K.
template <int F, int NT, int U>
__device__ __forceinline__ void up_sums(const MoeFew& p, const uint8_t* gp, const uint8_t* up, const uint16_t* const* xp,
                                        int wave, v4f* ag, v4f* au) {
    const int j16 = ((threadIdx.x & 63) >> 4) * 16;
    const int K = p.hidden, whole = K / (kStep * U);
    for (int b = wave; b < whole; b += kUpWaves) {
        const int k0 = b * (kStep * U) + j16;
        uint4 g[U], u[U], x[NT][U][2];
#pragma unroll
        for (int s = 0; s < U; ++s) {
            g[s] = load_weights(gp + k0 + s * kStep);
            u[s] = load_weights(up + k0 + s * kStep);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                x[n][s][0] = *reinterpret_cast<const uint4*>(xp[n] + k0 + s * kStep);
                x[n][s][1] = *reinterpret_cast<const uint4*>(xp[n] + k0 + s * kStep + 8);
            }
        }
#pragma unroll
        for (int s = 0; s < U; ++s) {
            const v8bf g0 = decode_bf16<F>(g[s].x, g[s].y), g1 = decode_bf16<F>(g[s].z, g[s].w);
            const v8bf u0 = decode_bf16<F>(u[s].x, u[s].y), u1 = decode_bf16<F>(u[s].z, u[s].w);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const v8bf x0 = __builtin_bit_cast(v8bf, x[n][s][0]), x1 = __builtin_bit_cast(v8bf, x[n][s][1]);
                ag[n] = mfma(g0, x0, ag[n]);
                au[n] = mfma(u0, x0, au[n]);
                ag[n] = mfma(g1, x1, ag[n]);
                au[n] = mfma(u1, x1, au[n]);
            }
        }
    }
    // what is left of K, 64 bytes a step, the last step's lanes past K zero on both sides
    const int left0 = whole * U, steps = (K + kStep - 1) / kStep;
    for (int st = left0 + (wave + kUpWaves - whole % kUpWaves) % kUpWaves; st < steps; st += kUpWaves) {
        const int k = st * kStep + j16;
        const bool in = k < K;
        const uint4 g = load_weights_if(in, gp + k), u = load_weights_if(in, up + k);
        const v8bf g0 = decode_bf16<F>(g.x, g.y), g1 = decode_bf16<F>(g.z, g.w);
        const v8bf u0 = decode_bf16<F>(u.x, u.y), u1 = decode_bf16<F>(u.z, u.w);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const v8bf x0 = load_bf16x8_if(in, xp[n] + k), x1 = load_bf16x8_if(in, xp[n] + k + 8);
            ag[n] = mfma(g0, x0, ag[n]);
            au[n] = mfma(u0, x0, au[n]);
            ag[n] = mfma(g1, x1, ag[n]);
            au[n] = mfma(u1, x1, au[n]);
        }
    }
}

struct Entries {
    int token[kMoeFewTokens];
    int slot[kMoeFewTokens];
    float share[kMoeFewTokens];
    int count;
};

template <int F, int NT, int U>
__device__ __forceinline__ void up_tile(const MoeFew& p, int e, int c0, const Entries& ent, float* red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint8_t* we = p.w1 + (int64_t)e * p.gs1;
    const uint8_t* gp = we + (int64_t)(c0 + (lane & 15)) * p.ld1;
    const uint8_t* up = we + (int64_t)(p.inter + c0 + (lane & 15)) * p.ld1;
    const uint16_t* xp[NT];
    v4f ag[NT], au[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int c = n * 16 + (lane & 15);
        xp[n] = p.x + (int64_t)ent.token[c < ent.count ? c : 0] * p.ldx;     // (columns past the entries are not used)
        ag[n] = au[n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    up_sums<F, NT, U>(p, gp, up, xp, wave, ag, au);
    // red[wave][tile][gate | up][column * 16 + row], row = 4 (lane / 16) + i
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float* r = red + ((wave * NT + n) * 2) * 256 + (lane & 15) * 16 + (lane >> 4) * 4;
        *reinterpret_cast<v4f*>(r) = ag[n];
        *reinterpret_cast<v4f*>(r + 256) = au[n];
    }
    __syncthreads();
    const int row = threadIdx.x & 15;
    const float sg = p.s1[(int64_t)e * 2 * p.inter + c0 + row], su = p.s1[(int64_t)e * 2 * p.inter + p.inter + c0 + row];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int c = n * 16 + (threadIdx.x >> 4);
        if (c >= ent.count) continue;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < kUpWaves; ++w) {
            g += red[((w * NT + n) * 2) * 256 + threadIdx.x];
            u += red[((w * NT + n) * 2 + 1) * 256 + threadIdx.x];
        }
        const float a = silu_fast(g * sg) * (u * su) * ent.share[c];
        const uint32_t hi = f32_to_bf16(a);
        const float rest = a - __uint_as_float(hi << 16);
        // (an Inf or NaN is carried by the high part alone)
        const uint32_t lo = __builtin_isfinite(a) && __builtin_isfinite(rest) ? f32_to_bf16(rest) : 0u;
        uint16_t* dst = p.ws + ((int64_t)ent.token[c] * p.topk + ent.slot[c]) * 2 * p.inter + c0 + row;
        dst[0] = (uint16_t)hi;
        dst[p.inter] = (uint16_t)lo;
    }
}

template <int F, int NTMAX>
__global__ __launch_bounds__(kUpWaves * 64) void k_moe_few_up(MoeFew p) {
    __shared__ uint32_t bits[kMaxWords];
    __shared__ Entries ent;
    __shared__ __attribute__((aligned(16))) float red[kUpWaves * NTMAX * 2 * 256];
    const int lane = threadIdx.x & 63;
    mark_experts(p, bits);
    const uint32_t word = lane < kMaxWords ? bits[lane] : 0u;
    int total;
    const int below = words_below(word, &total);
    const int a = blockIdx.y;
    if (a >= total) return;                                 // (uniform: every wavefront has the same bitmap)
    const bool mine = lane < kMaxWords && a >= below && a < below + __popc(word);
    uint32_t w = word;
    for (int i = below; mine && i < a; ++i) w &= w - 1u;    // drop the experts before it
    const int owner = __ffsll((unsigned long long)__ballot(mine)) - 1;
    const int e = __shfl(lane * 32 + __ffs((int)w) - 1, owner, 64);
    float share;
    const int slot = token_slot(p, e, &share);
    const uint64_t has = __ballot(slot >= 0);
    if (threadIdx.x < 64) {
        if (slot >= 0) {
            const int r = __popcll(has & ((1ull << lane) - 1ull));
            ent.token[r] = lane;
            ent.slot[r] = slot;
            ent.share[r] = share;
        }
        if (lane == 0) ent.count = __popcll(has);
    }
    __syncthreads();
    const int c0 = blockIdx.x * 16;
    if constexpr (NTMAX >= 4) {
        if (ent.count > 32) {
            up_tile<F, 4, 1>(p, e, c0, ent, red);
            return;
        }
    }
    if constexpr (NTMAX >= 2) {
        if (ent.count > 16) {
            up_tile<F, 2, 2>(p, e, c0, ent, red);
            return;
        }
    }
    up_tile<F, 1, 4>(p, e, c0, ent, red);
}

// -------------------------------------------------------------------- down --
// Workgroup: 16 output columns of every token. The units of work are pieces of
// K of the experts in use, dealt to the wavefronts in order; a wavefront adds
// an expert's sums, times the weight rows' factors, to the sums of the tokens
// that use the expert and to no others (the products of the others are with a
// token's values of another expert; NaN codes do not reach them). The
// wavefronts' sums meet in LDS and are added in order.
constexpr int kDownWaves = 8;

template <int F, int NT, int U>
__global__ __launch_bounds__(kDownWaves * 64) void k_moe_few_down(MoeFew p) {
    __shared__ uint32_t bits[kMaxWords];
    __shared__ uint16_t list[kMoeMaxExperts];
    __shared__ __attribute__((aligned(16))) float red[kDownWaves * NT * 256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    mark_experts(p, bits);
    uint32_t word = lane < kMaxWords ? bits[lane] : 0u;
    int total;
    int at = words_below(word, &total);
    if (wave == 0)
        for (; word; word &= word - 1u) list[at++] = (uint16_t)(lane * 32 + __ffs((int)word) - 1);
    __syncthreads();
    const int row0 = blockIdx.x * 16, K = p.inter, j16 = (lane >> 4) * 16;
    const int blocks = (K + kStep * U - 1) / (kStep * U);
    int pieces = total > 0 ? kDownWaves / total : 1;
    pieces = pieces < 1 ? 1 : (pieces > blocks ? blocks : pieces);
    v4f sum[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) sum[n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int unit = wave; unit < total * pieces; unit += kDownWaves) {
        const int e = list[unit / pieces];
        const int slot = token_slot(p, e, nullptr);         // of token `lane`
        const uint64_t has = __ballot(slot >= 0);
        const int any = __ffsll((unsigned long long)has) - 1;   // a token that uses it (there is one)
        const uint16_t* ap[NT];
        bool used[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int t = n * 16 + (lane & 15);
            used[n] = (has >> t) & 1ull;
            const int src = used[n] ? t : any;
            ap[n] = p.ws + ((int64_t)src * p.topk + __shfl(slot, src, 64)) * 2 * K;
        }
        const uint8_t* wp = p.w2 + (int64_t)e * p.gs2 + (int64_t)(row0 + (lane & 15)) * p.ld2;
        const float* sp = p.s2 + (int64_t)e * p.hidden + row0 + (lane >> 4) * 4;
        v4f acc[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int b = unit % pieces; b < blocks; b += pieces) {
            const int kb = b * (kStep * U);
            if (kb + kStep * U <= K) {
                uint4 w[U];
#pragma unroll
                for (int s = 0; s < U; ++s) w[s] = load_weights(wp + kb + s * kStep + j16);
#pragma unroll
                for (int s = 0; s < U; ++s) {
                    const int k = kb + s * kStep + j16;
                    const v8bf w0 = decode_bf16<F>(w[s].x, w[s].y), w1 = decode_bf16<F>(w[s].z, w[s].w);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const v8bf* hi = reinterpret_cast<const v8bf*>(ap[n] + k);
                        const v8bf* lo = reinterpret_cast<const v8bf*>(ap[n] + K + k);
                        acc[n] = mfma(w0, hi[0], acc[n]);
                        acc[n] = mfma(w0, lo[0], acc[n]);
                        acc[n] = mfma(w1, hi[1], acc[n]);
                        acc[n] = mfma(w1, lo[1], acc[n]);
                    }
                }
            } else {
                for (int k = kb + j16; k - j16 < K; k += kStep) {
                    const bool in = k < K;
                    const uint4 w = load_weights_if(in, wp + k);
                    const v8bf w0 = decode_bf16<F>(w.x, w.y), w1 = decode_bf16<F>(w.z, w.w);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        acc[n] = mfma(w0, load_bf16x8_if(in, ap[n] + k), acc[n]);
                        acc[n] = mfma(w0, load_bf16x8_if(in, ap[n] + K + k), acc[n]);
                        acc[n] = mfma(w1, load_bf16x8_if(in, ap[n] + k + 8), acc[n]);
                        acc[n] = mfma(w1, load_bf16x8_if(in, ap[n] + K + k + 8), acc[n]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float s = sp[i];
#pragma unroll
            for (int n = 0; n < NT; ++n) sum[n][i] = used[n] ? fmaf(acc[n][i], s, sum[n][i]) : sum[n][i];
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
        *reinterpret_cast<v4f*>(red + (wave * NT + n) * 256 + (lane & 15) * 16 + (lane >> 4) * 4) = sum[n];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 256; i += kDownWaves * 64) {
        const int n = i >> 8, t = n * 16 + ((i & 255) >> 4), row = i & 15;
        if (t >= p.tokens) continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) s += red[(w * NT + n) * 256 + (i & 255)];
        p.out[(int64_t)t * p.ldo + row0 + row] = (uint16_t)f32_to_bf16(s);
    }
}

}  // namespace

hipError_t launch_moe_few_tokens(const MoeFew& p, int f1, int f2, hipStream_t st) {
    if (p.tokens == 0) return hipSuccess;
    const int entries = p.tokens * p.topk;
    const dim3 gu((unsigned)(p.inter / 16), (unsigned)(entries < p.experts ? entries : p.experts));
    const dim3 gd((unsigned)(p.hidden / 16));
#define FP8_UP(F, N) hipLaunchKernelGGL((k_moe_few_up<F, N>), gu, dim3(kUpWaves * 64), 0, st, p)
#define FP8_DOWN(F, N, U) hipLaunchKernelGGL((k_moe_few_down<F, N, U>), gd, dim3(kDownWaves * 64), 0, st, p)
    if (f1 == kE4M3) {
        if (p.tokens <= 16) FP8_UP(kE4M3, 1);
        else if (p.tokens <= 32) FP8_UP(kE4M3, 2);
        else FP8_UP(kE4M3, 4);
    } else {
        if (p.tokens <= 16) FP8_UP(kE5M2, 1);
        else if (p.tokens <= 32) FP8_UP(kE5M2, 2);
        else FP8_UP(kE5M2, 4);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (f2 == kE4M3) {
        if (p.tokens <= 16) FP8_DOWN(kE4M3, 1, 4);
        else if (p.tokens <= 32) FP8_DOWN(kE4M3, 2, 4);
        else FP8_DOWN(kE4M3, 4, 2);
    } else {
        if (p.tokens <= 16) FP8_DOWN(kE5M2, 1, 4);
        else if (p.tokens <= 32) FP8_DOWN(kE5M2, 2, 4);
        else FP8_DOWN(kE5M2, 4, 2);
    }
#undef FP8_UP
#undef FP8_DOWN
    return hipGetLastError();
}

}  // namespace fp8amax
