// layer_device.hpp - device helpers of the layer kernels around the products
// (norm, SwiGLU, the MoE layer for a few tokens): MX blocks of fp32 values, MX
// decoding, wavefront sums, the logistic function (gfx950 only).
#pragma once

#include "fp8_device.hpp"

namespace fp8amax {

// base + a 32-bit byte offset: with a base that is uniform over the wavefront the
// access takes a scalar base and one offset register.
template <typename V>
__device__ __forceinline__ const V* at(const void* base, uint32_t bytes) {
    return reinterpret_cast<const V*>(static_cast<const char*>(base) + bytes);
}
template <typename V>
__device__ __forceinline__ V* at(void* base, uint32_t bytes) {
    return reinterpret_cast<V*>(static_cast<char*>(base) + bytes);
}

// Sum over the 64 lanes in every lane: neighbours, pairs, quads and eights by
// data-parallel moves, sixteens and thirty-twos by lane swaps, always the two
// halves' sums added: every lane ends with the same bits. (Six shuffles through
// LDS would take six index registers and their latency.)
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_move<0xB1>(v);       // quad_perm [1, 0, 3, 2]
    v += dpp_move<0x4E>(v);       // quad_perm [2, 3, 0, 1]
    v += dpp_move<0x141>(v);      // row_half_mirror
    v += dpp_move<0x140>(v);      // row_mirror
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const uint32_t w = __float_as_uint(v);
    const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// The larger magnitude; NaN if either is NaN (v_maximum3_f32: two values a
// step, where the order of magnitude bits takes an and and a maximum each).
__device__ __forceinline__ float absmax(float a, float b) {
    return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}
__device__ __forceinline__ float absmax8(const float* f) {
    float m = absmax(f[0], f[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2)
        m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(f[i]), __builtin_fabsf(f[i + 1])),
                                          m);
    return m;
}
// Largest of the 64 lanes (not negative, or NaN) in every lane.
__device__ __forceinline__ float wave_max(float v) {
    v = __builtin_elementwise_maximum(v, dpp_move<0xB1>(v));
    v = __builtin_elementwise_maximum(v, dpp_move<0x4E>(v));
    v = __builtin_elementwise_maximum(v, dpp_move<0x141>(v));
    v = __builtin_elementwise_maximum(v, dpp_move<0x140>(v));
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __builtin_elementwise_maximum(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const uint32_t w = __float_as_uint(v);
    const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return __builtin_elementwise_maximum(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// Sum and maximum of W wavefronts' values in LDS (after a barrier), in order.
template <int W>
__device__ __forceinline__ float sum_of(const float* r) {
    float s = r[0];
#pragma unroll
    for (int w = 1; w < W; ++w) s += r[w];
    return s;
}
template <int W>
__device__ __forceinline__ float max_of(const float* r) {
    float m = r[0];
#pragma unroll
    for (int w = 1; w < W; ++w) m = __builtin_elementwise_maximum(m, r[w]);
    return m;
}

// 1 / (1 + exp(-g)) and its complement, from t = exp(-|g|) <= 1, so that
// nothing overflows and the smaller of the two is not a difference:
// sigma(|g|) = 1 / (1 + t), sigma(-|g|) = t / (1 + t). exp(-|g|) =
// 2^(n + e), n + e = -|g| log2 e with the product's rounding error and log2 e's
// own tail carried in e: the relative error of t stays at 2^-22 for every g
// (without e it grows with |g|). t underflows to 0 below exp(-87.3) (the
// hardware exponential has no subnormal results). An Inf or NaN g: e would be
// NaN for Inf, so it is dropped there.
struct Logistic {
    float sig, com;   // sigma(g), 1 - sigma(g)
};
__device__ __forceinline__ Logistic logistic(float g) {
    const float a = __builtin_fabsf(g);
    const float n = a * -1.44269502f;                           // fl32(-log2 e)
    float e = fmaf(a, -1.44269502f, -n);
    e = fmaf(a, -1.92596303e-8f, e);                            // log2 e - fl32(log2 e)
    e = a < 128.0f ? e : 0.0f;                                  // (t is 0 there anyway)
    const float t0 = __builtin_amdgcn_exp2f(n);
    const float t = fmaf(t0, e * 0.693147181f, t0);             // 2^e = 1 + e ln 2, |e| < 2^-17
    const float d = 1.0f + t;
    float r = __builtin_amdgcn_rcpf(d);
    r = fmaf(fmaf(-d, r, 1.0f), r, r);                          // d in [1, 2]: one Newton step, no special cases
    const float s = t * r;
    const bool neg = g < 0.0f;
    return {neg ? s : r, neg ? r : s};
}
// g sigma(g). -Inf gives NaN, as in the definition's arithmetic (-Inf * 0).
__device__ __forceinline__ float silu_fast(float g) { return g * logistic(g).sig; }

// Block scale of the MX format from the fp32 magnitude bits of the block's
// largest element (NaN above Inf in this order): e = floor(log2 amax) - emax,
// clamped to -127 .. 127, byte e + 127; 255 for an Inf or NaN in the block,
// whose elements are then cast with scale 1. A subnormal amax is clamped to
// -127 whatever its exponent.
template <int F>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits, float* mul) {
    constexpr int emax = F == kE4M3 ? 8 : 15;
    if (amax_bits >= 0x7f800000u) {
        *mul = 1.0f;
        return 0xFFu;
    }
    int e = (int)(amax_bits >> 23) - 127 - emax;
    e = e < -127 ? -127 : e;
    *mul = __uint_as_float((uint32_t)(127 - e) << 23);          // 2^-e, a normal float: e <= 127 - emax
    return (uint32_t)(e + 127);
}

// 2^(byte - 127), NaN for 255 (byte 0 is the subnormal 2^-127).
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    if (b == 0xFFu) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(b == 0u ? 0x00400000u : b << 23);
}

// Four OCP codes of a word -> fp32 (exact).
template <int F>
__device__ __forceinline__ void decode4(uint32_t w, float* o) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    f32x2 lo, hi;
    if constexpr (F == kE4M3) {
        lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    } else {
        lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
        hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
    }
    o[0] = lo[0];
    o[1] = lo[1];
    o[2] = hi[0];
    o[3] = hi[1];
}

__device__ __forceinline__ void unpack8(uint4 v, float* o) {
    o[0] = bf16_lo(v.x);
    o[1] = bf16_hi(v.x);
    o[2] = bf16_lo(v.y);
    o[3] = bf16_hi(v.y);
    o[4] = bf16_lo(v.z);
    o[5] = bf16_hi(v.z);
    o[6] = bf16_lo(v.w);
    o[7] = bf16_hi(v.w);
}

// Two fp32 values -> bf16 (nearest even, NaN quiet), one instruction on gfx950.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}
// Eight fp32 values -> one 16-byte chunk of bf16.
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

template <int F, bool NAN_FREE>
__device__ __forceinline__ uint2 encode8f(const float* f, float s) {
    uint2 o;
    o.x = encode4<F, NAN_FREE>(f[0] * s, f[1] * s, f[2] * s, f[3] * s);
    o.y = encode4<F, NAN_FREE>(f[4] * s, f[5] * s, f[6] * s, f[7] * s);
    return o;
}

// Eight values times s = scale_from_amax of a finite amax of theirs -> codes.
// |value * s| ends at most two roundings above fmax, which the conversion
// rounds to fmax: no clamp.
template <int F>
__device__ __forceinline__ uint2 encode8_scaled(const float* f, float s) {
    if constexpr (F == kE4M3) {
        int a = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * s, f[1] * s, 0, false);
        a = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * s, f[3] * s, a, true);
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4] * s, f[5] * s, 0, false);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(f[6] * s, f[7] * s, b, true);
        return make_uint2((uint32_t)a, (uint32_t)b);
    } else if constexpr (F == kE5M2) {
        int a = __builtin_amdgcn_cvt_pk_bf8_f32(f[0] * s, f[1] * s, 0, false);
        a = __builtin_amdgcn_cvt_pk_bf8_f32(f[2] * s, f[3] * s, a, true);
        int b = __builtin_amdgcn_cvt_pk_bf8_f32(f[4] * s, f[5] * s, 0, false);
        b = __builtin_amdgcn_cvt_pk_bf8_f32(f[6] * s, f[7] * s, b, true);
        return make_uint2((uint32_t)a, (uint32_t)b);
    } else {
        return encode8f<F, true>(f, s);
    }
}

// One lane's chunk of 8 values of a row's MX checkpoint: the block of 32 is
// this lane's and its three neighbours' (lanes 4i .. 4i + 3), the record of
// four blocks that of 16 lanes. Every lane of the wavefront calls it (lanes
// past the row pass live = false; a block's four lanes are alike in that: the
// row is a multiple of 32). Returns the codes; *record is
// valid in lanes 16i, blocks past the row holding byte 0.
template <int F>
__device__ __forceinline__ uint2 mx_chunk(const float* f, bool live, uint32_t* record) {
    float m = absmax8(f);
    m = __builtin_elementwise_maximum(m, dpp_move<0xB1>(m));                // lane ^ 1
    m = __builtin_elementwise_maximum(m, dpp_move<0x4E>(m));                // lane ^ 2
    float mul;
    const uint32_t byte = mx_scale_byte<F>(__float_as_uint(m), &mul);
    const int mine = live ? (int)byte : 0;
    const uint32_t b1 = (uint32_t)__builtin_amdgcn_update_dpp(0, mine, 0x104, 0xf, 0xf, true),      // lanes + 4, 8, 12
                   b2 = (uint32_t)__builtin_amdgcn_update_dpp(0, mine, 0x108, 0xf, 0xf, true),
                   b3 = (uint32_t)__builtin_amdgcn_update_dpp(0, mine, 0x10C, 0xf, 0xf, true);
    *record = (uint32_t)mine | (b1 << 8) | (b2 << 16) | (b3 << 24);
    return byte != 0xFFu ? encode8f<F, true>(f, mul) : encode8f<F, false>(f, mul);
}

// Store of checkpoint codes: nontemporal, for they are read only in the backward
// pass, and what the next product reads (the cast's codes) then keeps its place
// in the caches (SwiGLU at 8192 x 7168: 80.8 -> 76.7 us).
__device__ __forceinline__ void store_checkpoint(uint8_t* p, uint2 v) {
    typedef unsigned int u32x2_nt __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store((u32x2_nt{v.x, v.y}), reinterpret_cast<u32x2_nt*>(p));
}

// Chunks of 8 values of a row of n: 16-byte accesses where the layout allows
// them (LOOSE = false: the row starts on 16 bytes and n is a multiple of 8), else
// 16 bytes at the row's own alignment (n >= 8). The last, cut chunk is loaded as
// the row's last 8 values and shifted into place when it is used, zeros behind
// it: no load waits in a branch (by elements in a branch, the gradient of 333 x
// 1111 took 17 us instead of 10).
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// A value whose address is a multiple of A bytes only. V is a scalar or one of the
// compiler's own vectors: a class (HIP's uint4, float4) would keep its alignment
// of 16 in here, and the access would promise it.
template <typename V, int A>
struct __attribute__((packed, aligned(A))) Loose {
    V v;
};
template <typename V, int A>
__device__ __forceinline__ V load_loose(const void* base, uint32_t bytes) {
    static_assert(alignof(Loose<V, A>) == A && sizeof(Loose<V, A>) == sizeof(V), "no more alignment than the layout has");
    return at<Loose<V, A>>(base, bytes)->v;
}
template <typename V, int A>
__device__ __forceinline__ void store_loose(void* base, uint32_t bytes, V v) {
    static_assert(alignof(Loose<V, A>) == A && sizeof(Loose<V, A>) == sizeof(V), "no more alignment than the layout has");
    at<Loose<V, A>>(base, bytes)->v = v;
}
// Eight values at any alignment, past the caches: what is met once leaves the place to
// what is read again.
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
__device__ __forceinline__ u32x4 load8(const uint16_t* base, uint32_t bytes) {
    return __builtin_nontemporal_load(at<u32x4_a2>(base, bytes));
}
__device__ __forceinline__ void store8(uint16_t* base, uint32_t bytes, u32x4 v) {
    __builtin_nontemporal_store(v, at<u32x4_a2>(base, bytes));
}
template <bool LOOSE>
__device__ __forceinline__ uint4 load_chunk(const uint16_t* row, uint32_t ch, uint32_t n) {
    if constexpr (!LOOSE) return load_stream(at<uint4>(row, ch * 16));
    const u32x4 v = load_loose<u32x4, 2>(row, (ch * 8 + 8 <= n ? ch * 8 : n - 8) * 2);
    return make_uint4(v.x, v.y, v.z, v.w);
}
// What load_chunk gave for chunk ch, its values in place.
template <bool LOOSE>
__device__ __forceinline__ void place_chunk(uint4* v, uint32_t ch, uint32_t n) {
    if constexpr (LOOSE) {
        if (ch * 8 + 8 > n) {
            const uint32_t s = ch * 8 + 8 - n;              // values to drop: 1 .. 7
            uint32_t x = v->x, y = v->y, z = v->z, w = v->w;
            x = s & 4 ? z : x;
            y = s & 4 ? w : y;
            z = s & 4 ? 0u : z;
            w = s & 4 ? 0u : w;
            x = s & 2 ? y : x;
            y = s & 2 ? z : y;
            z = s & 2 ? w : z;
            w = s & 2 ? 0u : w;
            const uint32_t odd = (s & 1) * 16;
            x = __builtin_amdgcn_alignbit(y, x, odd);
            y = __builtin_amdgcn_alignbit(z, y, odd);
            z = __builtin_amdgcn_alignbit(w, z, odd);
            w >>= odd;
            *v = make_uint4(x, y, z, w);
        }
    }
}
template <bool LOOSE>
__device__ __forceinline__ void store_chunk(uint16_t* row, uint32_t ch, uint32_t n, const float* f) {
    uint4 v = pack8(f);
    if constexpr (!LOOSE) {
        *at<uint4>(row, ch * 16) = v;
        return;
    }
    if (ch * 8 + 8 <= n) {
        store_loose<u32x4, 2>(row, ch * 16, u32x4{v.x, v.y, v.z, v.w});
        return;
    }
    const uint32_t m = n - ch * 8;                          // 4 + 2 + 1 of the 1 .. 7 values there
    uint32_t o = ch * 16;
    if (m & 4) {
        store_loose<u32x2, 2>(row, o, u32x2{v.x, v.y});
        v.x = v.z;
        v.y = v.w;
        o += 8;
    }
    if (m & 2) {
        store_loose<uint32_t, 2>(row, o, v.x);
        v.x = v.y;
        o += 4;
    }
    if (m & 1) *at<uint16_t>(row, o) = (uint16_t)v.x;
}
template <bool LOOSE>
__device__ __forceinline__ void store_codes(uint8_t* row, uint32_t ch, uint32_t n, uint2 v) {
    if constexpr (!LOOSE) {
        *at<uint2>(row, ch * 8) = v;
        return;
    }
    if (ch * 8 + 8 <= n) {
        store_loose<u32x2, 1>(row, ch * 8, u32x2{v.x, v.y});
        return;
    }
    const uint32_t m = n - ch * 8;
    uint32_t o = ch * 8;
    if (m & 4) {
        store_loose<uint32_t, 1>(row, o, v.x);
        v.x = v.y;
        o += 4;
    }
    if (m & 2) {
        store_loose<uint16_t, 1>(row, o, (uint16_t)v.x);
        v.x >>= 16;
        o += 2;
    }
    if (m & 1) row[o] = (uint8_t)v.x;
}

// Workgroup -> index of its rows such that the workgroups of one XCD (every
// eighth one in dispatch order) work on neighbouring rows at a time: what
// neighbouring rows write into one line (the scale records, 4 bytes a row) then
// meets in one L2 instead of leaving as partial lines of eight.
__device__ __forceinline__ int64_t xcd_block(int64_t b, int64_t n) {
    const int64_t per = n / 8, rest = n % 8, x = b % 8;
    return x * per + (x < rest ? x : rest) + b / 8;
}

}  // namespace fp8amax
