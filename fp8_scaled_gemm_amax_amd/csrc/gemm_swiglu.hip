// gemm_swiglu.hip - the gated feed-forward block's products with SwiGLU in the
// epilogue: the gate and up projections with silu(gate) * up, and the backward
// pass's product, which gives the activation's gradient, with SwiGLU's gradient.
//
//   forward: g = (A Wg^T) sa sb, u = (A Wu^T) sa sb, act = g sigma(g) u
//   backward: da = (A B^T) sa sb, s = sigma(g),
//     d(gate) = da u s (1 + g (1 - s)), d(up) = da g s, act = g s u
//
// The sums are fp32 and reach SwiGLU unrounded; each output is rounded once.
// B's rows are loaded such that a wavefront has the gate and the up columns of the
// same numbers: a lane then holds g and u of an element in two of its registers,
// and SwiGLU needs no exchange.
#include "block.hpp"
#include "gemm_device.hpp"

namespace fp8amax {
namespace {

// sigma(g) = 1 / (1 + 2^(-g log2 e)): the exponent's rounding is an error of |g|
// 2^-24 relative to the exponential, far below the outputs' 2^-9; 2^128 and more
// count as infinite (sigma 0), which the reciprocal of Inf gives.
__device__ __forceinline__ float sigma(float g) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}
__device__ __forceinline__ float swiglu(float g, float u) { return g * sigma(g) * u; }

struct SwigluGrad {
    float dg, du, act;
};
__device__ __forceinline__ SwigluGrad swiglu_grad(float da, float g, float u) {
    const float s = sigma(g), silu = g * s;
    return {da * u * (s * fmaf(g, 1.0f - s, 1.0f)), da * silu, silu * u};
}

__device__ __forceinline__ float bf16(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// ------------------------------------------------------- 128 x 128 tiles --
// Any sizes (k in steps of 16). Rows of B of a tile: 32 gate rows, the 32 up rows
// of the same columns, 32 gate rows, ..: block 0 of a wavefront is gate, block 1 up.
struct GluRows {
    const uint8_t* gate;        // of the tile's first column
    int64_t up, ld, valid;      // up: bytes from a gate row to its up row
    __device__ __forceinline__ int col(int row) const { return (row >> 6) * 32 + (row & 31); }
    __device__ __forceinline__ bool has(int row) const { return col(row) < valid; }
    __device__ __forceinline__ const uint8_t* at(int row) const {
        return gate + ((row >> 5) & 1) * up + (int64_t)col(row) * ld;
    }
};

template <int FA, int FB>
__global__ __launch_bounds__(kThreads) void k_glu(GluFwd p) {
    __shared__ uint4 As[BM * kChunksPerRow];
    __shared__ uint4 Bs[BN * kChunksPerRow];
    const int64_t tiles_n = (p.inter + 63) / 64;
    const int64_t row0 = (int64_t)(blockIdx.x / tiles_n) * BM, col0 = (int64_t)(blockIdx.x % tiles_n) * 64;
    v16f acc[2][2];
    mma_rows<FA, FB>(TileRows{p.a + row0 * p.lda, p.lda, p.m - row0},
                     GluRows{p.b + col0 * p.ldb, p.inter * p.ldb, p.ldb, p.inter - col0}, p.k, acc, As, Bs);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t col = col0 + (wave & 1) * 32 + (lane & 31);
    if (col >= p.inter) return;
    const float sg = p.sb[p.sb_vec ? col : 0], su = p.sb[p.sb_vec ? p.inter + col : 0];
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int64_t row = row0 + (wave >> 1) * 64 + mi * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
            if (row >= p.m) continue;
            const float sa = p.sa[p.sa_vec ? row : 0];
            const float g = acc[mi][0][r] * sa * sg, u = acc[mi][1][r] * sa * su;
            p.act[row * p.ldact + col] = (uint16_t)f32_to_bf16(swiglu(g, u));
            if (p.h) {
                p.h[row * p.ldh + col] = (uint16_t)f32_to_bf16(g);
                p.h[row * p.ldh + p.inter + col] = (uint16_t)f32_to_bf16(u);
            }
        }
}

template <int FA, int FB>
__global__ __launch_bounds__(kThreads) void k_glu_grad(GluBwd p) {
    __shared__ uint4 As[BM * kChunksPerRow];
    __shared__ uint4 Bs[BN * kChunksPerRow];
    const int64_t tiles_n = (p.inter + BN - 1) / BN;
    const int64_t row0 = (int64_t)(blockIdx.x / tiles_n) * BM, col0 = (int64_t)(blockIdx.x % tiles_n) * BN;
    v16f acc[2][2];
    mma_rows<FA, FB>(TileRows{p.a + row0 * p.lda, p.lda, p.m - row0},
                     TileRows{p.b + col0 * p.ldb, p.ldb, p.inter - col0}, p.k, acc, As, Bs);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int ni = 0; ni < 2; ++ni) {
        const int64_t col = col0 + (wave & 1) * 64 + ni * 32 + (lane & 31);
        if (col >= p.inter) continue;
        const float sb = p.sb[p.sb_vec ? col : 0];
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t row = row0 + (wave >> 1) * 64 + mi * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                if (row >= p.m) continue;
                const uint16_t* hr = p.h + row * p.ldh + col;
                const SwigluGrad d =
                    swiglu_grad(acc[mi][ni][r] * p.sa[p.sa_vec ? row : 0] * sb, bf16(hr), bf16(hr + p.inter));
                p.dh[row * p.lddh + col] = (uint16_t)f32_to_bf16(d.dg);
                p.dh[row * p.lddh + p.inter + col] = (uint16_t)f32_to_bf16(d.du);
                if (p.act) p.act[row * p.ldact + col] = (uint16_t)f32_to_bf16(d.act);
            }
    }
}

}  // namespace

template <int FA, int FB>
hipError_t glu_typed(const GluFwd& p, hipStream_t st) {
    const int64_t tiles = (p.m + BM - 1) / BM * ((p.inter + 63) / 64);
    hipLaunchKernelGGL((k_glu<FA, FB>), dim3((unsigned)tiles), dim3(kThreads), 0, st, p);
    return hipGetLastError();
}

template <int FA, int FB>
hipError_t glu_grad_typed(const GluBwd& p, hipStream_t st) {
    const int64_t tiles = (p.m + BM - 1) / BM * ((p.inter + BN - 1) / BN);
    hipLaunchKernelGGL((k_glu_grad<FA, FB>), dim3((unsigned)tiles), dim3(kThreads), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_gemm_swiglu(const GluFwd& p, int fa, int fb, hipStream_t st) {
    if (p.m == 0 || p.inter == 0) return hipSuccess;
    if (fa == kE4M3) return fb == kE4M3 ? glu_typed<kE4M3, kE4M3>(p, st) : glu_typed<kE4M3, kE5M2>(p, st);
    return fb == kE4M3 ? glu_typed<kE5M2, kE4M3>(p, st) : glu_typed<kE5M2, kE5M2>(p, st);
}

hipError_t launch_gemm_swiglu_backward(const GluBwd& p, int fa, int fb, hipStream_t st) {
    if (p.m == 0 || p.inter == 0) return hipSuccess;
    if (fa == kE4M3) return fb == kE4M3 ? glu_grad_typed<kE4M3, kE4M3>(p, st) : glu_grad_typed<kE4M3, kE5M2>(p, st);
    return fb == kE4M3 ? glu_grad_typed<kE5M2, kE4M3>(p, st) : glu_grad_typed<kE5M2, kE5M2>(p, st);
}

}  // namespace fp8amax
