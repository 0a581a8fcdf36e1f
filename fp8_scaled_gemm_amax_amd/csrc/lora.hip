// lora.hip - low-rank adapters of many requests at once, beside a projection that
// they share: out[t] = base[t] + c_e (x_t A_e^T) B_e^T, e = adapter[t].
//
// Two launches. The first forms v = x A^T, for tiles of 16 tokens and parts of k,
// in fp32; the second adds the parts, multiplies v with B and adds the base. A tile
// goes through the adapters that its tokens name, one after the other (or, for a few
// tokens, side by side in workgroups of their own), each multiplied with the whole
// tile on the matrix cores and kept for its own tokens alone: what another token or
// another adapter holds never enters a token's result. Tokens of one request next to
// each other share their adapter's loads; in any other order the result is the same.
// v c_e is kept as the sum of two bf16 numbers and multiplied in two products, so
// that the only rounding that counts is the output's.
#include "block.hpp"
#include "layer_device.hpp"

namespace fp8amax {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kBlock = 256, kWaves = 4;
constexpr int kTile = 16;                       // tokens of a tile
constexpr int kStepK = 64;                      // columns of x of one step of a wavefront

__device__ __forceinline__ v4f mfma(u32x4 a, u32x4 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}
// 16 bytes where `in`, zeros elsewhere (nothing is read there).
__device__ __forceinline__ u32x4 load_if(bool in, const uint16_t* p) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (in) v = *reinterpret_cast<const u32x4*>(p);
    return v;
}

// The adapters of a tile's tokens, in the order of their first tokens; every
// wavefront goes through the same ones.
struct Adapters {
    int mine;                                   // of token lane & 15: -1 for none
    uint32_t left;                              // tokens whose adapter is still to come
    __device__ __forceinline__ Adapters(const Lora& p, int64_t t0) {
        const int lane = threadIdx.x & 63;
        const int64_t t = t0 + (lane & 15);
        const int e = t < p.tokens ? p.adapter[t] : -1;
        mine = e >= 0 && e < p.adapters ? e : -1;
        left = (uint32_t)__ballot(mine >= 0) & 0xffffu;
    }
    // the next adapter, and a bit for each of its tokens
    __device__ __forceinline__ int next(uint32_t* tokens) {
        const int e = __builtin_amdgcn_readlane(mine, __ffs((int)left) - 1);
        *tokens = (uint32_t)__ballot(mine == e) & 0xffffu;
        left &= ~*tokens;
        return e;
    }
};

// ------------------------------------------------------------------ x A^T --
// Workgroup (tile, part, slot): the part's sums for every slot-th adapter of the
// tile. Its wavefronts share the part's steps; a lane's 32 bytes of a step are
// neighbours in memory (the order of k is the same on both sides, so any serves).
template <int RT>
__global__ __launch_bounds__(kBlock) void k_lora_down(Lora p) {
    __shared__ float red[kWaves][RT * 256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t0 = (int64_t)blockIdx.x * kTile;
    Adapters todo(p, t0);
    const int64_t steps = (p.k + kStepK - 1) / kStepK;
    const int64_t s0 = steps * blockIdx.y / p.parts, s1 = steps * (blockIdx.y + 1) / p.parts;
    const int64_t t = t0 + (lane & 15);
    const uint16_t* xr = p.x + (t < p.tokens ? t : p.tokens - 1) * p.ldx;
    const int kq = (lane >> 4) * 16;
    for (int j = 0; todo.left; ++j) {
        uint32_t tokens;
        const int e = todo.next(&tokens);
        if (j % (int)gridDim.z != (int)blockIdx.z) continue;
        const uint16_t* ar[RT];
        v4f acc[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int row = r * 16 + (lane & 15);
            ar[r] = p.a + e * p.gsa + (row < p.rank ? row : p.rank - 1) * p.lda;
            acc[r] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
        for (int64_t s = s0 + wave; s < s1; s += kWaves) {
            const int64_t k = s * kStepK + kq;
            const bool in0 = k < p.k, in1 = k + 8 < p.k;
            const u32x4 x0 = load_if(in0, xr + k), x1 = load_if(in1, xr + k + 8);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                acc[r] = mfma(load_if(in0, ar[r] + k), x0, acc[r]);
                acc[r] = mfma(load_if(in1, ar[r] + k + 8), x1, acc[r]);
            }
        }
        __syncthreads();                        // the adapter before is written
#pragma unroll
        for (int r = 0; r < RT; ++r)            // column (token) lane % 16, rows 4 (lane / 16) ..
            *reinterpret_cast<v4f*>(&red[wave][r * 256 + (lane & 15) * 16 + (lane >> 4) * 4]) = acc[r];
        __syncthreads();
        const int col = threadIdx.x >> 4;
        float* dst = p.ws + ((int64_t)blockIdx.y * p.tokens + t0 + col) * p.rank;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int row = r * 16 + (threadIdx.x & 15);
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += red[w][r * 256 + threadIdx.x];
            if (((tokens >> col) & 1u) && row < p.rank) dst[row] = v;
        }
    }
}

// ------------------------------------------------------------- base + v B^T --
// Workgroup: a tile's tokens, 256 columns; a wavefront 64 of them as four products
// of 16 rows of B with the 16 tokens. Row m of product i is column 32 (i / 2) +
// 8 (m / 4) + 4 (i % 2) + m % 4: a lane's four sums of products 2 j and 2 j + 1 are
// then 8 neighbouring columns of its token.
constexpr int kCols = 256;

__global__ __launch_bounds__(kBlock) void k_lora_up(Lora p, int64_t blocks_n, int vec) {
    __shared__ __attribute__((aligned(16))) uint16_t vs[2][kTile * (kLoraMaxRank + 8)];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t0 = (int64_t)(blockIdx.x / blocks_n) * kTile;
    const int64_t n0 = (int64_t)(blockIdx.x % blocks_n) * kCols + wave * 64;
    Adapters todo(p, t0);
    const int pitch = p.rank + 8;
    for (int i = threadIdx.x; i < kTile * p.rank; i += kBlock) {
        const int tok = i / p.rank, j = i % p.rank;
        const int e = __shfl(todo.mine, tok, 64);
        float v = 0.0f;
        if (e >= 0) {
            const float* src = p.ws + (t0 + tok) * p.rank + j;
#pragma unroll 4
            for (int q = 0; q < p.parts; ++q) v += src[(int64_t)q * p.tokens * p.rank];
            v *= p.scaling[e];
        }
        // (an Inf or NaN is carried by the high part alone; a finite value that bf16
        // would round to Inf is bf16's largest and the rest)
        const bool finite = __builtin_isfinite(v);
        uint32_t hi = f32_to_bf16(v);
        hi -= finite && (hi & 0x7fffu) == 0x7f80u ? 1u : 0u;
        vs[0][tok * pitch + j] = (uint16_t)hi;
        vs[1][tok * pitch + j] = (uint16_t)(finite ? f32_to_bf16(v - __uint_as_float(hi << 16)) : 0u);
    }
    __syncthreads();
    const int q = lane >> 4, m = lane & 15;
    v4f sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    while (todo.left) {
        uint32_t tokens;
        const int e = todo.next(&tokens);
        const uint16_t* br[4];
        v4f hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = n0 + (i >> 1) * 32 + (m >> 2) * 8 + (i & 1) * 4 + (m & 3);
            br[i] = p.b + e * p.gsb + (n < p.n ? n : p.n - 1) * p.ldb;
            hi[i] = lo[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
        for (int j = q * 8; j - q * 8 < p.rank; j += 32) {
            const bool in = j < p.rank;
            const u32x4 vh = load_if(in, &vs[0][m * pitch + j]), vl = load_if(in, &vs[1][m * pitch + j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4 w = load_if(in, br[i] + j);
                hi[i] = mfma(w, vh, hi[i]);
                lo[i] = mfma(w, vl, lo[i]);
            }
        }
        const bool mine = (tokens >> m) & 1u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // (an infinite weight: the low parts, of either sign or 0, would make NaN of Inf)
                const float v = __builtin_isfinite(hi[i][c]) ? hi[i][c] + lo[i][c] : hi[i][c];
                sum[i][c] = mine ? v : sum[i][c];
            }
    }
    const int64_t t = t0 + m;
    if (t >= p.tokens) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t n = n0 + h * 32 + q * 8;
        if (n >= p.n) continue;
        const uint16_t* src = p.base ? p.base + t * p.ldbase + n : nullptr;
        uint16_t* dst = p.out + t * p.ldout + n;
        float f[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            f[c] = sum[2 * h][c];
            f[4 + c] = sum[2 * h + 1][c];
        }
        if (vec && n + 8 <= p.n) {
            uint4 b = make_uint4(0u, 0u, 0u, 0u);
            if (src) b = *reinterpret_cast<const uint4*>(src);
            float g[8];
            unpack8(b, g);
#pragma unroll
            for (int c = 0; c < 8; ++c) g[c] += f[c];
            // (no adapter: the base's own bits)
            *reinterpret_cast<uint4*>(dst) = todo.mine >= 0 ? pack8(g) : b;
        } else {
            for (int c = 0; c < 8 && n + c < p.n; ++c) {
                const uint32_t b = src ? src[c] : 0u;
                dst[c] = (uint16_t)(todo.mine >= 0 ? f32_to_bf16(__uint_as_float(b << 16) + f[c]) : b);
            }
        }
    }
}

}  // namespace

hipError_t launch_lora_add(const Lora& p0, hipStream_t st) {
    Lora p = p0;
    if (p.tokens == 0 || p.n == 0) return hipSuccess;
    const int64_t tiles = (p.tokens + kTile - 1) / kTile, steps = (p.k + kStepK - 1) / kStepK;
    int64_t parts = kLoraPartRows / p.tokens;
    parts = parts < 16 ? parts : 16;
    parts = parts < (steps + kWaves - 1) / kWaves ? parts : (steps + kWaves - 1) / kWaves;
    p.parts = (int)(parts < 1 ? 1 : parts);
    const dim3 grid((unsigned)tiles, (unsigned)p.parts, p.tokens <= 1024 ? kTile : 2);
    if (p.rank <= 16) hipLaunchKernelGGL((k_lora_down<1>), grid, dim3(kBlock), 0, st, p);
    else if (p.rank <= 32) hipLaunchKernelGGL((k_lora_down<2>), grid, dim3(kBlock), 0, st, p);
    else if (p.rank <= 64) hipLaunchKernelGGL((k_lora_down<4>), grid, dim3(kBlock), 0, st, p);
    else hipLaunchKernelGGL((k_lora_down<8>), grid, dim3(kBlock), 0, st, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks_n = (p.n + kCols - 1) / kCols;
    const bool vec = chunk_aligned(p.base, p.ldbase) && chunk_aligned(p.out, p.ldout);
    hipLaunchKernelGGL(k_lora_up, dim3((unsigned)(tiles * blocks_n)), dim3(kBlock), 0, st, p, blocks_n, (int)vec);
    return hipGetLastError();
}

}  // namespace fp8amax
