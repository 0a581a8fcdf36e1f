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

typedef float f32x4 __attribute__((ext_vector_type(4)));

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

// ------------------------------------------------------- 256 x 256 tiles --
// The K128 loop's large tile, persistent: a workgroup takes tiles w, w + G, .., and
// the next tile's first two K steps load during the current one's last two. Tiles
// past the last row (column) are shifted back to end there (there are enough of both
// for a tile); what the tile before computes too is stored twice, the same bits.
// k % 256 == 0.
//
// The steps of one tile: sums of the tile at (at, bt) over nk steps; its last two
// load the first two of the tile at (nat, nbt).
template <int FA, int FB>
__device__ __forceinline__ void tile_steps(uint8_t* smem, v16f (&acc)[4][4], v8i (&f0)[8], const uint8_t* at,
                                           const uint32_t (&aoff)[8], const uint8_t* bt, const uint32_t (&boff)[8],
                                           const uint8_t* nat, const uint8_t* nbt, int64_t nk) {
    u32x4 sx[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
    {
        const bool last = 2 >= nk;
        const uint8_t* la = last ? nat : at;
        const uint8_t* lb = last ? nbt : bt;
        const int64_t kl = last ? 0 : 2 * k128::BK;
        k128_step<FA, FB, 0, true, true, false, true, true>(smem, acc, f0, sx, la, aoff, lb, boff, kl, nullptr, nullptr,
                                                            0, 0);
        k128_step<FA, FB, 1, true, true, false, true>(smem, acc, f0, sx, la, aoff, lb, boff, kl + k128::BK, nullptr,
                                                      nullptr, 0, 0);
    }
    for (int64_t p = 2; p < nk; p += 2) {
        const bool last = p + 2 >= nk;
        const uint8_t* la = last ? nat : at;
        const uint8_t* lb = last ? nbt : bt;
        const int64_t kl = last ? 0 : (p + 2) * k128::BK;
        k128_step<FA, FB, 0, true, true, false, true>(smem, acc, f0, sx, la, aoff, lb, boff, kl, nullptr, nullptr, 0, 0);
        k128_step<FA, FB, 1, true, true, false, true>(smem, acc, f0, sx, la, aoff, lb, boff, kl + k128::BK, nullptr,
                                                      nullptr, 0, 0);
    }
}

// The first two steps of the first tile, and its first fragments.
__device__ __forceinline__ void first_steps(uint8_t* smem, v8i (&f0)[8], const uint8_t* at, const uint32_t (&aoff)[8],
                                            const uint8_t* bt, const uint32_t (&boff)[8]) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint32_t base = __builtin_amdgcn_readfirstlane(lds_addr(smem + s * k128::kStage)) + wave * 8192;
#pragma unroll
        for (int i = 0; i < 8; ++i) lds_dma16_s(base + i * 1024, at + s * k128::BK, aoff[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) lds_dma16_s(base + k128::kOpBytes + i * 1024, bt + s * k128::BK, boff[i]);
    }
    wait_vmcnt<16>();                                    // (and the factors, issued before)
    __syncthreads();
#pragma unroll
    for (int f = 0; f < 8; ++f) {
        const int j = k128_frag(f);
        const uint8_t* tile = j < 4 ? smem : smem + k128::kOpBytes;
        f0[j] = big_join(k128_half<false>(tile, big_row(j), 0, 0), k128_half<false>(tile, big_row(j), 0, 1));
    }
}

// Four rows of one column -> 8 bytes of bf16.
__device__ __forceinline__ uint2 pack_rows(float a, float b, float c, float d) {
    uint2 w;
    w.x = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2bf));
    w.y = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{c, d}), v2bf));
    return w;
}
// Four 16-byte units of a staged block (4 rows x 8 columns) -> row r of the four.
__device__ __forceinline__ u32x4 unit_row(const u32x4 (&un)[4], int r) {
    const uint32_t sel = (r & 1) ? 0x07060302u : 0x05040100u;
    u32x4 row;
#pragma unroll
    for (int k = 0; k < 4; ++k) row[k] = __builtin_amdgcn_perm(un[k][2 + (r >> 1)], un[k][r >> 1], sel);
    return row;
}
// Eight columns of a row, at any alignment: a base that is uniform over the wavefront
// and the lane's offset in bytes. Nontemporal both ways: h, read once, would push the
// operand panels out of L2 (gradient at 8192 x 4096 x 14336: 519 us with ordinary
// loads, 484 with these).
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
__device__ __forceinline__ void store8(uint16_t* base, uint32_t bytes, u32x4 v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2*>(reinterpret_cast<char*>(base) + bytes));
}
__device__ __forceinline__ u32x4 load8(const uint16_t* base, uint32_t bytes) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(reinterpret_cast<const char*>(base) + bytes));
}

// A tile's outputs: 256 rows x 128 columns of act. A wavefront has 128 rows x 64
// columns: blocks 0 and 1 of its 128 columns of B are gate, 2 and 3 up. Staged
// through 4 KB of LDS a wavefront (its own: no barrier): with SAVE 16 rows of [gate |
// up], then 32 rows of act (row groups 2 j and 2 j + 1 side by side as one of 128
// columns).
template <bool SAVE>
__device__ __forceinline__ void glu_epilogue(uint8_t* smem, v16f (&acc)[4][4], const GluFwd& p, int64_t row0,
                                             int64_t col0) {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t wrow0 = row0 + wm * 128, wcol0 = col0 + wn * 64;
#pragma unroll
    for (int mi = 0; mi < 4; ++mi)
#pragma unroll
        for (int ni = 0; ni < 4; ++ni) asm volatile("" : "+a"(acc[mi][ni]));
    const float* s_rows = reinterpret_cast<const float*>(smem + big::kScaleOff);
    const float* s_cols = s_rows + 256;
    float sb[4];
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) sb[ni] = s_cols[wn * 128 + ni * 32 + (lane & 31)];
    uint8_t* ep = smem + persist::kEpiOff + wave * persist::kChunk;
    const int cc = lane & 15, gl = lane >> 4;
#pragma unroll
    for (int mi = 0; mi < 4; ++mi) {
        uint2 a[4][2];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int g4 = 8 * mi + 2 * q + (lane >> 5);            // rows 4 g4 .. + 3
            const u32x4 s4 = *reinterpret_cast<const u32x4*>(&s_rows[wm * 128 + 4 * g4]);
#pragma unroll
            for (int ni = 0; ni < 2; ++ni) {
                float g[4], u[4], act[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    g[i] = acc[mi][ni][4 * q + i] * __uint_as_float(s4[i]) * sb[ni];
                    u[i] = acc[mi][ni + 2][4 * q + i] * __uint_as_float(s4[i]) * sb[ni + 2];
                    act[i] = swiglu(g[i], u[i]);
                }
                a[q][ni] = pack_rows(act[0], act[1], act[2], act[3]);
                if constexpr (SAVE) {
                    const int at = 2 * (q & 1) + (lane >> 5), c = 32 * ni + (lane & 31);
                    *reinterpret_cast<uint2*>(ep + epi_off(at, c)) = pack_rows(g[0], g[1], g[2], g[3]);
                    *reinterpret_cast<uint2*>(ep + epi_off(at, 64 + c)) = pack_rows(u[0], u[1], u[2], u[3]);
                }
            }
            if constexpr (SAVE) {
                if ((q & 1) == 0) continue;
                wait_vmcnt<63, 0>();                     // this wavefront's staging writes are done
                __builtin_amdgcn_wave_barrier();
                u32x4 un[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) un[k] = *reinterpret_cast<const u32x4*>(ep + epi_off(gl, 8 * cc + 2 * k));
                const uint32_t off = (uint32_t)(4 * gl * p.ldh + 8 * (cc & 7) + (cc >= 8 ? p.inter : 0)) * 2;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    store8(p.h + (wrow0 + mi * 32 + 16 * (q >> 1) + r) * p.ldh + wcol0, off, unit_row(un, r));
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int ni = 0; ni < 2; ++ni)
                *reinterpret_cast<uint2*>(ep + epi_off(q, (lane >> 5) * 64 + 32 * ni + (lane & 31))) = a[q][ni];
        wait_vmcnt<63, 0>();
        __builtin_amdgcn_wave_barrier();
        u32x4 un[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) un[k] = *reinterpret_cast<const u32x4*>(ep + epi_off(gl, 8 * cc + 2 * k));
        const uint32_t off = (uint32_t)((8 * gl + 4 * (cc >> 3)) * p.ldact + 8 * (cc & 7)) * 2;
#pragma unroll
        for (int r = 0; r < 4; ++r) store8(p.act + (wrow0 + mi * 32 + r) * p.ldact + wcol0, off, unit_row(un, r));
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int FA, int FB, bool SAVE>
__global__ __launch_bounds__(256, 1) void k_glu_persist(GluFwd p) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[persist::kSmem];
    const int64_t tiles_m = (p.m + 255) / 256, tiles_n = (p.inter + 127) / 128, nt = tiles_m * tiles_n;
    const int64_t G = gridDim.x, nk = p.k / k128::BK;
    const int t = threadIdx.x, lane = t & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    auto lrow = [&](int64_t pm) { return pm * 256 + 256 > p.m ? p.m - 256 : pm * 256; };
    auto lcol = [&](int64_t pn) { return pn * 128 + 128 > p.inter ? p.inter - 128 : pn * 128; };
    // wavefront w loads rows 64 w .. of the tile's B: gate (w even) or up rows of the
    // columns 64 (w / 2) ..
    const int64_t brow = (wave & 1) * p.inter + (int64_t)(wave >> 1) * 64;
    uint32_t aoff[8], boff[8];
    k128_lane_offsets(aoff, p.lda, p.m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i * 8 + (lane >> 3);
        boff[i] = (uint32_t)row * (uint32_t)p.ldb + (uint32_t)(k128_slot(row, lane & 7) * 16);
    }
    int64_t id = blockIdx.x;                             // < nt (grid <= nt)
    int64_t pm, pn;
    tile_coords32((uint32_t)id, (uint32_t)tiles_m, (uint32_t)tiles_n, &pm, &pn);
    int64_t row0 = lrow(pm), col0 = lcol(pn);
    const uint32_t sbase = __builtin_amdgcn_readfirstlane(lds_addr(smem + big::kScaleOff)) + wave * 256;
    auto issue_scales = [&](int64_t r0, int64_t c0) {
        lds_dma4(sbase, p.sa + (p.sa_vec ? r0 + t : 0));
        lds_dma4(sbase + 1024, p.sb + (p.sb_vec ? brow + c0 + lane : 0));
    };
    const uint8_t* at = p.a + row0 * p.lda;
    const uint8_t* bt = p.b + (brow + col0) * p.ldb;
    issue_scales(row0, col0);
    v16f acc[4][4];
    v8i f0[8];
    first_steps(smem, f0, at, aoff, bt, boff);
    for (;;) {
        const int64_t nid = id + G, crow0 = row0, ccol0 = col0;
        const uint8_t* nat = at;                         // with no next tile: this tile's own first
        const uint8_t* nbt = bt;                         // steps (valid addresses, never used)
        if (nid < nt) {
            tile_coords32((uint32_t)nid, (uint32_t)tiles_m, (uint32_t)tiles_n, &pm, &pn);
            row0 = lrow(pm);
            col0 = lcol(pn);
            nat = p.a + row0 * p.lda;
            nbt = p.b + (brow + col0) * p.ldb;
        }
        tile_steps<FA, FB>(smem, acc, f0, at, aoff, bt, boff, nat, nbt, nk);
        at = nat;
        bt = nbt;
        glu_epilogue<SAVE>(smem, acc, p, crow0, ccol0);
        if (nid >= nt) break;
        id = nid;
        __syncthreads();                                 // every wavefront is done with the factors
        issue_scales(row0, col0);                        // (landed by the next tile's first mid-step wait)
    }
    wait_vmcnt<0>();
}

// A tile of the backward pass: 256 x 256 of da, a wavefront 128 x 128. Eight rows at
// a time go through LDS in fp32 (unit c of a group of four rows: their values of
// column c, at c ^ (c / 16 % 8), so that neither side meets a bank twice); a lane
// then has two rows x 8 columns, loads gate and up there in 16 bytes a row, and
// stores as much. h is loaded kAhead groups ahead.
template <bool ACT>
__device__ __forceinline__ void glu_grad_epilogue(uint8_t* smem, v16f (&acc)[4][4], const GluBwd& p, int64_t row0,
                                                  int64_t col0) {
    constexpr int kAhead = 2;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t wrow0 = row0 + wm * 128, wcol0 = col0 + wn * 128;
#pragma unroll
    for (int mi = 0; mi < 4; ++mi)
#pragma unroll
        for (int ni = 0; ni < 4; ++ni) asm volatile("" : "+a"(acc[mi][ni]));
    const float* s_rows = reinterpret_cast<const float*>(smem + big::kScaleOff);
    const float* s_cols = s_rows + 256;
    float sb[4];
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) sb[ni] = s_cols[wn * 128 + ni * 32 + (lane & 31)];
    uint8_t* ep = smem + persist::kEpiOff + wave * persist::kChunk;
    const int cc = lane & 15, rp = lane >> 4, c = 8 * cc;            // rows 2 rp, 2 rp + 1 of the eight
    u32x4 hg[kAhead + 1][2], hu[kAhead + 1][2];
    // (addresses: a base that is uniform over the wavefront and one offset a lane)
    const uint32_t oh = (uint32_t)(2 * rp * p.ldh + c) * 2, od = (uint32_t)(2 * rp * p.lddh + c) * 2,
                   oact = ACT ? (uint32_t)(2 * rp * p.ldact + c) * 2 : 0u;
    auto load_h = [&](int n) {                           // group n of eight rows
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint16_t* src = p.h + (wrow0 + 8 * n + j) * p.ldh + wcol0;
            hg[n % (kAhead + 1)][j] = load8(src, oh);
            hu[n % (kAhead + 1)][j] = load8(src + p.inter, oh);
        }
    };
#pragma unroll
    for (int n = 0; n < kAhead; ++n) load_h(n);
#pragma unroll
    for (int n = 0; n < 16; ++n) {
        const int mi = n >> 2, q = n & 3, g4 = 2 * n + (lane >> 5);
        if (n + kAhead < 16) load_h(n + kAhead);
        const u32x4 s4 = *reinterpret_cast<const u32x4*>(&s_rows[wm * 128 + 4 * g4]);
#pragma unroll
        for (int ni = 0; ni < 4; ++ni) {
            const int col = 32 * ni + (lane & 31);
            f32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = acc[mi][ni][4 * q + i] * __uint_as_float(s4[i]) * sb[ni];
            *reinterpret_cast<f32x4*>(ep + (lane >> 5) * 2048 + ((col ^ ((col >> 4) & 7)) << 4)) = v;
        }
        wait_vmcnt<63, 0>();                             // this wavefront's staging writes are done
        __builtin_amdgcn_wave_barrier();
        v2f da[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            da[e] = *reinterpret_cast<const v2f*>(ep + (rp >> 1) * 2048 + (((c + e) ^ (cc >> 1)) << 4) + (rp & 1) * 8);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const u32x4 wg = hg[n % (kAhead + 1)][j], wu = hu[n % (kAhead + 1)][j];
            u32x4 og, ou, oa;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const SwigluGrad lo = swiglu_grad(da[2 * e][j], bf16_lo(wg[e]), bf16_lo(wu[e]));
                const SwigluGrad hi = swiglu_grad(da[2 * e + 1][j], bf16_hi(wg[e]), bf16_hi(wu[e]));
                og[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo.dg, hi.dg}), v2bf));
                ou[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo.du, hi.du}), v2bf));
                if constexpr (ACT)
                    oa[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo.act, hi.act}), v2bf));
            }
            uint16_t* dst = p.dh + (wrow0 + 8 * n + j) * p.lddh + wcol0;
            store8(dst, od, og);
            store8(dst + p.inter, od, ou);
            if constexpr (ACT) store8(p.act + (wrow0 + 8 * n + j) * p.ldact + wcol0, oact, oa);
            __builtin_amdgcn_sched_barrier(0);           // (rows mixed: spills)
        }
    }
}

template <int FA, int FB, bool ACT>
__global__ __launch_bounds__(256, 1) void k_glu_grad_persist(GluBwd p) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[persist::kSmem];
    const int64_t tiles_m = (p.m + 255) / 256, tiles_n = (p.inter + 255) / 256, nt = tiles_m * tiles_n;
    const int64_t G = gridDim.x, nk = p.k / k128::BK;
    const int t = threadIdx.x;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    auto lrow = [&](int64_t pm) { return pm * 256 + 256 > p.m ? p.m - 256 : pm * 256; };
    auto lcol = [&](int64_t pn) { return pn * 256 + 256 > p.inter ? p.inter - 256 : pn * 256; };
    uint32_t aoff[8], boff[8];
    k128_lane_offsets(aoff, p.lda, p.m);
    k128_lane_offsets(boff, p.ldb, p.inter);
    int64_t id = blockIdx.x;                             // < nt (grid <= nt)
    int64_t pm, pn;
    tile_coords32((uint32_t)id, (uint32_t)tiles_m, (uint32_t)tiles_n, &pm, &pn);
    int64_t row0 = lrow(pm), col0 = lcol(pn);
    const uint32_t sbase = __builtin_amdgcn_readfirstlane(lds_addr(smem + big::kScaleOff)) + wave * 256;
    auto issue_scales = [&](int64_t r0, int64_t c0) {
        lds_dma4(sbase, p.sa + (p.sa_vec ? r0 + t : 0));
        lds_dma4(sbase + 1024, p.sb + (p.sb_vec ? c0 + t : 0));
    };
    const uint8_t* at = p.a + row0 * p.lda;
    const uint8_t* bt = p.b + col0 * p.ldb;
    issue_scales(row0, col0);
    v16f acc[4][4];
    v8i f0[8];
    first_steps(smem, f0, at, aoff, bt, boff);
    for (;;) {
        const int64_t nid = id + G, crow0 = row0, ccol0 = col0;
        const uint8_t* nat = at;
        const uint8_t* nbt = bt;
        if (nid < nt) {
            tile_coords32((uint32_t)nid, (uint32_t)tiles_m, (uint32_t)tiles_n, &pm, &pn);
            row0 = lrow(pm);
            col0 = lcol(pn);
            nat = p.a + row0 * p.lda;
            nbt = p.b + col0 * p.ldb;
        }
        tile_steps<FA, FB>(smem, acc, f0, at, aoff, bt, boff, nat, nbt, nk);
        at = nat;
        bt = nbt;
        glu_grad_epilogue<ACT>(smem, acc, p, crow0, ccol0);
        if (nid >= nt) break;
        id = nid;
        __syncthreads();                                 // every wavefront is done with the factors
        issue_scales(row0, col0);
    }
    wait_vmcnt<0>();
}

}  // namespace

// Workgroups of a persistent kernel: one a CU, as many of each XCD.
static int64_t persistent_grid(int64_t tiles) {
    const int64_t cus = current_device_props().cus, most = cus >= 8 ? cus / 8 * 8 : cus;
    return tiles < most ? tiles : most;
}
// (32-bit lane offsets: 256 rows of an operand, 32 of an output and its other half)
static bool large_operands(int64_t k, int64_t inter, int64_t lda, int64_t ldb, int64_t ldh, int64_t ldd, int64_t ldact) {
    return k > 0 && k % 256 == 0 && lda < (1 << 24) && ldb < (1 << 24) && inter < (1 << 25) && ldh < (1 << 25) &&
           ldd < (1 << 25) && ldact < (1 << 25);
}

template <int FA, int FB>
hipError_t glu_typed(const GluFwd& p, hipStream_t st) {
    const int64_t large = (p.m + 255) / 256 * ((p.inter + 127) / 128);
    if (large_operands(p.k, p.inter, p.lda, p.ldb, p.ldh, 0, p.ldact) && p.m >= 256 && p.inter >= 128 && large >= 128) {
        const dim3 grid((unsigned)persistent_grid(large));
        if (p.h) hipLaunchKernelGGL((k_glu_persist<FA, FB, true>), grid, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((k_glu_persist<FA, FB, false>), grid, dim3(256), 0, st, p);
        return hipGetLastError();
    }
    const int64_t tiles = (p.m + BM - 1) / BM * ((p.inter + 63) / 64);
    hipLaunchKernelGGL((k_glu<FA, FB>), dim3((unsigned)tiles), dim3(kThreads), 0, st, p);
    return hipGetLastError();
}

template <int FA, int FB>
hipError_t glu_grad_typed(const GluBwd& p, hipStream_t st) {
    const int64_t large = (p.m + 255) / 256 * ((p.inter + 255) / 256);
    if (large_operands(p.k, p.inter, p.lda, p.ldb, p.ldh, p.lddh, p.ldact) && p.m >= 256 && p.inter >= 256 && large >= 128) {
        const dim3 grid((unsigned)persistent_grid(large));
        if (p.act) hipLaunchKernelGGL((k_glu_grad_persist<FA, FB, true>), grid, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((k_glu_grad_persist<FA, FB, false>), grid, dim3(256), 0, st, p);
        return hipGetLastError();
    }
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
