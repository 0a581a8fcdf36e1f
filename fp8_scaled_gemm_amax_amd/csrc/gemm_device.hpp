// gemm_device.hpp - device code that the FP8 product kernels share (gemm.hip,
// gemm_swiglu.hip): the 128 x 128 tile's loads and K loop, and the large tile's
// direct global-to-LDS loads, K128 step and tile order (gfx950 only).
#pragma once

#include "fp8_device.hpp"

namespace fp8amax {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int BM = 128, BN = 128, BK = 128;
constexpr int kThreads = 256;
constexpr int kChunksPerRow = BK / 16;                            // 8
constexpr int kLoadsA = BM * kChunksPerRow / kThreads;            // 4
constexpr int kLoadsB = BN * kChunksPerRow / kThreads;            // 4

// Matrix-core operand format selectors: 0 = e4m3 (fp8), 1 = e5m2 (bf8).
template <int F> struct MfmaFmt;
template <> struct MfmaFmt<kE4M3> { static constexpr int v = 0; };
template <> struct MfmaFmt<kE5M2> { static constexpr int v = 1; };

struct TileArgs {
    const uint8_t* a;   // first row of the tile's row range
    const uint8_t* b;
    int64_t lda, ldb;
    int64_t m_rows;     // valid rows of a from `a` on (tile-relative upper bound)
    int64_t n_rows;     // valid rows of b
    int64_t k;
};

__device__ __forceinline__ int swz(int row, int chunk) { return row * kChunksPerRow + (chunk ^ (row & 7)); }

template <int LOADS>
__device__ __forceinline__ void load_tile(uint4 (&r)[LOADS], const uint8_t* base, int64_t ld, int64_t valid_rows,
                                          int64_t k0, int64_t k) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int c = threadIdx.x + i * kThreads;
        const int row = c >> 3, kc = c & 7;
        const int64_t kk = k0 + kc * 16;
        if (row < valid_rows && kk < k)
            r[i] = *reinterpret_cast<const uint4*>(base + (int64_t)row * ld + kk);
        else
            r[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

template <int LOADS>
__device__ __forceinline__ void store_tile(const uint4 (&r)[LOADS], uint4* lds) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int c = threadIdx.x + i * kThreads;
        lds[swz(c >> 3, c & 7)] = r[i];
    }
}

// Fragment of the 32x32x64 instruction: lane l supplies row (l % 32) of its
// 32-row block and 32 consecutive K bytes starting at (l / 32) * 32 of the
// 64-wide K slice kk. The same map is used for a and b, so the contraction
// pairs equal K indices whatever order the instruction sums them in.
__device__ __forceinline__ v8i load_frag(const uint4* lds, int row, int kk) {
    const int lane = threadIdx.x & 63;
    const int c0 = kk * 4 + (lane >> 5) * 2;
    const uint4 lo = lds[swz(row, c0)];
    const uint4 hi = lds[swz(row, c0 + 1)];
    v8i f;
    f[0] = (int)lo.x; f[1] = (int)lo.y; f[2] = (int)lo.z; f[3] = (int)lo.w;
    f[4] = (int)hi.x; f[5] = (int)hi.y; f[6] = (int)hi.z; f[7] = (int)hi.w;
    return f;
}

// One BM x BN output tile: acc[mi][ni] holds the wavefront's 32x32 block (mi, ni).
template <int FA, int FB>
__device__ __forceinline__ void mma_tile(const TileArgs& t, v16f (&acc)[2][2], uint4* As, uint4* Bs) {
    const int wave = threadIdx.x >> 6;
    const int lane = threadIdx.x & 63;
    const int wm = wave >> 1, wn = wave & 1;
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int ni = 0; ni < 2; ++ni)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[mi][ni][r] = 0.0f;

    const int64_t nk = (t.k + BK - 1) / BK;
    uint4 ra[kLoadsA], rb[kLoadsB];
    if (nk > 0) {
        load_tile<kLoadsA>(ra, t.a, t.lda, t.m_rows, 0, t.k);
        load_tile<kLoadsB>(rb, t.b, t.ldb, t.n_rows, 0, t.k);
    }
    for (int64_t kt = 0; kt < nk; ++kt) {
        __syncthreads();
        store_tile<kLoadsA>(ra, As);
        store_tile<kLoadsB>(rb, Bs);
        __syncthreads();
        if (kt + 1 < nk) {
            load_tile<kLoadsA>(ra, t.a, t.lda, t.m_rows, (kt + 1) * BK, t.k);
            load_tile<kLoadsB>(rb, t.b, t.ldb, t.n_rows, (kt + 1) * BK, t.k);
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            v8i fa[2], fb[2];
#pragma unroll
            for (int mi = 0; mi < 2; ++mi) fa[mi] = load_frag(As, wm * 64 + mi * 32 + (lane & 31), kk);
#pragma unroll
            for (int ni = 0; ni < 2; ++ni) fb[ni] = load_frag(Bs, wn * 64 + ni * 32 + (lane & 31), kk);
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                for (int ni = 0; ni < 2; ++ni)
                    acc[mi][ni] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        fa[mi], fb[ni], acc[mi][ni], MfmaFmt<FA>::v, MfmaFmt<FB>::v, 0, 0, 0, 0);
        }
    }
}

// ------------------------------------------------------------ large tiles --
namespace big {
constexpr int BM = 256, BN = 256;
constexpr int kEpiWave = 32 * 1024;                 // one wavefront's staged 128 x 128 bf16 block
constexpr int kMain = 4 * kEpiWave;                 // 128 KB: two K stages, or the staged output
constexpr int kScaleOff = kMain;                    // 256 row scales, then 256 column scales (fp32)
constexpr int kSmem = kMain + 2 * 256 * 4;
// MX operands: per K step, each of the 256 A rows and 256 B rows brings one
// dword of E8M0 block scales (its four 32-element blocks), in two stages
constexpr int kMxStage = 2 * 256 * 4;
constexpr int kMxOff = kSmem;
constexpr int kSmemMx = kSmem + 2 * kMxStage;       // 134 KB
}  // namespace big

// s_waitcnt immediates (gfx9 encoding: vmcnt in bits 3:0 and 15:14, expcnt
// 6:4, lgkmcnt 11:8): wait for vmcnt <= N (and lgkmcnt <= L), leave expcnt alone.
template <int N, int L = 15>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64 && L >= 0 && L < 16, "counter range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070 | (L << 8));
}

// One direct global->LDS load of 16 bytes per lane: lane l's bytes land at
// LDS address lds_base + 16 l (lds_base wave-uniform, set through M0; one
// wait state between the M0 write and the load). M0 is clobbered: the kernels
// that use this have no other M0 user (the build's ISA check test asserts it).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_dma16(uint32_t lds_base, const uint8_t* gptr) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(lds_base), "v"(gptr)
                 : "memory", "m0");
}
// The same load with the address split into a wave-uniform 64-bit base
// (SGPRs) and the lane's 32-bit byte offset (the instruction's SGPR-base
// form: one VGPR per lane instead of two). The base's halves go through
// v_readfirstlane, whose result is a signed int: each half is zero-extended
// before the two are joined (a sign-extended low half would set every bit of
// the high half for an address whose bit 31 is set). The s_nop gives the five
// wait states that a VMEM instruction reading an SGPR needs after a VALU
// instruction (such as v_readfirstlane) wrote it; the compiler does not
// account for the SGPR reads of an asm statement.
__device__ __forceinline__ void lds_dma16_s(uint32_t lds_base, const uint8_t* base, uint32_t voff) {
    const uint64_t b = (uint64_t)(uintptr_t)base;
    const uint64_t hi = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
    const uint64_t lo = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds_base), "v"(voff), "s"((hi << 32) | lo)
                 : "memory", "m0");
}
// Same with 4 bytes per lane: lane l's dword lands at lds_base + 4 l.
__device__ __forceinline__ void lds_dma4(uint32_t lds_base, const void* gptr) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                 :
                 : "s"(lds_base), "v"(gptr)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

__device__ __forceinline__ int big_row(int j) {   // j < 4: A block j; j >= 4: B block j-4 (row in its tile)
    const int w = threadIdx.x >> 6;
    return (j < 4 ? (w >> 1) * 128 + j * 32 : (w & 1) * 128 + (j - 4) * 32) + (threadIdx.x & 31);
}
__device__ __forceinline__ v8i big_join(u32x4 lo, u32x4 hi) {
    v8i f;
    f[0] = (int)lo[0]; f[1] = (int)lo[1]; f[2] = (int)lo[2]; f[3] = (int)lo[3];
    f[4] = (int)hi[0]; f[5] = (int)hi[1]; f[6] = (int)hi[2]; f[7] = (int)hi[3];
    return f;
}

// Logical tile of workgroup `bid` among `nt` tiles: the hardware deals
// workgroups to the 8 XCDs round-robin, so each XCD's share is mapped to a
// contiguous run of logical tiles (neighbouring tiles share A/B panels in that
// XCD's L2); within the run, groups of `gm` M-tiles sweep the N-tiles.
__device__ __forceinline__ void big_tile_coords(int64_t bid, int64_t tiles_m, int64_t tiles_n, int64_t* pm,
                                                int64_t* pn) {
    const int64_t nt = tiles_m * tiles_n;
    const int64_t q = nt / 8, rem = nt % 8;
    const int64_t xcd = bid % 8, idx = bid / 8;
    const int64_t t = xcd * q + (xcd < rem ? xcd : rem) + idx;
    constexpr int64_t gm = 4;
    const int64_t group = t / (gm * tiles_n);
    const int64_t first_m = group * gm;
    const int64_t gsize = tiles_m - first_m < gm ? tiles_m - first_m : gm;
    *pm = first_m + (t % (gm * tiles_n)) % gsize;
    *pn = (t % (gm * tiles_n)) / gsize;
}

// MX block scales of a step in LDS: row r of the tile (A, then B at +1 KB) at
// dword (r / 128) * 128 + (r % 32) * 4 + (r / 32) % 4, so the four rows
// wm*128 + 32 mi + l (mi = 0..3) that lane l needs are one 16-byte read. The
// thread that fills dword i (a wavefront's direct load fills 64 consecutive
// dwords) loads row mx_row(i).
__device__ __forceinline__ int mx_row(int i) { return (i >> 7) * 128 + (i & 3) * 32 + ((i & 127) >> 2); }

// The four scale dwords of lane l's rows, shifted by the lane half s = l / 32:
// lane half s supplies the scale of block s of each 64-deep half, so byte 0 is
// then block s of the step's first half and byte 2 block s of its second.
__device__ __forceinline__ u32x4 mx_scales(const uint8_t* stage, int half_sel) {
    const int lane = threadIdx.x & 63;
    const int w = (threadIdx.x >> 6);
    const int base = half_sel == 0 ? (w >> 1) * 128 : 256 + (w & 1) * 128;
    u32x4 v = *reinterpret_cast<const u32x4*>(stage + 4 * (base + (lane & 31) * 4));
    const int sh = 8 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] >>= sh;
    return v;
}

// MFMA of one 64-deep half: with MX the E8M0 scale bytes OPSEL of the lane's
// A and B scale dwords, else unscaled.
template <int FA, int FB, bool MX, int OPSEL>
__device__ __forceinline__ v16f mfma64(const v8i& fa, const v8i& fb, const v16f& c, uint32_t xa, uint32_t xb) {
    if constexpr (MX)
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa, fb, c, MfmaFmt<FA>::v, MfmaFmt<FB>::v, OPSEL,
                                                               (int)xa, OPSEL, (int)xb);
    else
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa, fb, c, MfmaFmt<FA>::v, MfmaFmt<FB>::v, 0, 0, 0, 0);
}

// K128 main loop of the large-tile kernels: K advances 128 bytes per step
// through two 64 KB LDS stages (A: 256 rows x 128 B, then B). Each direct load
// brings whole 128-byte row segments (8 lanes per row), so the L1 sends
// full-line requests to L2: on gfx950 the load path's throughput goes with the
// number of requests (a loop of 64-deep steps, whose loads move 64-byte row
// segments, was ~13% slower at these shapes). With two stages the loads of step p+2 are
// issued during the second half of step p and waited for in the middle of
// step p+1 (a barrier between the two halves of each step); step p's
// second-half fragments are read during its first 16 MFMAs and step p+1's
// first-half fragments during its last 16. 128-byte rows: chunk c of row r sits in slot c ^ ((r >> 1) & 7),
// so 16 consecutive rows reading one chunk hit 16 distinct 16-byte bank groups.
namespace k128 {
constexpr int BK = 128;
constexpr int kOpBytes = 256 * BK;                   // one operand of a stage: 32 KB
constexpr int kStage = 2 * kOpBytes;                 // 64 KB
static_assert(2 * kStage == big::kScaleOff, "two stages below the scale area");
}  // namespace k128

__device__ __forceinline__ int k128_slot(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// Per-lane byte offsets of this thread's 8 loads of one operand: load i of
// wavefront w fills rows w*64 + 8i .. w*64 + 8i + 7 (1 KB, 16 bytes per lane):
// lane l takes row + l / 8, slot l % 8, i.e. the chunk stored in that slot.
// 32-bit arithmetic (ld < 2^24); rows past the last valid one are clamped.
__device__ __forceinline__ void k128_lane_offsets(uint32_t (&off)[8], int64_t ld, int64_t valid_rows) {
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const uint32_t ld32 = (uint32_t)ld;
    const int last = (int)(valid_rows < 256 ? valid_rows : 256) - 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = wave * 64 + i * 8 + (lane >> 3);
        const int chunk = k128_slot(row, lane & 7);     // the slot map is an involution
        const uint32_t r = (uint32_t)(row < last ? row : last);
        off[i] = r * ld32 + (uint32_t)(chunk * 16);
    }
}

// Fragment half of the 32x32x64 instruction for K half h (bytes 64h ..
// 64h + 63 of the 128-byte row), in two 16-byte pieces hh. The instruction's
// own K order: lane half s = lane / 32 holds K 16s .. 16s + 15 in its bytes
// 0-15 and K 32 + 16s .. 32 + 16s + 15 in bytes 16-31, and with block scales
// the scale of lane half s covers K 32s .. 32s + 31, i.e. bytes 0-15 of both
// lane halves form the first 32-element block (measured on gfx950). That
// order is taken with MX. Without block scales any order common to A and B
// gives the same sums, and lane half s takes bytes 32s .. 32s + 31.
template <bool MX>
__device__ __forceinline__ u32x4 k128_half(const uint8_t* tile, int row, int h, int hh) {
    const int s = (threadIdx.x & 63) >> 5;
    const int c = MX ? h * 4 + s + 2 * hh : h * 4 + s * 2 + hh;
    return *reinterpret_cast<const u32x4*>(tile + row * 128 + (k128_slot(row, c) << 4));
}

// Fragment order of a step: A0, B0, B1, B2, B3, A1, A2, A3 (the order the MFMA
// sweep (mi, ni) = (0,0), (0,1), .. first needs them). j < 4: A block j, else B.
__device__ __forceinline__ int k128_frag(int f) { return f == 0 ? 0 : (f <= 4 ? 4 + (f - 1) : f - 4); }

// Step p with stage CUR = p % 2 (compile-time). On entry f0 holds step p's
// first-half fragments and sx its A and B scale dwords (MX), both read during
// step p-1 (or the prologue). The step:
//   16 MFMAs on f0, each followed by one read of step p's second-half
//   fragments from stage CUR
//   wait until this thread's loads have landed (those of step p+1, issued
//   during step p-1); barrier: stage CUR^1 is complete and every wavefront
//   has read stage CUR for the last time
//   16 MFMAs on f1, each followed (NEXT) by one read of step p+1's first-half
//   fragments from stage CUR^1 and (LOADS) by one of the 16 loads of step p+2
//   (K offset knext) into stage CUR; with MX also step p+2's two scale dwords
//   per thread (the records xa / xb of K step 0 advanced by knext / 128 steps
//   of xsa / xsb bytes), and step p+1's scales read into sx.
// A step's MFMAs thus never wait for LDS reads issued after the barrier, and
// the loads have a full step to land. With issue false (uniform) a LOADS step
// skips its loads: the same code, so a K loop whose last pair loads nothing
// needs no second copy of the steps. With ZERO the first 16 MFMAs start from
// zero instead of acc (a tile's first step: no zeroing pass). SADDR: the loads
// take the SGPR-base form (a, b wave-uniform bases, aoff / boff lane offsets).
template <int FA, int FB, int CUR, bool NEXT, bool LOADS, bool MX, bool SADDR = false, bool ZERO = false>
__device__ __forceinline__ void k128_step(uint8_t* smem, v16f (&acc)[4][4], v8i (&f0)[8], u32x4 (&sx)[2],
                                          const uint8_t* a, const uint32_t (&aoff)[8], const uint8_t* b,
                                          const uint32_t (&boff)[8], int64_t knext, const uint8_t* xa,
                                          const uint8_t* xb, int64_t xsa, int64_t xsb, bool issue = true) {
    const uint8_t* ta = smem + CUR * k128::kStage;
    const uint8_t* tb = ta + k128::kOpBytes;
    const uint8_t* na = smem + (CUR ^ 1) * k128::kStage;
    const uint8_t* nb = na + k128::kOpBytes;
    u32x4 h1[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int mi = i >> 2, ni = i & 3;
        acc[mi][ni] = mfma64<FA, FB, MX, 0>(f0[mi], f0[4 + ni], ZERO ? v16f{} : acc[mi][ni], sx[0][mi], sx[1][ni]);
        const int j = k128_frag(i >> 1);
        h1[i] = k128_half<MX>(j < 4 ? ta : tb, big_row(j), 1, i & 1);
        __builtin_amdgcn_sched_barrier(0);
    }
    v8i f1[8];
#pragma unroll
    for (int f = 0; f < 8; ++f) f1[k128_frag(f)] = big_join(h1[2 * f], h1[2 * f + 1]);
    wait_vmcnt<0, 0>();
    __syncthreads();
    const u32x4 sxc[2] = {sx[0], sx[1]};
    if constexpr (MX && NEXT) {
        const uint8_t* xs = smem + big::kMxOff + (CUR ^ 1) * big::kMxStage;
        sx[0] = mx_scales(xs, 0);
        sx[1] = mx_scales(xs, 1);
    }
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t dma_base = __builtin_amdgcn_readfirstlane(lds_addr(smem + CUR * k128::kStage)) + wave * 8192;
    u32x4 h0[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int mi = i >> 2, ni = i & 3;
        acc[mi][ni] = mfma64<FA, FB, MX, 2>(f1[mi], f1[4 + ni], acc[mi][ni], sxc[0][mi], sxc[1][ni]);
        if (NEXT) {
            const int j = k128_frag(i >> 1);
            h0[i] = k128_half<MX>(j < 4 ? na : nb, big_row(j), 0, i & 1);
        }
        if (LOADS && issue) {
            if constexpr (SADDR) {
                if (i < 8)
                    lds_dma16_s(dma_base + i * 1024, a + knext, aoff[i]);
                else
                    lds_dma16_s(dma_base + k128::kOpBytes + (i - 8) * 1024, b + knext, boff[i - 8]);
            } else {
                if (i < 8)
                    lds_dma16(dma_base + i * 1024, a + knext + aoff[i]);
                else
                    lds_dma16(dma_base + k128::kOpBytes + (i - 8) * 1024, b + knext + boff[i - 8]);
            }
            if constexpr (MX) {
                if (i == 3 || i == 11) {
                    const uint32_t xbase = __builtin_amdgcn_readfirstlane(
                                               lds_addr(smem + big::kMxOff + CUR * big::kMxStage)) +
                                           wave * 256 + (i == 3 ? 0 : 1024);
                    lds_dma4(xbase, i == 3 ? xa + (knext / k128::BK) * xsa : xb + (knext / k128::BK) * xsb);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    if (NEXT) {
#pragma unroll
        for (int f = 0; f < 8; ++f) f0[k128_frag(f)] = big_join(h0[2 * f], h0[2 * f + 1]);
    }
}

// The K loop of the large-tile kernels; k % 256 == 0, k > 0. The
// epilogue's row and column scales go to the scale area: sa_lane / sb_lane
// (thread t's row / column scale) or, with MX, 1 (the block scales are applied
// inside the MFMAs; xa / xb are the K-step-0 scale records of A row mx_row(t)
// and B row mx_row(t) of the tile, and a K step advances them by xsa / xsb
// bytes). Prologue: steps 0 and 1 in flight, wait for step 0, read its
// first-half fragments.
template <int FA, int FB, bool MX>
__device__ __forceinline__ void k128_mainloop(uint8_t* smem, const uint8_t* a, int64_t lda, int64_t a_rows,
                                              const uint8_t* b, int64_t ldb, int64_t b_rows, int64_t k,
                                              const float* sa_lane, const float* sb_lane, const uint8_t* xa,
                                              const uint8_t* xb, int64_t xsa, int64_t xsb, v16f (&acc)[4][4]) {
#pragma unroll
    for (int mi = 0; mi < 4; ++mi)
#pragma unroll
        for (int ni = 0; ni < 4; ++ni)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[mi][ni][r] = 0.0f;
    uint32_t aoff[8], boff[8];
    k128_lane_offsets(aoff, lda, a_rows);
    k128_lane_offsets(boff, ldb, b_rows);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t nk = k / k128::BK;
    constexpr int L = MX ? 18 : 16;                      // loads per thread per step
    v8i f0[8];
    u32x4 sx[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
    {
        if constexpr (MX) {
            float* s = reinterpret_cast<float*>(smem + big::kScaleOff);
            s[threadIdx.x] = 1.0f;
            s[256 + threadIdx.x] = 1.0f;
        } else {
            const uint32_t sbase = __builtin_amdgcn_readfirstlane(lds_addr(smem + big::kScaleOff)) + wave * 256;
            lds_dma4(sbase, sa_lane);
            lds_dma4(sbase + 1024, sb_lane);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t base = __builtin_amdgcn_readfirstlane(lds_addr(smem + s * k128::kStage)) + wave * 8192;
            const int64_t k0 = s * k128::BK;
#pragma unroll
            for (int i = 0; i < 8; ++i) lds_dma16(base + i * 1024, a + k0 + aoff[i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) lds_dma16(base + k128::kOpBytes + i * 1024, b + k0 + boff[i]);
            if constexpr (MX) {
                const uint32_t xbase =
                    __builtin_amdgcn_readfirstlane(lds_addr(smem + big::kMxOff + s * big::kMxStage)) + wave * 256;
                lds_dma4(xbase, xa + s * xsa);
                lds_dma4(xbase + 1024, xb + s * xsb);
            }
        }
        wait_vmcnt<L>();                                 // step 0 (and the scales) landed
        __syncthreads();
#pragma unroll
        for (int f = 0; f < 8; ++f) {
            const int j = k128_frag(f);
            f0[j] = big_join(k128_half<MX>(j < 4 ? smem : smem + k128::kOpBytes, big_row(j), 0, 0),
                             k128_half<MX>(j < 4 ? smem : smem + k128::kOpBytes, big_row(j), 0, 1));
        }
        if constexpr (MX) {
            sx[0] = mx_scales(smem + big::kMxOff, 0);
            sx[1] = mx_scales(smem + big::kMxOff, 1);
        }
    }
    // one loop over the step pairs: one path, so the sums keep one register
    // assignment from the zeroing to the epilogue. The last pair issues no
    // loads; with MX it loads the tile's steps 0 and 1 again instead (valid
    // addresses, never read: skipping the loads there costs registers)
    int64_t p = 0;
    do {                                                 // nk >= 2
        const bool more = p + 2 < nk;
        const int64_t kl = more ? (p + 2) * k128::BK : 0;
        k128_step<FA, FB, 0, true, true, MX>(smem, acc, f0, sx, a, aoff, b, boff, kl, xa, xb, xsa, xsb, more || MX);
        k128_step<FA, FB, 1, true, true, MX>(smem, acc, f0, sx, a, aoff, b, boff, kl + k128::BK, xa, xb, xsa, xsb,
                                             more || MX);
        p += 2;
    } while (p < nk);
    wait_vmcnt<0>();                                     // (MX: the last pair's loads landed)
}

// Staged bf16 block of the epilogue: group g of 4 rows, column c -> 8 bytes
// (the 4 rows' values) at g * 1024 + unit * 16 + (c % 2) * 8, where the 16-byte
// unit c / 2 = u is stored at (u & ~3) | ((u ^ (u >> 4)) & 3): the 16 lanes of
// one 16-byte read (units 4i + k, i = 0..15) then hit 16 distinct bank groups,
// and the 32 lanes of one 8-byte write still cover 256 contiguous bytes.
__device__ __forceinline__ int epi_off(int g, int c) {
    const int u = c >> 1;
    return g * 1024 + (((u & ~3) | ((u ^ (u >> 4)) & 3)) << 4) + ((c & 1) << 3);
}

// The persistent kernels' LDS behind the large tile's.
namespace persist {
constexpr int kChunk = 4 * 1024;                     // one wavefront's 16 staged rows
constexpr int kEpiOff = big::kSmem;                  // after the stages and the scale area
constexpr int kSmem = big::kSmem + 4 * kChunk;       // 146 KB
}  // namespace persist

// big_tile_coords in 32-bit arithmetic (tile counts below 2^31), its divisors
// made opaque at each call so that the divisions' setup is not kept live
// across the K loop.
__device__ __forceinline__ void tile_coords32(uint32_t bid, uint32_t tiles_m, uint32_t tiles_n, int64_t* pm,
                                              int64_t* pn) {
    asm volatile("" : "+s"(tiles_m), "+s"(tiles_n));
    const uint32_t nt = tiles_m * tiles_n;
    const uint32_t q = nt / 8, rem = nt % 8;
    const uint32_t xcd = bid % 8, idx = bid / 8;
    const uint32_t t = xcd * q + (xcd < rem ? xcd : rem) + idx;
    constexpr uint32_t gm = 4;
    const uint32_t span = gm * tiles_n;
    const uint32_t first_m = t / span * gm;
    const uint32_t gsize = tiles_m - first_m < gm ? tiles_m - first_m : gm;
    const uint32_t u = t % span;
    *pm = first_m + u % gsize;
    *pn = u / gsize;
}

}  // namespace fp8amax
