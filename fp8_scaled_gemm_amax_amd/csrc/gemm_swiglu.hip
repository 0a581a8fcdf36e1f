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
#include "layer_device.hpp"

namespace fp8amax {
namespace {

// sigma(g) = 1 / (1 + t) and 1 - sigma(g) = t sigma(g), t = exp(-g), with a relative error
// of 2^-20 at most for every g (1 - sigma as long as t 2^-24 is normal, g up to 70; what is
// less adds nothing to the 1 that it is added to). t = 2^n exp(e): n = -g log2 e as rounded, and e = -g - n ln 2,
// |e| < 2^-16, what that rounding lost (without it t's error grows with |g|, to 2^-17). The
// sum is formed times 2^-24, so that its reciprocal is normal as long as t is finite: the
// hardware's has no subnormal results, and sigma would vanish from t = 2^126. (A t of 2^128 and
// more is infinite, and sigma 0. Past +-200, where sigma is 1 or 0, g counts as that: e stays
// small. A NaN g gives any sigma; what it is multiplied with is NaN.)
struct Sigma {
    float sig, t, r;                                    // t 2^-24, sigma 2^24
    __device__ __forceinline__ explicit Sigma(float g) {
        constexpr float kDown = 5.9604644775390625e-8f; // 2^-24
        const float c = __builtin_amdgcn_fmed3f(g, -200.0f, 200.0f), n = c * -1.44269504f;
        const float e = fmaf(n, -0.693147182f, -c);
        t = __builtin_amdgcn_exp2f(n) * fmaf(e, kDown, kDown);
        r = __builtin_amdgcn_rcpf(t + kDown);
        sig = r * kDown;
    }
    // (t is infinite only with sigma 0)
    __device__ __forceinline__ float complement() const { return __builtin_fminf(t, 3.40282347e38f) * r; }
};
__device__ __forceinline__ float swiglu(float g, float u) { return g * Sigma(g).sig * u; }

struct SwigluGrad {
    float dg, du, act;
};
__device__ __forceinline__ SwigluGrad swiglu_grad(float da, float g, float u) {
    const Sigma s(g);
    const float silu = g * s.sig;
    return {da * u * (s.sig * fmaf(g, s.complement(), 1.0f)), da * silu, silu * u};
}

typedef float v4f __attribute__((ext_vector_type(4)));

// h, act and dh pass the caches (load8, store8): h, read once, would push the operand
// panels out of L2 (gradient at 8192 x 4096 x 14336: 519 us with ordinary loads, 484 so).

// --------------------------------------------------------------- few rows --
// Up to kFewRows rows of a (decoding; glu_few_rows): bound by the weights' bytes, each read once. A
// workgroup has 16 columns of act: its 16 gate rows and 16 up rows of b against tiles
// of 16 rows of a (16x16x128 products), its wavefronts taking K in turn in blocks of
// 256 bytes, their sums added in LDS. Weights are loaded in the order of the rows (16
// lanes a row) and turned into the matrix cores' order (lane l: 32 bytes of row l % 16)
// through LDS of the wavefront's own; the next block is on its way while one is
// multiplied. One row, 4096 x 14336: 24 us, 5 TB/s (8192 x 28672: 73 us, 6.4 TB/s; what
// a short call loses is the ramp-up and the drain).
constexpr int kFewBlock = 256;

template <int FA, int FB, int NT, int W>
__global__ __launch_bounds__(W * 64) void k_glu_few(GluFwd p) {
    // a wavefront's part: two tiles of 16 rows x 256 bytes, then its sums [2 NT][256]
    constexpr int kPart = 8192 > NT * 2048 ? 8192 : NT * 2048;
    __shared__ __attribute__((aligned(16))) uint8_t lds[W][kPart];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, m = lane & 15;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int cols = p.inter - n0 < 16 ? (int)(p.inter - n0) : 16;
    uint8_t* own = lds[wave];
    // loads: chunk m of rows q, q + 4, .. of each tile
    uint32_t wo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + q;
        wo[i] = (uint32_t)(row < cols ? row : cols - 1) * (uint32_t)p.ldb + (uint32_t)m * 16;
    }
    const uint8_t* wp[2] = {p.b + n0 * p.ldb, p.b + (p.inter + n0) * p.ldb};
    // chunk c of row r at c ^ r: 16 rows of one chunk meet 16 different groups of banks
    auto place = [](int row, int chunk) { return row * 256 + ((chunk ^ row) << 4); };
    uint32_t xo[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = n * 16 + m;
        xo[n] = (uint32_t)(row < p.m ? row : (int)p.m - 1) * (uint32_t)p.lda + (uint32_t)q * 32;
    }
    v4f acc[2][NT];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[w][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t blocks = (p.k + kFewBlock - 1) / kFewBlock;
    // chunks past k (in the last block) load the row's last one, for zeros
    auto load = [&](int64_t b, u32x4 (&w)[2][4]) {
        const int64_t left = p.k - b * kFewBlock;
        const int last = left < kFewBlock ? (int)left / 16 - 1 : 15;
        const uint32_t in = m <= last ? ~0u : 0u, back = m <= last ? 0u : (uint32_t)(m - last) * 16;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[t][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wp[t] + b * kFewBlock + (wo[i] - back))) & in;
    };
    auto work = [&](int64_t b, const u32x4 (&w)[2][4], u32x4 (*next)[2][4], int64_t nb) {
        const int64_t left = p.k - b * kFewBlock;
        u32x4 x[2][NT][2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = s * 128 + q * 32 + h * 16;
                    const uint32_t in = at < left ? ~0u : 0u;
                    x[s][n][h] = *reinterpret_cast<const u32x4*>(p.a + b * kFewBlock + (xo[n] + (at < left ? s * 128 + h * 16 : 0) -
                                                                                        (at < left ? 0 : q * 32))) & in;
                }
        __builtin_amdgcn_sched_barrier(0);              // (loads return in order: the rows of a first)
        if (next) load(nb, *next);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4*>(own + t * 4096 + place(4 * i + q, m)) = w[t][i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const v8i f = big_join(*reinterpret_cast<const u32x4*>(own + t * 4096 + place(m, 8 * s + 2 * q)),
                                       *reinterpret_cast<const u32x4*>(own + t * 4096 + place(m, 8 * s + 2 * q + 1)));
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[t][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f, big_join(x[s][n][0], x[s][n][1]), acc[t][n],
                                                                                 MfmaFmt<FB>::v, MfmaFmt<FA>::v, 0, 0, 0, 0);
            }
    };
    {
        u32x4 a[2][4], b[2][4];                         // in turn, so that no load waits to be copied
        int64_t i = wave;
        if (i < blocks) load(i, a);
        for (; i < blocks; i += 2 * W) {
            const int64_t j = i + W, k = j + W;
            work(i, a, j < blocks ? &b : nullptr, j);
            if (j >= blocks) break;
            work(j, b, k < blocks ? &a : nullptr, k);
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float* sums = reinterpret_cast<float*>(own);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < 2; ++t)                     // column (row of a) m, rows (of b) 4 q ..
            *reinterpret_cast<v4f*>(sums + (n * 2 + t) * 256 + m * 16 + q * 4) = acc[t][n];
    __syncthreads();
    const int col = threadIdx.x & 15;
    if (col >= cols) return;
    const float sg = p.sb[p.sb_vec ? n0 + col : 0], su = p.sb[p.sb_vec ? p.inter + n0 + col : 0];
#pragma unroll
    for (int i = threadIdx.x; i < NT * 256; i += W * 64) {
        const int64_t row = i >> 4;
        if (row >= p.m) break;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float* s = reinterpret_cast<const float*>(lds[w]) + (i >> 8) * 512 + (i & 255);
            g += s[0];
            u += s[256];
        }
        const float sa = p.sa[p.sa_vec ? row : 0];
        g = g * sa * sg;
        u = u * sa * su;
        p.act[row * p.ldact + n0 + col] = (uint16_t)f32_to_bf16(swiglu(g, u));
        if (p.h) {
            p.h[row * p.ldh + n0 + col] = (uint16_t)f32_to_bf16(g);
            p.h[row * p.ldh + p.inter + n0 + col] = (uint16_t)f32_to_bf16(u);
        }
    }
}

// ------------------------------------------------------- 128 x 128 tiles --
// Any sizes (k in steps of 16), and the kernel where large tiles are too few for the
// chip. Four wavefronts of 64 x 64 outputs (2 x 2 blocks of 32x32x64), K in steps of
// 128 through four stages in LDS, direct global-to-LDS loads three steps ahead (one
// step ahead in registers, 777 x 2048 x 1408 took 26 us), one half of a step read from
// LDS while the other multiplies (15.8 -> 15.0 us). An XCD takes neighbouring tiles,
// which share operand panels in its L2 (gradient of 1000 x 4112 x 14336 136 -> 130 us).
// Rows past the operand's last one are loaded as that one and not stored; the step that
// k ends in comes through registers, zeros behind k.
//
// MB: blocks of 32 rows a wavefront, 2 or, for tiles of 64 rows, 1 (glu_tiles_of_64_rows).
template <int MB>
struct Mid {
    static constexpr int kStages = 4, kA = MB * 64 * 128, kStage = kA + 128 * 128;
    static constexpr int kScaleOff = kStages * kStage;              // MB * 64 row factors, 128 column factors
    static constexpr int kSmem = kScaleOff + (MB * 64 + 128) * 4;   // 129 KB, 97 KB
};

// a, b: first rows (uniform over the wavefront: b may differ between wavefronts);
// ao, bo: offsets of this lane's rows, of which it loads chunk `slot` of each step.
template <int FA, int FB, int MB>
__device__ __forceinline__ void mid_sums(uint8_t* smem, const uint8_t* a, const uint32_t (&ao)[2 * MB], const uint8_t* b,
                                         const uint32_t (&bo)[4], int64_t k, v16f (&acc)[MB][2]) {
    using mid = Mid<MB>;
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    constexpr int kLoads = 2 * MB + 4;                  // of a thread and step
    const int64_t full = k / 128, nk = (k + 127) / 128;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
#pragma unroll
    for (int mi = 0; mi < MB; ++mi)
#pragma unroll
        for (int ni = 0; ni < 2; ++ni)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[mi][ni][r] = 0.0f;
    auto issue = [&](int64_t s) {
        const uint32_t base = lds0 + (uint32_t)(s & (mid::kStages - 1)) * mid::kStage;
        if (s < full) {
#pragma unroll
            for (int i = 0; i < 2 * MB; ++i) lds_dma16_s(base + wave * (MB * 2048) + i * 1024, a + s * 128, ao[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) lds_dma16_s(base + mid::kA + wave * 4096 + i * 1024, b + s * 128, bo[i]);
        } else if (s < nk) {
            // (the lane's chunk of the step: its offset modulo the row's 128 bytes)
            auto put = [&](uint8_t* to, const uint8_t* from, uint32_t off, int i) {
                const int chunk = k128_slot(8 * i + (lane >> 3), lane & 7);
                u32x4 v = {0u, 0u, 0u, 0u};
                if (s * 128 + chunk * 16 < k) v = *reinterpret_cast<const u32x4*>(from + s * 128 + off);
                *reinterpret_cast<u32x4*>(to + lane * 16 + i * 1024) = v;
            };
            uint8_t* to = smem + (s & (mid::kStages - 1)) * mid::kStage;
#pragma unroll
            for (int i = 0; i < 2 * MB; ++i) put(to + wave * (MB * 2048), a, ao[i], i);
#pragma unroll
            for (int i = 0; i < 4; ++i) put(to + mid::kA + wave * 4096, b, bo[i], i);
        }
    };
    struct Half {
        v8i a[MB], b[2];
    };
    auto read = [&](int64_t s, int h, Half& f) {
        const uint8_t* ta = smem + (s & (mid::kStages - 1)) * mid::kStage;
        const uint8_t* tb = ta + mid::kA;
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const int r = (wm * MB + i) * 32 + (lane & 31);
            f.a[i] = big_join(k128_half<false>(ta, r, h, 0), k128_half<false>(ta, r, h, 1));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (wn * 2 + i) * 32 + (lane & 31);
            f.b[i] = big_join(k128_half<false>(tb, r, h, 0), k128_half<false>(tb, r, h, 1));
        }
    };
    auto multiply = [&](const Half& f) {
#pragma unroll
        for (int mi = 0; mi < MB; ++mi)
#pragma unroll
            for (int ni = 0; ni < 2; ++ni) acc[mi][ni] = mfma64<FA, FB, false, 0>(f.a[mi], f.b[ni], acc[mi][ni], 0u, 0u);
    };
    // this thread's loads of step s have landed (those of two later steps may not have),
    // then everyone's, and everyone has read step s - 1
    auto arrive = [&](int64_t s) {
        if (s + 2 < full)
            wait_vmcnt<2 * kLoads>();
        else
            wait_vmcnt<0>();
        __syncthreads();
    };
    for (int s = 0; s < mid::kStages - 1; ++s) issue(s);
    if (nk > 0) {
        Half f0, f1;                                    // the halves of a step in turn: one is read while the other multiplies
        arrive(0);
        issue(mid::kStages - 1);
        read(0, 0, f0);
        for (int64_t s = 0; s + 1 < nk; ++s) {
            read(s, 1, f1);
            multiply(f0);
            arrive(s + 1);
            issue(s + mid::kStages);
            read(s + 1, 0, f0);
            multiply(f1);
        }
        read(nk - 1, 1, f1);
        multiply(f0);
        multiply(f1);
    }
    __syncthreads();                                    // (the stages are free, the factors in place)
}
// Offsets of this lane's N rows row0 + 8 i + l / 8, the last valid one instead of
// those past it, with the chunk that its slot holds.
template <int N>
__device__ __forceinline__ void mid_offsets(uint32_t (&off)[N], int row0, int64_t valid, int64_t ld) {
    const int lane = threadIdx.x & 63;
    const int last = valid < (1 << 20) ? (int)valid - 1 : 1 << 20;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = row0 + 8 * i + (lane >> 3);
        off[i] = (uint32_t)(row < last ? row : last) * (uint32_t)ld + (uint32_t)(k128_slot(8 * i + (lane >> 3), lane & 7) * 16);
    }
}

// Eight of the columns col .. of a row of bf16 outputs, `left` of them there.
__device__ __forceinline__ void store_chunk8(uint16_t* base, uint32_t bytes, int left, const float* f) {
    if (left >= 8) {
        store8(base, bytes, u32x4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])});
        return;
    }
    uint16_t* dst = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(base) + bytes);
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < left) dst[e] = (uint16_t)f32_to_bf16(f[e]);
}

// Tile: 64 MB rows x 64 columns of act; rows of b: 32 gate rows, the 32 up rows of the
// same columns, 32 gate rows, ..: block 0 of a wavefront is gate, block 1 up.
template <int FA, int FB, int MB>
__global__ __launch_bounds__(256) void k_glu_mid(GluFwd p) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[Mid<MB>::kSmem];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tiles_m = (p.m + MB * 64 - 1) / (MB * 64);
    int64_t pm, pn;
    big_tile_coords(blockIdx.x, tiles_m, (p.inter + 63) / 64, &pm, &pn);
    const int64_t row0 = pm * (MB * 64), col0 = pn * 64;
    const int64_t half = (int64_t)(wave & 1) * p.inter;         // wavefront w loads gate (w even) or up rows
    uint32_t ao[2 * MB], bo[4];
    mid_offsets(ao, wave * (MB * 16), p.m - row0, p.lda);
    mid_offsets(bo, (wave >> 1) * 32, p.inter - col0, p.ldb);
    float* s_rows = reinterpret_cast<float*>(smem + Mid<MB>::kScaleOff);
    float* s_cols = s_rows + MB * 64;
    if (threadIdx.x < 128) {
        const int64_t r = row0 + threadIdx.x, c = col0 + (threadIdx.x & 63);
        if (threadIdx.x < MB * 64) s_rows[threadIdx.x] = p.sa[p.sa_vec ? (r < p.m ? r : p.m - 1) : 0];
        // 64 gate factors, 64 up factors
        s_cols[threadIdx.x] = p.sb[p.sb_vec ? (threadIdx.x >> 6) * p.inter + (c < p.inter ? c : p.inter - 1) : 0];
    }
    v16f acc[MB][2];
    mid_sums<FA, FB, MB>(smem, p.a + row0 * p.lda, ao, p.b + (half + col0) * p.ldb, bo, p.k, acc);
    // the wavefront's 32 MB rows x 32 columns of g and of u in LDS, then a lane takes rows
    // of 8 columns
    constexpr int kPitch = 68;                          // fp32 values: 32 of g, 32 of u
    float* own = reinterpret_cast<float*>(smem) + wave * (MB * 32) * kPitch;
    const int wm = wave >> 1, wn = wave & 1;
    const float sg = s_cols[wn * 32 + (lane & 31)], su = s_cols[64 + wn * 32 + (lane & 31)];
#pragma unroll
    for (int mi = 0; mi < MB; ++mi)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = mi * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
            const float sa = s_rows[wm * (MB * 32) + row];
            own[row * kPitch + (lane & 31)] = acc[mi][0][r] * sa * sg;
            own[row * kPitch + 32 + (lane & 31)] = acc[mi][1][r] * sa * su;
        }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int64_t wcol = col0 + wn * 32 + 8 * (lane & 3);
    const int left = p.inter - wcol < 8 ? (int)(p.inter - wcol) : 8;
    if (left <= 0) return;
#pragma unroll
    for (int j = 0; j < 2 * MB; ++j) {
        const int row = j * 16 + (lane >> 2);
        const int64_t at = row0 + wm * (MB * 32) + row;
        if (at >= p.m) continue;
        float g[8], u[8], act[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const v4f vg = *reinterpret_cast<const v4f*>(own + row * kPitch + 8 * (lane & 3) + 4 * h);
            const v4f vu = *reinterpret_cast<const v4f*>(own + row * kPitch + 32 + 8 * (lane & 3) + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g[4 * h + e] = vg[e];
                u[4 * h + e] = vu[e];
                act[4 * h + e] = swiglu(vg[e], vu[e]);
            }
        }
        store_chunk8(p.act + at * p.ldact + wcol, 0, left, act);
        if (p.h) {
            store_chunk8(p.h + at * p.ldh + wcol, 0, left, g);
            store_chunk8(p.h + at * p.ldh + p.inter + wcol, 0, left, u);
        }
    }
}

// Tile: 64 MB x 128 of da, a wavefront 32 MB x 64.
template <int FA, int FB, int MB>
__global__ __launch_bounds__(256) void k_glu_grad_mid(GluBwd p) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[Mid<MB>::kSmem];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tiles_m = (p.m + MB * 64 - 1) / (MB * 64);
    int64_t pm, pn;
    big_tile_coords(blockIdx.x, tiles_m, (p.inter + 127) / 128, &pm, &pn);
    const int64_t row0 = pm * (MB * 64), col0 = pn * 128;
    uint32_t ao[2 * MB], bo[4];
    mid_offsets(ao, wave * (MB * 16), p.m - row0, p.lda);
    mid_offsets(bo, wave * 32, p.inter - col0, p.ldb);
    float* s_rows = reinterpret_cast<float*>(smem + Mid<MB>::kScaleOff);
    float* s_cols = s_rows + MB * 64;
    if (threadIdx.x < 128) {
        const int64_t r = row0 + threadIdx.x, c = col0 + threadIdx.x;
        if (threadIdx.x < MB * 64) s_rows[threadIdx.x] = p.sa[p.sa_vec ? (r < p.m ? r : p.m - 1) : 0];
        s_cols[threadIdx.x] = p.sb[p.sb_vec ? (c < p.inter ? c : p.inter - 1) : 0];
    }
    v16f acc[MB][2];
    mid_sums<FA, FB, MB>(smem, p.a + row0 * p.lda, ao, p.b + col0 * p.ldb, bo, p.k, acc);
    constexpr int kPitch = 68, kPasses = MB * 4;
    float* own = reinterpret_cast<float*>(smem) + wave * (MB * 32) * kPitch;
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t wcol = col0 + wn * 64 + 8 * (lane & 7);
    const int left = p.inter - wcol < 8 ? (int)(p.inter - wcol) : 8;
    const int64_t wrow = row0 + wm * (MB * 32);
    // h, two rows ahead
    u32x4 hg[3], hu[3];
    auto load_h = [&](int j) {
        const int64_t at = wrow + j * 8 + (lane >> 3);
        hg[j % 3] = hu[j % 3] = u32x4{0u, 0u, 0u, 0u};
        if (at >= p.m || left <= 0) return;
        const uint16_t* src = p.h + at * p.ldh + wcol;
        if (left >= 8) {
            hg[j % 3] = load8(src, 0);
            hu[j % 3] = load8(src + p.inter, 0);
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < left) {
                    hg[j % 3][e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
                    hu[j % 3][e >> 1] |= (uint32_t)src[p.inter + e] << (16 * (e & 1));
                }
        }
    };
    load_h(0);
    load_h(1);
#pragma unroll
    for (int ni = 0; ni < 2; ++ni) {
        const float sb = s_cols[(wn * 2 + ni) * 32 + (lane & 31)];
#pragma unroll
        for (int mi = 0; mi < MB; ++mi)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = mi * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                own[row * kPitch + ni * 32 + (lane & 31)] = acc[mi][ni][r] * s_rows[wm * (MB * 32) + row] * sb;
            }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int j = 0; j < kPasses; ++j) {
        if (j + 2 < kPasses) load_h(j + 2);
        const int row = j * 8 + (lane >> 3);
        float dg[8], du[8], act[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const v4f da = *reinterpret_cast<const v4f*>(own + row * kPitch + 8 * (lane & 7) + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t wg = hg[j % 3][2 * h + (e >> 1)], wu = hu[j % 3][2 * h + (e >> 1)];
                const SwigluGrad d = swiglu_grad(da[e], e & 1 ? bf16_hi(wg) : bf16_lo(wg), e & 1 ? bf16_hi(wu) : bf16_lo(wu));
                dg[4 * h + e] = d.dg;
                du[4 * h + e] = d.du;
                act[4 * h + e] = d.act;
            }
        }
        const int64_t at = wrow + row;
        if (at < p.m && left > 0) {
            store_chunk8(p.dh + at * p.lddh + wcol, 0, left, dg);
            store_chunk8(p.dh + at * p.lddh + p.inter + wcol, 0, left, du);
            if (p.act) store_chunk8(p.act + at * p.ldact + wcol, 0, left, act);
        }
    }
}

// ------------------------------------------------------- 256 x 256 tiles --
// The K128 loop's large tile, persistent: a workgroup takes tiles w, w + G, .., and
// the next tile's first two K steps load during the current one's last two. Tiles
// past the last row (column) are shifted back to end there (there are enough of both
// for a tile); what the tile before computes too is stored twice, the same bits.
// k % 256 == 0. 8192 x 4096 x 14336: product with h 735-760 us (2.6 PFLOP/s, matrix
// cores busy 71% at the 1.67 GHz that power allows; without h 690), gradient
// with act 480-494 us (without h, dh and act 356: their 1.2 GB are what bounds it).
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
    return make_uint2(pack2(a, b), pack2(c, d));
}
// Four 16-byte units of a staged block (4 rows x 8 columns) -> row r of the four.
__device__ __forceinline__ u32x4 unit_row(const u32x4 (&un)[4], int r) {
    const uint32_t sel = (r & 1) ? 0x07060302u : 0x05040100u;
    u32x4 row;
#pragma unroll
    for (int k = 0; k < 4; ++k) row[k] = __builtin_amdgcn_perm(un[k][2 + (r >> 1)], un[k][r >> 1], sel);
    return row;
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
            v4f v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = acc[mi][ni][4 * q + i] * __uint_as_float(s4[i]) * sb[ni];
            *reinterpret_cast<v4f*>(ep + (lane >> 5) * 2048 + ((col ^ ((col >> 4) & 7)) << 4)) = v;
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
                og[e] = pack2(lo.dg, hi.dg);
                ou[e] = pack2(lo.du, hi.du);
                if constexpr (ACT)
                    oa[e] = pack2(lo.act, hi.act);
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
template <int FA, int FB>
hipError_t glu_typed(const GluFwd& p, hipStream_t st) {
    const int64_t cus = current_device_props().cus, large = (p.m + 255) / 256 * ((p.inter + 127) / 128);
    if (p.k > 0 && p.k % 256 == 0 && p.m >= 256 && p.inter >= 128 && glu_large_tiles(large, cus)) {
        const dim3 grid((unsigned)persistent_grid(large));
        if (p.h) hipLaunchKernelGGL((k_glu_persist<FA, FB, true>), grid, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((k_glu_persist<FA, FB, false>), grid, dim3(256), 0, st, p);
        return hipGetLastError();
    }
    if (glu_few_rows(p.m, p.inter, cus)) {
        const dim3 grid((unsigned)((p.inter + 15) / 16));
        // Fewer workgroups than CUs: eight wavefronts each, else four. One row, 2048 x 1408
        // (88 workgroups) 4.4 and 4.9 us; 32 rows, 4096 x 4096 (256) 12.7 and 11.3.
#define CALL(NT, W) hipLaunchKernelGGL((k_glu_few<FA, FB, NT, W>), grid, dim3(W * 64), 0, st, p)
        if (grid.x < cus) {
            if (p.m <= 16) CALL(1, 8);
            else CALL(2, 8);
        } else {
            if (p.m <= 16) CALL(1, 4);
            else CALL(2, 4);
        }
#undef CALL
        return hipGetLastError();
    }
    const int64_t tiles_n = (p.inter + 63) / 64, tiles = (p.m + 127) / 128 * tiles_n;
    if (glu_tiles_of_64_rows(p.m, tiles, cus)) {
        const dim3 grid((unsigned)((p.m + 63) / 64 * tiles_n));
        hipLaunchKernelGGL((k_glu_mid<FA, FB, 1>), grid, dim3(256), 0, st, p);
    } else {
        hipLaunchKernelGGL((k_glu_mid<FA, FB, 2>), dim3((unsigned)tiles), dim3(256), 0, st, p);
    }
    return hipGetLastError();
}

template <int FA, int FB>
hipError_t glu_grad_typed(const GluBwd& p, hipStream_t st) {
    const int64_t cus = current_device_props().cus, large = (p.m + 255) / 256 * ((p.inter + 255) / 256);
    if (p.k > 0 && p.k % 256 == 0 && p.m >= 256 && p.inter >= 256 && glu_large_tiles(large, cus)) {
        const dim3 grid((unsigned)persistent_grid(large));
        if (p.act) hipLaunchKernelGGL((k_glu_grad_persist<FA, FB, true>), grid, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((k_glu_grad_persist<FA, FB, false>), grid, dim3(256), 0, st, p);
        return hipGetLastError();
    }
    const int64_t tiles_n = (p.inter + 127) / 128, tiles = (p.m + 127) / 128 * tiles_n;
    if (glu_tiles_of_64_rows(p.m, tiles, cus)) {
        const dim3 grid((unsigned)((p.m + 63) / 64 * tiles_n));
        hipLaunchKernelGGL((k_glu_grad_mid<FA, FB, 1>), grid, dim3(256), 0, st, p);
    } else {
        hipLaunchKernelGGL((k_glu_grad_mid<FA, FB, 2>), dim3((unsigned)tiles), dim3(256), 0, st, p);
    }
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
