// swiglu.hip - SwiGLU of a feed-forward layer in training: the forward pass
// fused with the rowwise cast and with an 8-bit checkpoint of its input
// h = [gate | up], and the backward pass from h or from the checkpoint.
//
//   forward: a = silu(g) u, silu(g) = g sigma(g), sigma(g) = 1 / (1 + exp(-g))
//   backward: du = da silu(g), dg = da u sigma(g) (1 + g (1 - sigma(g)))
//
// Bound by HBM: one read of the inputs, one write of the outputs.
#include "layer.hpp"
#include "layer_device.hpp"

namespace fp8amax {
namespace {

constexpr int kBlock = 256;   // 4 wavefronts
constexpr int kWaves = kBlock / 64;

// WPR wavefronts per row; a chunk of 8 gate columns and the same 8 up columns
// per lane and step. inter is a multiple of 32, so gate and up blocks of the
// checkpoint do not meet in one block; a record (four blocks) may hold blocks
// of both where inter is no multiple of 128, so each block's byte is stored
// by itself there.
template <int F, int MAXC, int WPR>
__global__ __launch_bounds__(WPR == 1 ? kBlock : WPR * 64) void k_swiglu_quant_row_mx(SwigluFwd p) {
    __shared__ float red[WPR];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = WPR == 1 ? lane : (int)threadIdx.x;
    constexpr int TPR = WPR * 64;
    const int64_t row = WPR == 1 ? xcd_block(blockIdx.x, gridDim.x) * kWaves + wave : xcd_block(blockIdx.x, gridDim.x);
    if (row >= p.rows) return;                              // (uniform over the wavefronts of a row)
    const int nch = (int)(p.inter >> 3);
    const uint4* gr = reinterpret_cast<const uint4*>(p.h + row * p.ldh);
    const uint4* ur = reinterpret_cast<const uint4*>(p.h + row * p.ldh + p.inter);
    uint4 gv[MAXC], uv[MAXC];
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
        const int ch = t + c * TPR;
        const int cc = ch < nch ? ch : nch - 1;
        gv[c] = load_stream(gr + cc);
        uv[c] = load_stream(ur + cc);
    }
    const bool whole = p.inter % 128 == 0;
    float a[MAXC][8];
    float mx = 0.0f;
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
        const int ch = t + c * TPR;
        const bool live = ch < nch;
        float g[8], u[8];
        unpack8(gv[c], g);
        unpack8(uv[c], u);
        uint32_t rg, ru;
        uint2 cg, cu;
        if (p.ckpt_e5m2) {
            cg = mx_chunk<kE5M2>(g, live, &rg);
            cu = mx_chunk<kE5M2>(u, live, &ru);
        } else {
            cg = mx_chunk<kE4M3>(g, live, &rg);
            cu = mx_chunk<kE4M3>(u, live, &ru);
        }
        if (live) {
            uint8_t* hr = p.hq + row * p.ldhq;
            store_checkpoint(hr + 8 * ch, cg);
            store_checkpoint(hr + p.inter + 8 * ch, cu);
            if (whole) {
                if ((lane & 15) == 0) {
                    *reinterpret_cast<uint32_t*>(p.hs + 4 * ((int64_t)(ch >> 4) * p.ldhs + row)) = rg;
                    *reinterpret_cast<uint32_t*>(p.hs + 4 * ((int64_t)((ch + nch) >> 4) * p.ldhs + row)) = ru;
                }
            } else if ((lane & 3) == 0) {
                // (the low byte of a record is the byte of the lane's own block)
                const int bg = ch >> 2, bu = (ch + nch) >> 2, last = (2 * nch) >> 2;
                p.hs[4 * ((int64_t)(bg >> 2) * p.ldhs + row) + (bg & 3)] = (uint8_t)rg;
                p.hs[4 * ((int64_t)(bu >> 2) * p.ldhs + row) + (bu & 3)] = (uint8_t)ru;
                if (bu == last - 1)                         // blocks past the row in the last record
                    for (int b = last; b & 3; ++b) p.hs[4 * ((int64_t)(b >> 2) * p.ldhs + row) + (b & 3)] = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) a[c][i] = silu_fast(g[i]) * u[i];
        mx = __builtin_elementwise_maximum(mx, absmax8(a[c]));      // (past the row: a duplicate of its last chunk)
    }
    mx = wave_max(mx);
    if (WPR > 1) {
        if (lane == 0) red[wave] = mx;
        __syncthreads();
        mx = max_of<WPR>(red);
    }
    const float s = scale_from_amax<F>(mx, p.margin);
    if (t == 0) p.scale_inv[row] = 1.0f / s;
    uint2* qr = reinterpret_cast<uint2*>(p.q + row * p.ldq);
    if (__builtin_isfinite(mx)) {
#pragma unroll
        for (int c = 0; c < MAXC; ++c) {
            const int ch = t + c * TPR;
            if (ch < nch) qr[ch] = encode8_scaled<F>(a[c], s);
        }
    } else {        // an Inf or NaN in the row (then the scale is 1): the bit-level encoder
#pragma unroll
        for (int c = 0; c < MAXC; ++c) {
            const int ch = t + c * TPR;
            if (ch < nch) qr[ch] = encode8f<F, false>(a[c], s);
        }
    }
}

// Chunks of one launch of the gradient (134 million values, a quarter of a
// millisecond): longer calls are cut, so that chunk numbers stay 32-bit.
constexpr int64_t kGradChunks = (int64_t)1 << 24;

// One chunk of 8 columns per thread; no reduction. SRC: 0 = h in bf16, 1 / 2 =
// the checkpoint in e4m3 / e5m2. Chunk i is chunk i % nch of row i / nch; the
// quotient is (mulhi(magic, i) + i) >> shift, exact for i < 2^31 (the launcher
// cuts larger calls into bands of rows).
template <int SRC>
__global__ __launch_bounds__(kBlock) void k_swiglu_grad(SwigluBwd p, uint32_t magic, int shift) {
    const uint32_t nch = (uint32_t)(p.inter >> 3);
    const uint32_t i = blockIdx.x * (uint32_t)kBlock + threadIdx.x;
    if (i < (uint32_t)(p.rows * nch)) {
        const uint32_t r = (__umulhi(magic, i) + i) >> shift;
        const int ch = (int)(i - r * nch);
        const int64_t row = r;
        const uint4 dv = load_stream(reinterpret_cast<const uint4*>(p.da + row * p.ldda) + ch);
        float g[8], u[8], da[8], o[8];
        if constexpr (SRC == 0) {
            const uint4 gv = load_stream(reinterpret_cast<const uint4*>(p.h + row * p.ldh) + ch);
            const uint4 uv = load_stream(reinterpret_cast<const uint4*>(p.h + row * p.ldh + p.inter) + ch);
            unpack8(gv, g);
            unpack8(uv, u);
        } else {
            constexpr int F = SRC == 1 ? kE4M3 : kE5M2;
            const uint8_t* hr = p.hq + row * p.ldhq;
            const uint2 gq = reinterpret_cast<const uint2*>(hr)[ch];
            const uint2 uq = reinterpret_cast<const uint2*>(hr + p.inter)[ch];
            const int bg = ch >> 2, bu = (ch + (int)nch) >> 2;
            const float sg = e8m0_value(p.hs[4 * ((int64_t)(bg >> 2) * p.ldhs + row) + (bg & 3)]);
            const float su = e8m0_value(p.hs[4 * ((int64_t)(bu >> 2) * p.ldhs + row) + (bu & 3)]);
            decode4<F>(gq.x, g);
            decode4<F>(gq.y, g + 4);
            decode4<F>(uq.x, u);
            decode4<F>(uq.y, u + 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[j] *= sg;
                u[j] *= su;
            }
        }
        unpack8(dv, da);
        float act[8], du[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Logistic l = logistic(g[j]);
            const float silu = g[j] * l.sig;
            act[j] = silu * u[j];
            du[j] = da[j] * silu;
            o[j] = da[j] * u[j] * fmaf(silu, l.com, l.sig);
        }
        uint16_t* dr = p.dh + row * p.lddh;
        reinterpret_cast<uint4*>(dr)[ch] = pack8(o);
        reinterpret_cast<uint4*>(dr + p.inter)[ch] = pack8(du);
        if (p.a) reinterpret_cast<uint4*>(p.a + row * p.lda)[ch] = pack8(act);
    }
}

}  // namespace

template <int F>
hipError_t swiglu_quant_fmt(const SwigluFwd& p, hipStream_t st) {
    const int64_t nch = p.inter / 8;
    // four wavefronts a row where the row is long (16384 x 2048: 40.9 us, with one
    // 46.5; 16384 x 1024: 37.3 and 24.9) or the rows are few (1000 x 2048: 5.4 and
    // 6.5). Longer rows take more wavefronts, two chunks a lane (with four, 92 VGPRs
    // leave 20 wavefronts a CU: 8192 x 7168 78 us, with two 75; 8192 x 14336 168 and
    // 163), as many as the row fills (8192 x 10240: 145 us with a third of the lanes
    // idle, 118 with ten wavefronts; x 5120 71 and 62), except fourteen, which are 175
    // at 14336
    const bool wide = nch > 128 || (nch > 64 && p.rows < 1024);
    const dim3 grid((unsigned)(wide ? p.rows : (p.rows + kWaves - 1) / kWaves));
#define FP8_SW_CASE(C, W) \
    hipLaunchKernelGGL((k_swiglu_quant_row_mx<F, C, W>), grid, dim3(W == 1 ? kBlock : W * 64), 0, st, p)
    if (wide) {
        if (nch <= 256) FP8_SW_CASE(1, 4);
        else if (nch <= 384) FP8_SW_CASE(2, 3);
        else if (nch <= 512) FP8_SW_CASE(2, 4);
        else if (nch <= 768) FP8_SW_CASE(2, 6);
        else if (nch <= 1024) FP8_SW_CASE(2, 8);
        else if (nch <= 1280) FP8_SW_CASE(2, 10);
        else if (nch <= 1536) FP8_SW_CASE(2, 12);
        else FP8_SW_CASE(2, 16);
    } else {
        if (nch <= 64) FP8_SW_CASE(1, 1);
        else FP8_SW_CASE(2, 1);
    }
#undef FP8_SW_CASE
    return hipGetLastError();
}

hipError_t launch_swiglu_quant_row_mx(const SwigluFwd& p0, int fmt, hipStream_t st) {
    if (p0.inter == 0) return hipSuccess;
    for (int64_t r0 = 0; r0 < p0.rows; r0 += kLaunchRows) {
        SwigluFwd p = p0;
        p.rows = p0.rows - r0 < kLaunchRows ? p0.rows - r0 : kLaunchRows;
        p.h += r0 * p.ldh;
        p.q += r0 * p.ldq;
        p.scale_inv += r0;
        p.hq += r0 * p.ldhq;
        p.hs += 4 * r0;
        hipError_t e;
        switch (fmt) {
            case kE4M3: e = swiglu_quant_fmt<kE4M3>(p, st); break;
            case kE5M2: e = swiglu_quant_fmt<kE5M2>(p, st); break;
            case kE4M3Fnuz: e = swiglu_quant_fmt<kE4M3Fnuz>(p, st); break;
            default: e = swiglu_quant_fmt<kE5M2Fnuz>(p, st); break;
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_swiglu_backward(const SwigluBwd& p0, hipStream_t st) {
    if (p0.rows == 0 || p0.inter == 0) return hipSuccess;
    const int64_t nch = p0.inter / 8;
    int shift = 0;                                          // magic division by nch: 2^shift >= nch
    while (((int64_t)1 << shift) < nch) ++shift;
    const uint32_t magic = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - (uint64_t)nch)) / (uint64_t)nch + 1);
    const int64_t band = kGradChunks / nch > 0 ? kGradChunks / nch : 1;
    for (int64_t r0 = 0; r0 < p0.rows; r0 += band) {
        SwigluBwd p = p0;
        p.rows = p0.rows - r0 < band ? p0.rows - r0 : band;
        p.da += r0 * p.ldda;
        p.dh += r0 * p.lddh;
        if (p.a) p.a += r0 * p.lda;
        if (p.hq) {
            p.hq += r0 * p.ldhq;
            p.hs += 4 * r0;
        } else {
            p.h += r0 * p.ldh;
        }
        const dim3 grid((unsigned)((p.rows * nch + kBlock - 1) / kBlock)), block(kBlock);
        if (!p.hq) hipLaunchKernelGGL((k_swiglu_grad<0>), grid, block, 0, st, p, magic, shift);
        else if (!p.ckpt_e5m2) hipLaunchKernelGGL((k_swiglu_grad<1>), grid, block, 0, st, p, magic, shift);
        else hipLaunchKernelGGL((k_swiglu_grad<2>), grid, block, 0, st, p, magic, shift);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace fp8amax
