// norm.hip - layer norm and its RMS form before an FP8 product: the forward
// pass fused with the rowwise cast (and with an 8-bit checkpoint of the
// normalised rows), the backward pass with the reduction of the weights'
// gradients, from x or from the checkpoint.
//
//   forward, row r of N columns: mu = sum x / N (RMS: 0), v = sum (x - mu)^2 / N,
//     rstd = 1 / sqrt(v + eps), xh = (x - mu) rstd, y = xh gamma + beta
//   backward: w = dy gamma, dx = rstd (w - mean(w) - xh mean(w xh))
//     (RMS: without mean(w)), dgamma = sum_r dy xh, dbeta = sum_r dy
//
// ADD: x is the sum of two inputs, s = bf16(x + r), formed in the same read and
// stored; the norm takes the stored (rounded) values, which the backward pass will
// read too. Backward, s's own gradient ds is added: dx = ds + the above, for both
// inputs. 16384 x 7168 with a checkpoint 160-182 us (5.2-5.9 TB/s); gradient of
// 8192 x 4096 from s 51 us, of 2050 x 7168 from the checkpoint 30.
//
// Everything here is bound by HBM: the rows are held in registers from their
// one read to their last use, and all statistics and sums are fp32.
#include "layer.hpp"
#include "layer_device.hpp"

namespace fp8amax {
namespace {

constexpr int kBlock = 256;   // 4 wavefronts
constexpr int kWaves = kBlock / 64;

// Eight of gamma's or beta's values (bf16 or fp32), chunk ch of n.
template <bool LOOSE>
__device__ __forceinline__ void load_weights8(const void* w, int w_f32, uint32_t ch, uint32_t n, float* o) {
    const uint32_t first = !LOOSE || ch * 8 + 8 <= n ? ch * 8 : n - 8;
    if (w_f32) {
        constexpr int A = LOOSE ? 4 : 16;
        const f32x4 a = load_loose<f32x4, A>(w, first * 4), b = load_loose<f32x4, A>(w, first * 4 + 16);
        o[0] = a.x;
        o[1] = a.y;
        o[2] = a.z;
        o[3] = a.w;
        o[4] = b.x;
        o[5] = b.y;
        o[6] = b.z;
        o[7] = b.w;
        if constexpr (LOOSE) {
            const uint32_t s = ch * 8 - first;
            if (s > 0) {
#pragma unroll
                for (int k = 4; k >= 1; k >>= 1)
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = s & k ? (i + k < 8 ? o[i + k] : 0.0f) : o[i];
            }
        }
    } else {
        const u32x4 r = load_loose<u32x4, LOOSE ? 2 : 16>(w, first * 2);
        uint4 v = make_uint4(r.x, r.y, r.z, r.w);
        place_chunk<LOOSE>(&v, ch, n);
        unpack8(v, o);
    }
}
__device__ __forceinline__ float load_weight(const void* w, int w_f32, int64_t c) {
    return w_f32 ? static_cast<const float*>(w)[c] : __uint_as_float((uint32_t) static_cast<const uint16_t*>(w)[c] << 16);
}

// ---------------------------------------------------------------- forward --
// WPR wavefronts per row. The variance is the second pass over the registers
// (sum of (x - mu)^2), so a row whose mean is large against its deviation
// loses nothing. y is formed in fp32 and cast from there.
template <int F, int MAXC, int WPR, bool LOOSE, bool ADD>
__global__ __launch_bounds__(WPR == 1 ? kBlock : WPR * 64) void k_norm_quant_row(NormFwd p) {
    __shared__ float red[3][WPR];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = WPR == 1 ? lane : (int)threadIdx.x;
    constexpr int TPR = WPR * 64;
    const int64_t row = WPR == 1 ? xcd_block(blockIdx.x, gridDim.x) * kWaves + wave : xcd_block(blockIdx.x, gridDim.x);
    if (row >= p.rows) return;                              // (uniform over the wavefronts of a row)
    const uint32_t n = (uint32_t)p.cols;
    const int nch = (int)((n + 7) >> 3);
    const float inv_n = 1.0f / (float)p.cols;
    const uint16_t* xr = p.x + row * p.ldx;
    uint4 raw[MAXC], res[ADD ? MAXC : 1];
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
        const int ch = t + c * TPR;
        raw[c] = load_chunk<LOOSE>(xr, (uint32_t)(ch < nch ? ch : nch - 1), n);
        if constexpr (ADD) res[c] = load_chunk<LOOSE>(p.res + row * p.ldres, (uint32_t)(ch < nch ? ch : nch - 1), n);
    }
    float v[MAXC][8];
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
        const int ch = t + c * TPR;
        place_chunk<LOOSE>(&raw[c], (uint32_t)ch, n);
        if constexpr (ADD) {
            place_chunk<LOOSE>(&res[c], (uint32_t)ch, n);
            float x[8], r[8];
            unpack8(raw[c], x);
            unpack8(res[c], r);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] += r[i];
            // (the sum may take an input's place: a lane reads of a chunk only what it
            // stores, the values of a cut chunk's neighbour aside, which it drops)
            if (ch < nch) store_chunk<LOOSE>(p.sum + row * p.ldsum, (uint32_t)ch, n, x);
            raw[c] = pack8(x);
        }
        if (ch >= nch) raw[c] = make_uint4(0u, 0u, 0u, 0u);                 // past the row: zeros
        unpack8(raw[c], v[c]);
    }
    float mean = 0.0f;
    if (!p.rms) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < MAXC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[c][i];
        s = wave_sum(s);
        if (WPR > 1) {
            if (lane == 0) red[0][wave] = s;
            __syncthreads();
            s = sum_of<WPR>(red[0]);
        }
        mean = s * inv_n;
#pragma unroll
        for (int c = 0; c < MAXC; ++c) {
            const int ch = t + c * TPR;
            const float m = ch < nch ? mean : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] -= !LOOSE || (uint32_t)(ch * 8 + i) < n ? m : 0.0f;
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < MAXC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
    ss = wave_sum(ss);
    if (WPR > 1) {
        if (lane == 0) red[1][wave] = ss;
        __syncthreads();
        ss = sum_of<WPR>(red[1]);
    }
    const float rstd = 1.0f / __builtin_sqrtf(ss * inv_n + p.eps);
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    float mx = 0.0f;
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
        const int ch = t + c * TPR;
        const bool live = ch < nch;
        const uint32_t cc = (uint32_t)(live ? ch : nch - 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= rstd;
        if (!LOOSE && p.xq) {
            uint32_t record;
            const uint2 code = p.ckpt_e5m2 ? mx_chunk<kE5M2>(v[c], live, &record) : mx_chunk<kE4M3>(v[c], live, &record);
            if (live) {
                store_checkpoint(p.xq + row * p.ldxq + 8 * ch, code);
                if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.xs + 4 * ((int64_t)(ch >> 4) * p.ldxs + row)) = record;
            }
        }
        if (p.gamma) {
            float g[8];
            load_weights8<LOOSE>(p.gamma, p.w_f32, cc, n, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] *= g[i];
        }
        if (p.beta) {
            float b[8];
            load_weights8<LOOSE>(p.beta, p.w_f32, cc, n, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] += b[i];
        }
        // (a chunk past the row holds a value of xh = 0 at the row's last
        // columns: kept out of the maximum)
        const float m = absmax8(v[c]);
        mx = __builtin_elementwise_maximum(mx, live ? m : 0.0f);
        if (p.y && live) store_chunk<LOOSE>(p.y + row * p.ldy, cc, n, v[c]);
    }
    if (!p.q) return;
    mx = wave_max(mx);
    if (WPR > 1) {
        if (lane == 0) red[2][wave] = mx;
        __syncthreads();
        mx = max_of<WPR>(red[2]);
    }
    const float sc = scale_from_amax<F>(mx, p.margin);
    if (t == 0) p.scale_inv[row] = 1.0f / sc;
    uint8_t* qr = p.q + row * p.ldq;
    if (__builtin_isfinite(mx)) {
#pragma unroll
        for (int c = 0; c < MAXC; ++c) {
            const int ch = t + c * TPR;
            if (ch < nch) store_codes<LOOSE>(qr, (uint32_t)ch, n, encode8_scaled<F>(v[c], sc));
        }
    } else {        // an Inf or NaN in the row (then the scale is 1): the bit-level encoder
#pragma unroll
        for (int c = 0; c < MAXC; ++c) {
            const int ch = t + c * TPR;
            if (ch < nch) store_codes<LOOSE>(qr, (uint32_t)ch, n, encode8f<F, false>(v[c], sc));
        }
    }
}

// Rows of fewer than 8 or more than kNormMaxVecCols columns, in any layout: one
// workgroup per row, element loads, the row read again from the
// caches for each pass.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}
__device__ __forceinline__ float load_bf16(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

template <int F, bool ADD>
__global__ __launch_bounds__(kBlock) void k_norm_quant_row_any(NormFwd p) {
    __shared__ float red[kWaves];
    __shared__ uint32_t redu[kWaves];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const uint16_t* xr = p.x + row * p.ldx;
    if constexpr (ADD) {                // (a thread reads of the sum what it wrote)
        const uint16_t* rr = p.res + row * p.ldres;
        uint16_t* sr = p.sum + row * p.ldsum;
        for (int64_t c = tid; c < p.cols; c += kBlock)
            sr[c] = (uint16_t)f32_to_bf16(load_bf16(xr + c) + load_bf16(rr + c));
        xr = sr;
    }
    const float inv_n = 1.0f / (float)p.cols;
    float mean = 0.0f, s = 0.0f;
    if (!p.rms) {
        for (int64_t c = tid; c < p.cols; c += kBlock) s += load_bf16(xr + c);
        mean = block_sum(s, red) * inv_n;
    }
    float ss = 0.0f;
    for (int64_t c = tid; c < p.cols; c += kBlock) {
        const float d = load_bf16(xr + c) - mean;
        ss = fmaf(d, d, ss);
    }
    const float rstd = 1.0f / __builtin_sqrtf(block_sum(ss, red) * inv_n + p.eps);
    if (tid == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    auto value = [&](int64_t c) {
        float y = (load_bf16(xr + c) - mean) * rstd;
        if (p.gamma) y *= load_weight(p.gamma, p.w_f32, c);
        if (p.beta) y += load_weight(p.beta, p.w_f32, c);
        return y;
    };
    uint32_t mx = 0;
    for (int64_t c = tid; c < p.cols; c += kBlock) {
        const float y = value(c);
        if (p.y) p.y[row * p.ldy + c] = (uint16_t)f32_to_bf16(y);
        const uint32_t b = __float_as_uint(y) & 0x7fffffffu;
        mx = b > mx ? b : mx;
    }
    if (!p.q) return;
    mx = wave_max_u32(mx);
    __syncthreads();
    if ((tid & 63) == 0) redu[tid >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mx = redu[w] > mx ? redu[w] : mx;
    const float sc = scale_from_amax<F>(__uint_as_float(mx), p.margin);
    if (tid == 0) p.scale_inv[row] = 1.0f / sc;
    for (int64_t c = tid; c < p.cols; c += kBlock) p.q[row * p.ldq + c] = (uint8_t)encode_sw<F>(value(c) * sc);
}

// --------------------------------------------------------------- backward --
// A workgroup owns a band of neighbouring rows; TPR threads work on one row (a
// team), each on the same MAXC chunks of 8 columns for every row, so that the
// sums over rows of the weights' gradients stay in registers. A row costs one
// barrier (its two sums meet in LDS, in one of two buffers); the next row's
// loads are issued before the current row is worked on. At the end the teams'
// sums are added in LDS in team order and the band's sums are written to the
// workspace; k_norm_weight_grad adds the bands in order. No atomics: results
// do not depend on timing.
// SRC: 0 = x in bf16 with mean and rstd, 1 / 2 = the checkpoint in e4m3 / e5m2.
template <int SRC, int MAXC, bool ADD>
struct RowData {
    uint4 dy[MAXC], ds[ADD && SRC == 0 ? MAXC : 1];
    uint32_t x[MAXC][SRC == 0 ? 4 : 2];
    uint32_t byte[MAXC];                // (SRC > 0: the block's scale)
    float mean, rstd;
};

template <int SRC, int TPR, int MAXC, bool LOOSE, bool ADD>
__device__ __forceinline__ void load_row(const NormBwd& p, int row, uint32_t tt, uint32_t nch,
                                         RowData<SRC, MAXC, ADD>* d) {
    const uint32_t n = (uint32_t)p.cols;
    d->rstd = p.rstd[row];
    d->mean = SRC == 0 && p.mean ? p.mean[row] : 0.0f;
    const uint16_t* dr = p.dy + row * p.lddy;
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
        const uint32_t ch = tt + c * TPR;
        const uint32_t cc = ch < nch ? ch : nch - 1;    // (past the row: a duplicate, never stored)
        d->dy[c] = load_chunk<LOOSE>(dr, cc, n);
        if constexpr (ADD && SRC == 0) d->ds[c] = load_chunk<LOOSE>(p.ds + row * p.ldds, cc, n);
        if constexpr (SRC == 0) {
            const uint4 x = load_chunk<LOOSE>(p.x + row * p.ldx, cc, n);
            d->x[c][0] = x.x;
            d->x[c][1] = x.y;
            d->x[c][2] = x.z;
            d->x[c][3] = x.w;
        } else {
            const uint2 q = *at<uint2>(p.xq + row * p.ldxq, cc * 8);
            d->x[c][0] = q.x;
            d->x[c][1] = q.y;
            d->byte[c] = (p.xs + 4 * (int64_t)row)[4 * (int64_t)(cc >> 4) * p.ldxs + ((cc >> 2) & 3u)];
        }
    }
}

// (dgamma and dbeta have no alignment but their type's)
template <bool LOOSE>
__device__ __forceinline__ void store_sums(float* p, uint32_t ch, uint32_t n, const float* v) {
    if (!LOOSE || ch * 8 + 8 <= n) {
        store_loose<f32x4, 4>(p, ch * 32, f32x4{v[0], v[1], v[2], v[3]});
        store_loose<f32x4, 4>(p, ch * 32 + 16, f32x4{v[4], v[5], v[6], v[7]});
        return;
    }
#pragma unroll
    for (uint32_t i = 0; i < 7; ++i)
        if (ch * 8 + i < n) p[ch * 8 + i] = v[i];
}

// Chunk c of the row as fp32.
template <int SRC, int MAXC, bool ADD>
__device__ __forceinline__ void row_values(const RowData<SRC, MAXC, ADD>& d, int c, float* xh, float* dy) {
    unpack8(d.dy[c], dy);
    if constexpr (SRC == 0) {
        unpack8(make_uint4(d.x[c][0], d.x[c][1], d.x[c][2], d.x[c][3]), xh);
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[i] = (xh[i] - d.mean) * d.rstd;
    } else {
        decode4<SRC == 1 ? kE4M3 : kE5M2>(d.x[c][0], xh);
        decode4<SRC == 1 ? kE4M3 : kE5M2>(d.x[c][1], xh + 4);
        const float bs = e8m0_value(d.byte[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[i] *= bs;
    }
}

template <int SRC, int TPR, int MAXC, int WG, bool LOOSE, bool ADD>
__global__ __launch_bounds__(WG, 4) void k_norm_grad(NormBwd p) {
    constexpr int TEAMS = WG / TPR, NW = TPR / 64;
    __shared__ float2 red[2][WG / 64];
    __shared__ float fold[TEAMS > 1 ? 2 * MAXC * 8 * TPR : 1];
    __shared__ float beta[SRC > 0 ? MAXC * 8 * TPR : 1];
    // (the team is uniform over a wavefront: row addresses stay in scalar registers)
    const int tid = threadIdx.x, team = __builtin_amdgcn_readfirstlane(tid / TPR);
    const int wave = tid >> 6, lane = tid & 63;
    uint32_t tt = (uint32_t)tid % TPR;
    const uint32_t n = (uint32_t)p.cols, nch = (n + 7) >> 3;
    const float inv_n = 1.0f / (float)p.cols;
    // the first `longer` bands have a row more than the others
    const int b = (int)blockIdx.x, r0 = b * (int)p.band + (b < (int)p.longer ? b : (int)p.longer);
    const int r1 = r0 + (int)p.band + (b < (int)p.longer ? 1 : 0);
    const bool want = p.dgamma || p.dbeta;
    float g[MAXC][8], dg[MAXC][8], db[MAXC][8];
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
        const uint32_t ch = tt + c * TPR, cc = ch < nch ? ch : nch - 1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[c][i] = 1.0f;
            dg[c][i] = db[c][i] = 0.0f;
        }
        if (p.gamma) load_weights8<LOOSE>(p.gamma, p.w_f32, cc, n, g[c]);
        // beta in LDS: the addresses of its two forms, kept over the loop, spilled
        if (SRC > 0 && p.y && p.beta && team == 0) {
            float b[8];
            load_weights8<LOOSE>(p.beta, p.w_f32, cc, n, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) beta[(c * TPR + tt) * 8 + i] = b[i];
        }
    }
    if (SRC > 0) __syncthreads();
    RowData<SRC, MAXC, ADD> cur, nxt;
    load_row<SRC, TPR, MAXC, LOOSE, ADD>(p, r0 + team < r1 ? r0 + team : r1 - 1, tt, nch, &cur);
    int buf = 0;
    for (int r = r0; r < r1; r += TEAMS, buf ^= 1) {
        const int row = r + team;
        const bool live_row = row < r1;
        const int next = row + TEAMS;
        // tt opaque in every step: offsets are then formed where they are used,
        // next to scalar bases, and not kept as 64-bit pairs over the loop
        asm volatile("" : "+v"(tt));
        // from a checkpoint, ds of the row at hand (a row ahead it spilled), asked for
        // before the next row, since loads return in order
        uint4 ds[ADD ? MAXC : 1];
        if constexpr (ADD) {
#pragma unroll
            for (int c = 0; c < MAXC; ++c) {
                const uint32_t ch = tt + c * TPR;
                if constexpr (SRC > 0)
                    ds[c] = load_chunk<LOOSE>(p.ds + (int64_t)(live_row ? row : r1 - 1) * p.ldds, ch < nch ? ch : nch - 1, n);
                else
                    ds[c] = cur.ds[c];
            }
        }
        load_row<SRC, TPR, MAXC, LOOSE, ADD>(p, next < r1 ? next : r1 - 1, tt, nch, &nxt);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int c = 0; c < MAXC; ++c) {
            const uint32_t ch = tt + c * TPR;
            const bool live = live_row && ch < nch;
            // (A row past the band is worked on and used nowhere.)
            if (LOOSE && live) {
                uint4 x = make_uint4(cur.x[c][0], cur.x[c][1], cur.x[c][SRC == 0 ? 2 : 0], cur.x[c][SRC == 0 ? 3 : 0]);
                place_chunk<LOOSE>(&cur.dy[c], ch, n);
                if constexpr (ADD) place_chunk<LOOSE>(&ds[c], ch, n);
                place_chunk<LOOSE>(&x, ch, n);
                cur.x[c][0] = x.x;
                cur.x[c][1] = x.y;
                cur.x[c][SRC == 0 ? 2 : 0] = x.z;
                cur.x[c][SRC == 0 ? 3 : 0] = x.w;
            }
            float xh[8], dy[8];
            row_values<SRC>(cur, c, xh, dy);
            // What stands past the row is selected out of the sums: as a term of 0
            // it would be 0 * Inf where a weight, xhat or rstd is infinite.
            float t1 = s1, t2 = s2;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = dy[i] * g[c][i], f1 = fmaf(w, xh[i], t1), f2 = t2 + w;
                const bool in = !LOOSE || ch * 8 + i < n;
                t1 = in ? f1 : t1;
                t2 = in ? f2 : t2;
            }
            s1 = ch < nch ? t1 : s1;
            s2 = ch < nch ? t2 : s2;
            if (SRC > 0 && p.y && live) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    xh[i] *= g[c][i];
                    if (p.beta) xh[i] += beta[(c * TPR + tt) * 8 + i];
                }
                *at<uint4>(p.y + row * p.ldy, ch * 16) = pack8(xh);
            }
        }
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if (NW > 1) {
            if (lane == 0) red[buf][wave] = make_float2(s1, s2);
            __syncthreads();
            s1 = s2 = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float2 f = red[buf][team * NW + w];
                s1 += f.x;
                s2 += f.y;
            }
        }
        const float c1 = s1 * inv_n, c2 = p.rms ? 0.0f : s2 * inv_n;
#pragma unroll
        for (int c = 0; c < MAXC; ++c) {
            const uint32_t ch = tt + c * TPR;
            const bool live = live_row && ch < nch;
            // the row's values again from its raw words (made opaque here, so
            // that they are not kept): holding them across the reduction took
            // 178 VGPRs, half the wavefronts a CU holds
            asm volatile("" : "+v"(cur.dy[c].x), "+v"(cur.dy[c].y), "+v"(cur.dy[c].z), "+v"(cur.dy[c].w));
            asm volatile("" : "+v"(cur.x[c][0]), "+v"(cur.x[c][1]));
            if constexpr (SRC == 0) asm volatile("" : "+v"(cur.x[c][2]), "+v"(cur.x[c][3]));
            float xh[8], dy[8], o[8];
            row_values<SRC>(cur, c, xh, dy);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = cur.rstd * (fmaf(-c1, xh[i], dy[i] * g[c][i]) - c2);
            if constexpr (ADD) {
                float d[8];
                unpack8(ds[c], d);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += d[i];
            }
            if (live) store_chunk<LOOSE>(p.dx + row * p.lddx, ch, n, o);
            if (live_row) {         // (uniform; the duplicate of a row could add 0 * Inf)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dg[c][i] = fmaf(dy[i], xh[i], dg[c][i]);
                    db[c][i] += dy[i];
                }
            }
        }
        cur = nxt;
    }
    if (!want) return;
    if constexpr (TEAMS > 1) {                              // word (2 c' + which) * TPR + tt: no bank conflicts
        for (int t = 1; t < TEAMS; ++t) {
            __syncthreads();
            if (team == t) {
#pragma unroll
                for (int c = 0; c < MAXC; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        fold[(2 * (c * 8 + i)) * TPR + tt] = dg[c][i];
                        fold[(2 * (c * 8 + i) + 1) * TPR + tt] = db[c][i];
                    }
            }
            __syncthreads();
            if (team == 0) {
#pragma unroll
                for (int c = 0; c < MAXC; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dg[c][i] += fold[(2 * (c * 8 + i)) * TPR + tt];
                        db[c][i] += fold[(2 * (c * 8 + i) + 1) * TPR + tt];
                    }
            }
        }
        if (team != 0) return;
    }
    // one band: its sums are the result
    float* og = p.bands == 1 ? p.dgamma : p.partial + (int64_t)blockIdx.x * 2 * p.cols;
    float* ob = p.bands == 1 ? p.dbeta : p.partial + (int64_t)blockIdx.x * 2 * p.cols + p.cols;
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
        const uint32_t ch = tt + c * TPR;
        if (ch >= nch) continue;
        if (p.dgamma) store_sums<LOOSE>(og, ch, n, dg[c]);
        if (p.dbeta) store_sums<LOOSE>(ob, ch, n, db[c]);
    }
}

// Sums of the bands, in order: 32 columns x 16 slices of the bands per
// workgroup, the slices added in order. blockIdx.y: 0 = dgamma, 1 = dbeta.
constexpr int kSliceCols = 32, kSlices = 16;
__global__ __launch_bounds__(kSliceCols * kSlices) void k_norm_weight_grad(const float* __restrict__ partial, int64_t bands,
                                                             int64_t cols, float* dgamma, float* dbeta) {
    __shared__ float red[kSlices][kSliceCols];
    float* out = blockIdx.y == 0 ? dgamma : dbeta;
    if (!out) return;
    const int cl = threadIdx.x % kSliceCols, sl = threadIdx.x / kSliceCols;
    const int64_t col = (int64_t)blockIdx.x * kSliceCols + cl;
    const int64_t per = (bands + kSlices - 1) / kSlices;
    const int64_t b0 = sl * per, b1 = b0 + per < bands ? b0 + per : bands;
    const float* src = partial + (int64_t)blockIdx.y * cols + (col < cols ? col : cols - 1);
    float s = 0.0f;
#pragma unroll 8
    for (int64_t b = b0; b < b1; ++b) s += src[b * 2 * cols];
    red[sl][cl] = s;
    __syncthreads();
    if (sl == 0 && col < cols) {
#pragma unroll
        for (int i = 1; i < kSlices; ++i) s += red[i][cl];
        out[col] = s;
    }
}

// Rows of fewer than 8 or more than kNormMaxVecCols columns, in any layout, from x:
// one workgroup per row for dx, another kernel for the weights' gradients.
__global__ __launch_bounds__(kBlock) void k_norm_grad_row_any(NormBwd p) {
    __shared__ float red[kWaves];
    const int tid = threadIdx.x;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const uint16_t *xr = p.x + row * p.ldx, *dr = p.dy + row * p.lddy;
        const float rstd = p.rstd[row], mean = p.mean ? p.mean[row] : 0.0f, inv_n = 1.0f / (float)p.cols;
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = tid; c < p.cols; c += kBlock) {
            const float w = load_bf16(dr + c) * (p.gamma ? load_weight(p.gamma, p.w_f32, c) : 1.0f);
            s1 = fmaf(w, (load_bf16(xr + c) - mean) * rstd, s1);
            s2 += w;
        }
        const float c1 = block_sum(s1, red) * inv_n, c2 = p.rms ? 0.0f : block_sum(s2, red) * inv_n;
        for (int64_t c = tid; c < p.cols; c += kBlock) {
            const float w = load_bf16(dr + c) * (p.gamma ? load_weight(p.gamma, p.w_f32, c) : 1.0f);
            const float xh = (load_bf16(xr + c) - mean) * rstd;
            const float ds = p.ds ? load_bf16(p.ds + row * p.ldds + c) : 0.0f;
            p.dx[row * p.lddx + c] = (uint16_t)f32_to_bf16(ds + rstd * (fmaf(-c1, xh, w) - c2));
        }
    }
}

// 32 columns x 32 slices of the band's rows per workgroup, the slices added in
// order. (One thread per column over bands of 32 rows: a third launch for every
// size, 333 x 1111: 4.6 + 2.6 us.)
__global__ __launch_bounds__(kAnyCols * kAnySlices) void k_norm_grad_cols_any(NormBwd p) {
    __shared__ float red[2][kAnySlices][kAnyCols];
    const int cl = threadIdx.x % kAnyCols, sl = threadIdx.x / kAnyCols;
    const int64_t c = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * kAnyCols + cl, cc = c < p.cols ? c : p.cols - 1;
    const int64_t r0 = (int64_t)blockIdx.y * p.band;
    const int64_t r1 = r0 + p.band < p.rows ? r0 + p.band : p.rows;
    float dg = 0.0f, db = 0.0f;
#pragma unroll 8
    for (int64_t r = r0 + sl; r < r1; r += kAnySlices) {
        const float xh = (load_bf16(p.x + r * p.ldx + cc) - (p.mean ? p.mean[r] : 0.0f)) * p.rstd[r];
        const float dy = load_bf16(p.dy + r * p.lddy + cc);
        dg = fmaf(dy, xh, dg);
        db += dy;
    }
    red[0][sl][cl] = dg;
    red[1][sl][cl] = db;
    __syncthreads();
    if (sl > 1 || c >= p.cols) return;
    float s = 0.0f;
#pragma unroll 8
    for (int i = 0; i < kAnySlices; ++i) s += red[sl][i][cl];
    float* out = sl == 0 ? p.dgamma : p.dbeta;
    if (out) (p.bands == 1 ? out : p.partial + ((int64_t)blockIdx.y * 2 + sl) * p.cols)[c] = s;
}

unsigned row_grid(int64_t rows) { return (unsigned)(rows < kLaunchRows ? rows : kLaunchRows); }

}  // namespace

template <int F, bool LOOSE, bool ADD>
hipError_t norm_quant_reg(const NormFwd& p, hipStream_t st) {
    const int64_t nch = (p.cols + 7) / 8;
    // One wavefront a row where it holds the row (16384 x 2048: 22.9 us, 31.0 with
    // the checkpoint; with four wavefronts 28.2 and 34.6) unless the rows are few
    // (1000 x 2048: 3.5 and 4.2 us with four wavefronts, 4.1 and 5.4 with one; 16 x
    // 2048: 2.8 and 3.0, 3.8 and 4.7); longer rows as many wavefronts as they fill
    // (8192 x 5120: 27.4 and 38.7 us with three, 29.9 and 42.1 with four; x 10240 49.0
    // and 68 with five, 54 and 76 with eight; two chunks a lane for these sizes, five
    // and ten wavefronts, 29.8 and 39.3, 63 and 80). RMS, on the device.
    const bool wide = nch > 256 || (nch > 64 && p.rows < 1024);
    const dim3 grid((unsigned)(wide ? p.rows : (p.rows + kWaves - 1) / kWaves));
#define FP8_NORM_CASE(C, W) \
    hipLaunchKernelGGL((k_norm_quant_row<F, C, W, LOOSE, ADD>), grid, dim3(W == 1 ? kBlock : W * 64), 0, st, p)
    if (wide) {
        if (nch <= 256) FP8_NORM_CASE(1, 4);
        else if (nch <= 384) FP8_NORM_CASE(2, 3);
        else if (nch <= 512) FP8_NORM_CASE(2, 4);
        else if (nch <= 768) FP8_NORM_CASE(4, 3);
        else if (nch <= 1024) FP8_NORM_CASE(4, 4);
        else if (nch <= 1280) FP8_NORM_CASE(4, 5);
        else if (nch <= 1536) FP8_NORM_CASE(4, 6);
        else FP8_NORM_CASE(4, 8);
    } else {
        if (nch <= 64) FP8_NORM_CASE(1, 1);
        else if (nch <= 128) FP8_NORM_CASE(2, 1);
        else FP8_NORM_CASE(4, 1);
    }
#undef FP8_NORM_CASE
    return hipGetLastError();
}

template <int F, bool ADD>
hipError_t norm_quant_add(const NormFwd& p, hipStream_t st) {
    if (norm_vector_layout(p)) return norm_quant_reg<F, false, ADD>(p, st);
    if (p.cols >= 8 && p.cols <= kNormMaxVecCols) return norm_quant_reg<F, true, ADD>(p, st);
    hipLaunchKernelGGL((k_norm_quant_row_any<F, ADD>), dim3((unsigned)p.rows), dim3(kBlock), 0, st, p);
    return hipGetLastError();
}

template <int F>
hipError_t norm_quant_fmt(const NormFwd& p, hipStream_t st) {
    return p.res ? norm_quant_add<F, true>(p, st) : norm_quant_add<F, false>(p, st);
}

hipError_t launch_norm_quant_row(const NormFwd& p0, int fmt, hipStream_t st) {
    for (int64_t r0 = 0; r0 < p0.rows; r0 += kLaunchRows) {
        NormFwd p = p0;
        p.rows = p0.rows - r0 < kLaunchRows ? p0.rows - r0 : kLaunchRows;
        p.x += r0 * p.ldx;
        if (p.res) {
            p.res += r0 * p.ldres;
            p.sum += r0 * p.ldsum;
        }
        if (p.q) p.q += r0 * p.ldq;
        if (p.scale_inv) p.scale_inv += r0;
        if (p.y) p.y += r0 * p.ldy;
        if (p.mean) p.mean += r0;
        if (p.rstd) p.rstd += r0;
        if (p.xq) {
            p.xq += r0 * p.ldxq;
            p.xs += 4 * r0;
        }
        hipError_t e;
        switch (fmt) {
            case kE4M3: e = norm_quant_fmt<kE4M3>(p, st); break;
            case kE5M2: e = norm_quant_fmt<kE5M2>(p, st); break;
            case kE4M3Fnuz: e = norm_quant_fmt<kE4M3Fnuz>(p, st); break;
            default: e = norm_quant_fmt<kE5M2Fnuz>(p, st); break;
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int SRC, bool LOOSE, bool ADD>
hipError_t norm_grad_add(NormBwd p, hipStream_t st) {
    const int64_t nch = (p.cols + 7) / 8;
    // 16 wavefronts a CU either way: as one workgroup they leave half as many
    // partial sums (8192 x 4096: 42.4 us with 1024 threads, 44.8 with 512), as two
    // they spread few rows wider (300 x 4096: 10.5 and 9.2 us) and need fewer
    // rounds to add up narrow teams (16384 x 1024: 28.1 and 26.5 us).
    const bool tall = p.rows >= 2048 && nch > 256;
    const int tpr = nch <= 128 ? 64 : (nch <= 256 ? 128 : (nch <= 512 ? 256 : (nch <= 1024 ? 512 : 1024)));
    const int wg = tall || tpr == 1024 ? 1024 : 512;
    const int64_t teams = wg / tpr, max_bands = wg == 512 ? kNormMaxBands : kNormMaxBands / 2;
    // bands of as many rows, to one (2050 x 7168 in bands of 10 left 51 CUs without
    // one: 30.5 us, in bands of 8 and 9 27.1)
    p.bands = (p.rows + teams - 1) / teams;
    if (p.bands > max_bands) p.bands = max_bands;
    p.band = p.rows / p.bands;
    p.longer = p.rows % p.bands;
    const dim3 grid((unsigned)p.bands);
#define FP8_NORM_CASE(T, C, W) hipLaunchKernelGGL((k_norm_grad<SRC, T, C, W, LOOSE, ADD>), grid, dim3(W), 0, st, p)
    if (nch <= 64) FP8_NORM_CASE(64, 1, 512);
    else if (nch <= 128) FP8_NORM_CASE(64, 2, 512);
    else if (nch <= 256) FP8_NORM_CASE(128, 2, 512);
    else if (nch <= 512 && !tall) FP8_NORM_CASE(256, 2, 512);
    else if (nch <= 512) FP8_NORM_CASE(256, 2, 1024);
    else if (nch <= 1024 && !tall) FP8_NORM_CASE(512, 2, 512);
    else if (nch <= 1024) FP8_NORM_CASE(512, 2, 1024);
    else FP8_NORM_CASE(1024, 2, 1024);
#undef FP8_NORM_CASE
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && (p.dgamma || p.dbeta) && p.bands > 1) {
        hipLaunchKernelGGL(k_norm_weight_grad, dim3((unsigned)((p.cols + kSliceCols - 1) / kSliceCols), 2),
                           dim3(kSliceCols * kSlices), 0, st, p.partial, p.bands, p.cols, p.dgamma, p.dbeta);
        e = hipGetLastError();
    }
    return e;
}

template <int SRC, bool LOOSE>
hipError_t norm_grad_src(const NormBwd& p, hipStream_t st) {
    return p.ds ? norm_grad_add<SRC, LOOSE, true>(p, st) : norm_grad_add<SRC, LOOSE, false>(p, st);
}

hipError_t launch_norm_backward(const NormBwd& p0, hipStream_t st) {
    NormBwd p = p0;
    hipError_t e = hipSuccess;
    if (p.cols == 0) return e;
    if (p.rows == 0) {                                      // empty sums
        if (p.dgamma) e = launch_fill(p.dgamma, p.cols, 0.0f, st);
        if (p.dbeta && e == hipSuccess) e = launch_fill(p.dbeta, p.cols, 0.0f, st);
        return e;
    }
    if (p.xq) return p.ckpt_e5m2 ? norm_grad_src<2, false>(p, st) : norm_grad_src<1, false>(p, st);
    if (norm_vector_layout(p)) return norm_grad_src<0, false>(p, st);
    if (p.cols >= 8 && p.cols <= kNormMaxVecCols) return norm_grad_src<0, true>(p, st);
    hipLaunchKernelGGL(k_norm_grad_row_any, dim3(row_grid(p.rows)), dim3(kBlock), 0, st, p);
    e = hipGetLastError();
    if (e != hipSuccess || (!p.dgamma && !p.dbeta)) return e;
    // one band up to 1024 rows (32 a thread); beyond, bands of as many rows until
    // they are kNormMaxBands
    p.band = (p.rows + kNormMaxBands - 1) / kNormMaxBands;
    if (p.band < kAnySlices * 32) p.band = kAnySlices * 32;
    p.bands = (p.rows + p.band - 1) / p.band;
    const ColsGrid grid = any_cols_grid(p.cols);
    hipLaunchKernelGGL(k_norm_grad_cols_any, dim3(grid.x, (unsigned)p.bands, grid.z), dim3(kAnyCols * kAnySlices), 0, st,
                       p);
    e = hipGetLastError();
    if (e == hipSuccess && p.bands > 1) {
        hipLaunchKernelGGL(k_norm_weight_grad, dim3((unsigned)((p.cols + kSliceCols - 1) / kSliceCols), 2),
                           dim3(kSliceCols * kSlices), 0, st, p.partial, p.bands, p.cols, p.dgamma, p.dbeta);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace fp8amax
