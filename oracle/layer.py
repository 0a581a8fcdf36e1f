"""Definitions, in numpy fp64, of the layer around the FP8 products: norm and its
gradient, SwiGLU's gradient, MX checkpoints, the MoE layer for a few tokens.
Test infrastructure only, independent of the HIP path. Every function that a
GPU result is compared with returns the exact values and, where the kernels
compute in fp32, how far fp32 arithmetic of the same formula may end from them
(worst-case bounds of the standard rounding analysis: a sum of n terms in any
order is off by at most n u times the sum of their magnitudes, u = 2^-24)."""
import numpy as np

from . import oracle as orc

U = 2.0 ** -24
BF16 = 2.0 ** -8                # half a step of bf16 relative to the value


def values(bits):
    """bf16 bit patterns -> fp64."""
    return orc.bf16_to_f64(bits)


def norm_forward(x, gamma, beta, eps, rms):
    """x fp64 [rows x cols]; gamma, beta fp64 [cols] or None. Returns dict of mean,
    rstd, xhat, y and the bounds mean_tol, rstd_tol (relative), xhat_tol, y_tol."""
    n = x.shape[1]
    mu = np.zeros(x.shape[0]) if rms else x.sum(1) / n
    d = x - mu[:, None]
    v = (d * d).sum(1) / n
    rstd = 1.0 / np.sqrt(v + eps)
    xhat = d * rstd[:, None]
    g = np.ones(n) if gamma is None else gamma
    b = np.zeros(n) if beta is None else beta
    y = xhat * g + b
    mean_tol = np.zeros(len(mu)) if rms else (n + 2) * U * np.abs(x).sum(1) / n
    # sum of d^2: each d off by mean_tol + U |d|, n additions, the products, eps added
    dtol = mean_tol[:, None] + U * np.abs(d)
    vtol = ((2 * np.abs(d) + dtol) * dtol).sum(1) / n + (n + 4) * U * v + U * (v + eps)
    rstd_rel = 0.5 * vtol / (v + eps) * (1 + vtol / (v + eps)) + 3 * U
    xhat_tol = rstd[:, None] * dtol * (1 + rstd_rel[:, None]) + np.abs(xhat) * (rstd_rel[:, None] + 2 * U)
    y_tol = np.abs(g) * xhat_tol + 2 * U * (np.abs(xhat * g) + np.abs(y) + np.abs(b))
    return dict(mean=mu, rstd=rstd, xhat=xhat, y=y, mean_tol=mean_tol, rstd_rel=rstd_rel, xhat_tol=xhat_tol,
                y_tol=y_tol)


def norm_backward(dy, xhat, gamma, rstd, rms, xhat_rel=0.0):
    """dy, xhat fp64 [rows x cols], rstd [rows]. xhat_rel: how far (relative) the
    kernel's own xhat is. Returns dict of dx, dgamma, dbeta and dx_tol (fp32
    arithmetic alone, without the output's rounding), dgamma_tol, dbeta_tol."""
    rows, n = dy.shape
    g = np.ones(n) if gamma is None else gamma
    w = dy * g
    c1 = (w * xhat).sum(1, keepdims=True) / n
    c2 = np.zeros((rows, 1)) if rms else w.sum(1, keepdims=True) / n
    dx = rstd[:, None] * (w - c2 - xhat * c1)
    c1_tol = ((n + 5) * U + xhat_rel) * np.abs(w * xhat).sum(1, keepdims=True) / n
    c2_tol = 0.0 if rms else (n + 4) * U * np.abs(w).sum(1, keepdims=True) / n
    terms = np.abs(w) + np.abs(c2) + np.abs(xhat * c1)
    dx_tol = rstd[:, None] * (np.abs(xhat) * c1_tol * (1 + xhat_rel) + c2_tol + np.abs(xhat * c1) * xhat_rel +
                              6 * U * terms)
    dgamma_tol = ((rows + 2) * U + xhat_rel) * np.abs(dy * xhat).sum(0)
    dbeta_tol = (rows + 1) * U * np.abs(dy).sum(0)
    return dict(dx=dx, dgamma=(dy * xhat).sum(0), dbeta=dy.sum(0), dx_tol=dx_tol, dgamma_tol=dgamma_tol,
                dbeta_tol=dbeta_tol)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


# fp32 evaluation of sigma(g) from t = exp(-|g|): t is off by at most 4 U (the
# exponent's product and its correction, the hardware exponential, one fma),
# 1 + t by U, the reciprocal after a Newton step by 2 U, the product by U.
SIGMOID_REL = 8 * U
# exp(-|g|) below the smallest normal number counts as zero.
TINY = 2.0 ** -126


def swiglu(g, u):
    """a = silu(g) u and how far an fp32 evaluation may be."""
    a = g * sigmoid(g) * u
    return a, (SIGMOID_REL + 2 * U) * np.abs(a) + np.abs(g * u) * TINY + TINY


def swiglu_backward(da, g, u):
    """dict of dg, du, a and their bounds (fp32 arithmetic, without the outputs' rounding)."""
    s = sigmoid(g)
    c = sigmoid(-g)
    silu = g * s
    dg = da * u * (s + silu * c)
    du = da * silu
    small = np.abs(g) * TINY
    # s + silu c: fma of factors off by SIGMOID_REL each and the product by U
    inner = np.abs(s) * SIGMOID_REL + np.abs(silu * c) * (2 * SIGMOID_REL + 2 * U) + U * np.abs(s + silu * c)
    return dict(dg=dg, du=du, a=silu * u,
                dg_tol=np.abs(da * u) * (inner + 2 * small + TINY) + 2 * U * np.abs(dg) + TINY,
                du_tol=np.abs(da) * (np.abs(silu) * (SIGMOID_REL + 2 * U) + small) + TINY,
                a_tol=np.abs(u) * (np.abs(silu) * (SIGMOID_REL + 2 * U) + small) + TINY)


def mx_values(codes, fmt, e8m0):
    """Values an MX checkpoint holds: codes [rows x cols], bytes [rows x cols / 32]."""
    s = orc.mx_scale_values(np.asarray(e8m0))
    return orc.decode(fmt, codes).astype(np.float64) * np.repeat(s, 32, axis=1)


def from_records(records, cols):
    """Scale records [J x rows x 4] -> bytes [rows x cols / 32]."""
    r = np.asarray(records, np.uint8)
    return r.transpose(1, 0, 2).reshape(r.shape[1], -1)[:, : cols // 32]


def half_step(fmt, v):
    """Half the distance of the format's neighbours around |v| (v within its range)."""
    fmax, _, mbits, bias = orc.fmt_info(fmt)
    mag = np.minimum(np.abs(v), fmax)
    e = np.maximum(np.floor(np.log2(np.maximum(mag, 1e-300))), 1 - bias)
    return 0.5 * np.exp2(e - mbits)


def codes_round(fmt, codes, v, tol):
    """Boolean array: code is the rounding (saturating) of some value within tol of
    v. A value that tol carries into the next binade is still off by no more
    than half the step of v's own binade plus tol."""
    fmax = orc.fmt_info(fmt)[0]
    dec = orc.decode(fmt, codes).astype(np.float64)
    err = np.abs(dec - np.clip(v, -fmax, fmax))
    with np.errstate(invalid="ignore"):
        ok = err <= half_step(fmt, v) * (1 + 1e-12) + tol
    return ok | (np.isnan(v) & np.isnan(dec))


def cast_ok(fmt, codes, scale_inv, y, y_tol, margin=0):
    """Checks a rowwise cast of fp32 values within y_tol of y: scale_inv against
    the rule, then every code against y / scale_inv. Rows with a NaN or Inf are
    the caller's."""
    fmax = orc.fmt_info(fmt)[0]
    amax = np.abs(y).max(1)
    at = np.abs(y).argmax(1)
    rel = np.array([y_tol[r, c] for r, c in enumerate(at)]) / np.maximum(amax, 1e-300)
    rel = np.maximum(rel, (np.abs(y) + y_tol).max(1) / np.maximum(amax, 1e-300) - 1)
    want = np.where(amax > 0, amax / fmax * 2.0 ** margin, 1.0)
    si = np.asarray(scale_inv, np.float64)
    assert np.all(np.abs(si - want) <= want * (rel + 3 * U)), "scale_inv"
    v = y / si[:, None]
    # the product with s = 1 / scale_inv: s, scale_inv and the product rounded
    ok = codes_round(fmt, codes, v, y_tol / si[:, None] + 4 * U * np.abs(v))
    assert ok.all(), f"{int((~ok).sum())} codes are no rounding of y * s; first {np.argwhere(~ok)[0]}"


def checkpoint_ok(fmt, codes, e8m0, v, tol):
    """Checks an MX checkpoint of fp32 values within tol of v: each byte the
    exponent rule's for an amax within tol, each code the cast with that byte."""
    rows, cols = v.shape
    emax = 8 if fmt == orc.E4M3 else 15
    b = np.abs(v).reshape(rows, cols // 32, 32)
    t = np.broadcast_to(tol, v.shape).reshape(b.shape)
    lo, hi = np.maximum(b - t, 0).max(2), (b + t).max(2)

    def byte(a):
        e = np.floor(np.log2(np.maximum(a, 2.0 ** -140))) - emax
        return np.clip(e, -127, 127) + 127

    e8 = np.asarray(e8m0, np.float64)
    ok = (e8 >= byte(lo)) & (e8 <= byte(hi))
    assert ok.all(), f"{int((~ok).sum())} scale bytes off the rule"
    s = np.repeat(np.exp2(e8 - 127), 32, axis=1)
    ok = codes_round(fmt, codes, v / s, tol / s + U * np.abs(v / s))
    assert ok.all(), f"{int((~ok).sum())} checkpoint codes are no rounding"


def moe_few(x, idx, weights, w1, w2, w1_abs=None, w2_abs=None):
    """x [T x H], idx, weights [T x k], w1 [E x 2I x H], w2 [E x H x I] (dequantised,
    fp64). Returns out [T x H] and how far the kernels may be before the output's
    rounding: fp32 sums (products of the matrix cores may be added with
    truncation, so 2 U an addition), a kept to 16 bits."""
    T, k = idx.shape
    E, I2, H = w1.shape
    inter = I2 // 2
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    mag = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if not 0 <= e < E:
                continue
            h = w1[e] @ x[t]
            ht = 2 * (H + 8) * U * (np.abs(w1[e]) @ np.abs(x[t]))
            g, u = h[:inter], h[inter:]
            gt, ut = ht[:inter], ht[inter:]
            a, at = swiglu(g, u)
            # |silu'| <= 1.1
            at = at + 1.1 * gt * (np.abs(u) + ut) + np.abs(g * sigmoid(g)) * ut
            w = float(weights[t, j])
            a, at = w * a, abs(w) * at + (2.0 ** -16 + 2 * U) * abs(w) * np.abs(a)
            out[t] += w2[e] @ a
            tol[t] += np.abs(w2[e]) @ at
            mag[t] += np.abs(w2[e]) @ np.abs(a)
    return out, tol + 2 * (inter * k + 16) * U * mag
