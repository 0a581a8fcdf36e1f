"""Definitions, in numpy fp64, of a feed-forward block's operators: the gated FP8
product and its gradient, adapters. Test infrastructure only, independent of the
HIP path. As in oracle/layer.py, each gives the exact values and how far fp32
arithmetic of the same formula may end from them.

A matrix-core sum of n products in fp32, in any order, each addition rounded or
cut to 24 bits: off by at most 2 n U times the sum of the magnitudes (U = 2^-24)."""
import numpy as np

from . import oracle as orc
from .layer import BF16, TINY, U, sigmoid, values  # noqa: F401


def codes(rng, rows, cols, fmt, std=1.0):
    """Random codes of an FP8 operand (a rowwise cast) and its factors."""
    x = (rng.standard_normal((rows, cols)) * std * np.exp2(rng.integers(-2, 3, (rows, 1)))).astype(np.float32)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    q, s, _ = orc.quantize_row(bits, fmt)
    return q, s


def product(qa, fa, sa, qb, fb, sb):
    """(a b^T) sa sb in fp64, and the bound of its fp32 evaluation."""
    a, b = (np.asarray(orc.decode(f, q), np.float64).reshape(q.shape) for f, q in ((fa, qa), (fb, qb)))
    sa, sb = np.asarray(sa, np.float64).reshape(-1, 1), np.asarray(sb, np.float64).reshape(1, -1)
    k = a.shape[1]
    y = a @ b.T * sa * sb
    mag = np.abs(a) @ np.abs(b).T * sa * sb
    return y, 2 * (k + 2) * U * mag + 2 * U * np.abs(y)


def exp_rel(g):
    """t = exp(-g) in fp32 as 2^n exp(e): the exponential 2 U, 1 + e and its product with it
    2 U, the constant of n ln 2 off by 1.9e-9: |n| 1.9e-9 < |g| U / 16."""
    return (4 + np.abs(g) / 16) * U


def sigma_rel(g):
    """sigma(g) = 1 / (1 + t): t's error in the share that t has of the sum, the sum U, the
    reciprocal 2 U."""
    return exp_rel(g) * sigmoid(-g) + 3 * U


def swiglu(g, u, g_tol, u_tol):
    """silu(g) u and its bound, g and u known to g_tol and u_tol (|silu'| <= 1.1)."""
    a = g * sigmoid(g) * u
    tol = 1.1 * np.abs(u) * g_tol + np.abs(g * sigmoid(g)) * u_tol + 1.1 * g_tol * u_tol
    return a, tol + np.abs(a) * (sigma_rel(g) + 3 * U) + (np.abs(g * u) + 1) * TINY


def swiglu_backward(da, g, u, da_tol):
    """dict of dg, du, a and their bounds, da known to da_tol, g and u exact."""
    s, c = sigmoid(g), sigmoid(-g)
    silu = g * s
    f = s * (1 + g * c)
    rel = sigma_rel(g)
    c_tol = c * (exp_rel(g) * s + 4 * U)        # 1 - sigma = t sigma: what t's error leaves, sigma's other 3 U, the product
    f_tol = np.abs(f) * (rel + 2 * U) + s * (np.abs(g) * c_tol + U * (1 + np.abs(g * c)))
    dg, du, a = da * u * f, da * silu, silu * u
    far = np.abs(da) + da_tol
    tiny = TINY * (1 + far) * (1 + np.abs(g)) ** 2 * (1 + np.abs(u))
    return dict(dg=dg, du=du, a=a,
                dg_tol=np.abs(u) * (np.abs(f) * da_tol + far * f_tol) + 4 * U * np.abs(dg) + tiny,
                du_tol=np.abs(silu) * da_tol + far * np.abs(silu) * (rel + 3 * U) + tiny,
                a_tol=np.abs(a) * (rel + 3 * U) + tiny)


def lora(x, a, b, scaling, idx, base):
    """base + scaling_e (x A_e^T) B_e^T and its bound: v = x A^T as a matrix-core sum
    (and up to 16 parts and 4 wavefronts added), v times the factor rounded to fp32, the
    second product as two sums, of up to 2 r products."""
    out = base.copy()
    tol = np.zeros_like(out)
    K, r = x.shape[1], a.shape[1]
    for e in range(a.shape[0]):
        t = np.nonzero(idx == e)[0]
        if t.size == 0:
            continue
        c = float(scaling[e])
        v = x[t] @ a[e].T
        v_tol = 2 * (K + 20) * U * (np.abs(x[t]) @ np.abs(a[e]).T)
        out[t] += c * (v @ b[e].T)
        w_tol = abs(c) * (v_tol + np.abs(v) * 2 * U)
        tol[t] = w_tol @ np.abs(b[e]).T + 2 * (2 * r + 4) * U * ((abs(c) * np.abs(v) + w_tol) @ np.abs(b[e]).T)
        tol[t] += 2 * U * (np.abs(base[t]) + np.abs(out[t]))
    return out, tol
