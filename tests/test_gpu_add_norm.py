"""GPU parity of the residual's addition with the norm and the rowwise cast, and of
its gradient, from the sum and from the 8-bit checkpoint, against the fp64
definitions of oracle/layer.py. The sum itself is exact to the bit (fp32, rounded
once); everything after it is the norm's of the stored sum. Sizes where the kernels
change their path, views with guard bands, the sum in an input's place, special rows."""
import numpy as np
import pytest
import torch

import workloads
from helpers import check_guard, dev_bf16, guarded, host_bits, say
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = layer.BF16


@pytest.fixture(scope="module")
def fp8():
    import fp8_scaled_gemm_amax_amd as m
    return m


def make(rng, rows, cols):
    """bf16 bits of x and of a residual of other sizes, and of their sum."""
    x = workloads.bf16_bits((rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-8, 4, (rows, cols)))).astype(np.float32))
    r = workloads.bf16_bits((rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-6, 7, (rows, 1)))
                             + rng.standard_normal((rows, 1))).astype(np.float32))
    s = workloads.bf16_bits((layer.values(x) + layer.values(r)).astype(np.float32))
    return x, r, s


def make_weights(rng, cols, kind):
    if kind == "none":
        return None, None
    v = (1 + 0.5 * rng.standard_normal(cols)).astype(np.float32)
    if kind == "f32":
        return torch.from_numpy(v).to(DEV), v.astype(np.float64)
    b = workloads.bf16_bits(v)
    return dev_bf16(b), layer.values(b)


def within(got, want, tol, what, rel=0.0):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - want) <= tol + rel * np.abs(want))
    assert not bad.any(), (f"{what}: {int(bad.sum())} values off, first {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]!r} for {want[bad][0]!r}")


def bf16_of(t):
    return layer.values(host_bits(t))


FORWARD = [  # rows, cols, rms, weights, fmt, where the sum goes
    (1, 8, False, "bf16", 0, "out"), (1, 4096, True, "bf16", 0, "res"), (5, 520, False, "f32", 1, "x"),
    (1030, 512, True, "f32", 0, "res"), (1025, 1000, False, "bf16", 2, "out"), (1024, 2048, False, "none", 3, "res"),
    (9, 2056, True, "none", 0, "out"), (33, 7168, True, "bf16", 0, "res"), (3, 16384, False, "bf16", 1, "x"),
    (4, 1, False, "bf16", 0, "res"), (7, 1111, False, "bf16", 0, "res"), (3, 20000, True, "f32", 1, "res"),
    (2, 17, True, "none", 3, "x"), (1030, 1021, False, "f32", 0, "out"), (2, 16383, True, "bf16", 0, "res"),
    (6, 2880, False, "bf16", 0, "out"), (5, 4104, False, "bf16", 0, "res"), (3, 8224, True, "none", 0, "out"),
    (2, 10240, True, "bf16", 2, "res"), (2, 12256, False, "bf16", 0, "out"), (5, 7, True, "none", 0, "out"),
    (2, 20003, False, "bf16", 0, "x"),
]


@pytest.mark.parametrize("rows,cols,rms,wk,fmt,where", FORWARD)
def test_forward(fp8, rows, cols, rms, wk, fmt, where):
    rng = np.random.default_rng(rows * 7 + cols)
    xb, rb, sb = make(rng, rows, cols)
    gamma, gv = make_weights(rng, cols, wk)
    beta, bv = (None, None) if rms else make_weights(rng, cols, wk)
    f = layer.norm_forward(layer.values(sb), gv, bv, np.float64(np.float32(1e-5)), rms)
    save = cols % 32 == 0 and cols <= 16384
    pad = 32 if cols % 8 == 0 else 3
    q, qbuf, qo = guarded(rows, cols, torch.uint8, ld=cols + pad)
    y, ybuf, yo = guarded(rows, cols, torch.bfloat16, ld=cols + pad)
    s, sbuf, so = guarded(rows, cols, torch.bfloat16, ld=cols + pad)
    x, res = dev_bf16(xb), dev_bf16(rb)
    if where != "out":
        s.copy_(res if where == "res" else x)
    x, res = (s if where == "x" else x), (s if where == "res" else res)
    si, mean, rstd = (torch.full((rows,), -7.0, device=DEV) for _ in range(3))
    xq = xs = None
    if save:
        xq, xqbuf, xqo = guarded(rows, cols, torch.uint8, ld=cols + 32)
        xs = fp8.mx_scale_records(rows, cols)
    ck = 1 if fmt == 1 else 0
    say("add norm", rows, cols, rms, wk, fmt, where)
    fp8.fp8_add_norm_quantize_row(x, res, s, gamma, beta, 1e-5, fp8.NORM_RMS if rms else fp8.NORM_LAYER, fmt, 0, q, si,
                                  y=y, mean_out=mean, rstd_out=rstd, xhat_q=xq, xhat_fmt=ck, xhat_scale=xs)
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(s), sb), "the sum is bf16(x + res)"
    within(mean.cpu().numpy(), f["mean"], f["mean_tol"], "mean")
    within(rstd.cpu().numpy(), f["rstd"], 0, "rstd", rel=f["rstd_rel"])
    within(bf16_of(y), f["y"], f["y_tol"] * (1 + BF), "y", rel=BF)
    layer.cast_ok(fmt, q.cpu().numpy(), si.cpu().numpy(), f["y"], f["y_tol"])
    for buf, o in ((qbuf, qo), (ybuf, yo), (sbuf, so)):
        check_guard(buf, o, rows, cols)
    if save:
        check_guard(xqbuf, xqo, rows, cols)
        layer.checkpoint_ok(ck, xq.cpu().numpy(), layer.from_records(xs.cpu().numpy(), cols), f["xhat"], f["xhat_tol"])


@pytest.mark.parametrize("rows,cols", [(70, 4096), (1200, 512), (9, 1111), (3, 20000)])
def test_forward_is_the_norm_of_the_sum(fp8, rows, cols):
    """Bit for bit what fp8_norm_quantize_row gives for the stored sum."""
    rng = np.random.default_rng(cols)
    xb, rb, _ = make(rng, rows, cols)
    gamma, _ = make_weights(rng, cols, "bf16")
    x, r = dev_bf16(xb), dev_bf16(rb)
    s = torch.empty_like(x)

    def outs():
        return (torch.zeros((rows, cols), dtype=torch.uint8, device=DEV), torch.zeros(rows, device=DEV),
                torch.zeros_like(x), torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV))

    a, b = outs(), outs()
    say("add norm against the norm", rows, cols)
    fp8.fp8_add_norm_quantize_row(x, r, s, gamma, gamma, 1e-6, 0, 0, 1, a[0], a[1], y=a[2], mean_out=a[3], rstd_out=a[4])
    fp8.fp8_norm_quantize_row(s, gamma, gamma, 1e-6, 0, 0, 1, b[0], b[1], y=b[2], mean_out=b[3], rstd_out=b[4])
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_forward_special_rows(fp8):
    """Inf - Inf and an overflowing sum in a row reach that row alone; x = -res gives a
    row of zeros."""
    rng = np.random.default_rng(1)
    xb, rb, _ = make(rng, 6, 256)
    x, r = dev_bf16(xb), dev_bf16(rb)
    q0, si0 = torch.zeros((6, 256), dtype=torch.uint8, device=DEV), torch.zeros(6, device=DEV)
    q1, si1 = torch.zeros_like(q0), torch.zeros_like(si0)
    s = torch.empty_like(x)
    say("add norm, special rows")
    fp8.fp8_add_norm_quantize_row(x, r, s, None, None, 1e-5, 1, 0, 0, q0, si0)
    x[1, 3], r[1, 3] = float("inf"), float("-inf")
    x[2, 4] = r[2, 4] = 3.3e38
    x[3] = -r[3]
    fp8.fp8_add_norm_quantize_row(x, r, s, None, None, 1e-5, 1, 0, 0, q1, si1)
    torch.cuda.synchronize()
    for i in (0, 4, 5):
        assert torch.equal(q0[i], q1[i]) and si0[i] == si1[i]
    assert torch.isnan(s[1, 3]) and torch.isinf(s[2, 4]) and not s[3].any()
    assert (q1[1] & 0x7F == 0x7F).all() and si1[1] == 1.0
    assert not (q1[3] & 0x7F).any() and si1[3] == 1.0


BACKWARD = [  # rows, cols, rms, gamma, dx in dsum's place
    (1, 8, False, "bf16", False), (1, 512, True, "none", True), (3, 520, False, "f32", False), (700, 1024, False, "bf16", True),
    (65, 2048, True, "bf16", False), (1100, 2056, False, "none", True), (40, 4096, False, "f32", False),
    (515, 7168, True, "bf16", True), (5, 8200, False, "bf16", False), (300, 16384, True, "f32", True),
    (333, 1111, False, "bf16", True), (2, 1, False, "none", False), (1, 20000, False, "bf16", True), (70, 33, True, "f32", True),
    (2100, 2051, True, "bf16", False), (3, 16381, False, "f32", True), (2050, 4096, False, "bf16", True),
    (1100, 16392, True, "bf16", False),
]


@pytest.mark.parametrize("rows,cols,rms,gk,in_place", BACKWARD)
def test_backward_from_the_sum(fp8, rows, cols, rms, gk, in_place):
    rng = np.random.default_rng(rows + cols * 3)
    _, _, sb = make(rng, rows, cols)
    dyb = workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32) * 1e-3)
    dsb = workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32) * 1e-3)
    gamma, gv = make_weights(rng, cols, gk)
    x = layer.values(sb)
    f = layer.norm_forward(x, None, None, 1e-5, rms)
    mean, rstd = f["mean"].astype(np.float32), f["rstd"].astype(np.float32)
    xhat = (x - (0 if rms else mean.astype(np.float64)[:, None])) * rstd.astype(np.float64)[:, None]
    want = layer.norm_backward(layer.values(dyb), xhat, gv, rstd.astype(np.float64), rms, xhat_rel=2 * layer.U)
    dsum = layer.values(dsb)
    dx_want = dsum + want["dx"]
    dx_tol = want["dx_tol"] + layer.U * (np.abs(dx_want) + want["dx_tol"])
    pad = 32 if cols % 8 == 0 else 5
    dx, buf, o = guarded(rows, cols, torch.bfloat16, ld=cols + pad)
    ds = dev_bf16(dsb)
    if in_place:
        dx.copy_(ds)
        ds = dx
    dg, db = torch.full((cols,), 9.0, device=DEV), torch.full((cols,), 9.0, device=DEV)
    say("add norm backward", rows, cols, rms, gk, in_place)
    args = (dev_bf16(dyb), dev_bf16(sb), gamma, None if rms else torch.from_numpy(mean).to(DEV),
            torch.from_numpy(rstd).to(DEV), fp8.NORM_RMS if rms else fp8.NORM_LAYER)
    ws = fp8.norm_workspace(rows, cols)
    fp8.fp8_add_norm_backward(ds, *args, dx, dgamma=dg, dbeta=db, workspace=ws)
    torch.cuda.synchronize()
    within(bf16_of(dx), dx_want, dx_tol * (1 + BF), "dx", rel=BF)
    within(dg.cpu().numpy(), want["dgamma"], want["dgamma_tol"], "dgamma")
    within(db.cpu().numpy(), want["dbeta"], want["dbeta_tol"], "dbeta")
    check_guard(buf, o, rows, cols)
    # the weights' gradients are the norm's own, bit for bit
    other, dg2, db2 = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV), torch.empty_like(dg), torch.empty_like(db)
    fp8.fp8_norm_backward(*args, other, dgamma=dg2, dbeta=db2, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(dg, dg2) and torch.equal(db, db2)


SAVED = [(1, 32, True, 0, False, False), (3, 544, False, 1, True, True), (1030, 1024, True, 0, True, False),
         (67, 2048, False, 0, True, True), (40, 4096, True, 1, False, True), (515, 7168, False, 0, True, False),
         (9, 16384, False, 0, True, True), (2050, 7168, True, 0, True, True)]


@pytest.mark.parametrize("rows,cols,rms,fmt,with_y,in_place", SAVED)
def test_backward_from_checkpoint(fp8, orc, rows, cols, rms, fmt, with_y, in_place):
    rng = np.random.default_rng(rows + cols * 5)
    xhb = workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32))
    codes, e8 = orc.mx_quantize_row(xhb, fmt)
    xhat = layer.mx_values(codes, fmt, e8)
    dyb = workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32) * 1e-3)
    dsb = workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32) * 1e-3)
    gamma, gv = make_weights(rng, cols, "bf16")
    beta, bv = make_weights(rng, cols, "bf16")
    rstd = (0.5 + rng.random(rows)).astype(np.float32)
    want = layer.norm_backward(layer.values(dyb), xhat, gv, rstd.astype(np.float64), rms)
    dx_want = layer.values(dsb) + want["dx"]
    dx_tol = want["dx_tol"] + layer.U * (np.abs(dx_want) + want["dx_tol"])
    J = (cols + 127) // 128
    rec = torch.zeros((J, rows + 3, 4), dtype=torch.uint8, device=DEV)
    pad = np.zeros((rows, J * 4), np.uint8)
    pad[:, :cols // 32] = e8
    rec[:, :rows] = torch.from_numpy(np.ascontiguousarray(pad.reshape(rows, J, 4).transpose(1, 0, 2))).to(DEV)
    xq = torch.from_numpy(codes).to(DEV)
    dx, buf, o = guarded(rows, cols, torch.bfloat16)
    ds = dev_bf16(dsb)
    if in_place:
        dx.copy_(ds)
        ds = dx
    y, ybuf, yo = guarded(rows, cols, torch.bfloat16)
    dg, db = torch.full((cols,), 9.0, device=DEV), torch.full((cols,), 9.0, device=DEV)
    say("add norm backward from checkpoint", rows, cols, rms, fmt, with_y, in_place)
    fp8.fp8_mx_add_norm_backward(ds, dev_bf16(dyb), xq, fmt, rec[:, :rows], gamma, beta, torch.from_numpy(rstd).to(DEV),
                                 fp8.NORM_RMS if rms else fp8.NORM_LAYER, dx, dgamma=dg, dbeta=db,
                                 y=y if with_y else None, workspace=fp8.norm_workspace(rows, cols))
    torch.cuda.synchronize()
    within(bf16_of(dx), dx_want, dx_tol * (1 + BF), "dx", rel=BF)
    within(dg.cpu().numpy(), want["dgamma"], want["dgamma_tol"], "dgamma")
    within(db.cpu().numpy(), want["dbeta"], want["dbeta_tol"], "dbeta")
    check_guard(buf, o, rows, cols)
    if with_y:
        v = xhat * gv + bv
        within(bf16_of(y), v, 2 * layer.U * (np.abs(xhat * gv) + np.abs(v)), "y", rel=BF)
        check_guard(ybuf, yo, rows, cols)


def test_no_rows(fp8):
    say("add norm, no rows")
    x = torch.empty((0, 96), dtype=torch.bfloat16, device=DEV)
    q = torch.empty((0, 96), dtype=torch.uint8, device=DEV)
    z = torch.empty(0, device=DEV)
    fp8.fp8_add_norm_quantize_row(x, x, x, None, None, 0.0, fp8.NORM_LAYER, 0, 0, q, z, xhat_q=q,
                                  xhat_scale=fp8.mx_scale_records(0, 96))
    dg, db = torch.ones(96, device=DEV), torch.ones(96, device=DEV)
    fp8.fp8_add_norm_backward(x, x, x, None, z, z, fp8.NORM_LAYER, x, dgamma=dg, dbeta=db)
    torch.cuda.synchronize()
    assert not dg.any() and not db.any()
