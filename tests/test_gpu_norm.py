"""GPU parity of the norm with the rowwise cast and of its gradient, from x and
from the 8-bit checkpoint, against the fp64 definitions of oracle/layer.py:
every output within fp32 rounding of the formula (the bounds are worked out
there) plus half a step of its own type. Sizes where the kernels change their
path (one and four wavefronts a row, 1 to 8 chunks a lane, teams of 64 to 1024
threads, the scalar path), views with guard bands, special rows."""
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


def make_x(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-6, 7, (rows, 1))) + rng.standard_normal((rows, 1))
    return workloads.bf16_bits(x.astype(np.float32))


def make_weights(rng, cols, kind):
    """(device tensor or None, fp64 values or None) for kind "none", "bf16", "f32"."""
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


FORWARD = [  # rows, cols, rms, gamma, beta, fmt
    (1, 8, False, "bf16", "bf16", 0), (1, 4096, True, "bf16", "none", 0), (5, 520, False, "f32", "f32", 1),
    (1030, 512, True, "f32", "none", 0), (1025, 1000, False, "bf16", "bf16", 2), (1024, 2048, False, "none", "none", 3),
    (9, 2056, True, "none", "f32", 0), (33, 7168, True, "bf16", "none", 0), (3, 16384, False, "bf16", "bf16", 1),
    (4, 1, False, "bf16", "bf16", 0), (7, 1111, False, "bf16", "bf16", 0), (3, 20000, True, "f32", "none", 1),
    (2, 17, True, "none", "none", 3), (1030, 1021, False, "f32", "bf16", 0), (2, 16383, True, "bf16", "none", 0),
    (6, 2880, False, "bf16", "bf16", 0), (5, 4104, False, "bf16", "bf16", 0), (4, 6144, True, "f32", "none", 1),
    (3, 8224, False, "none", "bf16", 0), (2, 10240, True, "bf16", "none", 2), (2, 12256, False, "bf16", "bf16", 0),
    (2, 12320, True, "bf16", "none", 0), (3, 2999, False, "bf16", "bf16", 0), (2, 9001, True, "none", "none", 0),
    (2, 11003, False, "f32", "f32", 1),
]


@pytest.mark.parametrize("rows,cols,rms,gk,bk,fmt", FORWARD)
def test_norm_forward(fp8, rows, cols, rms, gk, bk, fmt):
    rng = np.random.default_rng(rows * 7 + cols)
    xb = make_x(rng, rows, cols)
    gamma, gv = make_weights(rng, cols, gk)
    beta, bv = make_weights(rng, cols, bk)
    if gamma is not None and beta is not None:
        beta = beta.to(gamma.dtype)
    eps = 1e-5
    f = layer.norm_forward(layer.values(xb), gv, bv, np.float64(np.float32(eps)), rms)
    save = cols % 32 == 0 and cols <= 16384
    pad = 32 if cols % 8 == 0 else 3
    q, qbuf, qo = guarded(rows, cols, torch.uint8, ld=cols + pad)
    y, ybuf, yo = guarded(rows, cols, torch.bfloat16, ld=cols + pad)
    si, mean, rstd = (torch.full((rows,), -7.0, device=DEV) for _ in range(3))
    xq = xs = None
    if save:
        xq, xqbuf, xqo = guarded(rows, cols, torch.uint8, ld=cols + 32)
        xs = fp8.mx_scale_records(rows, cols)
    ck = 1 if fmt == 1 else 0
    say("norm forward", rows, cols, rms, gk, bk, fmt)
    fp8.fp8_norm_quantize_row(dev_bf16(xb), gamma, beta, eps, fp8.NORM_RMS if rms else fp8.NORM_LAYER, fmt, 0, q, si,
                              y=y, mean_out=mean, rstd_out=rstd, xhat_q=xq, xhat_fmt=ck, xhat_scale=xs)
    torch.cuda.synchronize()
    within(mean.cpu().numpy(), f["mean"], f["mean_tol"], "mean")
    within(rstd.cpu().numpy(), f["rstd"], 0, "rstd", rel=f["rstd_rel"])
    within(bf16_of(y), f["y"], f["y_tol"] * (1 + BF), "y", rel=BF)
    layer.cast_ok(fmt, q.cpu().numpy(), si.cpu().numpy(), f["y"], f["y_tol"])
    check_guard(qbuf, qo, rows, cols)
    check_guard(ybuf, yo, rows, cols)
    if save:
        check_guard(xqbuf, xqo, rows, cols)
        rec = xs.cpu().numpy()
        layer.checkpoint_ok(ck, xq.cpu().numpy(), layer.from_records(rec, cols), f["xhat"], f["xhat_tol"])
        spare = rec.transpose(1, 0, 2).reshape(rows, -1)[:, cols // 32:]
        assert not spare.any(), "bytes of blocks past the row"


def test_norm_forward_outputs_are_optional(fp8):
    """q alone and y alone give what both together give; margin halves the scale; a
    strided x (rows of a wider tensor, an odd row stride) gives the same as a copy."""
    rng = np.random.default_rng(0)
    xb = make_x(rng, 40, 1024)
    x = dev_bf16(xb)
    gamma, _ = make_weights(rng, 1024, "bf16")
    say("norm optional outputs")

    def call(x, want_q, want_y, margin=0):
        q = torch.zeros((40, 1024), dtype=torch.uint8, device=DEV) if want_q else None
        si = torch.zeros(40, device=DEV) if want_q else None
        y = torch.zeros((40, 1024), dtype=torch.bfloat16, device=DEV) if want_y else None
        fp8.fp8_norm_quantize_row(x, gamma, None, 1e-6, fp8.NORM_RMS, 0, margin, q, si, y=y)
        torch.cuda.synchronize()
        return q, si, y

    q, si, y = call(x, True, True)
    q1, si1, _ = call(x, True, False)
    _, _, y1 = call(x, False, True)
    assert torch.equal(q, q1) and torch.equal(si, si1) and torch.equal(y, y1)
    _, si2, _ = call(x, True, False, margin=1)
    assert torch.equal(si2, si * 2)
    wide = torch.empty((40, 1024 + 64), dtype=torch.bfloat16, device=DEV)
    wide[:, 64:] = x
    assert all(torch.equal(a, b) for a, b in zip(call(wide[:, 64:], True, True), (q, si, y)))
    # an odd stride and start: the scalar path, whose sums run in another order (the values agree to rounding)
    odd = torch.empty(40 * 1029 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(40, 1029)
    odd[:, :1024] = x
    qs, sis, ys = call(odd[:, :1024], True, True)
    assert torch.allclose(sis, si, rtol=1e-5) and (ys.float() - y.float()).abs().max() <= y.float().abs().max() * 2 * BF


def test_norm_forward_special_rows(fp8):
    """A constant row (variance 0), a zero row with eps = 0 (rstd Inf, xhat NaN), a NaN
    and an Inf in a row, a row whose mean is large against its deviation; rows of
    their neighbours are not touched by them. The checkpoint marks NaN rows by
    byte 255."""
    cols = 64
    rng = np.random.default_rng(1)
    xb = workloads.bf16_bits(rng.standard_normal((8, cols)).astype(np.float32))
    plain = xb.copy()
    xb[1] = workloads.bf16_bits(np.full((1, cols), 3.0, np.float32))
    xb[2, 5] = 0x7FC0
    xb[3, 6] = 0x7F80
    xb[4] = 0
    xb[5] = workloads.bf16_bits((1000 + 8 * np.arange(cols, dtype=np.float32) % 64)[None])
    say("norm special rows")
    for eps, zero_nan in ((1e-5, False), (0.0, True)):
        out = []
        for b in (xb, plain):
            q = torch.empty((8, cols), dtype=torch.uint8, device=DEV)
            si, rstd = torch.empty(8, device=DEV), torch.empty(8, device=DEV)
            xq, xs = torch.empty((8, cols), dtype=torch.uint8, device=DEV), fp8.mx_scale_records(8, cols)
            fp8.fp8_norm_quantize_row(dev_bf16(b), None, None, eps, fp8.NORM_LAYER, 0, 0, q, si, rstd_out=rstd,
                                      xhat_q=xq, xhat_scale=xs)
            torch.cuda.synchronize()
            out.append((q.cpu().numpy(), si.cpu().numpy(), layer.from_records(xs.cpu().numpy(), cols)))
        (q, si, e8), (q0, si0, _) = out
        for r in (0, 6, 7):
            assert np.array_equal(q[r], q0[r]) and si[r] == si0[r]
        nan = lambda r: np.all((q[r] & 0x7F) == 0x7F) and si[r] == 1.0 and np.all(e8[r] == 255)  # noqa: E731
        assert nan(2) and nan(3)
        assert nan(4) == zero_nan and nan(1) == zero_nan
        if not zero_nan:
            assert not q[4].any() and not (q[1] & 0x7F).any()
        v = layer.values(xb[5:6])
        f = layer.norm_forward(v, None, None, np.float64(np.float32(eps)), False)
        layer.cast_ok(0, q[5:6], si[5:6], f["y"], f["y_tol"])


BACKWARD = [  # rows, cols, rms, gamma
    (1, 8, False, "bf16"), (1, 512, True, "none"), (3, 520, False, "f32"), (700, 1024, False, "bf16"),
    (65, 2048, True, "bf16"), (1100, 2056, False, "none"), (40, 4096, False, "f32"), (515, 7168, True, "bf16"),
    (5, 8200, False, "bf16"), (300, 16384, True, "f32"), (333, 1111, False, "bf16"), (2, 1, False, "none"),
    (1, 20000, False, "bf16"), (70, 33, True, "f32"), (2100, 2051, True, "bf16"), (3, 16381, False, "f32"),
    (2050, 4096, False, "bf16"), (1100, 16392, True, "bf16"),
]


@pytest.mark.parametrize("rows,cols,rms,gk", BACKWARD)
def test_norm_backward_from_x(fp8, rows, cols, rms, gk):
    rng = np.random.default_rng(rows + cols * 3)
    xb = make_x(rng, rows, cols)
    dyb = workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32) * 1e-3)
    gamma, gv = make_weights(rng, cols, gk)
    x = layer.values(xb)
    f = layer.norm_forward(x, None, None, 1e-5, rms)
    mean, rstd = f["mean"].astype(np.float32), f["rstd"].astype(np.float32)
    xhat = (x - (0 if rms else mean.astype(np.float64)[:, None])) * rstd.astype(np.float64)[:, None]
    want = layer.norm_backward(layer.values(dyb), xhat, gv, rstd.astype(np.float64), rms, xhat_rel=2 * layer.U)
    pad = 32 if cols % 8 == 0 else 5
    dx, buf, o = guarded(rows, cols, torch.bfloat16, ld=cols + pad)
    dg, db = torch.full((cols,), 9.0, device=DEV), torch.full((cols,), 9.0, device=DEV)
    say("norm backward", rows, cols, rms, gk)
    args = (dev_bf16(dyb), dev_bf16(xb), gamma, None if rms else torch.from_numpy(mean).to(DEV),
            torch.from_numpy(rstd).to(DEV), fp8.NORM_RMS if rms else fp8.NORM_LAYER)
    ws = fp8.norm_workspace(rows, cols)
    guard = torch.full((ws.numel() + 64,), 3.0, device=DEV)
    fp8.fp8_norm_backward(*args, dx, dgamma=dg, dbeta=db, workspace=guard[:ws.numel()])
    torch.cuda.synchronize()
    assert (guard[ws.numel():] == 3.0).all(), "writes past the workspace"
    within(bf16_of(dx), want["dx"], want["dx_tol"] * (1 + BF), "dx", rel=BF)
    within(dg.cpu().numpy(), want["dgamma"], want["dgamma_tol"], "dgamma")
    within(db.cpu().numpy(), want["dbeta"], want["dbeta_tol"], "dbeta")
    check_guard(buf, o, rows, cols)
    # the same bits again, and with one gradient or none
    dx2, dg2 = torch.empty_like(dx), torch.empty_like(dg)
    fp8.fp8_norm_backward(*args, dx2, dgamma=dg2, workspace=ws)
    dx3, db3 = torch.empty_like(dx), torch.empty_like(db)
    fp8.fp8_norm_backward(*args, dx3, dbeta=db3, workspace=ws)
    dx4 = torch.empty_like(dx)
    fp8.fp8_norm_backward(*args, dx4)
    torch.cuda.synchronize()
    assert torch.equal(dg2, dg) and torch.equal(db3, db)
    assert torch.equal(dx2, dx) and torch.equal(dx3, dx) and torch.equal(dx4, dx)


SAVED = [(1, 32, True, 0, False), (3, 544, False, 1, True), (1030, 1024, True, 0, True), (67, 2048, False, 0, True),
         (40, 4096, True, 1, False), (515, 7168, False, 0, True), (9, 16384, False, 0, True)]


@pytest.mark.parametrize("rows,cols,rms,fmt,with_y", SAVED)
def test_norm_backward_from_checkpoint(fp8, orc, rows, cols, rms, fmt, with_y):
    rng = np.random.default_rng(rows + cols * 5)
    xhb = workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32))
    codes, e8 = orc.mx_quantize_row(xhb, fmt)
    xhat = layer.mx_values(codes, fmt, e8)
    dyb = workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32) * 1e-3)
    gamma, gv = make_weights(rng, cols, "bf16")
    beta, bv = make_weights(rng, cols, "bf16")
    rstd = (0.5 + rng.random(rows)).astype(np.float32)
    want = layer.norm_backward(layer.values(dyb), xhat, gv, rstd.astype(np.float64), rms)
    # records with three spare ones per K step
    J = (cols + 127) // 128
    rec = torch.zeros((J, rows + 3, 4), dtype=torch.uint8, device=DEV)
    pad = np.zeros((rows, J * 4), np.uint8)
    pad[:, :cols // 32] = e8
    rec[:, :rows] = torch.from_numpy(np.ascontiguousarray(pad.reshape(rows, J, 4).transpose(1, 0, 2))).to(DEV)
    xq = torch.zeros((rows, cols + 32), dtype=torch.uint8, device=DEV)[:, :cols]
    xq.copy_(torch.from_numpy(codes))
    dx, buf, o = guarded(rows, cols, torch.bfloat16)
    y, ybuf, yo = guarded(rows, cols, torch.bfloat16)
    dg, db = torch.full((cols,), 9.0, device=DEV), torch.full((cols,), 9.0, device=DEV)
    say("norm backward from checkpoint", rows, cols, rms, fmt)
    fp8.fp8_mx_norm_backward(dev_bf16(dyb), xq, fmt, rec[:, :rows], gamma, beta, torch.from_numpy(rstd).to(DEV),
                             fp8.NORM_RMS if rms else fp8.NORM_LAYER, dx, dgamma=dg, dbeta=db,
                             y=y if with_y else None, workspace=fp8.norm_workspace(rows, cols))
    torch.cuda.synchronize()
    within(bf16_of(dx), want["dx"], want["dx_tol"] * (1 + BF), "dx", rel=BF)
    within(dg.cpu().numpy(), want["dgamma"], want["dgamma_tol"], "dgamma")
    within(db.cpu().numpy(), want["dbeta"], want["dbeta_tol"], "dbeta")
    check_guard(buf, o, rows, cols)
    if with_y:
        v = xhat * gv + bv
        within(bf16_of(y), v, 2 * layer.U * (np.abs(xhat * gv) + np.abs(v)), "y", rel=BF)
        check_guard(ybuf, yo, rows, cols)


def test_norm_backward_checkpoint_nan_block(fp8):
    """A NaN scale byte makes its own row NaN (and the gradients of the block's
    columns' weights), and no other row."""
    rows, cols = 6, 256
    rng = np.random.default_rng(2)
    xq = torch.from_numpy(rng.integers(0, 0x70, (rows, cols)).astype(np.uint8)).to(DEV)
    rec = torch.full((2, rows, 4), 120, dtype=torch.uint8, device=DEV)
    rec[1, 2, 1] = 255                                      # row 2, block 5
    dy = dev_bf16(workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32)))
    dx, dg = torch.empty_like(dy), torch.empty(cols, device=DEV)
    say("norm backward NaN block")
    fp8.fp8_mx_norm_backward(dy, xq, 0, rec, None, None, torch.ones(rows, device=DEV), fp8.NORM_RMS, dx, dgamma=dg,
                             workspace=fp8.norm_workspace(rows, cols))
    torch.cuda.synchronize()
    bad = torch.isnan(dx.float()).cpu().numpy()
    assert bad[2].all() and not np.delete(bad, 2, 0).any()
    assert np.array_equal(torch.isnan(dg).cpu().numpy(), np.arange(cols) // 32 == 5)


def test_norm_backward_inf_in_an_odd_row(fp8):
    """An Inf in the last columns of a band's last row (RMS: rstd is 0 there and xhat
    NaN in that column alone): dgamma is NaN in that column alone, also where
    threads without a row of their own read that row again."""
    rows, cols, bad = 333, 1111, 1108
    rng = np.random.default_rng(11)
    x = make_x(rng, rows, cols)
    x[rows - 1, bad] = 0x7F80
    dyb = workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32))
    v = layer.values(x)
    rstd = 1 / np.sqrt(np.mean(np.where(np.isinf(v), 0, v) ** 2, axis=1) + 1e-5)
    rstd[rows - 1] = 0
    rstd = rstd.astype(np.float32)
    dx = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    dg, db = (torch.empty(cols, device=DEV) for _ in range(2))
    fp8.fp8_norm_backward(dev_bf16(dyb), dev_bf16(x), None, None, torch.from_numpy(rstd).to(DEV), fp8.NORM_RMS, dx, dg, db,
                          fp8.norm_workspace(rows, cols))
    dg = dg.cpu().numpy()
    assert np.array_equal(np.nonzero(np.isnan(dg))[0], [bad])
    terms = layer.values(dyb)[:-1] * (v[:-1] * rstd[:-1, None].astype(np.float64))
    keep = np.arange(cols) != bad
    # xhat rounded once, then a sum of rows terms in some order: rows + 1 roundings a term
    tol = (rows + 4) * 2.0**-24 * np.abs(terms).sum(axis=0)
    within(dg[keep], terms.sum(axis=0)[keep], tol[keep], "dgamma")
    assert torch.isnan(dx[rows - 1].float()).all() and torch.isfinite(dx[:rows - 1].float()).all()
    assert torch.isfinite(db).all()


def test_norm_no_rows(fp8):
    """No rows: nothing to cast, and the weights' gradients are 0."""
    say("norm no rows")
    x = torch.empty((0, 96), dtype=torch.bfloat16, device=DEV)
    q = torch.empty((0, 96), dtype=torch.uint8, device=DEV)
    z = torch.empty(0, device=DEV)
    fp8.fp8_norm_quantize_row(x, None, None, 0.0, fp8.NORM_LAYER, 0, 0, q, z, xhat_q=q,
                              xhat_scale=fp8.mx_scale_records(0, 96))
    dg, db = torch.ones(96, device=DEV), torch.ones(96, device=DEV)
    fp8.fp8_norm_backward(x, x, None, z, z, fp8.NORM_LAYER, x, dgamma=dg, dbeta=db)
    torch.cuda.synchronize()
    assert not dg.any() and not db.any()


def test_norm_gradient_against_differences(fp8):
    """dx of a layer norm against central differences of its own forward pass (y in
    bf16): with a perturbation of 2^-3 and rows of 16 values near 1 the
    differences' error is the two outputs' half steps over the perturbation,
    summed with |dy|, plus the third derivative's h^2 / 6 part."""
    rng = np.random.default_rng(8)
    cols, h = 16, 2.0 ** -3
    x = workloads.bf16_to_f32(workloads.bf16_bits(rng.standard_normal((1, cols)).astype(np.float32)))
    x = np.round(x * 8) / 8                                 # +-h stays exact in bf16
    assert np.abs(x - x.mean()).max() + 2 * h < 3.5
    dy = np.zeros((1, cols), np.float32)
    dy[0, 3] = 1.0
    xs = np.concatenate([x] * (2 * cols), 0).astype(np.float32)
    for c in range(cols):
        xs[2 * c, c] += h
        xs[2 * c + 1, c] -= h
    say("norm differences")
    y = torch.empty((2 * cols, cols), dtype=torch.bfloat16, device=DEV)
    fp8.fp8_norm_quantize_row(dev_bf16(workloads.bf16_bits(xs)), None, None, 0.5, fp8.NORM_LAYER, 0, 0, None, None, y=y)
    xb, mean, rstd = dev_bf16(workloads.bf16_bits(x)), torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    y0, dx = torch.empty((1, cols), dtype=torch.bfloat16, device=DEV), torch.empty((1, cols), dtype=torch.bfloat16,
                                                                                 device=DEV)
    fp8.fp8_norm_quantize_row(xb, None, None, 0.5, fp8.NORM_LAYER, 0, 0, None, None, y=y0, mean_out=mean, rstd_out=rstd)
    fp8.fp8_norm_backward(dev_bf16(workloads.bf16_bits(dy)), xb, None, mean, rstd, fp8.NORM_LAYER, dx)
    torch.cuda.synchronize()
    yv = y.double().cpu().numpy()[:, 3]
    diff = (yv[0::2] - yv[1::2]) / (2 * h)
    # rounding: 2 half steps of y over 2 h, dx's own half step. Third derivative of
    # y_3 = d s, s = (v + eps)^-0.5, in x_c, with v + eps >= 0.5, |d| <= 3.5, N = 16:
    # |v'| <= 2 |d| / N < 0.44, v'' < 2 / N; s'' <= 0.75 * 5.66 * 0.44^2 + 0.5 * 2.83 /
    # 8 < 1.01, s3 = s's third derivative <= 1.875 * 11.3 * 0.44^3 + 2.25 * 5.66 * 0.44 / 8 < 2.51, so
    # |y's third| <= 3.5 s3 + 3 s'' < 12; times h^2 / 6.
    tol = np.abs(yv).max() * BF / h + np.abs(diff) * BF + 12 * h * h / 6
    assert np.all(np.abs(dx.double().cpu().numpy()[0] - diff) <= tol)


def test_norm_many_rows(fp8):
    """More rows than one launch takes (2^20): the rows on either side of the cut and
    the last ones are those of a call on them alone."""
    rows, cols = (1 << 20) + 37, 64
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn((rows, cols), device=DEV, generator=g, dtype=torch.bfloat16)
    say("norm many rows")

    def call(x):
        n = x.shape[0]
        q, si, rstd = torch.empty((n, cols), dtype=torch.uint8, device=DEV), torch.empty(n, device=DEV), torch.empty(
            n, device=DEV)
        y, xq, xs = torch.empty_like(x), torch.empty_like(q), fp8.mx_scale_records(n, cols)
        fp8.fp8_norm_quantize_row(x, None, None, 1e-5, fp8.NORM_LAYER, 0, 0, q, si, y=y, rstd_out=rstd, xhat_q=xq,
                                  xhat_scale=xs)
        return q, si, rstd, y, xq, xs[0]

    whole = call(x)
    for lo, hi in ((0, 40), ((1 << 20) - 8, (1 << 20) + 8), (rows - 9, rows)):
        part = call(x[lo:hi])
        torch.cuda.synchronize()
        assert all(torch.equal(a[lo:hi], b) for a, b in zip(whole, part)), (lo, hi)
    dx, dg, db = torch.empty_like(x), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    mean = torch.zeros(rows, device=DEV)
    fp8.fp8_norm_backward(x, x, None, mean, whole[2], fp8.NORM_LAYER, dx, dgamma=dg, dbeta=db,
                          workspace=fp8.norm_workspace(rows, cols))
    part = torch.empty((9, cols), dtype=torch.bfloat16, device=DEV)
    fp8.fp8_norm_backward(x[-9:], x[-9:], None, mean[-9:], whole[2][-9:], fp8.NORM_LAYER, part)
    torch.cuda.synchronize()
    assert torch.equal(dx[-9:], part)
    xd = x.double()
    want, mag = xd.sum(0), xd.abs().sum(0)
    # a band of 2049 rows is added by 8 teams, 257 rows each in turn, then 512 bands in 16 slices
    assert torch.all((db.double() - want).abs() <= (257 + 8 + 32 + 16) * layer.U * mag)


def test_norm_tensors_of_two_devices_are_refused(fp8):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    z = torch.zeros(4, device=DEV)
    with pytest.raises(ValueError, match="on one GPU"):
        fp8.fp8_norm_backward(x, x, None, z, z, fp8.NORM_LAYER, torch.empty_like(x), dgamma=torch.zeros(64, device=DEV),
                              workspace=torch.zeros(1024))
    with pytest.raises(fp8.Fp8Error, match="workspace of 2048 bytes"):
        fp8.fp8_norm_backward(x, x, None, z, z, fp8.NORM_LAYER, torch.empty_like(x), dgamma=torch.zeros(64, device=DEV),
                              workspace=torch.zeros(511, device=DEV))


def test_norm_backward_of_the_most_columns(fp8):
    """One row of 2^27 - 1 columns, the most that is accepted: the grid of the weights'
    gradients is in two layers. dbeta is dy and dgamma the rounded product, bit for bit;
    dx within the rounding of its sums (256 threads add 2^19 terms each, in order)."""
    n = (1 << 27) - 1
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    x, dy = (torch.randn((1, n), device=DEV, generator=gen, dtype=torch.bfloat16) for _ in range(2))
    rstd = torch.full((1,), 1.25, device=DEV)
    dx = torch.zeros_like(x)
    dgamma, dbeta = (torch.full((n,), float("nan"), device=DEV) for _ in range(2))
    say("norm gradient", 1, n)
    fp8.fp8_norm_backward(dy, x, None, None, rstd, fp8.NORM_RMS, dx, dgamma, dbeta, fp8.norm_workspace(1, n))
    torch.cuda.synchronize()
    assert torch.equal(dbeta, dy[0].float())
    xh = x[0].float() * rstd
    assert torch.equal(dgamma, xh * dy[0].float())
    d64, x64 = dy[0].double(), xh.double()
    c1 = (d64 * x64).sum() / n
    c1_tol = (2.0 ** 19 + 16) * layer.U * (d64 * x64).abs().sum() / n
    want = 1.25 * (d64 - x64 * c1)
    tol = 1.25 * (x64.abs() * c1_tol + 6 * layer.U * (d64.abs() + (x64 * c1).abs()))
    assert ((dx[0].double() - want).abs() <= tol * (1 + BF) + BF * want.abs()).all()


def special_gradient(dy, xh, g, rstd, rms):
    """dx of one row in the arithmetic of the definition (fp64, Inf and NaN included)."""
    with np.errstate(invalid="ignore", over="ignore"):
        w = dy * g
        c1, c2 = (w * xh).sum() / len(dy), 0.0 if rms else w.sum() / len(dy)
        return rstd * (w - xh * c1 - c2)


def same_specials(got, want, what):
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(np.isposinf(got), np.isposinf(want)) and np.array_equal(np.isneginf(got), np.isneginf(want)), what


@pytest.mark.parametrize("cols", [520, 512, 1030, 1111, 2560, 2999, 4104, 8224])
@pytest.mark.parametrize("rms", [True, False])
def test_norm_backward_infinite_weight(fp8, cols, rms):
    """An infinite gamma among the row's last columns makes the row's means infinite, not
    NaN, whether or not the width fills the lanes of its team: dx is the definition's."""
    rng = np.random.default_rng(cols)
    rows, at = 3, cols - 2
    x = workloads.bf16_bits(rng.uniform(0.5, 2.0, (rows, cols)).astype(np.float32))
    dy = workloads.bf16_bits(rng.uniform(0.5, 2.0, (rows, cols)).astype(np.float32))
    gamma = np.ones(cols, np.float32)
    gamma[at] = np.inf
    mean, rstd = np.array([0.25, -1.0, 0.0], np.float32), np.array([1.0, 0.5, 2.0], np.float32)
    dx = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    say("norm gradient, infinite gamma", cols, rms)
    fp8.fp8_norm_backward(dev_bf16(dy), dev_bf16(x), torch.from_numpy(gamma).to(DEV), torch.from_numpy(mean).to(DEV),
                          torch.from_numpy(rstd).to(DEV), fp8.NORM_RMS if rms else fp8.NORM_LAYER, dx)
    got = dx.float().cpu().numpy()
    for r in range(rows):
        xh = (layer.values(x)[r] - (0.0 if rms else mean[r])) * rstd[r]
        same_specials(got[r], special_gradient(layer.values(dy)[r], xh, gamma.astype(np.float64), rstd[r], rms), (r, cols))


@pytest.mark.parametrize("cols", [1032, 1111, 2047, 4099])
def test_norm_backward_infinite_rstd(fp8, cols):
    """rstd = Inf (eps = 0 and squares that underflow): xhat is infinite and so is dx; the
    zeros behind a row that ends inside a chunk of 8 add nothing (0 * Inf)."""
    rng = np.random.default_rng(cols)
    x = workloads.bf16_bits(rng.uniform(0.5, 2.0, (2, cols)).astype(np.float32))
    dy = workloads.bf16_bits(rng.uniform(0.5, 2.0, (2, cols)).astype(np.float32))
    dx = torch.zeros((2, cols), dtype=torch.bfloat16, device=DEV)
    say("norm gradient, infinite rstd", cols)
    fp8.fp8_norm_backward(dev_bf16(dy), dev_bf16(x), None, None, torch.full((2,), float("inf"), device=DEV),
                          fp8.NORM_RMS, dx)
    got = dx.float().cpu().numpy()
    for r in range(2):
        same_specials(got[r], special_gradient(layer.values(dy)[r], layer.values(x)[r] * np.inf, 1.0, np.inf, True), r)
    assert np.isneginf(got).all()


@pytest.mark.parametrize("cols", [544, 512, 1056, 2592, 8224])
@pytest.mark.parametrize("with_y", [False, True])
def test_norm_backward_infinite_checkpoint(fp8, cols, with_y):
    """An Inf code (e5m2) of a checkpoint in the row's last columns, its block's byte an
    ordinary one: the mean is infinite and dx the definition's at every width."""
    rng = np.random.default_rng(cols)
    rows, at = 2, cols - 3
    dy = workloads.bf16_bits(rng.uniform(0.5, 2.0, (rows, cols)).astype(np.float32))
    q = np.full((rows, cols), 0x3C, np.uint8)                       # 1.0
    q[:, at] = 0x7C                                                 # Inf
    xs = fp8.mx_scale_records(rows, cols)
    xs.fill_(127)
    dx = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros_like(dx) if with_y else None
    say("norm gradient, infinite checkpoint", cols, with_y)
    fp8.fp8_mx_norm_backward(dev_bf16(dy), torch.from_numpy(q).to(DEV), 1, xs, None, None,
                             torch.ones(rows, device=DEV), fp8.NORM_RMS, dx, y=y)
    got = dx.float().cpu().numpy()
    xh = np.ones(cols)
    xh[at] = np.inf
    for r in range(rows):
        same_specials(got[r], special_gradient(layer.values(dy)[r], xh, 1.0, 1.0, True), (r, cols))
    if with_y:
        assert np.array_equal(bf16_of(y), np.tile(xh, (rows, 1)))
