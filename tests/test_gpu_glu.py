"""GPU parity of the gated FP8 products (gate and up with SwiGLU, and the backward
pass's product with SwiGLU's gradient) against the fp64 definitions of
oracle/block.py: every output within the fp32 evaluation's bound plus half a step
of bf16. Sizes around every kernel's tile and every rule that chooses one, odd
sizes, views with guard bands, scalar and vector factors, both formats."""
import numpy as np
import pytest
import torch

import workloads
from helpers import check_guard, dev_bf16, dev_f32, dev_u8, guarded, host_bits, say
from oracle import block, layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = block.BF16


@pytest.fixture(scope="module")
def fp8():
    import fp8_scaled_gemm_amax_amd as m
    return m


def within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol * (1 + BF) + BF * np.abs(want) + 2.0 ** -133)
    assert not bad.any(), (f"{what}: {int(bad.sum())} values off, first {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]!r} for {want[bad][0]!r} +- {tol[bad][0]!r}")


def bf16_of(t):
    return layer.values(host_bits(t))


def operand(rng, rows, cols, fmt, mode, std):
    """(codes on the host, factors on the host [rows], codes and factors on the device)."""
    q, s = block.codes(rng, rows, cols, fmt, std) if cols else (np.zeros((rows, 0), np.uint8), np.ones(rows, np.float32))
    if mode == 0:
        s = np.full(rows, np.float32(0.37 * std / max(cols, 1) ** 0.25), np.float32)
    return q, s, s[:1] if mode == 0 else s


def padded(codes, pad):
    """codes on the device with pad more bytes a row, those 0x7F (NaN)."""
    rows, cols = codes.shape
    t = torch.full((rows, cols + pad), 0x7F, dtype=torch.uint8, device=DEV)
    t[:, :cols] = dev_u8(codes)
    return t[:, :cols]


FORWARD = [  # m, k, inter, fa, fb, a_mode, b_mode, h, output row padding
    (1, 16, 1, 0, 0, 1, 1, True, 0), (1, 4096, 64, 0, 0, 1, 1, False, 0), (1, 7168, 136, 0, 1, 0, 1, True, 8),
    (3, 272, 40, 1, 0, 1, 0, True, 3), (16, 512, 72, 0, 0, 1, 1, True, 8), (17, 1040, 33, 1, 1, 1, 1, True, 1),
    (31, 2048, 1408, 0, 0, 0, 0, False, 8), (64, 1024, 520, 0, 0, 1, 1, True, 8), (65, 768, 96, 0, 1, 1, 1, True, 8),
    (128, 128, 64, 0, 0, 1, 1, True, 0), (129, 1024, 200, 1, 0, 1, 1, False, 24), (300, 512, 641, 0, 0, 1, 1, True, 7),
    (777, 256, 1408, 0, 0, 0, 0, True, 8), (256, 256, 16384, 0, 0, 1, 1, False, 8),
    (4000, 512, 1100, 0, 0, 1, 1, True, 4), (4097, 256, 1100, 1, 0, 1, 1, True, 0), (2049, 768, 2056, 0, 1, 0, 1, False, 8),
    (8200, 256, 1026, 0, 0, 1, 0, True, 2), (5000, 272, 900, 0, 0, 1, 1, True, 4), (40, 0, 72, 0, 0, 1, 1, True, 8),
    (300, 0, 200, 0, 0, 0, 0, True, 8), (48, 1296, 24, 0, 0, 1, 1, True, 8), (33, 256, 7, 1, 0, 1, 1, True, 2),
    (5, 2304, 50, 0, 0, 1, 0, True, 8), (70, 128, 5, 0, 0, 1, 1, True, 1), (200, 384, 64, 0, 1, 1, 1, False, 8),
    (130, 1008, 4233, 0, 0, 1, 1, True, 3), (1030, 144, 1000, 0, 1, 0, 1, False, 8), (63, 640, 8300, 1, 0, 1, 1, True, 4),
    (129, 400, 72, 0, 0, 1, 1, True, 8), (500, 1008, 136, 1, 0, 0, 1, True, 8), (255, 4096, 16392, 0, 0, 1, 1, False, 8),
]


@pytest.mark.parametrize("m,k,inter,fa,fb,am,bm,want_h,pad", FORWARD)
def test_forward(fp8, m, k, inter, fa, fb, am, bm, want_h, pad):
    rng = np.random.default_rng(m * 3 + k + inter)
    qa, sa, sad = operand(rng, m, k, fa, am, 1.0)
    qb, sb, sbd = operand(rng, 2 * inter, k, fb, bm, 1.3 / max(k, 1) ** 0.5)
    h, tol = block.product(qa, fa, sa, qb, fb, sb)
    g, u, gt, ut = h[:, :inter], h[:, inter:], tol[:, :inter], tol[:, inter:]
    act, act_tol = block.swiglu(g, u, gt, ut)
    d, dbuf, do = guarded(m, inter, torch.bfloat16, ld=inter + pad)
    hd = None
    if want_h:
        hd, hbuf, ho = guarded(m, 2 * inter, torch.bfloat16, ld=2 * inter + pad)
    say("gated product", m, k, inter, fa, fb, am, bm, want_h, pad)
    args = (padded(qa, 16), fa, padded(qb, 32), fb, dev_f32(sad), am, dev_f32(sbd), bm)
    fp8.fp8_gemm_swiglu(*args, d, h=hd)
    torch.cuda.synchronize()
    within(bf16_of(d), act, act_tol, "act")
    check_guard(dbuf, do, m, inter)
    if want_h:
        within(bf16_of(hd), h, tol, "h")
        check_guard(hbuf, ho, m, 2 * inter)
    again = torch.empty((m, inter), dtype=torch.bfloat16, device=DEV)
    fp8.fp8_gemm_swiglu(*args, again)
    torch.cuda.synchronize()
    assert torch.equal(again, d), "act depends on whether h is stored, or on its layout"


BACKWARD = [  # m, k, inter, fa, fb, a_mode, b_mode, act, row padding
    (1, 16, 1, 1, 0, 1, 1, True, 0), (3, 272, 40, 1, 0, 1, 0, True, 3), (64, 512, 136, 1, 0, 1, 1, False, 8),
    (130, 1008, 8261, 1, 0, 1, 1, True, 3), (1100, 144, 2060, 0, 1, 0, 1, False, 8), (63, 640, 8300, 1, 0, 1, 1, True, 4),
    (130, 1024, 200, 1, 0, 1, 1, True, 24), (300, 512, 641, 0, 1, 0, 1, True, 7), (1001, 256, 1408, 1, 0, 1, 1, False, 8),
    (4000, 512, 2100, 1, 0, 1, 1, True, 4), (4097, 256, 2200, 0, 0, 1, 1, True, 0), (2049, 768, 4104, 1, 1, 0, 0, False, 8),
    (8200, 256, 1026, 1, 0, 1, 0, True, 2), (5000, 272, 900, 0, 0, 1, 1, True, 4), (300, 0, 72, 0, 0, 1, 1, True, 8),
    (256, 256, 32768, 1, 0, 1, 1, True, 8), (129, 400, 72, 1, 0, 1, 1, True, 8), (70, 128, 5, 0, 0, 1, 1, True, 1),
    (200, 1520, 129, 1, 0, 1, 1, True, 3),
]


@pytest.mark.parametrize("m,k,inter,fa,fb,am,bm,want_act,pad", BACKWARD)
def test_backward(fp8, m, k, inter, fa, fb, am, bm, want_act, pad):
    rng = np.random.default_rng(m * 5 + k + inter)
    qa, sa, sad = operand(rng, m, k, fa, am, 1e-3)
    qb, sb, sbd = operand(rng, inter, k, fb, bm, 1.3 / max(k, 1) ** 0.5)
    da, tol = block.product(qa, fa, sa, qb, fb, sb)
    hb = workloads.bf16_bits((1.5 * rng.standard_normal((m, 2 * inter))).astype(np.float32))
    hv = layer.values(hb)
    want = block.swiglu_backward(da, hv[:, :inter], hv[:, inter:], tol)
    h = torch.full((m, 2 * inter + pad), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :2 * inter]
    h.copy_(dev_bf16(hb))
    dh, buf, o = guarded(m, 2 * inter, torch.bfloat16, ld=2 * inter + pad)
    act = None
    if want_act:
        act, abuf, ao = guarded(m, inter, torch.bfloat16, ld=inter + pad)
    say("gated product's gradient", m, k, inter, fa, fb, am, bm, want_act, pad)
    args = (padded(qa, 16), fa, padded(qb, 32), fb, dev_f32(sad), am, dev_f32(sbd), bm, h)
    fp8.fp8_gemm_swiglu_backward(*args, dh, act=act)
    torch.cuda.synchronize()
    got = bf16_of(dh)
    within(got[:, :inter], want["dg"], want["dg_tol"], "d(gate)")
    within(got[:, inter:], want["du"], want["du_tol"], "d(up)")
    check_guard(buf, o, m, 2 * inter)
    if want_act:
        within(bf16_of(act), want["a"], want["a_tol"], "act")
        check_guard(abuf, ao, m, inter)
    again = torch.empty((m, 2 * inter), dtype=torch.bfloat16, device=DEV)
    fp8.fp8_gemm_swiglu_backward(*args, again)
    torch.cuda.synchronize()
    assert torch.equal(again, dh), "dh depends on whether act is stored, or on its layout"


@pytest.mark.parametrize("m,k,inter", [(4, 256, 80), (40, 1024, 64), (20, 272, 33), (130, 256, 200), (130, 400, 72), (4200, 256, 1100)])
def test_rows_and_columns_stay_apart(fp8, m, k, inter):
    """A NaN in a row of a, in a gate row and in an up row of b reaches that row and
    those columns alone, in both directions; large gates give silu of 0 and g."""
    rng = np.random.default_rng(k)
    qa, sa, _ = operand(rng, m, k, 0, 1, 1.0)
    qb, sb, _ = operand(rng, 2 * inter, k, 0, 1, 1.0)
    a, b = dev_u8(qa), dev_u8(qb)
    row, gate, up = m // 2, inter // 3, inter - 1
    a[row, 3], b[gate, 5], b[inter + up, k - 1] = 0x7F, 0xFF, 0x7F
    act = torch.empty((m, inter), dtype=torch.bfloat16, device=DEV)
    h = torch.empty((m, 2 * inter), dtype=torch.bfloat16, device=DEV)
    say("gated product, NaN", m, k, inter)
    fp8.fp8_gemm_swiglu(a, 0, b, 0, dev_f32(sa), 1, dev_f32(sb), 1, act, h=h)
    torch.cuda.synchronize()
    bad = torch.zeros((m, 2 * inter), dtype=torch.bool, device=DEV)
    bad[row] = True
    bad[:, gate] = bad[:, inter + up] = True
    assert torch.equal(torch.isnan(h), bad)
    assert torch.equal(torch.isnan(act), bad[:, :inter] | bad[:, inter:])
    hv = torch.randn((m, 2 * inter), device=DEV).to(torch.bfloat16)
    hv[0, 0], hv[1, 1], hv[2, inter + 2] = float("nan"), 300.0, float("nan")
    hv[1, 2] = -300.0
    dh = torch.empty((m, 2 * inter), dtype=torch.bfloat16, device=DEV)
    say("gated product's gradient, NaN", m, k, inter)
    fp8.fp8_gemm_swiglu_backward(a, 0, b[:inter], 0, dev_f32(sa), 1, dev_f32(sb[:inter]), 1, hv, dh, act=act)
    torch.cuda.synchronize()
    da = torch.zeros((m, inter), dtype=torch.bool, device=DEV)
    da[row] = True
    da[:, gate] = True
    nan_g, nan_u = torch.isnan(hv[:, :inter]), torch.isnan(hv[:, inter:])
    assert torch.equal(torch.isnan(act), nan_g | nan_u)
    assert torch.equal(torch.isnan(dh[:, :inter]), da | nan_g | nan_u)
    assert torch.equal(torch.isnan(dh[:, inter:]), da | nan_g)
    assert act[1, 1] == (300.0 * hv[1, inter + 1].float()).to(torch.bfloat16) and act[1, 2] == 0
    if row != 1 and gate != 2:
        assert dh[1, 2] == 0 and dh[1, inter + 2] == 0


def test_empty(fp8):
    say("gated product, no rows")
    e = torch.empty
    z = e((0, 64), dtype=torch.uint8, device=DEV)
    b = torch.zeros((16, 64), dtype=torch.uint8, device=DEV)
    one = torch.ones(1, device=DEV)
    fp8.fp8_gemm_swiglu(z, 0, b, 0, one, 0, one, 0, e((0, 8), dtype=torch.bfloat16, device=DEV))
    fp8.fp8_gemm_swiglu_backward(z, 0, b, 0, one, 0, one, 0, e((0, 32), dtype=torch.bfloat16, device=DEV),
                                 e((0, 32), dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()


def test_gradient_against_differences(fp8):
    """dh against central differences of act, in fp64 from the exact product: the
    objective sum(act * da) of one element is act * da; the difference over a step
    of 2^-6 is off by the third derivative's part, h^2 / 6 of at most |da u| (|silu'''| < 1)."""
    rng = np.random.default_rng(5)
    m, k, inter = 24, 64, 48
    qa, sa, _ = operand(rng, m, k, 1, 1, 1.0)
    qb, sb, _ = operand(rng, inter, k, 0, 1, 0.2)
    da, tol = block.product(qa, 1, sa, qb, 0, sb)
    hb = workloads.bf16_bits(rng.standard_normal((m, 2 * inter)).astype(np.float32))
    hv = layer.values(hb)
    g, u = hv[:, :inter], hv[:, inter:]
    f = lambda g, u: g * layer.sigmoid(g) * u  # noqa: E731
    step = 2.0 ** -6
    dg = da * (f(g + step, u) - f(g - step, u)) / (2 * step)
    du = da * (f(g, u + step) - f(g, u - step)) / (2 * step)
    dh = torch.empty((m, 2 * inter), dtype=torch.bfloat16, device=DEV)
    say("gated product's gradient against differences")
    fp8.fp8_gemm_swiglu_backward(dev_u8(qa), 1, dev_u8(qb), 0, dev_f32(sa), 1, dev_f32(sb), 1, dev_bf16(hb), dh)
    torch.cuda.synchronize()
    want = block.swiglu_backward(da, g, u, tol)
    got = bf16_of(dh)
    within(got[:, :inter], dg, want["dg_tol"] + step ** 2 / 6 * np.abs(da * u), "d(gate)")
    within(got[:, inter:], du, want["du_tol"] + 1e-9 * np.abs(du), "d(up)")


def spread(t, ld):
    """t with its rows ld elements apart."""
    rows, cols = t.shape
    far = torch.empty((rows - 1) * ld + cols, dtype=t.dtype, device=DEV).as_strided((rows, cols), (ld, 1))
    return far.copy_(t)


@pytest.mark.parametrize("m,k,inter", [(7, 272, 24), (70, 272, 24), (300, 256, 4300)])
def test_rows_far_apart(fp8, m, k, inter):
    """Leading dimensions at their limits: the rows of one tile span 4 GiB and more."""
    rng = np.random.default_rng(m)
    qa, sa, sad = operand(rng, m, k, 0, 1, 1.0)
    qb, sb, sbd = operand(rng, 2 * inter, k, 0, 1, 0.1)
    qd, sd, sdd = operand(rng, inter, k, 0, 1, 0.1)
    ldf, ldo = (1 << 24) - 16, (1 << 25) - 8
    a, b, d = padded(qa, 16), padded(qb, 32), padded(qd, 32)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    say("gated product, rows far apart", m, k, inter)
    fa, fb, fd = spread(a, ldf), (spread(b, ldf) if inter < 100 else b), (spread(d, ldf) if inter < 100 else d)
    near = [torch.zeros((m, w * inter), **bf) for w in (1, 2, 2, 1)]
    far = [spread(t, ldo) for t in near]
    for q, w, v, o in ((a, b, d, near), (fa, fb, fd, far)):
        fp8.fp8_gemm_swiglu(q, 0, w, 0, dev_f32(sad), 1, dev_f32(sbd), 1, o[0], h=o[1])
        fp8.fp8_gemm_swiglu_backward(q, 0, v, 0, dev_f32(sad), 1, dev_f32(sdd), 1, o[1], o[2], act=o[3])
    torch.cuda.synchronize()
    for n, f in zip(near, far):
        assert torch.equal(n, f)


@pytest.mark.parametrize("m,k,inter,fa,fb,am,bm,want_h,pad", [
    (4100, 768, 2184, 0, 1, 1, 1, True, 8), (4100, 512, 3976, 0, 0, 1, 1, True, 0)])
def test_forward_of_many_tiles(fp8, m, k, inter, fa, fb, am, bm, want_h, pad):
    """More large tiles than CUs: a workgroup goes on to its second (306 tiles, six steps
    of K) and third one (544 tiles), with h and without."""
    test_forward(fp8, m, k, inter, fa, fb, am, bm, want_h, pad)


def test_backward_of_many_tiles(fp8):
    """The same of the gradient (306 tiles, six steps of K), with act and without."""
    test_backward(fp8, 4100, 768, 4360, 1, 0, 1, 1, True, 8)


@pytest.mark.parametrize("m,k,inter,fa,fb,am,bm,want_h,pad", [
    (1, 1040, 4104, 0, 0, 1, 1, True, 3), (2, 4096, 8200, 0, 1, 1, 0, True, 8), (16, 528, 4120, 1, 0, 0, 1, True, 8),
    (17, 2304, 4097, 0, 0, 1, 1, True, 1), (32, 768, 5000, 1, 1, 1, 1, True, 8), (32, 1040, 14336, 0, 0, 1, 1, True, 0),
    (24, 512, 8192, 0, 0, 1, 1, True, 8)])
def test_forward_of_few_rows_and_many_columns(fp8, m, k, inter, fa, fb, am, bm, want_h, pad):
    """A decoding batch at the widths that are served: as many workgroups as CUs and more."""
    test_forward(fp8, m, k, inter, fa, fb, am, bm, want_h, pad)


# What the epilogue makes of exact sums: a and b have a single column that is not 0, so
# that a sum is a product of factors, any fp32 number. The other factor of an output is
# then set such that the exact output lies 32 or 48 U (U = 2^-24) beside the middle
# between two bf16 numbers, and the output has to be the nearer one: an error of more
# than that in sigma, 1 - sigma or a product gives another.
def unit_codes(rows, k):
    q = torch.zeros((rows, k), dtype=torch.uint8, device=DEV)
    q[:, 0] = 0x38                              # 1 in e4m3
    return q


def beside_middle(rng, factor, shift):
    """(other factor in fp32, the nearest bf16 of the product) for exact factors."""
    at = (np.floor(rng.random(factor.shape) * 128) + 0.5) / 128 + 1
    side = np.where(rng.random(factor.shape) < 0.5, -1.0, 1.0)
    other = (at * (1 + side * shift * block.U) / np.abs(factor)).astype(np.float32)
    exact = other.astype(np.float64) * factor
    assert (np.abs(np.abs(exact) - at) >= (shift - 2) * block.U * at).all()
    return other, np.sign(factor) * (at + side / 256)


def check_nearest(got, want, g, what):
    bad = got != want
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} not the nearest, the first at gate "
                           f"{np.broadcast_to(g, bad.shape)[bad][0]!r}: {got[bad][0]!r} for {want[bad][0]!r}")


@pytest.mark.parametrize("m,k,inter", [(3, 16, 1000), (3, 16, 4096), (70, 16, 4096), (200, 16, 4608), (600, 256, 4096)])
def test_sigma_of_exact_gates(fp8, m, k, inter):
    """act = g sigma(g) u of gates from -88.7, where exp(-g) is just finite, to 88. sigma is
    off by 15 U at most: exp(-g) 2 U by the exponential, 2 by its two products and 4 by ln
    2's constant, the sum 1, the reciprocal 2, 4 where sigma is subnormal; then two products."""
    rng = np.random.default_rng(m + inter)
    g = np.concatenate([rng.uniform(-88.72, -87.3, inter // 4), rng.uniform(-88, 88, inter - inter // 4)]).astype(np.float32)
    u, want = beside_middle(rng, g.astype(np.float64) * layer.sigmoid(g.astype(np.float64)), 32)
    one = torch.ones(1, device=DEV)
    act = torch.empty((m, inter), dtype=torch.bfloat16, device=DEV)
    say("gated product, exact gates", m, k, inter)
    fp8.fp8_gemm_swiglu(unit_codes(m, k), 0, unit_codes(2 * inter, k), 0, one, 0, dev_f32(np.concatenate([g, u])), 1, act)
    torch.cuda.synchronize()
    check_nearest(bf16_of(act), np.broadcast_to(want, (m, inter)), g, "act")


@pytest.mark.parametrize("m,k,inter", [(3, 16, 4096), (300, 16, 6000), (600, 256, 5632)])
def test_sigma_of_exact_gates_backward(fp8, m, k, inter):
    """d(gate) = da u sigma (1 + g (1 - sigma)) and d(up) = da g sigma of gates that bf16
    holds. Where 1 + g (1 - sigma) is no small difference (gates past -3 or -0.6) it is off by
    1.5 (4 + 8 sigma) U + U, sigma by 15 U, and three products: 26 U at most."""
    rng = np.random.default_rng(m + inter)
    h = layer.values(workloads.bf16_bits(np.concatenate(
        [rng.uniform(-88.5, -87.4, inter // 8), rng.uniform(-88, -3.1, inter // 2),
         rng.uniform(-0.59, 88, inter - inter // 8 - inter // 2)]).astype(np.float32)))
    up = layer.values(workloads.bf16_bits(rng.uniform(0.5, 2, inter).astype(np.float32)))
    hd = torch.from_numpy(np.concatenate([h, up])).to(DEV).to(torch.bfloat16).repeat(m, 1)
    s, c = layer.sigmoid(h), layer.sigmoid(-h)
    dh = torch.empty((m, 2 * inter), dtype=torch.bfloat16, device=DEV)
    one = torch.ones(1, device=DEV)
    for what, factor, part in (("d(gate)", up * s * (1 + h * c), slice(0, inter)), ("d(up)", h * s, slice(inter, None))):
        da, want = beside_middle(rng, factor, 48)
        say("gated product's gradient, exact gates", m, k, inter, what)
        fp8.fp8_gemm_swiglu_backward(unit_codes(m, k), 0, unit_codes(inter, k), 0, one, 0, dev_f32(da), 1, hd, dh)
        torch.cuda.synchronize()
        check_nearest(bf16_of(dh)[:, part], np.broadcast_to(want, (m, inter)), h, what)
