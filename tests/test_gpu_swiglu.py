"""GPU parity of SwiGLU with an 8-bit checkpoint and of its gradient against the
fp64 definitions of oracle/layer.py. The checkpoint is bit for bit what
fp8_mx_quantize_row gives for h; the codes are roundings of a value within fp32
rounding of silu(gate) up; the gradients are within fp32 rounding plus half a
step of bf16."""
import numpy as np
import pytest
import torch

import workloads
from helpers import check_guard, dev_bf16, guarded, host_bits, say
from oracle import layer
from test_gpu_norm import within

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = layer.BF16


@pytest.fixture(scope="module")
def fp8():
    import fp8_scaled_gemm_amax_amd as m
    return m


def make_h(rng, rows, inter):
    h = rng.standard_normal((rows, 2 * inter)) * np.exp2(rng.integers(-5, 6, (rows, 1)))
    return workloads.bf16_bits(h.astype(np.float32))


SAVE = [(1, 32, 0, 0), (37, 256, 1, 1), (1030, 512, 0, 0), (1025, 1024, 2, 0), (1024, 2048, 0, 1), (3, 2080, 3, 0),
        (300, 4096, 0, 0), (65, 4128, 1, 0), (20, 14336, 0, 0), (5, 16384, 0, 1), (6, 96, 0, 0),
        (4, 3008, 0, 0), (3, 6112, 1, 1), (2, 8192, 0, 0), (3, 10240, 0, 0), (2, 11008, 2, 1), (3, 12320, 0, 0)]


@pytest.mark.parametrize("rows,inter,fmt,ck", SAVE)
def test_swiglu_save(fp8, rows, inter, fmt, ck):
    rng = np.random.default_rng(rows + inter)
    hb = make_h(rng, rows, inter)
    wide = torch.zeros((rows, 2 * inter + 64), dtype=torch.bfloat16, device=DEV)
    wide[:, :2 * inter] = dev_bf16(hb)
    h = wide[:, :2 * inter]
    q, qbuf, qo = guarded(rows, inter, torch.uint8)
    hq, hbuf, ho = guarded(rows, 2 * inter, torch.uint8)
    si = torch.full((rows,), -7.0, device=DEV)
    J = (2 * inter + 127) // 128
    rec = torch.full((J, rows + 2, 4), 0x5A, dtype=torch.uint8, device=DEV)
    say("swiglu save", rows, inter, fmt, ck)
    fp8.fp8_swiglu_quantize_row_mx(h, fmt, 0, q, si, hq, ck, rec[:, :rows])
    hq0, rec0 = torch.empty((rows, 2 * inter), dtype=torch.uint8, device=DEV), fp8.mx_scale_records(rows, 2 * inter)
    fp8.fp8_mx_quantize_row(h, ck, hq0, rec0)
    torch.cuda.synchronize()
    assert torch.equal(hq, hq0), "checkpoint codes"
    assert torch.equal(rec[:, :rows], rec0), "checkpoint records"
    assert (rec[:, rows:] == 0x5A).all(), "records past the rows"
    v = layer.values(hb)
    a, tol = layer.swiglu(v[:, :inter], v[:, inter:])
    layer.cast_ok(fmt, q.cpu().numpy(), si.cpu().numpy(), a, tol)
    check_guard(qbuf, qo, rows, inter)
    check_guard(hbuf, ho, rows, 2 * inter)


def test_swiglu_save_special_rows(fp8, orc):
    """NaN and Inf in gate and up, a zero row, gates where exp overflows or
    underflows; the checkpoint stays fp8_mx_quantize_row's, a NaN row's codes are
    cast with scale 1, the other rows are untouched."""
    inter = 64
    rng = np.random.default_rng(3)
    hb = make_h(rng, 8, inter)
    plain = hb.copy()
    hb[1, 3] = 0x7FC0
    hb[2, inter + 9] = 0xFF80                               # -Inf up: an infinite value saturates
    hb[3] = 0
    hb[4, :8] = workloads.bf16_bits(np.array([[-200, -90, -88, -87, 87, 90, 200, -1e30]], np.float32))
    hb[5, 7] = 0xFF80                                       # -Inf gate: NaN
    out = []
    say("swiglu special rows")
    for b in (hb, plain):
        q, si = torch.empty((8, inter), dtype=torch.uint8, device=DEV), torch.empty(8, device=DEV)
        hq, rec = torch.empty((8, 2 * inter), dtype=torch.uint8, device=DEV), fp8.mx_scale_records(8, 2 * inter)
        fp8.fp8_swiglu_quantize_row_mx(dev_bf16(b), 0, 0, q, si, hq, 0, rec)
        hq0, rec0 = torch.empty_like(hq), torch.empty_like(rec)
        fp8.fp8_mx_quantize_row(dev_bf16(b), 0, hq0, rec0)
        torch.cuda.synchronize()
        assert torch.equal(hq, hq0) and torch.equal(rec, rec0)
        out.append((q.cpu().numpy(), si.cpu().numpy()))
    (q, si), (q0, si0) = out
    for r in (0, 6, 7):
        assert np.array_equal(q[r], q0[r]) and si[r] == si0[r]
    assert (q[1, 3] & 0x7F) == 0x7F and si[1] == 1.0 and np.count_nonzero((q[1] & 0x7F) == 0x7F) == 1
    assert (q[2, 9] & 0x7F) == 0x7E and si[2] == 1.0
    assert not q[3].any() and si[3] == 1.0
    assert (q[5, 7] & 0x7F) == 0x7F and si[5] == 1.0
    v = layer.values(hb[4:5])
    a, tol = layer.swiglu(v[:, :inter], v[:, inter:])
    layer.cast_ok(0, q[4:5], si[4:5], a, tol)


GRAD = [(1, 8, False), (3, 40, True), (1001, 256, True), (37, 4096, False), (64, 2056, True), (513, 1408, True),
        (2, 14336, True)]


@pytest.mark.parametrize("rows,inter,with_a", GRAD)
def test_swiglu_backward(fp8, rows, inter, with_a):
    rng = np.random.default_rng(rows * 3 + inter)
    hb = make_h(rng, rows, inter)
    dab = workloads.bf16_bits(rng.standard_normal((rows, inter)).astype(np.float32) * 1e-3)
    v = layer.values(hb)
    want = layer.swiglu_backward(layer.values(dab), v[:, :inter], v[:, inter:])
    dh, buf, o = guarded(rows, 2 * inter, torch.bfloat16)
    a, abuf, ao = guarded(rows, inter, torch.bfloat16)
    say("swiglu backward", rows, inter, with_a)
    fp8.fp8_swiglu_backward(dev_bf16(dab), dev_bf16(hb), dh, a=a if with_a else None)
    torch.cuda.synchronize()
    got = layer.values(host_bits(dh))
    within(got[:, :inter], want["dg"], want["dg_tol"] * (1 + BF), "d(gate)", rel=BF)
    within(got[:, inter:], want["du"], want["du_tol"] * (1 + BF), "d(up)", rel=BF)
    check_guard(buf, o, rows, 2 * inter)
    if with_a:
        within(layer.values(host_bits(a)), want["a"], want["a_tol"] * (1 + BF), "a", rel=BF)
        check_guard(abuf, ao, rows, inter)


@pytest.mark.parametrize("rows,inter,fmt,blockwise", [(1, 32, 0, False), (300, 2048, 0, False), (33, 1056, 1, False),
                                                      (7, 96, 0, False), (40, 512, 0, True)])
def test_swiglu_backward_from_checkpoint(fp8, rows, inter, fmt, blockwise):
    """From the checkpoint of the forward call, and from a blockwise cast of h (its
    records are read the same way)."""
    rng = np.random.default_rng(rows + inter * 3)
    hb = make_h(rng, rows, inter)
    dab = workloads.bf16_bits(rng.standard_normal((rows, inter)).astype(np.float32) * 1e-3)
    h = dev_bf16(hb)
    hq, rec = torch.empty((rows, 2 * inter), dtype=torch.uint8, device=DEV), fp8.mx_scale_records(rows, 2 * inter)
    say("swiglu backward from checkpoint", rows, inter, fmt, blockwise)
    if blockwise:
        fp8.fp8_blockwise_quantize_act(h, fmt, hq, rec)
    else:
        fp8.fp8_swiglu_quantize_row_mx(h, 0, 0, torch.empty((rows, inter), dtype=torch.uint8, device=DEV),
                                       torch.empty(rows, device=DEV), hq, fmt, rec)
    dh, buf, o = guarded(rows, 2 * inter, torch.bfloat16)
    a = torch.empty((rows, inter), dtype=torch.bfloat16, device=DEV)
    fp8.fp8_mx_swiglu_backward(dev_bf16(dab), hq, fmt, rec, dh, a=a)
    torch.cuda.synchronize()
    v = layer.mx_values(hq.cpu().numpy(), fmt, layer.from_records(rec.cpu().numpy(), 2 * inter))
    want = layer.swiglu_backward(layer.values(dab), v[:, :inter], v[:, inter:])
    got = layer.values(host_bits(dh))
    within(got[:, :inter], want["dg"], want["dg_tol"] * (1 + BF), "d(gate)", rel=BF)
    within(got[:, inter:], want["du"], want["du_tol"] * (1 + BF), "d(up)", rel=BF)
    within(layer.values(host_bits(a)), want["a"], want["a_tol"] * (1 + BF), "a", rel=BF)
    check_guard(buf, o, rows, 2 * inter)


def test_swiglu_backward_every_gate(fp8):
    """Every finite bf16 gate with up = da = 1: the gradients' shape over the whole
    range (no overflow at either end), and the infinities as the formula gives them."""
    g = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    hb = np.full((1 << 16, 16), 0x3F80, np.uint16)
    hb[:, 0] = g
    da = np.full((1 << 16, 8), 0x3F80, np.uint16)
    dh = torch.empty((1 << 16, 16), dtype=torch.bfloat16, device=DEV)
    say("swiglu backward, every gate")
    fp8.fp8_swiglu_backward(dev_bf16(da), dev_bf16(hb), dh)
    torch.cuda.synchronize()
    got = layer.values(host_bits(dh))
    v = layer.values(g)
    fin = np.isfinite(v)
    want = layer.swiglu_backward(np.ones(fin.sum()), v[fin], np.ones(fin.sum()))
    within(got[fin, 0], want["dg"], want["dg_tol"] * (1 + BF), "d(gate)", rel=BF)
    within(got[fin, 8], want["du"], want["du_tol"] * (1 + BF), "d(up)", rel=BF)
    assert np.all(np.isnan(got[~fin, 0]))
    inf = np.nonzero(g == 0x7F80)[0][0]
    assert got[inf, 8] == np.inf                            # silu(Inf) = Inf
    assert np.all(np.isnan(got[np.isnan(v), 8]))


def test_swiglu_backward_against_differences(fp8):
    """d(gate) and d(up) with da = 1 against central differences of the library's own
    a (bf16): error of the differences is a's half steps over the perturbation and
    the third derivative of silu (below 0.5) times h^2 / 6."""
    n, h = 64, 2.0 ** -3
    rng = np.random.default_rng(5)
    g = np.round(rng.uniform(-4, 4, n) * 8) / 8
    u = np.round(rng.uniform(-2, 2, n) * 8) / 8
    rows = np.stack([np.concatenate(r) for r in ((g + h, u), (g - h, u), (g, u + h), (g, u - h), (g, u))])
    hb = workloads.bf16_bits(rows.astype(np.float32))
    dh, a = torch.empty((5, 2 * n), dtype=torch.bfloat16, device=DEV), torch.empty((5, n), dtype=torch.bfloat16,
                                                                                 device=DEV)
    say("swiglu differences")
    fp8.fp8_swiglu_backward(torch.ones((5, n), dtype=torch.bfloat16, device=DEV), dev_bf16(hb), dh, a=a)
    torch.cuda.synchronize()
    a, d = a.double().cpu().numpy(), dh.double().cpu().numpy()[4]
    dg, du = (a[0] - a[1]) / (2 * h), (a[2] - a[3]) / (2 * h)
    step = np.abs(a[:4]).max(0) * BF / h
    assert np.all(np.abs(d[:n] - dg) <= step + np.abs(dg) * BF + np.abs(u) * 0.5 * h * h / 6)
    assert np.all(np.abs(d[n:] - du) <= step + np.abs(du) * BF)


def test_swiglu_no_rows(fp8):
    say("swiglu no rows")
    h = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    q, hq = torch.empty((0, 64), dtype=torch.uint8, device=DEV), torch.empty((0, 128), dtype=torch.uint8, device=DEV)
    fp8.fp8_swiglu_quantize_row_mx(h, 0, 0, q, torch.empty(0, device=DEV), hq, 0, fp8.mx_scale_records(0, 128))
    fp8.fp8_swiglu_backward(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), h, torch.empty_like(h))
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", [0, 1])
def test_swiglu_checkpoint_of_every_value(fp8, fmt):
    """Every bf16 pattern, 32 neighbours a block (subnormal, Inf and NaN blocks among
    them), and blocks of one loud value among tiny ones: the checkpoint is
    fp8_mx_quantize_row's, bit for bit."""
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16).reshape(1024, 64)
    mixed = bits.copy()
    mixed[:, ::32] = np.random.default_rng(1).permutation(bits.reshape(-1))[:2048].reshape(1024, 2)
    h = dev_bf16(np.concatenate([bits, mixed]))
    say("swiglu checkpoint of every value", fmt)
    q, si = torch.empty((2048, 32), dtype=torch.uint8, device=DEV), torch.empty(2048, device=DEV)
    hq, rec = torch.empty((2048, 64), dtype=torch.uint8, device=DEV), fp8.mx_scale_records(2048, 64)
    hq0, rec0 = torch.empty_like(hq), torch.empty_like(rec)
    fp8.fp8_swiglu_quantize_row_mx(h, 0, 0, q, si, hq, fmt, rec)
    fp8.fp8_mx_quantize_row(h, fmt, hq0, rec0)
    torch.cuda.synchronize()
    assert torch.equal(rec, rec0) and torch.equal(hq, hq0)


def test_swiglu_many_rows(fp8):
    """More rows than one launch takes, forward (2^20 rows) and backward (2^24 chunks
    of 8): the rows at the cut and the last ones are those of a call on them alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    say("swiglu many rows")
    rows = (1 << 20) + 21
    h = torch.randn((rows, 64), device=DEV, generator=g, dtype=torch.bfloat16)

    def save(h):
        n = h.shape[0]
        q, si = torch.empty((n, 32), dtype=torch.uint8, device=DEV), torch.empty(n, device=DEV)
        hq, rec = torch.empty((n, 64), dtype=torch.uint8, device=DEV), fp8.mx_scale_records(n, 64)
        fp8.fp8_swiglu_quantize_row_mx(h, 0, 0, q, si, hq, 0, rec)
        return q, si, hq, rec[0]

    whole = save(h)
    for lo, hi in (((1 << 20) - 8, (1 << 20) + 8), (rows - 9, rows)):
        part = save(h[lo:hi])
        torch.cuda.synchronize()
        assert all(torch.equal(a[lo:hi], b) for a, b in zip(whole, part)), (lo, hi)
    rows = (1 << 24) + 300
    h = torch.randn((rows, 16), device=DEV, generator=g, dtype=torch.bfloat16)
    dh, a = torch.empty_like(h), torch.empty((rows, 8), dtype=torch.bfloat16, device=DEV)
    fp8.fp8_swiglu_backward(h[:, :8], h, dh, a=a)
    for lo, hi in ((0, 8), ((1 << 24) - 8, (1 << 24) + 8), (rows - 9, rows)):
        pd, pa = torch.empty((hi - lo, 16), dtype=torch.bfloat16, device=DEV), torch.empty(
            (hi - lo, 8), dtype=torch.bfloat16, device=DEV)
        fp8.fp8_swiglu_backward(h[lo:hi, :8], h[lo:hi], pd, a=pa)
        torch.cuda.synchronize()
        assert torch.equal(dh[lo:hi], pd) and torch.equal(a[lo:hi], pa), (lo, hi)
