"""The layer's operators together, as a training step uses them: norm (its
checkpoint saved) -> FP8 product -> SwiGLU (its checkpoint saved) -> FP8
product, then the backward pass through the library alone, the checkpoints
taking the place of the bf16 activations. Each operator's outputs are checked
against its fp64 definition on the inputs that it got in the run, and the
gradients against the fp64 gradient of the same layer; the backward pass is
also captured into a graph and replayed."""
import numpy as np
import pytest
import torch

import workloads
from helpers import dev_bf16, host_bits, say
from oracle import layer
from test_gpu_norm import within

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = layer.BF16


@pytest.fixture(scope="module")
def fp8():
    import fp8_scaled_gemm_amax_amd as m
    return m


def u8(*shape):
    return torch.empty(shape, dtype=torch.uint8, device=DEV)


def bf(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV)


def f32(*shape):
    return torch.empty(shape, device=DEV)


class Layer:
    """A feed-forward layer y = W2 (silu(G n) * (U n)), n = norm(x), on the library."""

    def __init__(self, fp8, m, hidden, inter, rms, seed):
        rng = np.random.default_rng(seed)
        self.fp8, self.m, self.H, self.I, self.rms = fp8, m, hidden, inter, rms
        bits = lambda *s, std=1.0: workloads.bf16_bits((rng.standard_normal(s) * std).astype(np.float32))  # noqa: E731
        self.host = {"x": bits(m, hidden), "gamma": workloads.bf16_bits(
            (1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32)), "beta": bits(hidden, std=0.1),
            "w1": bits(2 * inter, hidden, std=hidden ** -0.5), "w2": bits(hidden, inter, std=inter ** -0.5),
            "dout": bits(m, hidden, std=1e-3)}
        self.d = {k: dev_bf16(v) for k, v in self.host.items()}
        self.kind = fp8.NORM_RMS if rms else fp8.NORM_LAYER
        self.beta = None if rms else self.d["beta"]
        self.buf = {"nq": u8(m, hidden), "ns": f32(m), "rstd": f32(m), "mean": f32(m), "xq": u8(m, hidden),
                    "xs": fp8.mx_scale_records(m, hidden), "w1q": u8(2 * inter, hidden), "w1s": f32(2 * inter),
                    "h": bf(m, 2 * inter), "aq": u8(m, inter), "as": f32(m), "hq": u8(m, 2 * inter),
                    "hs": fp8.mx_scale_records(m, 2 * inter), "w2q": u8(hidden, inter), "w2s": f32(hidden),
                    "out": bf(m, hidden)}
        b = self.buf
        for n, (r, c) in {"dout": (m, hidden), "dh": (m, 2 * inter)}.items():
            b.update({n + "q": u8(r, c), n + "s": f32(r), n + "a": f32(r), n + "t": u8(c, r), n + "ts": f32(c),
                      n + "ta": f32(c)})
        for n, (r, c) in {"w1": (2 * inter, hidden), "w2": (hidden, inter), "a": (m, inter), "n": (m, hidden)}.items():
            b.update({n + "t": u8(c, r), n + "ts": f32(c), n + "ta": f32(c)})
        b.update({"da": bf(m, inter), "dh": bf(m, 2 * inter), "a": bf(m, inter), "dn": bf(m, hidden), "n": bf(m, hidden),
                  "dx": bf(m, hidden), "dgamma": f32(hidden), "dbeta": f32(hidden), "dw1": bf(2 * inter, hidden),
                  "dw2": bf(hidden, inter), "ws": fp8.norm_workspace(m, hidden)})

    def product(self, a, sa, b, sb, d, fa=0, fb=0):
        f = self.fp8
        f.fp8_gemm_scaled(a, fa, b, fb, sa, f.SCALE_VECTOR, sb, f.SCALE_VECTOR, d)

    def forward(self):
        f, b, d = self.fp8, self.buf, self.d
        f.fp8_norm_quantize_row(d["x"], d["gamma"], self.beta, 1e-5, self.kind, f.E4M3, 0, b["nq"], b["ns"],
                                mean_out=None if self.rms else b["mean"], rstd_out=b["rstd"], xhat_q=b["xq"],
                                xhat_fmt=f.E4M3, xhat_scale=b["xs"])
        f.fp8_quantize_row(d["w1"], f.E4M3, 0, b["w1q"], b["w1s"])
        self.product(b["nq"], b["ns"], b["w1q"], b["w1s"], b["h"])
        f.fp8_swiglu_quantize_row_mx(b["h"], f.E4M3, 0, b["aq"], b["as"], b["hq"], f.E4M3, b["hs"])
        f.fp8_quantize_row(d["w2"], f.E4M3, 0, b["w2q"], b["w2s"])
        self.product(b["aq"], b["as"], b["w2q"], b["w2s"], b["out"])

    def backward(self):
        """dout e5m2; every weight gradient from checkpoints (h itself is not read)."""
        f, b, d = self.fp8, self.buf, self.d
        f.fp8_quantize_rowcol(d["dout"], f.E5M2, 0, b["doutq"], b["douts"], b["douta"], b["doutt"], b["doutts"],
                              b["doutta"])
        f.fp8_quantize_col(d["w2"], f.E4M3, 0, b["w2t"], b["w2ts"], b["w2ta"])
        self.product(b["doutq"], b["douts"], b["w2t"], b["w2ts"], b["da"], fa=f.E5M2)
        f.fp8_mx_swiglu_backward(b["da"], b["hq"], f.E4M3, b["hs"], b["dh"], a=b["a"])
        f.fp8_quantize_col(b["a"], f.E4M3, 0, b["at"], b["ats"], b["ata"])
        self.product(b["doutt"], b["doutts"], b["at"], b["ats"], b["dw2"], fa=f.E5M2)
        f.fp8_quantize_rowcol(b["dh"], f.E5M2, 0, b["dhq"], b["dhs"], b["dha"], b["dht"], b["dhts"], b["dhta"])
        f.fp8_quantize_col(d["w1"], f.E4M3, 0, b["w1t"], b["w1ts"], b["w1ta"])
        self.product(b["dhq"], b["dhs"], b["w1t"], b["w1ts"], b["dn"], fa=f.E5M2)
        f.fp8_mx_norm_backward(b["dn"], b["xq"], f.E4M3, b["xs"], d["gamma"], self.beta, b["rstd"], self.kind, b["dx"],
                               dgamma=b["dgamma"], dbeta=None if self.rms else b["dbeta"], y=b["n"],
                               workspace=b["ws"])
        f.fp8_quantize_col(b["n"], f.E4M3, 0, b["nt"], b["nts"], b["nta"])
        self.product(b["dht"], b["dhts"], b["nt"], b["nts"], b["dw1"], fa=f.E5M2)

    def exact(self):
        v = {k: layer.values(a) for k, a in self.host.items()}
        f = layer.norm_forward(v["x"], v["gamma"], None if self.rms else v["beta"], 1e-5, self.rms)
        h = f["y"] @ v["w1"].T
        g, u = h[:, :self.I], h[:, self.I:]
        a = layer.swiglu(g, u)[0]
        s = layer.swiglu_backward(v["dout"] @ v["w2"], g, u)
        dh = np.concatenate([s["dg"], s["du"]], 1)
        n = layer.norm_backward(dh @ v["w1"], f["xhat"], v["gamma"], f["rstd"], self.rms)
        return {"out": a @ v["w2"].T, "dw2": v["dout"].T @ a, "dw1": dh.T @ f["y"], "dx": n["dx"],
                "dgamma": n["dgamma"], "dbeta": n["dbeta"]}


@pytest.mark.parametrize("rms", [True, False])
def test_training_step(fp8, rms):
    say("layer training step", rms)
    L = Layer(fp8, 256, 512, 384, rms, 3)
    L.forward()
    L.backward()
    torch.cuda.synchronize()
    b, H, inter = L.buf, L.H, L.I
    val = lambda t: layer.values(host_bits(t))  # noqa: E731
    gv, bv = layer.values(L.host["gamma"]), None if rms else layer.values(L.host["beta"])
    # each operator on the inputs that it got
    f = layer.norm_forward(layer.values(L.host["x"]), gv, bv, np.float64(np.float32(1e-5)), rms)
    layer.cast_ok(0, b["nq"].cpu().numpy(), b["ns"].cpu().numpy(), f["y"], f["y_tol"])
    e8 = layer.from_records(b["xs"].cpu().numpy(), H)
    layer.checkpoint_ok(0, b["xq"].cpu().numpy(), e8, f["xhat"], f["xhat_tol"])
    h = val(b["h"])
    a, tol = layer.swiglu(h[:, :inter], h[:, inter:])
    layer.cast_ok(0, b["aq"].cpu().numpy(), b["as"].cpu().numpy(), a, tol)
    hv = layer.mx_values(b["hq"].cpu().numpy(), 0, layer.from_records(b["hs"].cpu().numpy(), 2 * inter))
    s = layer.swiglu_backward(val(b["da"]), hv[:, :inter], hv[:, inter:])
    within(val(b["dh"])[:, :inter], s["dg"], s["dg_tol"] * (1 + BF), "d(gate)", rel=BF)
    within(val(b["dh"])[:, inter:], s["du"], s["du_tol"] * (1 + BF), "d(up)", rel=BF)
    within(val(b["a"]), s["a"], s["a_tol"] * (1 + BF), "a", rel=BF)
    xh = layer.mx_values(b["xq"].cpu().numpy(), 0, e8)
    n = layer.norm_backward(val(b["dn"]), xh, gv, b["rstd"].double().cpu().numpy(), rms)
    within(val(b["dx"]), n["dx"], n["dx_tol"] * (1 + BF), "dx", rel=BF)
    within(b["dgamma"].cpu().numpy(), n["dgamma"], n["dgamma_tol"], "dgamma")
    y = xh * gv + (0 if rms else bv)
    within(val(b["n"]), y, 2 * layer.U * (np.abs(xh * gv) + np.abs(y)), "y", rel=BF)
    # the whole step against fp64: every product's operands are cast to 8 bits
    # (relative error at most 2^-4 an element for e4m3, 2^-3 for e5m2, of either
    # sign) and the checkpoints add 2^-4 (2^-3 where the largest codes saturate).
    # A gradient has at most six such casts on its way; were they all to add up,
    # 3 * 2^-3 + 5 * 2^-4 = 0.69 of the norm; errors of independent sign stay
    # below half of that.
    want = L.exact()
    for name in ("out", "dw2", "dw1", "dx", "dgamma") + (() if rms else ("dbeta",)):
        got = val(b[name]) if b[name].dtype == torch.bfloat16 else b[name].double().cpu().numpy()
        rel = np.linalg.norm(got - want[name]) / np.linalg.norm(want[name])
        say(name, "relative error against fp64", round(float(rel), 4))
        assert rel < 0.35, (name, rel)


def test_training_step_in_a_graph(fp8):
    """The step captured once and replayed with new inputs, eager work of the same
    buffers' shapes between the replays: the bits of an eager step."""
    say("layer graph")
    L, E = Layer(fp8, 128, 256, 256, False, 5), Layer(fp8, 128, 256, 256, False, 5)
    L.forward()
    L.backward()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward()
        L.backward()
    rng = np.random.default_rng(9)
    for it in range(4):
        new = dev_bf16(workloads.bf16_bits(rng.standard_normal((128, 256)).astype(np.float32)))
        for o in (L, E):
            o.d["x"].copy_(new)
        for n in ("out", "dx", "dw1", "dw2", "dgamma", "dbeta"):
            L.buf[n].zero_()
        g.replay()
        torch.cuda.synchronize()
        E.forward()
        E.backward()
        torch.cuda.synchronize()
        for n in ("out", "dx", "dw1", "dw2", "dgamma", "dbeta", "xq", "xs", "hq", "hs"):
            assert torch.equal(L.buf[n], E.buf[n]), (it, n)


def test_operators_on_side_streams(fp8):
    """Two streams run the norm's gradient at the same time, each with its own
    workspace: the bits of a run alone."""
    say("layer side streams")
    rng = np.random.default_rng(6)
    rows, cols = 3000, 1024
    dy, x = (dev_bf16(workloads.bf16_bits(rng.standard_normal((rows, cols)).astype(np.float32))) for _ in range(2))
    mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)

    def run(ws):
        dx, dg, db = torch.empty_like(x), f32(cols), f32(cols)
        fp8.fp8_norm_backward(dy, x, None, mean, rstd, fp8.NORM_LAYER, dx, dgamma=dg, dbeta=db, workspace=ws)
        return dx, dg, db

    want = run(fp8.norm_workspace(rows, cols))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [fp8.norm_workspace(rows, cols) for _ in range(2)]
    got = []
    for s, w in zip(streams, wss):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got += [run(w) for _ in range(3)]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
