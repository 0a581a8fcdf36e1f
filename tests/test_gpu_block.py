"""A feed-forward block's operators together. Training: residual + norm + cast ->
gate and up products with SwiGLU -> down product -> residual + norm, and the
backward pass through the library, against the fp64 gradient of the same block.
Serving: the same forward with adapters beside the down projection, for one token,
a decode batch and a prompt. Both captured into graphs and replayed with new
inputs, and on side streams at the same time: the bits of an eager run."""
import numpy as np
import pytest
import torch

import workloads
from helpers import dev_bf16, host_bits, say
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


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


def bits(rng, *shape, std=1.0):
    return workloads.bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))


class Block:
    """s1 = x + res, out = W2 (silu(G n) * (U n)), n = rms(s1) gamma1, y = layer(s1 + out) gamma2."""

    def __init__(self, fp8, m, hidden, inter, seed):
        rng = np.random.default_rng(seed)
        self.fp8, self.m, self.H, self.I = fp8, m, hidden, inter
        self.host = {"x": bits(rng, m, hidden), "res": bits(rng, m, hidden, std=2.0),
                     "g1": workloads.bf16_bits((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32)),
                     "g2": workloads.bf16_bits((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32)),
                     "w1": bits(rng, 2 * inter, hidden, std=hidden ** -0.5),
                     "w2": bits(rng, hidden, inter, std=inter ** -0.5),
                     "dy": bits(rng, m, hidden, std=1e-3), "ds2": bits(rng, m, hidden, std=1e-3)}
        self.d = d = {k: dev_bf16(v) for k, v in self.host.items()}
        self.buf = b = {"s1": bf(m, hidden), "s2": bf(m, hidden), "y": bf(m, hidden), "nq": u8(m, hidden), "ns": f32(m),
                        "r1": f32(m), "xq": u8(m, hidden), "xs": fp8.mx_scale_records(m, hidden), "act": bf(m, inter),
                        "h": bf(m, 2 * inter), "aq": u8(m, inter), "as": f32(m), "out": bf(m, hidden), "m2": f32(m),
                        "r2": f32(m), "yq": u8(m, hidden), "ys": f32(m), "w1q": u8(2 * inter, hidden), "w1s": f32(2 * inter),
                        "w2q": u8(hidden, inter), "w2s": f32(hidden), "dx2": bf(m, hidden), "dg2": f32(hidden),
                        "db2": f32(hidden), "dh": bf(m, 2 * inter), "dact": bf(m, inter), "dn": bf(m, hidden), "n": bf(m, hidden),
                        "dx": bf(m, hidden), "dg1": f32(hidden), "dw1": bf(2 * inter, hidden), "dw2": bf(hidden, inter),
                        "ws": fp8.norm_workspace(m, hidden)}
        for n, (r, c) in {"dx2": (m, hidden), "dh": (m, 2 * inter)}.items():
            b.update({n + "q": u8(r, c), n + "s": f32(r), n + "a": f32(r)})
        for n, (r, c) in {"dx2": (m, hidden), "dh": (m, 2 * inter), "w1": (2 * inter, hidden), "w2": (hidden, inter),
                          "act": (m, inter), "n": (m, hidden)}.items():
            b.update({n + "t": u8(c, r), n + "ts": f32(c), n + "ta": f32(c)})
        fp8.fp8_quantize_row(d["w1"], fp8.E4M3, 0, b["w1q"], b["w1s"])
        fp8.fp8_quantize_row(d["w2"], fp8.E4M3, 0, b["w2q"], b["w2s"])
        torch.cuda.synchronize()

    def product(self, a, sa, b, sb, d, fa=0):
        f = self.fp8
        f.fp8_gemm_scaled(a, fa, b, f.E4M3, sa, f.SCALE_VECTOR, sb, f.SCALE_VECTOR, d)

    def forward(self, lora=None):
        f, b, d = self.fp8, self.buf, self.d
        V = f.SCALE_VECTOR
        f.fp8_add_norm_quantize_row(d["x"], d["res"], b["s1"], d["g1"], None, 1e-5, f.NORM_RMS, f.E4M3, 0, b["nq"], b["ns"],
                                    rstd_out=b["r1"], xhat_q=b["xq"], xhat_scale=b["xs"])
        f.fp8_gemm_swiglu(b["nq"], f.E4M3, b["w1q"], f.E4M3, b["ns"], V, b["w1s"], V, b["act"], h=b["h"])
        f.fp8_quantize_row(b["act"], f.E4M3, 0, b["aq"], b["as"])
        self.product(b["aq"], b["as"], b["w2q"], b["w2s"], b["out"])
        if lora is not None:
            f.fp8_lora_add(b["act"], lora["a"], lora["b"], lora["c"], lora["idx"], b["out"], b["out"], lora["ws"])
        f.fp8_add_norm_quantize_row(b["out"], b["s1"], b["s2"], d["g2"], None, 1e-5, f.NORM_LAYER, f.E4M3, 0, b["yq"], b["ys"],
                                    y=b["y"], mean_out=b["m2"], rstd_out=b["r2"])

    def backward(self):
        f, b, d = self.fp8, self.buf, self.d
        V = f.SCALE_VECTOR
        f.fp8_add_norm_backward(d["ds2"], d["dy"], b["s2"], d["g2"], b["m2"], b["r2"], f.NORM_LAYER, b["dx2"],
                                dgamma=b["dg2"], dbeta=b["db2"], workspace=b["ws"])
        f.fp8_quantize_rowcol(b["dx2"], f.E5M2, 0, b["dx2q"], b["dx2s"], b["dx2a"], b["dx2t"], b["dx2ts"], b["dx2ta"])
        f.fp8_quantize_col(d["w2"], f.E4M3, 0, b["w2t"], b["w2ts"], b["w2ta"])
        f.fp8_gemm_swiglu_backward(b["dx2q"], f.E5M2, b["w2t"], f.E4M3, b["dx2s"], V, b["w2ts"], V, b["h"], b["dh"],
                                   act=b["dact"])
        f.fp8_quantize_col(b["dact"], f.E4M3, 0, b["actt"], b["actts"], b["actta"])
        self.product(b["dx2t"], b["dx2ts"], b["actt"], b["actts"], b["dw2"], fa=f.E5M2)
        f.fp8_quantize_rowcol(b["dh"], f.E5M2, 0, b["dhq"], b["dhs"], b["dha"], b["dht"], b["dhts"], b["dhta"])
        f.fp8_quantize_col(d["w1"], f.E4M3, 0, b["w1t"], b["w1ts"], b["w1ta"])
        self.product(b["dhq"], b["dhs"], b["w1t"], b["w1ts"], b["dn"], fa=f.E5M2)
        f.fp8_mx_add_norm_backward(b["dx2"], b["dn"], b["xq"], f.E4M3, b["xs"], d["g1"], None, b["r1"], f.NORM_RMS, b["dx"],
                                   dgamma=b["dg1"], y=b["n"], workspace=b["ws"])
        f.fp8_quantize_col(b["n"], f.E4M3, 0, b["nt"], b["nts"], b["nta"])
        self.product(b["dht"], b["dhts"], b["nt"], b["nts"], b["dw1"], fa=f.E5M2)

    def exact(self):
        v = {k: layer.values(a) for k, a in self.host.items()}
        s1 = v["x"] + v["res"]
        f1 = layer.norm_forward(s1, v["g1"], None, 1e-5, True)
        h = f1["y"] @ v["w1"].T
        g, u = h[:, :self.I], h[:, self.I:]
        act = layer.swiglu(g, u)[0]
        out = act @ v["w2"].T
        f2 = layer.norm_forward(s1 + out, v["g2"], None, 1e-5, False)
        n2 = layer.norm_backward(v["dy"], f2["xhat"], v["g2"], f2["rstd"], False)
        dx2 = v["ds2"] + n2["dx"]
        s = layer.swiglu_backward(dx2 @ v["w2"], g, u)
        dh = np.concatenate([s["dg"], s["du"]], 1)
        n1 = layer.norm_backward(dh @ v["w1"], f1["xhat"], v["g1"], f1["rstd"], True)
        return {"s1": s1, "act": act, "out": out, "y": f2["y"], "dx2": dx2, "dg2": n2["dgamma"], "db2": n2["dbeta"], "dh": dh,
                "dw2": dx2.T @ act, "dw1": dh.T @ f1["y"], "dx": dx2 + n1["dx"], "dg1": n1["dgamma"]}


def test_training_step_against_fp64(fp8):
    """Every product's operands are cast to 8 bits (relative error at most 2^-4 an
    element for e4m3, 2^-3 for e5m2, of either sign), the checkpoint adds 2^-4. A
    gradient has at most eight such casts on its way; were they all to add up, 2 *
    2^-3 + 6 * 2^-4 = 0.63 of the norm; errors of independent sign stay below half
    of that."""
    say("block training step")
    B = Block(fp8, 384, 512, 640, 3)
    B.forward()
    B.backward()
    torch.cuda.synchronize()
    want = B.exact()
    for name, w in want.items():
        t = B.buf[name]
        got = layer.values(host_bits(t)) if t.dtype == torch.bfloat16 else t.double().cpu().numpy()
        rel = np.linalg.norm(got - w) / np.linalg.norm(w)
        say(name, "relative error against fp64", round(float(rel), 4))
        assert rel < (2.0 ** -8 if name == "s1" else 0.32), (name, rel)


NAMES = ("s1", "act", "h", "out", "s2", "y", "yq", "ys", "dx2", "dg2", "db2", "dh", "dact", "dw2", "dw1", "dx", "dg1")


def test_training_step_in_a_graph(fp8):
    """Captured once and replayed with new inputs, eager work between the replays."""
    say("block graph")
    L, E = Block(fp8, 256, 256, 384, 5), Block(fp8, 256, 256, 384, 5)
    for o in (L, E):
        o.forward()
        o.backward()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward()
        L.backward()
    rng = np.random.default_rng(9)
    for it in range(4):
        new = dev_bf16(bits(rng, 256, 256))
        for o in (L, E):
            o.d["x"].copy_(new)
        for n in NAMES:
            L.buf[n].zero_()
        g.replay()
        torch.cuda.synchronize()
        E.forward()
        E.backward()
        torch.cuda.synchronize()
        for n in NAMES:
            assert torch.equal(L.buf[n], E.buf[n]), (it, n)


def adapters(fp8, rng, m, hidden, inter, rank=16, E=5):
    return {"a": dev_bf16(bits(rng, E * rank, inter, std=inter ** -0.5)).view(E, rank, inter),
            "b": dev_bf16(bits(rng, E * hidden, rank, std=rank ** -0.5)).view(E, hidden, rank),
            "c": torch.from_numpy((0.5 + rng.random(E)).astype(np.float32)).to(DEV),
            "idx": torch.from_numpy(rng.integers(-1, E, m).astype(np.int32)).to(DEV), "ws": fp8.lora_workspace(m, rank)}


@pytest.mark.parametrize("m", [1, 24, 100, 700])
def test_serving_in_a_graph(fp8, m):
    """The forward pass with adapters, captured once and replayed with new tokens and
    other adapters: the bits of an eager run, and the adapters' share is there."""
    say("block serving", m)
    rng = np.random.default_rng(m)
    L, E = Block(fp8, m, 512, 640, 7), Block(fp8, m, 512, 640, 7)
    la = adapters(fp8, rng, m, 512, 640)
    lb = dict(la, ws=fp8.lora_workspace(m, 16), idx=la["idx"].clone())
    L.forward(la)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward(la)
    names = ("s1", "act", "out", "s2", "y", "yq", "ys")
    for it in range(3):
        new = dev_bf16(bits(rng, m, 512))
        idx = torch.from_numpy(rng.integers(-1, 5, m).astype(np.int32)).to(DEV)
        for o, lo in ((L, la), (E, lb)):
            o.d["x"].copy_(new)
            lo["idx"].copy_(idx)
        for n in names:
            L.buf[n].zero_()
        g.replay()
        torch.cuda.synchronize()
        E.forward(lb)
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(L.buf[n], E.buf[n]), (it, n)
        with_adapters = E.buf["out"].clone()
        E.forward()
        torch.cuda.synchronize()
        changed = (E.buf["out"] != with_adapters).any(1)
        assert torch.equal(changed, idx >= 0)


def test_on_side_streams(fp8):
    """Two streams run a block each at the same time, each with its own buffers: the bits of a run alone."""
    say("block side streams")
    rng = np.random.default_rng(6)
    pairs = []
    for seed in (1, 2):
        pairs.append((Block(fp8, 304, 256, 384, seed), adapters(fp8, rng, 304, 256, 384)))
    want = []
    for B, lo in pairs:
        B.forward(lo)
        B.backward()
        torch.cuda.synchronize()
        want.append({n: B.buf[n].clone() for n in NAMES})
        for n in NAMES:
            B.buf[n].zero_()
    streams = [torch.cuda.Stream() for _ in pairs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, (B, lo) in zip(streams, pairs):
            with torch.cuda.stream(s):
                B.forward(lo)
                B.backward()
    torch.cuda.synchronize()
    for (B, _), w in zip(pairs, want):
        for n in NAMES:
            assert torch.equal(B.buf[n], w[n]), n
