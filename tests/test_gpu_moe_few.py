"""GPU parity of the MoE layer for a few tokens against its fp64 definition
(oracle/layer.py): every output within fp32 rounding of the sums plus half a
step of bf16. One to 64 tokens (every tile count), one to 64 slots, experts
that nobody names, names out of range, names twice; lengths of K that end
inside a load block; strided weights; NaN rows and NaN codes; graphs."""
import numpy as np
import pytest
import torch

import workloads
from helpers import check_guard, dev_bf16, dev_f32, dev_u8, guarded, host_bits, say
from oracle import layer
from test_gpu_norm import within

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = layer.BF16


@pytest.fixture(scope="module")
def fp8():
    import fp8_scaled_gemm_amax_amd as m
    return m


def make(orc, rng, T, k, E, H, inter, f1=0, f2=0):
    """Inputs on the host: bf16 x, indices, weights, codes and factors; the fp64
    weights they stand for."""
    d = {"x": workloads.bf16_bits(rng.standard_normal((T, H)).astype(np.float32)),
         "idx": np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(T)]).astype(
             np.int32).reshape(T, k),
         "w": rng.uniform(-1, 1, (T, k)).astype(np.float32)}
    for name, fmt, rows, cols in (("w1", f1, 2 * inter, H), ("w2", f2, H, inter)):
        b = workloads.bf16_bits(rng.standard_normal((E * rows, cols)).astype(np.float32) / np.sqrt(cols))
        q, si, _ = orc.quantize_row(b, fmt)
        d[name], d["s" + name] = q.reshape(E, rows, cols), si.reshape(E, rows)
        d["v" + name] = (orc.decode(fmt, q).astype(np.float64) * si.astype(np.float64)[:, None]).reshape(E, rows, cols)
    return d


def call(fp8, d, f1=0, f2=0, out=None, ws=None, w1=None, w2=None):
    T, H = d["x"].shape
    k, inter = d["idx"].shape[1], d["w2"].shape[2]
    if out is None:
        out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = fp8.moe_few_workspace(T, k, inter) if ws is None else ws
    fp8.fp8_moe_few_tokens(dev_bf16(d["x"]), torch.from_numpy(d["idx"]).to(DEV), dev_f32(d["w"]),
                           dev_u8(d["w1"]) if w1 is None else w1, f1, dev_f32(d["sw1"]),
                           dev_u8(d["w2"]) if w2 is None else w2, f2, dev_f32(d["sw2"]), out, ws)
    torch.cuda.synchronize()
    return out


def check(d, out, what):
    want, tol = layer.moe_few(layer.values(d["x"]), d["idx"], d["w"], d["vw1"], d["vw2"])
    within(layer.values(host_bits(out)), want, tol * (1 + BF), what, rel=BF)


CASES = [  # T, k, E, H, inter, f1, f2
    (1, 1, 1, 16, 16, 0, 0), (1, 8, 32, 256, 128, 0, 0), (5, 2, 16, 1024, 512, 1, 1), (3, 2, 8, 272, 80, 0, 1),
    (16, 4, 8, 512, 272, 1, 0), (17, 2, 4, 304, 144, 0, 0), (32, 8, 32, 256, 256, 0, 0), (33, 3, 4, 528, 64, 0, 0),
    (64, 2, 3, 1040, 112, 0, 1), (64, 64, 64, 64, 32, 0, 0), (2, 64, 1024, 32, 16, 0, 0), (7, 3, 2, 96, 48, 0, 0),
    (1, 2, 2, 7168, 2048, 0, 0), (4, 1, 8, 2064, 1040, 0, 0),
    (64, 2, 3, 5152, 80, 0, 1), (20, 3, 4, 5120, 336, 1, 0), (9, 8, 8, 5152, 272, 0, 0), (40, 1, 2, 5184, 592, 0, 0),
]


@pytest.mark.parametrize("T,k,E,H,inter,f1,f2", CASES)
def test_moe_few_parity(fp8, orc, T, k, E, H, inter, f1, f2):
    rng = np.random.default_rng(T * 5 + H)
    d = make(orc, rng, T, k, E, H, inter, f1, f2)
    out, buf, o = guarded(T, H, torch.bfloat16)
    n = T * k * inter
    ws = torch.full((n + 64,), 5.0, device=DEV)
    say("moe few", T, k, E, H, inter, f1, f2)
    call(fp8, d, f1, f2, out, ws[:n])
    check(d, out, "out")
    check_guard(buf, o, T, H)
    assert (ws[n:] == 5.0).all(), "writes past the workspace"
    # the same bits whatever the workspace held before
    again = call(fp8, d, f1, f2, ws=torch.full((n,), float("nan"), device=DEV))
    assert torch.equal(again, out)


@pytest.mark.parametrize("T,k,f1", [(16, 16, 0), (31, 9, 1), (64, 4, 0)])
def test_moe_few_many_experts(fp8, orc, T, k, f1):
    """64 experts with four tokens or more on average, where the gate and up product
    takes two row tiles a workgroup; one expert has every token, another half of
    them (both also by chance in other slots)."""
    rng = np.random.default_rng(T)
    d = make(orc, rng, T, k, 64, 176, 544, f1, 0)
    d["idx"][:, 0] = 5
    d["idx"][:T // 2 + 1, 1] = 6
    say("moe few, many experts", T, k, f1)
    out = call(fp8, d, f1, 0)
    check(d, out, "out")
    assert torch.equal(call(fp8, d, f1, 0, ws=torch.full((T * k * 544,), float("nan"), device=DEV)), out)


@pytest.mark.parametrize("T", [17, 24, 25, 33, 40, 41, 56, 57])
def test_moe_few_tiles_without_tokens(fp8, orc, T):
    """Every token at the last expert, one slot each: the down product's instance has
    tiles without tokens (17..24 and 33..56 tokens), the workspace no spare row
    (tests/test_moe_few_layout.py has the addresses)."""
    rng = np.random.default_rng(T + 100)
    d = make(orc, rng, T, 1, 2, 96, 336)
    d["idx"][:] = 1
    say("moe few, tiles without tokens", T)
    out = call(fp8, d)
    check(d, out, "out")
    assert torch.equal(call(fp8, d, ws=torch.full((T, 336), float("nan"), device=DEV)), out)


def test_moe_few_every_code(fp8, orc):
    """Every finite code of both formats decodes exactly: one-hot tokens read the
    columns of W1 = all codes back through a large gate (silu = identity)."""
    for fmt in (0, 1):
        table = orc.decode_table(fmt)
        codes = np.arange(256, dtype=np.uint8)
        codes = codes[np.isfinite(table)]
        n = len(codes)
        inter, H, T = 16, 256, 16
        w1 = np.zeros((1, 2 * inter, H), np.uint8)
        one = orc.encode(fmt, np.array([1.0], np.float32))[0]
        top = orc.encode(fmt, np.array([64.0], np.float32))[0]
        w1[0, :inter, :] = top                                          # gate 64: silu(64) = 64 in fp32
        w1[0, inter, :n] = codes
        w2 = np.zeros((1, H, inter), np.uint8)
        w2[0, 0, 0] = one
        got = []
        for t0 in range(0, H, T):
            x = np.zeros((T, H), np.float32)
            x[np.arange(T), t0 + np.arange(T)] = 1.0
            d = {"x": workloads.bf16_bits(x), "idx": np.zeros((T, 1), np.int32), "w": np.full((T, 1), 1 / 64, np.float32),
                 "w1": w1, "w2": w2, "sw1": np.ones((1, 2 * inter), np.float32), "sw2": np.ones((1, H), np.float32)}
            say("moe few codes", fmt, t0)
            got.append(call(fp8, d, fmt, fmt).float().cpu().numpy()[:, 0])
        got = np.concatenate(got)[:n]
        assert np.array_equal(got.astype(np.float64), table[codes].astype(np.float64))


def test_moe_few_indices(fp8, orc):
    """Indices out of range add nothing (a token with no valid one gets zeros), an
    expert named twice counts with both weights."""
    rng = np.random.default_rng(11)
    d = make(orc, rng, 9, 3, 5, 128, 64)
    d["idx"][0] = [-1, 5, 1 << 30]
    d["idx"][1] = [2, 2, 2]
    d["idx"][2] = [4, -7, 4]
    d["idx"][3] = [0, 1, 0]
    say("moe few indices")
    out = call(fp8, d)
    check(d, out, "out")
    assert not out[0].any()
    # no valid index at all
    d["idx"][:] = -1
    assert not call(fp8, d).any()


def test_moe_few_nan_stays_in_its_token(fp8, orc):
    """A NaN in one token's row and a NaN code in one expert's W1 and another's W2
    reach the tokens that use them and no others, for every tile of tokens."""
    rng = np.random.default_rng(12)
    T, k, E, H, inter = 40, 2, 6, 128, 64
    d = make(orc, rng, T, k, E, H, inter)
    say("moe few NaN")
    clean = call(fp8, d).float().cpu().numpy()
    d["x"][7, 3] = 0x7FC0
    d["w1"][1, 5, 9] = 0x7F
    d["w2"][2, 3, 4] = 0x7F
    got = call(fp8, d).float().cpu().numpy()
    uses1 = (d["idx"] == 1).any(1)
    uses1[7] = True
    uses2 = (d["idx"] == 2).any(1)
    assert np.isnan(got[uses1]).all()
    assert np.isnan(got[uses2 & ~uses1, 3]).all()
    rest = np.ones_like(got, bool)
    rest[uses1] = False
    rest[uses2, 3] = False
    assert np.array_equal(got[rest], clean[rest])


def test_moe_few_strided_operands(fp8, orc):
    """x and out as columns of wider tensors, weights with padded rows, experts
    apart or shared (stride 0): the same bits as contiguous ones."""
    rng = np.random.default_rng(13)
    T, k, E, H, inter = 6, 2, 4, 160, 96
    d = make(orc, rng, T, k, E, H, inter)
    say("moe few strides")
    want = call(fp8, d)
    w1 = torch.zeros((E, 2 * inter + 3, H + 16), dtype=torch.uint8, device=DEV)
    w1[:, :2 * inter, :H] = dev_u8(d["w1"])
    w2 = torch.zeros((E, H, inter + 32), dtype=torch.uint8, device=DEV)
    w2[:, :, :inter] = dev_u8(d["w2"])
    got = call(fp8, d, w1=w1[:, :2 * inter, :H], w2=w2[:, :, :inter])
    assert torch.equal(got, want)
    shared = dict(d, w1=np.repeat(d["w1"][:1], E, 0), w2=np.repeat(d["w2"][:1], E, 0))
    a = call(fp8, shared)
    b = call(fp8, shared, w1=dev_u8(d["w1"][:1]).expand(E, -1, -1), w2=dev_u8(d["w2"][:1]).expand(E, -1, -1))
    assert torch.equal(a, b)


def test_moe_few_token_alone(fp8, orc):
    """A token's result does not depend on the other tokens of the call beyond the
    order of the experts' sums: alone and in a batch of 20 both are within the bound."""
    rng = np.random.default_rng(14)
    d = make(orc, rng, 20, 2, 8, 256, 128)
    say("moe few alone")
    check(d, call(fp8, d), "batch")
    one = dict(d, x=d["x"][3:4], idx=d["idx"][3:4].copy(), w=d["w"][3:4].copy())
    check(one, call(fp8, one), "alone")


def test_moe_few_no_tokens(fp8):
    say("moe few empty")
    z = torch.empty((0, 32), dtype=torch.bfloat16, device=DEV)
    fp8.fp8_moe_few_tokens(z, torch.empty((0, 2), dtype=torch.int32, device=DEV), torch.empty((0, 2), device=DEV),
                           torch.zeros((2, 32, 32), dtype=torch.uint8, device=DEV), 0, torch.ones((2, 32), device=DEV),
                           torch.zeros((2, 32, 16), dtype=torch.uint8, device=DEV), 0, torch.ones((2, 32), device=DEV),
                           z, fp8.moe_few_workspace(0, 2, 16))
    torch.cuda.synchronize()


def test_moe_few_in_graphs(fp8, orc):
    """Captured and replayed: two graphs that share a workspace, replayed in turn with
    eager calls and new inputs in the same buffers between, give the eager bits."""
    rng = np.random.default_rng(15)
    T, k, E, H, inter = 4, 2, 6, 256, 128
    d = make(orc, rng, T, k, E, H, inter)
    x, idx, w = dev_bf16(d["x"]), torch.from_numpy(d["idx"]).to(DEV), dev_f32(d["w"])
    w1, s1, w2, s2 = dev_u8(d["w1"]), dev_f32(d["sw1"]), dev_u8(d["w2"]), dev_f32(d["sw2"])
    ws = fp8.moe_few_workspace(T, k, inter)
    outs = [torch.empty((T, H), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    say("moe few graphs")

    def run(n, out, ws):
        fp8.fp8_moe_few_tokens(x[:n], idx[:n], w[:n], w1, 0, s1, w2, 0, s2, out[:n], ws)

    sizes = (4, 1)
    for n, o in zip(sizes, outs):
        run(n, o, ws)
    torch.cuda.synchronize()
    graphs = []
    for n, o in zip(sizes, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(n, o, ws)
        graphs.append(g)
    for it in range(4):
        x.copy_(dev_bf16(workloads.bf16_bits(rng.standard_normal((T, H)).astype(np.float32))))
        idx.copy_(torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)))
        for o in outs:
            o.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for n, o in zip(sizes, outs):
            eager = torch.empty_like(o)
            run(n, eager, fp8.moe_few_workspace(T, k, inter))
            torch.cuda.synchronize()
            assert torch.equal(o[:n], eager[:n]), (it, n)


def test_moe_few_two_streams(fp8, orc):
    """Two calls at once, each with its own workspace, give the bits of a call alone."""
    rng = np.random.default_rng(16)
    d = [make(orc, rng, 12, 2, 6, 512, 256) for _ in range(2)]
    say("moe few two streams")
    want = [call(fp8, x) for x in d]
    args = []
    for x in d:
        args.append((dev_bf16(x["x"]), torch.from_numpy(x["idx"]).to(DEV), dev_f32(x["w"]), dev_u8(x["w1"]), 0,
                     dev_f32(x["sw1"]), dev_u8(x["w2"]), 0, dev_f32(x["sw2"])))
    outs = [[torch.empty((12, 512), dtype=torch.bfloat16, device=DEV) for _ in range(5)] for _ in d]
    wss = [fp8.moe_few_workspace(12, 2, 256) for _ in d]
    streams = [torch.cuda.Stream() for _ in d]
    torch.cuda.synchronize()
    for i in range(5):
        for a, o, w, s in zip(args, outs, wss, streams):
            with torch.cuda.stream(s):
                fp8.fp8_moe_few_tokens(*a, o[i], w)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in o)


@pytest.mark.parametrize("T,inter", [(1, 336), (12, 336), (20, 272), (40, 80), (64, 16)])
def test_moe_few_infinite_codes(fp8, orc, T, inter):
    """Infinite codes (e5m2) of W1 and W2 give what the definition's arithmetic gives: an
    infinite output of the activation's sign from W2, whichever sign the activation's low
    part has, NaN where two of them meet with opposite signs; infinite gates and ups from
    W1 (a gate of -Inf is NaN). Every other output stays within its bound."""
    rng = np.random.default_rng(T + inter)
    k, E, H = 2, 4, 64
    d = make(orc, rng, T, k, E, H, inter, 1, 1)
    d["x"] = np.where((d["x"] & 0x7FFF) == 0, 0x3F80, d["x"]).astype(np.uint16)

    def put(name, e, row, col, code):
        d[name][e, row, col] = code
        d["v" + name][e, row, col] = np.inf if code == 0x7C else -np.inf

    for row in range(0, 40):                                        # every place of K in turn
        put("w2", 0, row, (row * 37) % inter, 0x7C if row % 3 else 0xFC)
    put("w2", 1, 50, 3, 0x7C)
    put("w2", 1, 50, 7, 0xFC)                                       # Inf or NaN, as the activations' signs meet
    put("w1", 3, 5, 9, 0x7C)                                        # a gate
    put("w1", 2, inter + 2, 17, 0xFC)                               # an up
    say("moe few, infinite codes", T, inter)
    got = layer.values(host_bits(call(fp8, d, 1, 1)))
    with np.errstate(invalid="ignore", over="ignore"):
        want, tol = layer.moe_few(layer.values(d["x"]), d["idx"], d["w"], d["vw1"], d["vw2"])
    assert np.isinf(want).any()
    for same in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(same(got), same(want)), (same.__name__, np.argwhere(same(got) != same(want))[:3])
    fin = np.isfinite(want)
    if fin.any():
        within(got[fin], want[fin], tol[fin] * (1 + BF), "finite outputs", rel=BF)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_moe_few_largest_activations(fp8, orc, sign):
    """An activation between bf16's largest value and fp32's is finite: its parts are bf16's
    largest value and the rest, and the output follows the definition."""
    H = inter = 16
    one = orc.encode(1, np.array([1.0], np.float32))[0]
    d = {"x": np.zeros((1, H), np.uint16), "idx": np.zeros((1, 1), np.int32), "w": np.ones((1, 1), np.float32),
         "w1": np.zeros((1, 2 * inter, H), np.uint8), "w2": np.zeros((1, H, inter), np.uint8),
         "sw1": np.ones((1, 2 * inter), np.float32), "sw2": np.full((1, H), 2.0 ** -100, np.float32)}
    d["x"][0, 0] = 0x3F80
    d["w1"][0, 0, 0] = d["w1"][0, inter, 0] = d["w2"][0, 5, 0] = one
    gate, up = np.float32(1.8432e19), np.float32(sign * 3.4e38 / 1.8432e19)
    d["sw1"][0, 0], d["sw1"][0, inter] = gate, up
    want = float(gate) * float(up)
    assert 3.3962e38 < abs(want) < 3.4028e38
    say("moe few, largest activations", sign)
    got = layer.values(host_bits(call(fp8, d, 1, 1)))[0]
    want *= 2.0 ** -100
    # two roundings of the activation, its two parts to 2^-16, the output's half step
    assert abs(got[5] - want) <= (BF + 2.0 ** -16 + 4 * layer.U) * abs(want) * (1 + BF)
    assert not got[:5].any() and not got[6:].any()


@pytest.mark.parametrize("T,k", [(9, 2), (40, 3)])
def test_moe_few_other_tokens_values(fp8, orc, T, k):
    """With the same routing a token's bits do not depend on the other tokens' values,
    NaN and Inf among them."""
    rng = np.random.default_rng(T + 21)
    d = make(orc, rng, T, k, 4, 144, 80)
    say("moe few, other tokens' values", T, k)
    want = call(fp8, d)
    for t in (0, 5, T - 1):
        x = workloads.bf16_bits(rng.standard_normal((T, 144)).astype(np.float32) * 100)
        x[::2, 3], x[1::2, 4] = 0x7FC0, 0xFF80
        x[t] = d["x"][t]
        assert torch.equal(call(fp8, dict(d, x=x))[t], want[t]), t
