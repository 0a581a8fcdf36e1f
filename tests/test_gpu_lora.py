"""GPU parity of the adapters of many requests against the fp64 definition of
oracle/block.py: every output within the bound of an fp32 evaluation plus half a
step of bf16. Ranks, odd lengths, requests in any order, tokens without an adapter,
views with guard bands, in place, NaN and Inf in other requests' data."""
import numpy as np
import pytest
import torch

import workloads
from helpers import check_guard, dev_bf16, guarded, host_bits, say
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


def normal(rng, *shape, std=1.0):
    b = workloads.bf16_bits((std * rng.standard_normal(shape)).astype(np.float32).reshape(-1, shape[-1])).reshape(shape)
    return b, layer.values(b)


def adapters_of(rng, how, tokens, E):
    if how == "one":
        return np.zeros(tokens, np.int32)
    if how == "none":
        return np.full(tokens, -1, np.int32)
    if how == "each":                           # every token another, out of range ones among them
        return rng.integers(-2, E + 2, tokens).astype(np.int32)
    idx = np.empty(tokens, np.int32)            # requests of neighbouring tokens of odd lengths
    t = 0
    while t < tokens:
        n = int(rng.integers(1, 40))
        idx[t:t + n] = rng.integers(-1, E)
        t += n
    return idx


CASES = [  # tokens, k, n, rank, adapters, how, base, row padding of base and out
    (1, 8, 1, 8, 1, "one", True, 0), (1, 4096, 4096, 16, 4, "each", True, 8), (1, 1024, 200, 128, 2, "one", False, 8),
    (2, 72, 17, 24, 3, "each", True, 3), (15, 512, 256, 8, 40, "each", True, 8), (16, 520, 264, 16, 2, "each", True, 8),
    (17, 4096, 512, 32, 64, "each", True, 0), (33, 1000, 1001, 40, 5, "runs", True, 1), (64, 2048, 640, 64, 7, "each", False, 8),
    (100, 264, 130, 104, 3, "runs", True, 6), (300, 640, 392, 16, 9, "runs", True, 8), (257, 136, 96, 128, 4, "each", True, 8),
    (40, 256, 128, 16, 3, "none", True, 8), (1025, 520, 264, 64, 3, "runs", True, 8), (2100, 264, 520, 16, 20, "each", True, 8),
    (1300, 1024, 300, 8, 2, "one", True, 4), (9000, 64, 40, 16, 5, "runs", True, 8), (600, 2048, 72, 48, 1, "one", False, 8),
    (64, 128, 520, 32, 70, "each", True, 8), (65, 136, 1032, 64, 70, "each", True, 8), (512, 328, 776, 16, 3, "each", True, 8),
    (513, 200, 264, 32, 2, "runs", True, 8), (514, 1032, 2000, 112, 1, "one", True, 8), (700, 64, 520, 16, 3, "none", True, 8),
    (200, 64, 130, 8, 4, "one", True, 2),
]


@pytest.mark.parametrize("tokens,k,n,rank,E,how,with_base,pad", CASES)
def test_lora_add(fp8, tokens, k, n, rank, E, how, with_base, pad):
    rng = np.random.default_rng(tokens + k * 3 + n)
    xb, x = normal(rng, tokens, k)
    ab, a = normal(rng, E, rank, k, std=k ** -0.5)
    bb, b = normal(rng, E, n, rank, std=rank ** -0.5)
    baseb, base = normal(rng, tokens, n)
    if not with_base:
        base = np.zeros_like(base)
    scaling = (0.25 + rng.random(E)).astype(np.float32)
    idx = adapters_of(rng, how, tokens, E)
    want, tol = block.lora(x, a, b, scaling, idx, base)
    xd = torch.full((tokens, k + 8), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :k]
    xd.copy_(dev_bf16(xb))
    ad = torch.full((E, rank + 1, k + 16), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :rank, :k]
    ad.copy_(dev_bf16(ab))
    bd = torch.full((E, n + 2, rank + 8), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :n, :rank]
    bd.copy_(dev_bf16(bb))
    based = None
    if with_base:
        based = torch.full((tokens, n + pad), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :n]
        based.copy_(dev_bf16(baseb))
    out, buf, o = guarded(tokens, n, torch.bfloat16, ld=n + pad)
    ws = fp8.lora_workspace(tokens, rank)
    guard = torch.full((ws.numel() + 64,), 3.0, device=DEV)
    say("adapters", tokens, k, n, rank, E, how, with_base, pad)
    args = (xd, ad, bd, torch.from_numpy(scaling).to(DEV), torch.from_numpy(idx).to(DEV))
    fp8.fp8_lora_add(*args, based, out, guard[:ws.numel()])
    torch.cuda.synchronize()
    assert (guard[ws.numel():] == 3.0).all(), "writes past the workspace"
    got = layer.values(host_bits(out))
    within(got, want, tol, "out")
    none = (idx < 0) | (idx >= E)
    assert np.array_equal(got[none], base[none]), "a token without an adapter keeps its base"
    check_guard(buf, o, tokens, n)
    # the same bits again, and in place
    again = torch.empty((tokens, n), dtype=torch.bfloat16, device=DEV)
    if with_base:
        again.copy_(based)
        fp8.fp8_lora_add(*args, again, again, ws)
    else:
        fp8.fp8_lora_add(*args, None, again, ws)
    torch.cuda.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("tokens", [5, 40, 300, 1100])
def test_requests_stay_apart(fp8, tokens):
    """NaN and Inf in a token, in an adapter and in a factor reach only the tokens
    that they belong to; an infinite weight of B gives Inf, not NaN."""
    rng = np.random.default_rng(tokens)
    k, n, rank, E = 136, 72, 16, 6
    idx = rng.integers(-1, E, tokens).astype(np.int32)
    idx[:5] = [0, 1, 2, 3, 4]
    x = torch.randn((tokens, k), device=DEV).to(torch.bfloat16)
    a = torch.randn((E, rank, k), device=DEV).to(torch.bfloat16)
    b = torch.randn((E, n, rank), device=DEV).to(torch.bfloat16)
    base = torch.randn((tokens, n), device=DEV).to(torch.bfloat16)
    base[3] = -0.0
    sc = torch.ones(E, device=DEV)
    ids = torch.from_numpy(idx).to(DEV)
    ws = fp8.lora_workspace(tokens, rank)
    clean, out = torch.empty_like(base), torch.empty_like(base)
    say("adapters, NaN", tokens)
    fp8.fp8_lora_add(x, a, b, sc, ids, base, clean, ws)
    x[0, 7] = float("nan")
    a[1, 3, k - 1] = float("inf")
    sc[2] = float("nan")
    b[4, n - 1, 2] = float("inf")
    fp8.fp8_lora_add(x, a, b, sc, ids, base, out, ws)
    torch.cuda.synchronize()
    assert torch.isnan(out[0]).all()
    hit = torch.isin(ids, torch.tensor([1, 2, 4], device=DEV, dtype=torch.int32))
    hit[0] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert torch.isnan(out[2]).all() and not torch.isfinite(out[1]).any()
    four = (ids == 4).nonzero()[:, 0]
    assert torch.isinf(out[four, n - 1]).all() and torch.equal(out[four, :n - 1], clean[four, :n - 1])


def test_negative_zero_base(fp8):
    """The base of a token without an adapter is copied bit for bit."""
    base = torch.tensor([[-0.0, 1.0, float("inf"), -0.0]], device=DEV).to(torch.bfloat16).repeat(3, 5)
    x = torch.zeros((3, 8), dtype=torch.bfloat16, device=DEV)
    a, b = torch.zeros((1, 8, 8), dtype=torch.bfloat16, device=DEV), torch.zeros((1, 20, 8), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(base)
    say("adapters, -0")
    fp8.fp8_lora_add(x, a, b, torch.ones(1, device=DEV), torch.full((3,), -1, dtype=torch.int32, device=DEV), base, out,
                     fp8.lora_workspace(3, 8))
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(out), host_bits(base))


def test_empty(fp8):
    say("adapters, no tokens")
    bf = dict(dtype=torch.bfloat16, device=DEV)
    fp8.fp8_lora_add(torch.empty((0, 16), **bf), torch.zeros((1, 8, 16), **bf), torch.zeros((1, 32, 8), **bf),
                     torch.ones(1, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), torch.empty((0, 32), **bf),
                     torch.empty((0, 32), **bf), torch.empty(0, device=DEV))
    torch.cuda.synchronize()


def spread(t, ld):
    """t with its rows ld elements apart."""
    rows, cols = t.shape
    far = torch.empty((rows - 1) * ld + cols, dtype=t.dtype, device=DEV).as_strided((rows, cols), (ld, 1))
    return far.copy_(t)


def test_rows_far_apart(fp8):
    """Leading dimensions at their limit: the rows of one workgroup span 2 GiB."""
    tokens, k, n, rank, E, ld = 130, 72, 43, 16, 3, (1 << 24) - 8
    x = torch.randn((tokens, k), device=DEV).to(torch.bfloat16)
    a = torch.randn((E, rank, k), device=DEV).to(torch.bfloat16)
    b = torch.randn((E, n, rank), device=DEV).to(torch.bfloat16)
    base = torch.randn((tokens, n), device=DEV).to(torch.bfloat16)
    ids = (torch.arange(tokens, device=DEV, dtype=torch.int32) * 7) % 5 - 1
    sc, ws = torch.rand(E, device=DEV), fp8.lora_workspace(tokens, rank)
    near = torch.empty_like(base)
    say("adapters, rows far apart")
    fp8.fp8_lora_add(x, a, b, sc, ids, base, near, ws)
    af = spread(a.reshape(E * rank, k), ld).as_strided((E, rank, k), (rank * ld, ld, 1))
    bf = spread(b.reshape(E * n, rank), ld).as_strided((E, n, rank), (n * ld, ld, 1))
    out = spread(torch.zeros_like(base), ld)
    fp8.fp8_lora_add(spread(x, ld), af, bf, sc, ids, spread(base, ld), out, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, near)


@pytest.mark.parametrize("index", [-(1 << 31), -1, 3, (1 << 31) - 1])
def test_indices_without_an_adapter(fp8, index):
    tokens, k, n, rank, E = 70, 64, 300, 8, 3
    x = torch.full((tokens, k), float("nan"), dtype=torch.bfloat16, device=DEV)
    a = torch.full((E, rank, k), float("nan"), dtype=torch.bfloat16, device=DEV)
    b = torch.full((E, n, rank), float("nan"), dtype=torch.bfloat16, device=DEV)
    base = torch.randn((tokens, n), device=DEV).to(torch.bfloat16)
    out = torch.full_like(base, 3.0)
    ids = torch.full((tokens,), index, dtype=torch.int32, device=DEV)
    say("adapters, index", index)
    fp8.fp8_lora_add(x, a, b, torch.ones(E, device=DEV), ids, base, out, fp8.lora_workspace(tokens, rank))
    torch.cuda.synchronize()
    assert torch.equal(out, base)


@pytest.mark.parametrize("tokens", [1, 20, 300])
def test_largest_values(fp8, tokens):
    """A value between bf16's largest and fp32's stays finite (the definition's output is 64
    times its quotient by 2^126); past fp32's it is Inf, for that adapter's tokens alone."""
    k, n, rank = 8, 40, 8
    x = torch.zeros((tokens, k), device=DEV)
    x[:, 1] = 2.0 ** 63
    a, b = torch.zeros((3, rank, k), device=DEV), torch.zeros((3, n, rank), device=DEV)
    a[:, 3, 1] = 2.0 ** 63
    b[:, :, 3] = 2.0 ** -120
    sc = torch.tensor([4 * (1 - 2.0 ** -24), 4.5, -4 * (1 - 2.0 ** -10)], device=DEV)
    ids = torch.arange(tokens, device=DEV, dtype=torch.int32) % 3
    out = torch.empty((tokens, n), dtype=torch.bfloat16, device=DEV)
    say("adapters, largest values", tokens)
    fp8.fp8_lora_add(x.to(torch.bfloat16), a.to(torch.bfloat16), b.to(torch.bfloat16), sc, ids, None, out,
                     fp8.lora_workspace(tokens, rank))
    torch.cuda.synchronize()
    want = torch.tensor([256.0, float("inf"), -256.0], device=DEV)      # (255.99998 and 255.75 in bf16, whose step there is 1)
    assert torch.equal(out.float(), want[ids.long()][:, None].expand(tokens, n))


@pytest.mark.parametrize("tokens,k,n,rank", [(5, 4096, 4096, 16), (300, 4096, 4096, 16), (1000, 2048, 1024, 40), (2100, 1024, 512, 8)])
def test_bits_do_not_depend_on_the_adapters_loaded(fp8, tokens, k, n, rank):
    """An adapter that is loaded beside the others changes no request's bits."""
    x = torch.randn((tokens, k), device=DEV).to(torch.bfloat16)
    a = (torch.randn((200, rank, k), device=DEV) * k ** -0.5).to(torch.bfloat16)
    b = (torch.randn((200, n, rank), device=DEV) * rank ** -0.5).to(torch.bfloat16)
    base = torch.randn((tokens, n), device=DEV).to(torch.bfloat16)
    sc, ws = torch.rand(200, device=DEV) + 0.5, fp8.lora_workspace(tokens, rank)
    ids = torch.randint(-1, 8, (tokens,), device=DEV, dtype=torch.int32)
    ids[ids < 0] = -1
    outs = []
    for E in (8, 9, 64, 200):
        out = torch.empty_like(base)
        say("adapters loaded", tokens, k, n, rank, E)
        fp8.fp8_lora_add(x, a[:E], b[:E], sc[:E], ids, base, out, ws)
        torch.cuda.synchronize()
        outs.append(out)
    for out in outs[1:]:
        assert torch.equal(out, outs[0])


@pytest.mark.parametrize("tokens,n,rank", [(1, 64, 8), (40, 300, 24), (70, 264, 64), (600, 72, 128)])
def test_rank_wide_values_keep_24_bits(fp8, tokens, n, rank):
    """Two values of x A^T that differ in their 18th bit, subtracted by B: each sum of the
    definition is exact in fp32, and so is the difference."""
    k = 72
    x = torch.zeros((tokens, k), device=DEV)
    x[:, :3] = torch.tensor([1.0, 2.0 ** -9, 2.0 ** -18], device=DEV)
    a, b = torch.zeros((1, rank, k), device=DEV), torch.zeros((1, n, rank), device=DEV)
    a[0, 0, :3], a[0, rank - 1, :2] = 1.0, 1.0
    b[0, :, 0], b[0, :, rank - 1] = 3.0, -3.0
    out = torch.empty((tokens, n), dtype=torch.bfloat16, device=DEV)
    say("adapters, 24 bits", tokens, n, rank)
    fp8.fp8_lora_add(x.to(torch.bfloat16), a.to(torch.bfloat16), b.to(torch.bfloat16), torch.ones(1, device=DEV),
                     torch.zeros(tokens, dtype=torch.int32, device=DEV), None, out, fp8.lora_workspace(tokens, rank))
    torch.cuda.synchronize()
    assert (out.float() == 3 * 2.0 ** -18).all(), out.float().unique()


@pytest.mark.parametrize("tokens", [1, 3, 63, 64, 65, 130, 520, 2000, 5003])
@pytest.mark.parametrize("E", [1, 5, 64])
def test_every_block_of_columns_is_reached(fp8, tokens, E):
    """However a group's workgroups are shared out among its adapters: with x of 1 in one
    column, A of 1 and B of 1 for the token's adapter number, every output is that number."""
    k, rank = 8, 8
    x = torch.ones((tokens, k), dtype=torch.bfloat16, device=DEV)
    a = torch.zeros((E, rank, k), dtype=torch.bfloat16, device=DEV)
    a[:, 2, 5] = 1
    for how, ids in (("each", torch.arange(tokens, device=DEV) * 7 % (E + 1) - 1), ("runs", torch.arange(tokens, device=DEV) // 37 % E),
                     ("one", torch.full((tokens,), E - 1, device=DEV))):
        for n in (24, 256, 2000, 14336):
            b = torch.zeros((E, n, rank), dtype=torch.bfloat16, device=DEV)
            b[:, :, 2] = torch.arange(1, E + 1, device=DEV)[:, None]
            out = torch.full((tokens, n), float("nan"), dtype=torch.bfloat16, device=DEV)
            say("adapters, blocks of columns", tokens, E, how, n)
            fp8.fp8_lora_add(x, a, b, torch.ones(E, device=DEV), ids.to(torch.int32), None, out, fp8.lora_workspace(tokens, rank))
            torch.cuda.synchronize()
            assert torch.equal(out, (ids + 1).to(torch.bfloat16)[:, None].expand(tokens, n)), (how, n)
