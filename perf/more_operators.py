"""Cases that measure the operators of a feed-forward block between two points of the residual stream:

  add_norm       the residual's addition, the norm of the sum (RMS or layer norm) and the rowwise FP8 cast in one pass, the
                 normalised rows saved as an 8-bit checkpoint where the backward pass wants them
  add_norm_grad  its backward pass: the residual's own gradient added to the norm's, and the weights' gradients, from the
                 sum in bf16 or from the checkpoint
  glu            the gated block's FP8 products, gate and up, with silu(gate) * up in the same kernel
  glu_grad       its backward pass: the FP8 product that gives the activation's gradient, with SwiGLU's gradient in the
                 same kernel
  lora           low-rank adapters of many requests at once, added to what a shared projection gave

`run` computes them in plain torch operations, or, with `own`, through the library.
8-bit results are returned as float8 tensors: the values the codes hold, and the block scales they are multiplied by.
"""
import math

import torch

own = False

DEV = "cuda:0"
FMT = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
EPS = 1e-5


def listed():
    return [
        # between two layers for one decoded token: latency
        {"name": "add_norm_one_token", "op": "add_norm", "rows": 1, "cols": 4096, "rms": True, "save": False,
         "fmt": "e4m3"},
        # a training step of a wide model, checkpoint saved: the largest call
        {"name": "add_norm_save_large", "op": "add_norm", "rows": 16384, "cols": 7168, "rms": True, "save": True,
         "fmt": "e4m3"},
        # the gradients from the sum, a training step
        {"name": "add_norm_grad_x", "op": "add_norm_grad", "rows": 8192, "cols": 4096, "rms": False, "mx": False},
        # the same from the 8-bit checkpoint, rows of a ragged batch, y recomputed
        {"name": "add_norm_grad_saved", "op": "add_norm_grad", "rows": 2050, "cols": 7168, "rms": True, "mx": True},
        # one decoded token through a dense layer's gate and up projections: every weight is read for it
        {"name": "glu_one_token", "op": "glu", "m": 1, "k": 4096, "inter": 14336, "rowwise": True, "h": False,
         "fa": "e4m3", "fb": "e4m3"},
        # a ragged batch through a small expert, scalar scales, h kept for the backward pass
        {"name": "glu_ragged", "op": "glu", "m": 777, "k": 2048, "inter": 1408, "rowwise": False, "h": True,
         "fa": "e4m3", "fb": "e4m3"},
        # a dense layer's training step: the largest product
        {"name": "glu_train", "op": "glu", "m": 8192, "k": 4096, "inter": 14336, "rowwise": True, "h": True,
         "fa": "e4m3", "fb": "e4m3"},
        # its backward pass, the output's gradient in e5m2
        {"name": "glu_grad_train", "op": "glu_grad", "m": 8192, "k": 4096, "inter": 14336, "rowwise": True, "act": True,
         "fa": "e5m2", "fb": "e4m3"},
        # the backward pass of a ragged batch of a small expert
        {"name": "glu_grad_ragged", "op": "glu_grad", "m": 1001, "k": 2048, "inter": 1408, "rowwise": True, "act": False,
         "fa": "e5m2", "fb": "e4m3"},
        # one decoded token and its adapter: latency
        {"name": "lora_one_token", "op": "lora", "tokens": 1, "requests": 1, "k": 4096, "n": 4096, "rank": 16,
         "adapters": 4},
        # a decode batch: every token of another request, nearly every request with an adapter of its own
        {"name": "lora_decode", "op": "lora", "tokens": 32, "requests": 32, "k": 4096, "n": 14336, "rank": 16,
         "adapters": 64},
        # prompts of a few requests of odd lengths at once
        {"name": "lora_prefill", "op": "lora", "tokens": 5003, "requests": 9, "k": 4096, "n": 14336, "rank": 64,
         "adapters": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["add_norm", "add_norm_grad", "glu", "glu_grad", "lora"])
    if op in ("add_norm", "add_norm_grad"):
        marked = rng.random() < 0.5         # from or to a checkpoint: whole blocks of 32
        cols = _log(rng, 256, 8192)
        cols = (cols + 31) // 32 * 32 if marked else cols + rng.choice([0, 8 - cols % 8, 1])
        case = {"op": op, "rows": _log(rng, 1, min(16384, (1 << 26) // cols)), "cols": cols,
                "rms": rng.random() < 0.6, ("save" if op == "add_norm" else "mx"): marked}
        if op == "add_norm":
            case["fmt"] = rng.choice(["e4m3", "e5m2"])
        return case
    if op in ("glu", "glu_grad"):
        step = rng.choice([16, 256])
        k, inter = max(step, _log(rng, 256, 7168) // step * step), _log(rng, 256, 14336) // 8 * 8
        most = min(8192, 8192 * 4096 * 14336 // (k * inter))
        case = {"op": op, "m": _log(rng, 1 if op == "glu" else 64, most), "k": k, "inter": inter,
                "rowwise": rng.random() < 0.7, ("h" if op == "glu" else "act"): rng.random() < 0.5}
        case["fa"], case["fb"] = rng.choice([("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")])
        return case
    tokens = _log(rng, 1, 5003)
    return {"op": op, "tokens": tokens, "requests": _log(rng, 1, min(tokens, 64)), "k": _log(rng, 512, 4096) // 8 * 8,
            "n": _log(rng, 512, 14336) // 8 * 8, "rank": rng.choice([8, 16, 32, 64]),
            "adapters": rng.choice([1, 4, 8, 32])}


def _records_shape(rows, cols):
    return ((cols + 127) // 128, rows, 4)


def _to_records(b):
    """[rows x blocks] block bytes -> [ceil(blocks / 4) x rows x 4] records, zero bytes past the last block."""
    rows, blocks = b.shape
    j = (blocks + 3) // 4
    full = torch.zeros((rows, j * 4), dtype=torch.uint8, device=b.device)
    full[:, :blocks] = b
    return full.view(rows, j, 4).transpose(0, 1).contiguous()


def _mx_random(gen, rows, cols):
    """A checkpoint of random rows: e4m3 codes and its records (a power of two for each block of 32)."""
    v = torch.randn((rows, cols // 32, 32), device=DEV, generator=gen)
    e = (torch.floor(torch.log2(v.abs().amax(2))) - 8).clamp(-127, 127)
    codes = (v * torch.exp2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).reshape(rows, cols)
    return codes.view(torch.uint8), _to_records((e + 127).to(torch.uint8))


def _operand(gen, rows, cols, std, fmt, rowwise):
    """A random operand of an FP8 product: codes [rows x cols] and its factors, one a row or one."""
    dtype, fmax = FMT[fmt]
    x = torch.randn((rows, cols), device=DEV, generator=gen).mul_(std)
    amax = x.abs().amax(1) if rowwise else x.abs().amax().view(1)
    codes = x.mul_((fmax / amax)[:, None] if rowwise else fmax / amax).clamp_(-fmax, fmax).to(dtype)
    return codes.view(torch.uint8), amax / fmax


def _requests(case, gen):
    """The adapter of each token: requests of neighbouring tokens of odd lengths, one in eight without an adapter."""
    t, r = case["tokens"], case["requests"]
    cuts = torch.randperm(t - 1, device=DEV, generator=gen)[: r - 1] + 1 if r > 1 else torch.empty(
        0, dtype=torch.int64, device=DEV)
    of = torch.zeros(t, dtype=torch.int64, device=DEV)
    of[cuts] = 1
    who = torch.randint(case["adapters"], (r,), device=DEV, generator=gen)
    if r > 1:
        who[torch.rand(r, device=DEV, generator=gen) < 0.125] = -1
    return who[of.cumsum(0)].to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, c = case["op"], case

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, device=DEV, generator=gen).mul_(std).to(dtype)

    s = {"case": c}
    if op in ("add_norm", "add_norm_grad"):
        rows, cols = c["rows"], c["cols"]
        s["gamma"] = (1 + randn(cols, std=0.1, dtype=torch.float32)).to(torch.bfloat16)
        s["beta"] = None if c["rms"] else randn(cols, std=0.1)
        if op == "add_norm" or not c["mx"]:
            r = torch.randn((rows, cols), device=DEV, generator=gen)
            r[:, :: max(1, cols // 5)] *= 8         # a few loud channels, as in a residual stream
            r.add_(0.1)
        if op == "add_norm":
            s["x"], s["res"] = randn(rows, cols, std=0.5), r.to(torch.bfloat16)
            s["sum"] = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
            s["q"] = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
            s["scale_inv"] = torch.empty(rows, device=DEV)
            s["rstd"] = torch.empty(rows, device=DEV)
            s["mean"] = None if c["rms"] else torch.empty(rows, device=DEV)
            s["xq"] = torch.empty((rows, cols), dtype=torch.uint8, device=DEV) if c["save"] else None
            s["xs"] = torch.empty(_records_shape(rows, cols), dtype=torch.uint8, device=DEV) if c["save"] else None
            return s
        s["dsum"], s["dy"] = randn(rows, cols, std=1e-3), randn(rows, cols, std=1e-3)
        if c["mx"]:
            s["xq"], s["xs"] = _mx_random(gen, rows, cols)
            s["rstd"] = torch.rand(rows, device=DEV, generator=gen) + 0.5
            s["y"] = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
        else:
            s["sum"] = r.to(torch.bfloat16)
            xd = s["sum"].double()
            m = torch.zeros(rows, dtype=torch.float64, device=DEV) if c["rms"] else xd.mean(1)
            s["mean"] = None if c["rms"] else m.float()
            s["rstd"] = ((xd - m[:, None]).square().mean(1) + EPS).rsqrt().float()
        s["dx"] = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
        s["dgamma"] = torch.empty(cols, device=DEV)
        s["dbeta"] = None if c["rms"] else torch.empty(cols, device=DEV)
        # partial sums of the weights' gradients: at most 512 bands of rows, two sums a column
        s["workspace"] = torch.empty(512 * 2 * cols, device=DEV)
        return s
    if op in ("glu", "glu_grad"):
        m, k, inter = c["m"], c["k"], c["inter"]
        s["a"], s["sa"] = _operand(gen, m, k, 1.0 if op == "glu" else 1e-3, c["fa"], c["rowwise"])
        s["b"], s["sb"] = _operand(gen, 2 * inter if op == "glu" else inter, k, 1.3 / math.sqrt(k), c["fb"],
                                   c["rowwise"])
        wants = c["h"] if op == "glu" else c["act"]
        if op == "glu":
            s["act"] = torch.empty((m, inter), dtype=torch.bfloat16, device=DEV)
            s["h"] = torch.empty((m, 2 * inter), dtype=torch.bfloat16, device=DEV) if wants else None
        else:
            s["h"] = randn(m, 2 * inter, std=1.5)
            s["dh"] = torch.empty((m, 2 * inter), dtype=torch.bfloat16, device=DEV)
            s["act"] = torch.empty((m, inter), dtype=torch.bfloat16, device=DEV) if wants else None
        return s
    T, K, N, r, E = c["tokens"], c["k"], c["n"], c["rank"], c["adapters"]
    s["x"], s["base"] = randn(T, K), randn(T, N)
    s["lora_a"] = randn(E, r, K, std=1 / math.sqrt(K))
    s["lora_b"] = randn(E, N, r, std=0.5 / math.sqrt(r))
    s["scaling"] = 0.5 + torch.rand(E, device=DEV, generator=gen)
    s["adapter"] = _requests(c, gen)
    s["out"] = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    # partial sums of the down projections: at most 64 parts a token, 8192 rows of them in all or one a token
    s["workspace"] = torch.empty(r * max(T, min(64 * T, 8192)), device=DEV)
    return s


# ---------------------------------------------------------------- plain form --
def _cast(y, fmt):
    """Rows of fp32 values -> (codes, factor that gives the values back)."""
    dtype, fmax = FMT[fmt]
    amax = y.abs().amax(1)
    scale = torch.where(amax > 0, fmax / amax, torch.ones_like(amax))
    return (y * scale[:, None]).clamp(-fmax, fmax).to(dtype), 1.0 / scale


def _blocks(v):
    """fp32 rows -> e4m3 codes with a power of two for each block of 32, as records."""
    rows, cols = v.shape
    b = v.view(rows, cols // 32, 32)
    amax = b.abs().amax(2)
    e = torch.frexp(amax)[1] - 1 - 8
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    codes = torch.ldexp(b, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(rows, cols)
    return codes, _to_records((e + 127).to(torch.uint8)).view(torch.float8_e8m0fnu)


def _unblock(codes, records):
    """Codes and records -> fp32 values."""
    rows, cols = codes.shape
    e = records.transpose(0, 1).reshape(rows, -1)[:, : cols // 32].int() - 127
    v = codes.view(torch.float8_e4m3fn).float().view(rows, cols // 32, 32)
    return torch.ldexp(v, e[..., None]).view(rows, cols)


def _plain_add_norm(s):
    c = s["case"]
    out = {"sum": (s["x"].float() + s["res"].float()).to(torch.bfloat16)}
    d = out["sum"].float()          # the norm is the stored sum's
    if not c["rms"]:
        out["mean"] = d.mean(1)
        d = d - out["mean"][:, None]
    out["rstd"] = 1.0 / torch.sqrt(d.square().mean(1) + EPS)
    xhat = d * out["rstd"][:, None]
    y = xhat * s["gamma"].float()
    if not c["rms"]:
        y = y + s["beta"].float()
    out["q"], out["scale_inv"] = _cast(y, c["fmt"])
    if c["save"]:
        out["xq"], out["xs"] = _blocks(xhat)
    return out


def _plain_add_norm_grad(s):
    c, dy, gamma = s["case"], s["dy"].float(), s["gamma"].float()
    out = {}
    if c["mx"]:
        xhat = _unblock(s["xq"], s["xs"])
        y = xhat * gamma
        out["y"] = (y if c["rms"] else y + s["beta"].float()).to(torch.bfloat16)
    else:
        x = s["sum"].float()
        xhat = (x if c["rms"] else x - s["mean"][:, None]) * s["rstd"][:, None]
    w = dy * gamma
    d = w - xhat * (w * xhat).mean(1, keepdim=True)
    if not c["rms"]:
        d = d - w.mean(1, keepdim=True)
        out["dbeta"] = dy.sum(0)
    out["dx"] = (s["dsum"].float() + d * s["rstd"][:, None]).to(torch.bfloat16)
    out["dgamma"] = (dy * xhat).sum(0)
    return out


def _values(codes, factors, fmt):
    return codes.view(FMT[fmt][0]).float() * factors[:, None]


def _plain_glu(s):
    c = s["case"]
    h = _values(s["a"], s["sa"], c["fa"]) @ _values(s["b"], s["sb"], c["fb"]).t()
    g, u = h.chunk(2, dim=1)
    out = {"act": (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)}
    if c["h"]:
        out["h"] = h.to(torch.bfloat16)
    return out


def _plain_glu_grad(s):
    c = s["case"]
    da = _values(s["a"], s["sa"], c["fa"]) @ _values(s["b"], s["sb"], c["fb"]).t()
    g, u = s["h"].float().chunk(2, dim=1)
    sig = 1.0 / (1.0 + torch.exp(-g))
    silu = g * sig
    out = {"dh": torch.cat([da * u * sig * (1.0 + g * (1.0 - sig)), da * silu], 1).to(torch.bfloat16)}
    if c["act"]:
        out["act"] = (silu * u).to(torch.bfloat16)
    return out


def _plain_lora(s):
    c = s["case"]
    E, r = c["adapters"], c["rank"]
    v = (s["x"].float() @ s["lora_a"].float().view(E * r, -1).t()).view(-1, E, r)      # every adapter for every token
    of = s["adapter"][:, None] == torch.arange(E, device=DEV)
    v = torch.where(of[..., None], v * s["scaling"][:, None], torch.zeros_like(v))
    b = s["lora_b"].float().transpose(1, 2).reshape(E * r, -1)
    return (s["base"].float() + v.view(-1, E * r) @ b).to(torch.bfloat16)


# ------------------------------------------------------------- library calls --
def _own_add_norm(s):
    import fp8_scaled_gemm_amax_amd as fp8
    c = s["case"]
    fp8.fp8_add_norm_quantize_row(s["x"], s["res"], s["sum"], s["gamma"], s["beta"], EPS,
                                  fp8.NORM_RMS if c["rms"] else fp8.NORM_LAYER,
                                  fp8.E4M3 if c["fmt"] == "e4m3" else fp8.E5M2, 0, s["q"], s["scale_inv"],
                                  mean_out=s["mean"], rstd_out=s["rstd"], xhat_q=s["xq"], xhat_fmt=fp8.E4M3,
                                  xhat_scale=s["xs"])
    out = {"sum": s["sum"], "q": s["q"].view(FMT[c["fmt"]][0]), "scale_inv": s["scale_inv"], "rstd": s["rstd"]}
    if not c["rms"]:
        out["mean"] = s["mean"]
    if c["save"]:
        out["xq"], out["xs"] = s["xq"].view(torch.float8_e4m3fn), s["xs"].view(torch.float8_e8m0fnu)
    return out


def _own_add_norm_grad(s):
    import fp8_scaled_gemm_amax_amd as fp8
    c = s["case"]
    kind = fp8.NORM_RMS if c["rms"] else fp8.NORM_LAYER
    out = {"dx": s["dx"], "dgamma": s["dgamma"]}
    if c["mx"]:
        fp8.fp8_mx_add_norm_backward(s["dsum"], s["dy"], s["xq"], fp8.E4M3, s["xs"], s["gamma"], s["beta"], s["rstd"],
                                     kind, s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"], y=s["y"],
                                     workspace=s["workspace"])
        out["y"] = s["y"]
    else:
        fp8.fp8_add_norm_backward(s["dsum"], s["dy"], s["sum"], s["gamma"], s["mean"], s["rstd"], kind, s["dx"],
                                  dgamma=s["dgamma"], dbeta=s["dbeta"], workspace=s["workspace"])
    if not c["rms"]:
        out["dbeta"] = s["dbeta"]
    return out


def _product(fp8, c):
    fmt = {"e4m3": fp8.E4M3, "e5m2": fp8.E5M2}
    return fmt[c["fa"]], fmt[c["fb"]], fp8.SCALE_VECTOR if c["rowwise"] else fp8.SCALE_TENSOR


def _own_glu(s):
    import fp8_scaled_gemm_amax_amd as fp8
    fa, fb, mode = _product(fp8, s["case"])
    fp8.fp8_gemm_swiglu(s["a"], fa, s["b"], fb, s["sa"], mode, s["sb"], mode, s["act"], h=s["h"])
    return {"act": s["act"], "h": s["h"]} if s["case"]["h"] else {"act": s["act"]}


def _own_glu_grad(s):
    import fp8_scaled_gemm_amax_amd as fp8
    fa, fb, mode = _product(fp8, s["case"])
    fp8.fp8_gemm_swiglu_backward(s["a"], fa, s["b"], fb, s["sa"], mode, s["sb"], mode, s["h"], s["dh"], act=s["act"])
    return {"dh": s["dh"], "act": s["act"]} if s["case"]["act"] else {"dh": s["dh"]}


def _own_lora(s):
    import fp8_scaled_gemm_amax_amd as fp8
    fp8.fp8_lora_add(s["x"], s["lora_a"], s["lora_b"], s["scaling"], s["adapter"], s["base"], s["out"], s["workspace"])
    return s["out"]


PLAIN = {"add_norm": _plain_add_norm, "add_norm_grad": _plain_add_norm_grad, "glu": _plain_glu,
         "glu_grad": _plain_glu_grad, "lora": _plain_lora}
OWN = {"add_norm": _own_add_norm, "add_norm_grad": _own_add_norm_grad, "glu": _own_glu, "glu_grad": _own_glu_grad,
       "lora": _own_lora}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


def work(case):
    c, op = case, case["op"]
    if op in ("add_norm", "add_norm_grad"):
        n, rows, cols = c["rows"] * c["cols"], c["rows"], c["cols"]
        ckpt = n + n // 32
        if op == "add_norm":
            per_row = 8 if c["rms"] else 12
            return {"bytes": 7 * n + (ckpt if c["save"] else 0) + per_row * rows + (2 if c["rms"] else 4) * cols,
                    "flops": 9 * n}
        read = 4 * n + (ckpt if c["mx"] else 2 * n) + (4 if c["rms"] or c["mx"] else 8) * rows
        grads = (4 if c["rms"] else 8) * cols
        weights = 2 * cols + (2 * cols if c["mx"] and not c["rms"] else 0)
        return {"bytes": read + 2 * n + (2 * n if c["mx"] else 0) + grads + weights, "flops": 13 * n}
    if op in ("glu", "glu_grad"):
        m, k, inter = c["m"], c["k"], c["inter"]
        n = 2 * inter if op == "glu" else inter
        factors = 4 * (m + n) if c["rowwise"] else 8
        if op == "glu":
            out = 2 * m * inter + (4 * m * inter if c["h"] else 0)
        else:
            out = 8 * m * inter + (2 * m * inter if c["act"] else 0)
        return {"bytes": (m + n) * k + factors + out, "flops": 2.0 * m * n * k}
    T, K, N, r, E = c["tokens"], c["k"], c["n"], c["rank"], c["adapters"]
    used = E * (1 - (1 - 1 / E) ** c["requests"]) if E > 1 else 1       # adapters that a random choice reaches
    return {"bytes": used * 2 * r * (K + N) + T * (2 * K + 4 * N + 4), "flops": 2.0 * T * r * (K + N)}


# ------------------------------------------------------------------- 64 bits --
def _round_to(v, mbits, emin, fmax):
    """Nearest value of a format with mbits fraction bits and smallest normal exponent emin, ties to even."""
    v = v.clamp(-fmax, fmax)
    e = torch.floor(torch.log2(v.abs().clamp_min(1e-300))).clamp_min(emin)
    e = torch.where(torch.exp2(e) > v.abs(), (e - 1).clamp_min(emin), e)
    step = torch.exp2(e - mbits)
    return torch.round(v / step) * step


ROUND = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0), "bf16": (7, -126, 3.3895313892515355e38)}


def _exact_cast(y, fmt):
    s = ROUND[fmt][2] / y.abs().max(dim=1, keepdim=True)[0]
    return _round_to(y * s, *ROUND[fmt]), (1 / s)[:, 0]


def _exact_blocks(v):
    rows, cols = v.shape
    b = v.reshape(rows, cols // 32, 32)
    p = torch.exp2(torch.floor(torch.log2(b.abs().max(dim=2, keepdim=True)[0])) - 8)
    codes = _round_to(b / p, *ROUND["e4m3"]).reshape(rows, cols)
    rec = torch.full((rows, (cols + 127) // 128 * 4), 2.0 ** -127, dtype=torch.float64, device=v.device)
    rec[:, : cols // 32] = p[..., 0]
    return codes, rec.reshape(rows, -1, 4).permute(1, 0, 2).contiguous()


def _exact_values(codes, records):
    rows, cols = codes.shape
    p = torch.exp2(records.permute(1, 0, 2).reshape(rows, -1)[:, : cols // 32].double() - 127)
    return codes.view(torch.float8_e4m3fn).double() * p.repeat_interleave(32, dim=1)


def _exact_product(s, c):
    a = s["a"].view(FMT[c["fa"]][0]).double().mul_(s["sa"].double()[:, None])
    b = s["b"].view(FMT[c["fb"]][0]).double().mul_(s["sb"].double()[:, None])
    return a @ b.T


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op in ("add_norm", "add_norm_grad"):
        gamma = s["gamma"].double()
        beta = 0.0 if c["rms"] else s["beta"].double()
        if op == "add_norm":
            x = _round_to(s["x"].double() + s["res"].double(), *ROUND["bf16"])
            mu = torch.zeros_like(x[:, 0]) if c["rms"] else x.sum(1) / c["cols"]
            rstd = ((x - mu[:, None]).pow(2).sum(1) / c["cols"] + EPS).pow(-0.5)
            xhat = (x - mu[:, None]) * rstd[:, None]
            out = {"sum": x, "rstd": rstd}
            if not c["rms"]:
                out["mean"] = mu
            out["q"], out["scale_inv"] = _exact_cast(xhat * gamma + beta, c["fmt"])
            if c["save"]:
                out["xq"], out["xs"] = _exact_blocks(xhat)
            return out
        rstd = s["rstd"].double()[:, None]
        if c["mx"]:
            xhat = _exact_values(s["xq"], s["xs"])
        else:
            xhat = (s["sum"].double() - (0.0 if c["rms"] else s["mean"].double()[:, None])) * rstd
        dy = s["dy"].double()
        g = dy * gamma
        dot = (g * xhat).sum(1, keepdim=True) / c["cols"]
        shift = 0.0 if c["rms"] else g.sum(1, keepdim=True) / c["cols"]
        out = {"dx": rstd * (g - shift - xhat * dot) + s["dsum"].double(), "dgamma": (dy * xhat).sum(0)}
        if not c["rms"]:
            out["dbeta"] = dy.sum(0)
        if c["mx"]:
            out["y"] = xhat * gamma + beta
        return out
    if op == "glu":
        h = _exact_product(s, c)
        g, u = h[:, : c["inter"]], h[:, c["inter"]:]
        out = {"act": g * torch.sigmoid(g) * u}
        if c["h"]:
            out["h"] = h
        return out
    if op == "glu_grad":
        da, n = _exact_product(s, c), c["inter"]
        g, u = s["h"][:, :n].double(), s["h"][:, n:].double()
        e = torch.exp(-g)
        dh = torch.empty((c["m"], 2 * n), dtype=torch.float64, device=DEV)
        dh[:, :n] = da * u * (1 + e + g * e) / (1 + e).pow(2)
        dh[:, n:] = da * g / (1 + e)
        return {"dh": dh, "act": g * u / (1 + e)} if c["act"] else {"dh": dh}
    out = s["base"].double()
    for e in range(c["adapters"]):
        rows = torch.nonzero(s["adapter"] == e)[:, 0]
        if rows.numel():
            v = s["x"][rows].double() @ s["lora_a"][e].double().T
            out[rows] += s["scaling"][e].double() * (v @ s["lora_b"][e].double().T)
    return out
