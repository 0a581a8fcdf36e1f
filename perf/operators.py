"""Cases that measure the feed-forward layer's operators around its FP8 products:

  norm         layer norm (or its RMS form) fused with the rowwise FP8 cast, with the normalised rows saved as an
               8-bit checkpoint where the backward pass wants them
  norm_grad    its backward pass with the reduction of the weights' gradients, from x in bf16 or from the checkpoint
               (then with y recomputed for the weight gradient of the product that follows)
  swiglu       SwiGLU fused with the rowwise FP8 cast, [gate | up] saved as an 8-bit checkpoint
  swiglu_grad  its backward pass, from [gate | up] in bf16 or from the checkpoint
  moe          a whole mixture-of-experts layer with FP8 weights for a few tokens

`run` computes them in plain torch operations, or, with `own`, through the library.
8-bit results are returned as float8 tensors: the values the codes hold, and the block scales they are multiplied by.
"""
import math

import torch

own = False

DEV = "cuda:0"
FMT = {"e4m3": (torch.float8_e4m3fn, 448.0, 8), "e5m2": (torch.float8_e5m2, 57344.0, 15)}
EPS = 1e-5


def listed():
    return [
        # the norm of one decoded token: latency
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "rms": True, "save": False, "fmt": "e4m3"},
        # the norm of a training step of a wide model, checkpoint saved
        {"name": "norm_save_large", "op": "norm", "rows": 16384, "cols": 7168, "rms": True, "save": True,
         "fmt": "e4m3"},
        # the norm's gradients from x, a training step
        {"name": "norm_grad_x", "op": "norm_grad", "rows": 8192, "cols": 4096, "rms": False, "mx": False},
        # the same from the 8-bit checkpoint, rows of a ragged batch, y recomputed
        {"name": "norm_grad_saved", "op": "norm_grad", "rows": 2050, "cols": 7168, "rms": True, "mx": True},
        # a small odd width: nothing aligned to vectors
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 333, "cols": 1111, "rms": False, "mx": False},
        # a dense feed-forward layer's activation, a training step: the largest call
        {"name": "swiglu_save_large", "op": "swiglu", "rows": 8192, "inter": 14336, "fmt": "e4m3"},
        # the tokens of one small expert
        {"name": "swiglu_save_small", "op": "swiglu", "rows": 48, "inter": 2048, "fmt": "e5m2"},
        # the routed tokens of a MoE layer, from the checkpoint
        {"name": "swiglu_grad_saved", "op": "swiglu_grad", "rows": 16384, "inter": 2048, "mx": True},
        # a ragged batch from bf16
        {"name": "swiglu_grad_h", "op": "swiglu_grad", "rows": 1001, "inter": 4096, "mx": False},
        # one decoded token through one GPU's share of a large MoE layer
        {"name": "moe_one_token", "op": "moe", "tokens": 1, "topk": 8, "experts": 32, "hidden": 7168, "inter": 2048,
         "fmt": "e4m3"},
        # a few tokens through a small MoE layer: latency
        {"name": "moe_small", "op": "moe", "tokens": 5, "topk": 2, "experts": 16, "hidden": 1024, "inter": 512,
         "fmt": "e5m2"},
        # a decode batch: every expert is read
        {"name": "moe_batch", "op": "moe", "tokens": 32, "topk": 8, "experts": 32, "hidden": 7168, "inter": 2048,
         "fmt": "e4m3"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "swiglu", "swiglu_grad", "moe"])
    if op in ("norm", "norm_grad"):
        marked = rng.random() < 0.5         # from or to a checkpoint: whole blocks of 32
        cols = _log(rng, 256, 8192)
        cols = (cols + 31) // 32 * 32 if marked else cols + rng.choice([0, 8 - cols % 8, 1])
        case = {"op": op, "rows": _log(rng, 1, min(16384, (1 << 26) // cols)), "cols": cols,
                "rms": rng.random() < 0.5, ("save" if op == "norm" else "mx"): marked}
        if op == "norm":
            case["fmt"] = rng.choice(["e4m3", "e5m2"])
        return case
    if op in ("swiglu", "swiglu_grad"):
        inter = _log(rng, 256, 14336) // 32 * 32
        case = {"op": op, "rows": _log(rng, 1, min(16384, (1 << 26) // inter)), "inter": inter}
        if op == "swiglu":
            case["fmt"] = rng.choice(["e4m3", "e5m2"])
        else:
            case["mx"] = rng.random() < 0.5
        return case
    hidden, inter = _log(rng, 512, 7168) // 16 * 16, _log(rng, 256, 2048) // 16 * 16
    experts = rng.choice([4, 8, 16, 32])
    return {"op": op, "tokens": _log(rng, 1, 32), "topk": rng.choice([1, 2, 4, min(8, experts)]), "experts": experts,
            "hidden": hidden, "inter": inter, "fmt": rng.choice(["e4m3", "e5m2"])}


def _records_shape(rows, cols):
    return ((cols + 127) // 128, rows, 4)


def _mx_random(gen, rows, cols):
    """A checkpoint of random rows: e4m3 codes and its records (a power of two for each block of 32)."""
    v = torch.randn((rows, cols // 32, 32), device=DEV, generator=gen)
    e = (torch.floor(torch.log2(v.abs().amax(2))) - 8).clamp(-127, 127)
    codes = (v * torch.exp2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).reshape(rows, cols)
    return codes.view(torch.uint8), _to_records((e + 127).to(torch.uint8))


def _to_records(b):
    """[rows x blocks] block bytes -> [ceil(blocks / 4) x rows x 4] records, zero bytes past the last block."""
    rows, blocks = b.shape
    j = (blocks + 3) // 4
    full = torch.zeros((rows, j * 4), dtype=torch.uint8, device=b.device)
    full[:, :blocks] = b
    return full.view(rows, j, 4).transpose(0, 1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, c = case["op"], case

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, device=DEV, generator=gen).mul_(std).to(dtype)

    s = {"case": c}
    if op in ("norm", "norm_grad"):
        rows, cols = c["rows"], c["cols"]
        s["gamma"] = (1 + randn(cols, std=0.1, dtype=torch.float32)).to(torch.bfloat16)
        s["beta"] = None if c["rms"] else randn(cols, std=0.1)
        if op == "norm" or not c["mx"]:
            x = torch.randn((rows, cols), device=DEV, generator=gen)
            x[:, :: max(1, cols // 5)] *= 8         # a few loud channels, as in a residual stream
            s["x"] = x.add_(0.1).to(torch.bfloat16)
        if op == "norm":
            s["q"] = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
            s["scale_inv"] = torch.empty(rows, device=DEV)
            s["rstd"] = torch.empty(rows, device=DEV)
            s["mean"] = None if c["rms"] else torch.empty(rows, device=DEV)
            s["xq"] = torch.empty((rows, cols), dtype=torch.uint8, device=DEV) if c["save"] else None
            s["xs"] = torch.empty(_records_shape(rows, cols), dtype=torch.uint8, device=DEV) if c["save"] else None
            return s
        s["dy"] = randn(rows, cols, std=1e-3)
        if c["mx"]:
            s["xq"], s["xs"] = _mx_random(gen, rows, cols)
            s["rstd"] = torch.rand(rows, device=DEV, generator=gen) + 0.5
            s["y"] = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
        else:
            xd = s["x"].double()
            m = torch.zeros(rows, dtype=torch.float64, device=DEV) if c["rms"] else xd.mean(1)
            s["mean"] = None if c["rms"] else m.float()
            s["rstd"] = ((xd - m[:, None]).square().mean(1) + EPS).rsqrt().float()
        s["dx"] = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
        s["dgamma"] = torch.empty(cols, device=DEV)
        s["dbeta"] = None if c["rms"] else torch.empty(cols, device=DEV)
        # partial sums of the weights' gradients: at most 512 bands of rows, two sums a column
        s["workspace"] = torch.empty(512 * 2 * cols, device=DEV)
        return s
    if op in ("swiglu", "swiglu_grad"):
        rows, inter = c["rows"], c["inter"]
        if op == "swiglu":
            s["h"] = randn(rows, 2 * inter, std=1.5)
            s["q"] = torch.empty((rows, inter), dtype=torch.uint8, device=DEV)
            s["scale_inv"] = torch.empty(rows, device=DEV)
            s["hq"] = torch.empty((rows, 2 * inter), dtype=torch.uint8, device=DEV)
            s["hs"] = torch.empty(_records_shape(rows, 2 * inter), dtype=torch.uint8, device=DEV)
            return s
        s["da"] = randn(rows, inter, std=1e-3)
        if c["mx"]:
            s["hq"], s["hs"] = _mx_random(gen, rows, 2 * inter)
        else:
            s["h"] = randn(rows, 2 * inter, std=1.5)
        s["dh"] = torch.empty((rows, 2 * inter), dtype=torch.bfloat16, device=DEV)
        s["a"] = torch.empty((rows, inter), dtype=torch.bfloat16, device=DEV)
        return s
    T, k, E, H, inter = c["tokens"], c["topk"], c["experts"], c["hidden"], c["inter"]
    dtype, fmax, _ = FMT[c["fmt"]]

    def weight(rows, cols):
        w = torch.randn((E * rows, cols), device=DEV, generator=gen, dtype=torch.bfloat16)
        amax = w.abs().amax(1, keepdim=True)
        codes = w.mul_(fmax / amax).clamp_(-fmax, fmax).to(dtype).view(torch.uint8).view(E, rows, cols)
        return codes, (amax.float().flatten() * (1.0 / math.sqrt(cols) / fmax)).view(E, rows)

    s["x"] = randn(T, H)
    s["w1"], s["s1"] = weight(2 * inter, H)
    s["w2"], s["s2"] = weight(H, inter)
    s["idx"] = torch.rand((T, E), device=DEV, generator=gen).argsort(1)[:, :k].to(torch.int32).contiguous()
    s["weights"] = torch.randn((T, k), device=DEV, generator=gen).softmax(1)
    s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    s["workspace"] = torch.empty((T * k, inter), device=DEV)
    return s


# ---------------------------------------------------------------- plain form --
def _cast(y, fmt):
    """Rows of fp32 values -> (codes, factor that gives the values back)."""
    dtype, fmax, _ = FMT[fmt]
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


def _plain_norm(s):
    c, x = s["case"], s["x"].float()
    out = {}
    if c["rms"]:
        d = x
    else:
        out["mean"] = x.mean(1)
        d = x - out["mean"][:, None]
    out["rstd"] = 1.0 / torch.sqrt(d.square().mean(1) + EPS)
    xhat = d * out["rstd"][:, None]
    y = xhat * s["gamma"].float()
    if not c["rms"]:
        y = y + s["beta"].float()
    out["q"], out["scale_inv"] = _cast(y, c["fmt"])
    if c["save"]:
        out["xq"], out["xs"] = _blocks(xhat)
    return out


def _plain_norm_grad(s):
    c, dy, gamma = s["case"], s["dy"].float(), s["gamma"].float()
    out = {}
    if c["mx"]:
        xhat = _unblock(s["xq"], s["xs"])
        y = xhat * gamma
        out["y"] = (y if c["rms"] else y + s["beta"].float()).to(torch.bfloat16)
    else:
        x = s["x"].float()
        xhat = (x if c["rms"] else x - s["mean"][:, None]) * s["rstd"][:, None]
    w = dy * gamma
    d = w - xhat * (w * xhat).mean(1, keepdim=True)
    if not c["rms"]:
        d = d - w.mean(1, keepdim=True)
        out["dbeta"] = dy.sum(0)
    out["dx"] = (d * s["rstd"][:, None]).to(torch.bfloat16)
    out["dgamma"] = (dy * xhat).sum(0)
    return out


def _plain_swiglu(s):
    h = s["h"].float()
    g, u = h.chunk(2, dim=1)
    out = {}
    out["q"], out["scale_inv"] = _cast(g / (1.0 + torch.exp(-g)) * u, s["case"]["fmt"])
    out["hq"], out["hs"] = _blocks(h)
    return out


def _plain_swiglu_grad(s):
    h = _unblock(s["hq"], s["hs"]) if s["case"]["mx"] else s["h"].float()
    g, u = h.chunk(2, dim=1)
    da = s["da"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    silu = g * sig
    dg = da * u * sig * (1.0 + g * (1.0 - sig))
    return {"dh": torch.cat([dg, da * silu], 1).to(torch.bfloat16), "a": (silu * u).to(torch.bfloat16)}


def _plain_moe(s):
    c, idx, x = s["case"], s["idx"].long(), s["x"].float()
    T, k, E = c["tokens"], c["topk"], c["experts"]
    dtype = FMT[c["fmt"]][0]
    if T * k < E:       # the entries' experts alone
        e = idx.flatten()
        w1 = s["w1"][e].view(dtype).float() * s["s1"][e][..., None]
        h = torch.bmm(w1, x.repeat_interleave(k, 0)[..., None])[..., 0]
        g, u = h.chunk(2, dim=1)
        w2 = s["w2"][e].view(dtype).float() * s["s2"][e][..., None]
        y = torch.bmm(w2, (g / (1.0 + torch.exp(-g)) * u)[..., None])[..., 0]
        return (y.view(T, k, -1) * s["weights"][..., None]).sum(1).to(torch.bfloat16)
    w1 = s["w1"].view(dtype).float() * s["s1"][..., None]
    h = torch.bmm(w1, x.t().expand(E, -1, -1))                              # [E, 2I, T]
    g, u = h.chunk(2, dim=1)
    share = torch.zeros((T, E), device=x.device).scatter_add_(1, idx, s["weights"])
    w2 = s["w2"].view(dtype).float() * s["s2"][..., None]
    y = torch.bmm(w2, g / (1.0 + torch.exp(-g)) * u)                        # [E, H, T]
    return (y * share.t()[:, None]).sum(0).t().to(torch.bfloat16)


# ------------------------------------------------------------- library calls --
def _own_norm(s):
    import fp8_scaled_gemm_amax_amd as fp8
    c = s["case"]
    fp8.fp8_norm_quantize_row(s["x"], s["gamma"], s["beta"], EPS, fp8.NORM_RMS if c["rms"] else fp8.NORM_LAYER,
                              fp8.E4M3 if c["fmt"] == "e4m3" else fp8.E5M2, 0, s["q"], s["scale_inv"],
                              mean_out=s["mean"], rstd_out=s["rstd"], xhat_q=s["xq"], xhat_fmt=fp8.E4M3,
                              xhat_scale=s["xs"])
    out = {"q": s["q"].view(FMT[c["fmt"]][0]), "scale_inv": s["scale_inv"], "rstd": s["rstd"]}
    if not c["rms"]:
        out["mean"] = s["mean"]
    if c["save"]:
        out["xq"], out["xs"] = s["xq"].view(torch.float8_e4m3fn), s["xs"].view(torch.float8_e8m0fnu)
    return out


def _own_norm_grad(s):
    import fp8_scaled_gemm_amax_amd as fp8
    c = s["case"]
    kind = fp8.NORM_RMS if c["rms"] else fp8.NORM_LAYER
    out = {"dx": s["dx"], "dgamma": s["dgamma"]}
    if c["mx"]:
        fp8.fp8_mx_norm_backward(s["dy"], s["xq"], fp8.E4M3, s["xs"], s["gamma"], s["beta"], s["rstd"], kind, s["dx"],
                                 dgamma=s["dgamma"], dbeta=s["dbeta"], y=s["y"], workspace=s["workspace"])
        out["y"] = s["y"]
    else:
        fp8.fp8_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], kind, s["dx"], dgamma=s["dgamma"],
                              dbeta=s["dbeta"], workspace=s["workspace"])
    if not c["rms"]:
        out["dbeta"] = s["dbeta"]
    return out


def _own_swiglu(s):
    import fp8_scaled_gemm_amax_amd as fp8
    fmt = s["case"]["fmt"]
    fp8.fp8_swiglu_quantize_row_mx(s["h"], fp8.E4M3 if fmt == "e4m3" else fp8.E5M2, 0, s["q"], s["scale_inv"],
                                   s["hq"], fp8.E4M3, s["hs"])
    return {"q": s["q"].view(FMT[fmt][0]), "scale_inv": s["scale_inv"], "hq": s["hq"].view(torch.float8_e4m3fn),
            "hs": s["hs"].view(torch.float8_e8m0fnu)}


def _own_swiglu_grad(s):
    import fp8_scaled_gemm_amax_amd as fp8
    if s["case"]["mx"]:
        fp8.fp8_mx_swiglu_backward(s["da"], s["hq"], fp8.E4M3, s["hs"], s["dh"], a=s["a"])
    else:
        fp8.fp8_swiglu_backward(s["da"], s["h"], s["dh"], a=s["a"])
    return {"dh": s["dh"], "a": s["a"]}


def _own_moe(s):
    import fp8_scaled_gemm_amax_amd as fp8
    fmt = fp8.E4M3 if s["case"]["fmt"] == "e4m3" else fp8.E5M2
    fp8.fp8_moe_few_tokens(s["x"], s["idx"], s["weights"], s["w1"], fmt, s["s1"], s["w2"], fmt, s["s2"], s["out"],
                           s["workspace"])
    return s["out"]


PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "swiglu": _plain_swiglu,
         "swiglu_grad": _plain_swiglu_grad, "moe": _plain_moe}
OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "swiglu": _own_swiglu, "swiglu_grad": _own_swiglu_grad,
       "moe": _own_moe}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


def work(case):
    c, op = case, case["op"]
    if op in ("norm", "norm_grad"):
        n, rows, cols = c["rows"] * c["cols"], c["rows"], c["cols"]
        ckpt = n + n // 32
        if op == "norm":
            per_row = 8 if c["rms"] else 12
            return {"bytes": 3 * n + (ckpt if c["save"] else 0) + per_row * rows + (2 if c["rms"] else 4) * cols,
                    "flops": 8 * n}
        read = 2 * n + (ckpt if c["mx"] else 2 * n) + (4 if c["rms"] or c["mx"] else 8) * rows
        grads = (4 if c["rms"] else 8) * cols
        weights = 2 * cols + (2 * cols if c["mx"] and not c["rms"] else 0)
        return {"bytes": read + 2 * n + (2 * n if c["mx"] else 0) + grads + weights, "flops": 12 * n}
    if op in ("swiglu", "swiglu_grad"):
        n = c["rows"] * c["inter"]
        ckpt = 2 * n + 2 * n // 32
        if op == "swiglu":
            return {"bytes": 4 * n + n + ckpt + 4 * c["rows"], "flops": 12 * n}
        return {"bytes": 2 * n + (ckpt if c["mx"] else 4 * n) + 4 * n + 2 * n, "flops": 16 * n}
    T, k, E, H, inter = c["tokens"], c["topk"], c["experts"], c["hidden"], c["inter"]
    used = E * (1 - (1 - k / E) ** T)           # experts that a random choice reaches
    return {"bytes": used * (3 * inter * H + 4 * (2 * inter + H)) + 4 * T * H + 8 * T * k,
            "flops": 6.0 * T * k * inter * H}


# ------------------------------------------------------------------- 64 bits --
def _round_to(v, mbits, emin, fmax):
    """Nearest value of a format with mbits fraction bits and smallest normal exponent emin, ties to even."""
    v = v.clamp(-fmax, fmax)
    e = torch.floor(torch.log2(v.abs().clamp_min(1e-300))).clamp_min(emin)
    e = torch.where(torch.exp2(e) > v.abs(), (e - 1).clamp_min(emin), e)
    step = torch.exp2(e - mbits)
    return torch.round(v / step) * step


ROUND = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}


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


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op in ("norm", "norm_grad"):
        gamma = s["gamma"].double()
        beta = 0.0 if c["rms"] else s["beta"].double()
        if op == "norm":
            x = s["x"].double()
            mu = torch.zeros_like(x[:, 0]) if c["rms"] else x.sum(1) / c["cols"]
            rstd = ((x - mu[:, None]).pow(2).sum(1) / c["cols"] + EPS).pow(-0.5)
            xhat = (x - mu[:, None]) * rstd[:, None]
            out = {"rstd": rstd}
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
            xhat = (s["x"].double() - (0.0 if c["rms"] else s["mean"].double()[:, None])) * rstd
        dy = s["dy"].double()
        g = dy * gamma
        dot = (g * xhat).sum(1, keepdim=True) / c["cols"]
        shift = 0.0 if c["rms"] else g.sum(1, keepdim=True) / c["cols"]
        out = {"dx": rstd * (g - shift - xhat * dot), "dgamma": (dy * xhat).sum(0)}
        if not c["rms"]:
            out["dbeta"] = dy.sum(0)
        if c["mx"]:
            out["y"] = xhat * gamma + beta
        return out
    if op in ("swiglu", "swiglu_grad"):
        n = c["inter"]
        h = _exact_values(s["hq"], s["hs"]) if c.get("mx") else s["h"].double()
        g, u = h[:, :n], h[:, n:]
        a = g * torch.sigmoid(g) * u
        if op == "swiglu":
            out = {}
            out["q"], out["scale_inv"] = _exact_cast(a, c["fmt"])
            out["hq"], out["hs"] = _exact_blocks(h)
            return out
        da = s["da"].double()
        e = torch.exp(-g)
        dh = torch.empty_like(h)
        dh[:, :n] = da * u * (1 + e + g * e) / (1 + e).pow(2)
        dh[:, n:] = da * g / (1 + e)
        return {"dh": dh, "a": a}
    dtype = FMT[c["fmt"]][0]
    out = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device=DEV)
    for e in range(c["experts"]):
        token, slot = torch.nonzero(s["idx"] == e, as_tuple=True)
        if token.numel():
            w1 = s["w1"][e].view(dtype).double() * s["s1"][e].double()[:, None]
            w2 = s["w2"][e].view(dtype).double() * s["s2"][e].double()[:, None]
            h = s["x"][token].double() @ w1.T
            a = h[:, : c["inter"]] * torch.sigmoid(h[:, : c["inter"]]) * h[:, c["inter"]:]
            out.index_add_(0, token, s["weights"][token, slot].double()[:, None] * (a @ w2.T))
    return out
