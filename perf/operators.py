"""Cases of the routing and 4-bit operators: expert routing from logits, its gradient, microscaled FP4
quantisation, and the FP4 product (one matrix, or one per expert).

Each case runs in two forms, chosen by the module's `own`: the plain form in elementary torch operations, and
the framework's entry points. `exact` computes the same outputs in 64 bits, in code of its own.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def _route(name, op, T, E, k, score, dtype, groups=1, kept=1, bias=False, renorm=True, scale=1.0, off=0):
    """off: experts whose logit is -inf (taken out of service) in every row."""
    return dict(name=name, op=op, T=T, E=E, k=k, score=score, dtype=dtype, groups=groups, kept=kept, bias=bias,
                renorm=renorm, scale=scale, off=off)


def _quant(name, rows, cols, fmt, dtype):
    return dict(name=name, op="quantize", rows=rows, cols=cols, fmt=fmt, dtype=dtype)


def _linear(name, T, N, K, fmt, dtype, E=0, pad=0, skew=0.0):
    """E = 0: one weight matrix; E > 0: one per expert, the T rows sorted by expert, `pad` unused rows behind
    them; skew: the spread of the experts' loads (0: uniform)."""
    return dict(name=name, op="linear", T=T, N=N, K=K, fmt=fmt, dtype=dtype, E=E, pad=pad, skew=skew)


def listed():
    return [
        # a decode step of the 384-expert layer, the router's own score
        _route("route decode", "route", 32, 384, 6, "sqrtsoftplus", "fp32", scale=1.5),
        # a prefill batch, sigmoid scores with a balancing bias, experts in groups
        _route("route prefill groups", "route", 8192, 256, 8, "sigmoid", "fp32", 8, 4, True, scale=2.5),
        # a ragged training batch of the 128-expert layer, softmax over all experts, some of them out of service
        _route("route softmax", "route", 4099, 128, 3, "softmax", "bf16", renorm=False, off=3),
        # the gradients that belong to the last two
        _route("route grad sigmoid", "route_grad", 8192, 384, 6, "sigmoid", "fp32", scale=2.5),
        _route("route grad softmax", "route_grad", 4099, 128, 3, "softmax", "bf16", renorm=False, off=3),
        # a prefill batch's tokens and a few rows of an expert's width
        _quant("quantize prefill", 8192, 5120, "mxfp4", "bf16"),
        _quant("quantize few rows", 33, 2304, "nvfp4", "fp16"),
        # one expert-sized matrix: one token, a ragged batch, a prefill batch
        _linear("linear one token", 1, 4608, 5120, "mxfp4", "bf16"),
        _linear("linear ragged", 517, 2304, 1312, "nvfp4", "fp16"),
        _linear("linear prefill", 8192, 4608, 5120, "nvfp4", "bf16"),
        # 32 tokens times 6 experts against 384 experts: the weights are read once
        _linear("experts decode", 192, 5120, 2304, "mxfp4", "bf16", E=384, pad=0, skew=0.5),
        # a prefill batch against 64 experts, loads uneven, unused rows at the end
        _linear("experts prefill", 12288, 2304, 5120, "mxfp4", "bf16", E=64, pad=37, skew=0.7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "route_grad", "quantize", "linear", "experts"))
    if op in ("route", "route_grad"):
        score = rng.choice(("softmax", "sigmoid", "sqrtsoftplus"))
        groups = rng.choice((1, 1, 2, 4, 8)) if op == "route" else 1
        E = groups * _log(rng, 8, 512 // groups)
        kept = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(16, E // groups * kept - 1))
        c = _route("", op, _log(rng, 1, 16384), E, k, score, rng.choice(("fp32", "bf16", "fp16")), groups, kept,
                   op == "route" and rng.random() < 0.5, rng.random() < 0.6, rng.choice((1.0, 1.5, 2.5)),
                   rng.choice((0, 0, 1, 3)))
    elif op == "quantize":
        cols = 32 * _log(rng, 1, 256)
        c = _quant("", _log(rng, 1, (8192 * 5120) // cols), cols, rng.choice(("mxfp4", "nvfp4")),
                   rng.choice(("bf16", "fp16", "fp32")))
    elif op == "linear":
        N, K = _log(rng, 32, 8192), 32 * _log(rng, 2, 256)
        T = _log(rng, 1, max(1, min(16384, 8192 * 4608 * 5120 // (N * K))))
        c = _linear("", T, N, K, rng.choice(("mxfp4", "nvfp4")), rng.choice(("bf16", "fp16")))
    else:
        E, N, K = _log(rng, 2, 128), _log(rng, 64, 4096), 32 * _log(rng, 4, 160)
        c = _linear("", _log(rng, 1, 8192), N, K, rng.choice(("mxfp4", "nvfp4")), rng.choice(("bf16", "fp16")), E=E,
                    pad=rng.choice((0, 0, 5, 64)), skew=rng.choice((0.0, 0.5, 1.0)))
        # the plain form pads every expert to the largest: keep that within the listed cases' work
        c["T"] = max(1, min(c["T"], 12288 * 2304 * 5120 // (N * K)))
    del c["name"]
    return c


def work(case):
    c = case
    if c["op"] == "route":
        # logits and bias in, an index and a weight for each slot out; a score (exp, reciprocal) per expert and
        # k passes of comparisons
        n = c["T"] * c["E"]
        return {"bytes": n * BYTES[c["dtype"]] + c["bias"] * c["E"] * 4 + c["T"] * c["k"] * 8, "flops": n * (8 + c["k"])}
    if c["op"] == "route_grad":
        # the selected logits (all of them where the scores are normalised over all), indices and the weights'
        # gradients in, the logits' gradients out
        n = c["T"] * c["E"]
        dense = c["score"] == "softmax" and not c["renorm"]
        read = n if dense else c["T"] * c["k"]
        return {"bytes": (n + read) * BYTES[c["dtype"]] + c["T"] * c["k"] * 8, "flops": (8 * n if dense else 0) + 20 * c["T"] * c["k"]}
    if c["op"] == "quantize":
        # values in; codes and scales out and in again; the values they stand for out
        n = c["rows"] * c["cols"]
        return {"bytes": n * (2 * BYTES[c["dtype"]] + 2 * (0.5 + 1.0 / BLOCK[c["fmt"]])), "flops": 6 * n}
    wbytes = c["N"] * c["K"] * (0.5 + 1.0 / BLOCK[c["fmt"]])
    # experts that at least one of T rows meets (uniform loads)
    touched = c["E"] * (1.0 - (1.0 - 1.0 / c["E"]) ** c["T"]) if c["E"] else 1
    return {"bytes": touched * wbytes + c["T"] * (c["K"] + c["N"]) * BYTES[c["dtype"]], "flops": 2.0 * c["T"] * c["N"] * c["K"]}


# ------------------------------------------------------------------ inputs
def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 101)
    return g


def prepare(case, seed):
    c, dev = case, torch.device("cuda", torch.cuda.current_device())
    g = _gen(seed, dev)
    s = {"case": c}
    if c["op"] in ("route", "route_grad"):
        z = torch.randn((c["T"], c["E"]), generator=g, device=dev) * 1.5
        if c["off"]:
            z[:, torch.randperm(c["E"], generator=g, device=dev)[:c["off"]]] = -math.inf
        s["logits"] = z.to(DTYPES[c["dtype"]])
        s["bias"] = torch.randn(c["E"], generator=g, device=dev) * 0.05 if c["bias"] else None
        if c["op"] == "route_grad":
            s["idx"] = _plain_route(c, s["logits"], s["bias"])[0]
            s["grad"] = torch.randn((c["T"], c["k"]), generator=g, device=dev)
        return s
    if c["op"] == "quantize":
        x = torch.randn((c["rows"], c["cols"]), generator=g, device=dev)
        x.mul_(torch.exp(torch.randn((1, c["cols"]), generator=g, device=dev)))  # channels of unlike size
        s["x"] = x.to(DTYPES[c["dtype"]])
        s["tensor_scale"] = _tensor_scale(s["x"], c["fmt"])
        return s
    E, N, K, T = max(1, c["E"]), c["N"], c["K"], c["T"]
    x = torch.randn((T + c["pad"], K), generator=g, device=dev).to(DTYPES[c["dtype"]])
    s["x"] = x
    s["x_scale"] = _tensor_scale(x, c["fmt"])
    bs = BLOCK[c["fmt"]]
    s["w"] = torch.empty((E, N, K // 2), dtype=torch.uint8, device=dev)
    s["w_scales"] = torch.empty((E, N, K // bs), dtype=torch.uint8, device=dev)
    s["w_scale"] = torch.empty(E, device=dev) if c["fmt"] == "nvfp4" else None
    some = max(1, (1 << 26) // (N * K))  # experts made together
    for e in range(0, E, some):
        n = min(some, E - e)
        w = (torch.randn((n * N, K), generator=g, device=dev) / math.sqrt(K)).to(torch.bfloat16)
        ts = None
        if c["fmt"] == "nvfp4":
            s["w_scale"][e:e + n] = 0.01 / 6.0 * torch.rand(n, generator=g, device=dev) + 0.001
            ts = s["w_scale"][e:e + n].repeat_interleave(N)[:, None]
        codes, scales = _plain_quantize(w, c["fmt"], ts)
        s["w"][e:e + n] = codes.view(n, N, K // 2)
        s["w_scales"][e:e + n] = scales.view(n, N, K // bs)
    if c["E"] == 0:
        s["w"], s["w_scales"] = s["w"][0], s["w_scales"][0]
        return s
    p = torch.softmax(torch.randn(E, generator=g, device=dev) * c["skew"], 0)
    who = torch.multinomial(p, T, replacement=True, generator=g)
    count = torch.bincount(who, minlength=E)
    s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
    s["most"] = int(count.max())
    s["out"] = torch.zeros((T + c["pad"], N), dtype=x.dtype, device=dev)
    return s


def _tensor_scale(x, fmt):
    """The largest value becomes 6 (the largest element) times 448 (the largest scale), as a calibrated scale does."""
    return (x.abs().max().float() / (6.0 * 448.0)).reshape(1) if fmt == "nvfp4" else None


# ------------------------------------------------------------------ plain forms
def _plain_scores(z, score):
    if score == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    return torch.sqrt(z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())))


def _plain_route(c, logits, bias):
    z = logits.double()  # two scores may be nearer to each other than 32 bits tell
    off = torch.isneginf(z)
    s = _plain_scores(z, c["score"])
    key = s if bias is None else s + bias.double()
    key = key.masked_fill(off, -math.inf)
    if c["groups"] > 1:
        kg = key.view(c["T"], c["groups"], -1)
        top = torch.sort(kg, dim=2, descending=True)[0][:, :, :2]
        gs = top[:, :, 0] + top[:, :, 1:].masked_fill(torch.isneginf(top[:, :, 1:]), 0.0).sum(2)
        order = torch.sort(gs, dim=1, descending=True, stable=True)[1][:, :c["kept"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, order, True)
        key = kg.masked_fill(~keep[:, :, None], -math.inf).reshape(key.shape)
    key, idx = torch.sort(key, dim=1, descending=True, stable=True)
    key, idx = key[:, :c["k"]], idx[:, :c["k"]]
    none = torch.isneginf(key)
    w = torch.gather(s, 1, idx).masked_fill(none, 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.masked_fill(none, -1).to(torch.int32), (w * c["scale"]).float()


def _plain_route_grad(c, logits, idx, grad):
    z = logits.float()
    i = idx.long().clamp(min=0)
    sel = idx >= 0
    g = (grad * c["scale"]).masked_fill(~sel, 0.0)
    s = _plain_scores(z, c["score"])
    ss = torch.gather(s, 1, i).masked_fill(~sel, 0.0)
    if c["renorm"]:
        total = ss.sum(1, keepdim=True)
        ds = (g - (g * ss).sum(1, keepdim=True) / total) / total
    else:
        ds = g
    if c["score"] == "softmax":
        # the sum over the selected experts of ds * s vanishes where the weights are renormalised
        d = torch.zeros_like(z).scatter_add_(1, i, ds.masked_fill(~sel, 0.0))
        dz = s * (d - (ds * ss).sum(1, keepdim=True))
        if c["renorm"]:
            dz = torch.zeros_like(z).scatter_add_(1, i, (ss * ds).masked_fill(~sel, 0.0))
        return dz.to(logits.dtype)
    zs = torch.gather(z, 1, i)
    slope = ss * (1.0 - ss) if c["score"] == "sigmoid" else 1.0 / (1.0 + torch.exp(-zs)) / (2.0 * ss)
    return torch.zeros_like(z).scatter_add_(1, i, (ds * slope).masked_fill(~sel, 0.0)).to(logits.dtype)


def _codes_of(a):
    """E2M1 code of magnitudes on the format's own grid: nearest, ties to the even code, at most 6."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))


def _plain_quantize(x, fmt, tensor_scale):
    """Codes [rows, cols / 2] (even element in the low nibble) and scales [rows, cols / block] as bytes."""
    rows, cols = x.shape
    b = x.view(rows, cols // BLOCK[fmt], BLOCK[fmt])
    if fmt == "mxfp4":
        b = b.float()
        amax = b.abs().amax(2)
        e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        unit = torch.ldexp(torch.ones_like(amax), e)
        scales = (e + 127).to(torch.uint8)
    else:
        # in 64 bits: the 4- and 8-bit grids' borders times a scale have more digits than 32 bits hold
        b = b.double()
        g = torch.ones(1, device=x.device) if tensor_scale is None else tensor_scale
        v = b.abs().amax(2) / (6.0 * g.double())
        step = torch.ldexp(torch.ones_like(v), (torch.frexp(v)[1] - 1).clamp(min=-6) - 3)
        v = (torch.round(v / step) * step).clamp(max=448.0)
        scales = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
        unit = (v.float() * g).double()
    a = b.abs() / unit[:, :, None]
    a = torch.where(unit[:, :, None] > 0, a, torch.zeros_like(a))
    code = _codes_of(a) | (torch.signbit(b).to(torch.uint8) << 3)
    code = code.view(rows, cols // 2, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), scales


def _plain_values(codes, scales, fmt, tensor_scale):
    """The values in 32 bits of codes [..., K / 2] with their scales."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pairs = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)  # both values of each byte
    bs = BLOCK[fmt]
    v = pairs[codes.int()].view(*scales.shape, bs)
    if fmt == "mxfp4":
        d = torch.ldexp(torch.ones(scales.shape, device=codes.device), scales.int() - 127)
    else:
        d = scales.view(torch.float8_e4m3fn).float()
        if tensor_scale is not None:
            d = d * tensor_scale
    return v.mul_(d[..., None]).flatten(-2)


def _plain_linear(c, s):
    x, fmt = s["x"][:c["T"]], c["fmt"]
    q = _plain_values(*_plain_quantize(x, fmt, s["x_scale"]), fmt, s["x_scale"])
    ts = s["w_scale"]
    w = _plain_values(s["w"], s["w_scales"], fmt, None if ts is None else ts.view((-1, 1, 1) if c["E"] else (-1, 1)))
    if not c["E"]:
        return torch.matmul(q, w.t()).to(x.dtype)
    # one product per expert, each padded to the largest load
    off = s["offsets"].long()
    row = torch.arange(c["T"], device=x.device)
    e = torch.searchsorted(off[1:], row, right=True)
    xp = q.new_zeros((c["E"], s["most"], c["K"]))
    xp[e, row - off[e]] = q
    y = torch.bmm(xp, w.transpose(1, 2))
    s["out"][:c["T"]] = y[e, row - off[e]].to(x.dtype)
    return s["out"]


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        import routed_expert_ffn_sqrtsoftplus_b200 as moe
        if c["op"] == "route":
            return moe.route(state["logits"], c["k"], score=c["score"], bias=state["bias"], n_groups=c["groups"],
                             topk_groups=c["kept"], renormalize=c["renorm"], route_scale=c["scale"])
        if c["op"] == "route_grad":
            return moe.route_backward(state["grad"], state["logits"], state["idx"], score=c["score"],
                                      renormalize=c["renorm"], route_scale=c["scale"])
        if c["op"] == "quantize":
            codes, scales = moe.quantize_fp4(state["x"], c["fmt"], tensor_scale=state["tensor_scale"])
            return moe.dequantize_fp4(codes, scales, c["fmt"], tensor_scale=state["tensor_scale"], dtype=state["x"].dtype)
        return moe.fp4_linear(state["x"], state["w"], state["w_scales"], c["fmt"], x_tensor_scale=state["x_scale"],
                              w_tensor_scale=state["w_scale"], offsets=state.get("offsets"), out=state.get("out"))
    if c["op"] == "route":
        return _plain_route(c, state["logits"], state["bias"])
    if c["op"] == "route_grad":
        return _plain_route_grad(c, state["logits"], state["idx"], state["grad"])
    if c["op"] == "quantize":
        codes, scales = _plain_quantize(state["x"], c["fmt"], state["tensor_scale"])
        return _plain_values(codes, scales, c["fmt"], state["tensor_scale"]).to(state["x"].dtype)
    return _plain_linear(c, state)


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_score(z, score):
    if score == "softmax":
        return torch.softmax(z, 1)
    if score == "sigmoid":
        return torch.sigmoid(z)
    return torch.logaddexp(z, torch.zeros((), dtype=z.dtype, device=z.device)).sqrt()


def _exact_nearest(v, grid):
    """Index of the nearest value of an ascending grid; a tie goes to the even index."""
    hi = torch.bucketize(v, grid).clamp(1, grid.numel() - 1)
    lo = hi - 1
    below, above = v - grid[lo], grid[hi] - v
    return torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def _exact_quantized(x, fmt, ts):
    """Values that x's 4-bit form stands for; the tensor's scale enters as a factor in 64 bits."""
    dev = x.device
    grid = torch.tensor(E2M1, dtype=torch.float64, device=dev)
    b = x.double().unflatten(1, (-1, BLOCK[fmt]))
    amax = b.abs().max(2, keepdim=True)[0]
    if fmt == "mxfp4":
        powers = torch.tensor([2.0 ** e for e in range(-127, 128)], dtype=torch.float64, device=dev)
        # the largest power of two at most amax / 4
        unit = powers[(torch.bucketize(amax / 4.0, powers, right=True) - 1).clamp(0, 254)]
    else:
        # every finite value of the 8-bit scale format, ascending
        all8 = torch.arange(0, 127, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        g = 1.0 if ts is None else ts.double()
        unit = (all8[_exact_nearest(amax / (6.0 * g), all8)] * g).float().double()
    a = torch.where(unit > 0, b.abs() / unit, torch.zeros_like(b))
    return (grid[_exact_nearest(a, grid)] * torch.sign(b) * unit).flatten(1)


def _exact_weights(codes, scales, fmt):
    lut = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    d = torch.pow(2.0, scales.double() - 127.0) if fmt == "mxfp4" else scales.view(torch.float8_e4m3fn).double()
    return lut[n & 7] * (1.0 - 2.0 * (n >> 3)) * d.repeat_interleave(BLOCK[fmt], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        z = s["logits"].double()
        p = _exact_score(z, c["score"])
        key = (p if s["bias"] is None else p + s["bias"].double()).masked_fill(z == -math.inf, -math.inf)
        G = c["groups"]
        two = torch.topk(key.unflatten(1, (G, -1)), 2, 2)[0]
        worth = torch.where(two[..., 1] == -math.inf, two[..., 0], two.sum(2))
        # rank of a group: how many are worth more, or as much with a lower number
        before = (worth[:, None, :] > worth[:, :, None]) | ((worth[:, None, :] == worth[:, :, None]) & torch.tril(
            torch.ones(G, G, dtype=torch.bool, device=z.device), -1))
        key = key.masked_fill((before.sum(2) >= c["kept"]).repeat_interleave(c["E"] // G, 1), -math.inf)
        idx = torch.argsort(-key, dim=1, stable=True)[:, :c["k"]]
        dead = torch.gather(key, 1, idx) == -math.inf
        w = torch.where(dead, 0.0, torch.gather(p, 1, idx))
        return torch.where(dead, -1, idx).to(torch.int32), w * c["scale"] / (w.sum(1, keepdim=True) if c["renorm"] else 1.0)
    if c["op"] == "route_grad":
        z = s["logits"].double().requires_grad_(True)
        used = s["idx"] >= 0
        p = torch.gather(_exact_score(z, c["score"]), 1, s["idx"].long().clamp(min=0)) * used
        w = c["scale"] * (p / p.sum(1, keepdim=True) if c["renorm"] else p)
        return torch.autograd.grad(w, z, s["grad"].double())[0].masked_fill(z == -math.inf, 0.0).detach()
    if c["op"] == "quantize":
        return _exact_quantized(s["x"], c["fmt"], s["tensor_scale"])
    x = _exact_quantized(s["x"][:c["T"]], c["fmt"], s["x_scale"])
    if not c["E"]:
        y = x @ _exact_weights(s["w"], s["w_scales"], c["fmt"]).t()
        return y if s["w_scale"] is None else y * s["w_scale"].double()
    y = torch.zeros((c["T"] + c["pad"], c["N"]), dtype=torch.float64, device=x.device)
    off = s["offsets"].tolist()
    for e in range(c["E"]):
        if off[e + 1] > off[e]:
            r = x[off[e]:off[e + 1]] @ _exact_weights(s["w"][e], s["w_scales"][e], c["fmt"]).t()
            y[off[e]:off[e + 1]] = r if s["w_scale"] is None else r * s["w_scale"][e].double()
    return y
