"""Cases of the row normalisation (``wan.rmsnorm``) and of the linear layer
(``wan.linear``), each with a plain form in elementary torch operations.

    rmsnorm   h = x + r,  y = h / sqrt(mean(h^2) + eps) * g, stored as bf16, as
              float32, or as e4m3 codes with one scale (amax / 448) per row
    linear    out = act((a w^T) [a_scale[m] w_scale[n]] + b) + r, on bf16
              operands or on e4m3 codes with their scales

A case gives the operator, the sizes and the types; ``own`` chooses between
the plain form and the library's entry points. Widths and token counts are
those of the library's block configurations (dim 1536 and 5120, ffn 8960 and
13824, 7800 and 32760 tokens, 512 text tokens of 4096 features) or generic.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZE = {"none": 0, "fp8": 1, "bf16": 2, "f32": 4}


def _norm(name, rows, width, x, res, out):
    return {"name": name, "op": "rmsnorm", "rows": rows, "width": width, "x": x, "res": res, "out": out}


def _linear(name, m, n, k, a, act, bias, res, out, wscale="tensor"):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "a": a, "act": act, "bias": bias, "res": res,
            "out": out, "wscale": wscale}


def listed():
    return [
        # one token entering an FP8 projection: all latency
        _norm("norm 1x5120 fp8", 1, 5120, "bf16", "f32", "fp8"),
        # the text tokens of one prompt, everything in bf16
        _norm("norm 512x4096 bf16", 512, 4096, "bf16", "bf16", "bf16"),
        # an odd width: rows that start at any multiple of two bytes
        _norm("norm 2011x1037 odd", 2011, 1037, "bf16", "bf16", "f32"),
        # q or k normalised head by head: many short rows, no residual
        _norm("norm 93600x128 heads", 93600, 128, "bf16", "none", "bf16"),
        # the stream of the short clip, kept in float32, into an FP8 projection
        _norm("norm 7800x1536 fp8", 7800, 1536, "bf16", "f32", "fp8"),
        # the stream of the long clip at the large width
        _norm("norm 32760x5120 fp8", 32760, 5120, "bf16", "f32", "fp8"),
        # one token through a square projection: the weights' bytes alone
        _linear("linear 1x5120x5120", 1, 5120, 5120, "bf16", "silu", True, "none", "bf16"),
        # a handful of tokens through the FP8 FFN's first matrix, a scale for each weight row
        _linear("linear 24x13824x5120 fp8", 24, 13824, 5120, "fp8", "gelu", True, "none", "bf16", "row"),
        # odd sizes, an output whose rows are not aligned
        _linear("linear 333x1003x1000 odd", 333, 1003, 1000, "bf16", "relu", True, "bf16", "bf16"),
        # the text features' first projection
        _linear("linear 512x5120x4096", 512, 5120, 4096, "bf16", "gelu", True, "none", "bf16"),
        # the short clip through the FFN's first matrix
        _linear("linear 7800x8960x1536", 7800, 8960, 1536, "bf16", "gelu", True, "none", "bf16"),
        # the long clip through the FP8 FFN's second matrix, onto the float32 stream
        _linear("linear 32760x5120x13824 fp8", 32760, 5120, 13824, "fp8", "none", True, "f32", "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        width = _log(rng, 64, 16384)
        if rng.random() < 0.7:                       # most widths are multiples of 8, the others any
            width -= width % 8
        rows = min(_log(rng, 1, 120000), 32760 * 5120 // width)
        return {"op": "rmsnorm", "rows": rows, "width": width, "x": rng.choice(["bf16", "f32"]),
                "res": rng.choice(["none", "bf16", "f32"]), "out": rng.choice(["bf16", "f32", "fp8"])}
    a = rng.choice(["bf16", "bf16", "fp8"])
    unit = 16 if a == "fp8" else 8                   # matrix rows are whole multiples of 16 bytes
    k = max(unit, _log(rng, 64, 16384) // unit * unit)
    n = _log(rng, 32, 16384)
    if rng.random() < 0.7:
        n -= n % 8
    m = min(_log(rng, 1, 32760), 32760 * 5120 * 13824 // (n * k))
    return {"op": "linear", "m": m, "n": n, "k": k, "a": a, "act": rng.choice(["none", "gelu", "silu", "relu"]),
            "bias": rng.random() < 0.75, "res": rng.choice(["none", "bf16", "f32"]), "out": rng.choice(["bf16", "f32"]),
            "wscale": rng.choice(["tensor", "row"])}


# ---------------------------------------------------------------- inputs
def _quantized(t, dim):
    """e4m3 codes and float32 scales of t, one scale per row (dim=1) or one for all (dim=None)."""
    amax = t.abs().amax() if dim is None else t.abs().amax(dim, keepdim=True)
    codes = (t * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, (amax / E4M3_MAX).reshape(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = {"case": case}
    if case["op"] == "rmsnorm":
        rows, width = case["rows"], case["width"]
        # a few channels are larger than the others, as in a trained stream
        channel = torch.exp(0.5 * normal(width))
        s["x"] = (normal(rows, width) * channel).to(TYPES[case["x"]])
        s["r"] = None if case["res"] == "none" else (2.0 * normal(rows, width) * channel).to(TYPES[case["res"]])
        s["g"] = 1.0 + 0.1 * normal(width)
        s["h"] = None if s["r"] is None else torch.empty_like(s["r"])
        s["y"] = torch.empty(rows, width, device="cuda", dtype=TYPES[case["out"]])
        s["scale"] = torch.empty(rows, device="cuda") if case["out"] == "fp8" else None
        return s
    m, n, k = case["m"], case["n"], case["k"]
    a, w = normal(m, k), 0.02 * normal(n, k)
    if case["a"] == "fp8":
        s["a"], s["as"] = _quantized(a, 1)
        s["w"], s["ws"] = _quantized(w, 1 if case["wscale"] == "row" else None)
    else:
        s["a"], s["as"], s["w"], s["ws"] = a.bfloat16(), None, w.bfloat16(), None
    s["b"] = (0.1 * normal(n)).bfloat16() if case["bias"] else None
    # the stream that a branch is added to is larger than the branch
    s["r"] = None if case["res"] == "none" else (4.0 * normal(m, n)).to(TYPES[case["res"]])
    s["out"] = torch.empty(m, n, device="cuda", dtype=TYPES[case["out"]])
    return s


# ---------------------------------------------------------------- one pass
ACTS = {"none": "none", "gelu": "gelu_tanh", "silu": "silu", "relu": "relu"}


def run(s):
    case = s["case"]
    if own:
        from video_diffusion_transformer_fwd_b200 import wan
        if case["op"] == "rmsnorm":
            y, scale, h = wan.rmsnorm(s["x"], s["g"], residual=s["r"], eps=EPS, out=s["y"], row_scale=s["scale"],
                                      h_out=s["h"])
            return _norm_outputs(y, scale, h if s["r"] is not None else None)
        return wan.linear(s["a"], s["w"], bias=s["b"], activation=ACTS[case["act"]], residual=s["r"], a_scale=s["as"],
                          w_scale=s["ws"], out=s["out"])
    return _plain_norm(s) if case["op"] == "rmsnorm" else _plain_linear(s)


def _norm_outputs(y, scale, h):
    return {k: v for k, v in (("y", y), ("scale", scale), ("h", h)) if v is not None}


def _plain_norm(s):
    case = s["case"]
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * s["g"] * rstd
    scale = None
    if case["out"] == "fp8":
        amax = y.abs().amax(1, keepdim=True)
        inv = torch.where(amax > 0, E4M3_MAX / amax, torch.zeros_like(amax))
        y = (y * inv).clamp(-E4M3_MAX, E4M3_MAX)
        scale = (amax / E4M3_MAX).reshape(-1)
    return _norm_outputs(y.to(TYPES[case["out"]]), scale, None if s["r"] is None else h.to(s["r"].dtype))


def _plain_linear(s):
    case = s["case"]
    v = torch.matmul(s["a"].float(), s["w"].float().t())
    if s["as"] is not None:
        v = v * (s["as"][:, None] * s["ws"][None, :])
    if s["b"] is not None:
        v = v + s["b"].float()
    if case["act"] == "gelu":
        v = 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    elif case["act"] == "silu":
        v = v / (1.0 + torch.exp(-v))
    elif case["act"] == "relu":
        v = torch.maximum(v, torch.zeros_like(v))
    if s["r"] is not None:
        v = v + s["r"].float()
    return v.to(s["out"].dtype)


# ---------------------------------------------------------------- work and exact values
def work(case):
    if case["op"] == "rmsnorm":
        rows, width = case["rows"], case["width"]
        per = SIZE[case["x"]] + 2 * SIZE[case["res"]] + SIZE[case["out"]]
        return {"bytes": rows * width * per + 4 * width + (4 * rows if case["out"] == "fp8" else 0),
                "flops": 5 * rows * width}
    m, n, k = case["m"], case["n"], case["k"]
    e = SIZE[case["a"]]
    b = (m + n) * k * e + m * n * (SIZE[case["res"]] + SIZE[case["out"]]) + (2 * n if case["bias"] else 0)
    if case["a"] == "fp8":
        b += 4 * m + (4 * n if case["wscale"] == "row" else 4)
    return {"bytes": b, "flops": 2 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rmsnorm":
        x = s["x"].double()
        h = x if s["r"] is None else x + s["r"].double()
        y = h * torch.rsqrt(h.square().sum(-1, keepdim=True) / case["width"] + EPS) * s["g"].double()
        scale = None
        if case["out"] == "fp8":                     # the codes before their rounding
            top = torch.linalg.vector_norm(y, math.inf, dim=-1)
            scale = top / E4M3_MAX
            y = y / scale[:, None]
        return _norm_outputs(y, scale, None if s["r"] is None else h)
    v = torch.einsum("mk,nk->mn", s["a"].double(), s["w"].double())
    if s["as"] is not None:
        v = v * s["as"].double().outer(s["ws"].double().expand(case["n"]))
    if s["b"] is not None:
        v += s["b"].double()
    if case["act"] == "gelu":
        v = v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v.pow(3)))
    elif case["act"] == "silu":
        v = v * torch.sigmoid(v)
    elif case["act"] == "relu":
        v = v.clamp_min(0.0)
    return v if s["r"] is None else v + s["r"].double()
