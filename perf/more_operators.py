"""Measured cases of the operators around a quantized layer: block norms, and products with an epilogue.

Five kinds of pass, each in a plain form (elementary torch operations in 32 bits) and through the
package's entry points:

* ``norm``: a block's output y joins the residual stream r (normalized, gated and scaled), and the
  stream is normalized for the next block (``block_norm``, ``block_norm_w8a8``, ``block_norm_mxfp4``):

      u = y, or y / rms(y) * post_weight;  r' = r + scale * gate * u;  out = r' / rms(r') * weight

  with rms(v) = sqrt(mean(v^2) + eps) along the row. The gate is absent, one fp32 value per channel,
  or a row per token. out is of the rows' type, or int8 rows (one scale per row), or MXFP4 rows;
  quantized rows are returned as the values that they stand for;
* ``norm_backward``: its gradients, from those of out and r' (``block_norm_backward``);
* ``linear``: 16-bit rows and weights, act(x w^T + bias) + residual, and for training
  pre = x w^T + bias beside it (``w16a16_linear``);
* ``linear_backward``: d_pre = d_out * act'(pre) in the rows' type, d_bias its column sums before that
  rounding, and d_x = d_pre w, d_w = d_pre^T x (``w16a16_linear_backward``);
* ``w8a8``: the int8 product with row and channel scales, bias, activation and residual
  (``w8a8_gemm_act``).
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
ACTIVATIONS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 16 sequences before a W8A8 layer: latency
        {"name": "norm_decode", "kind": "norm", "dtype": "bf16", "rows": 16, "width": 4096, "post": False,
         "gate": "none", "out": "int8"},
        # a vision transformer's block, 64 images of 257 tokens, with a learned gate per channel
        {"name": "norm_images", "kind": "norm", "dtype": "bf16", "rows": 16448, "width": 1280, "post": True,
         "gate": "channel", "out": "same"},
        # an odd width, a gate row for every token, in 32 bits
        {"name": "norm_odd", "kind": "norm", "dtype": "f32", "rows": 1285, "width": 1031, "post": True,
         "gate": "token", "out": "same"},
        # a small training batch of an odd width in binary16
        {"name": "norm_backward_odd", "kind": "norm_backward", "dtype": "f16", "rows": 257, "width": 1031,
         "post": True, "gate": "channel"},
        # a training batch of 8192 tokens with a gate row for every token
        {"name": "norm_backward_large", "kind": "norm_backward", "dtype": "bf16", "rows": 8192, "width": 4096,
         "post": True, "gate": "token"},
        # one sequence decoding: the weight is read for a single row
        {"name": "linear_token", "kind": "linear", "dtype": "bf16", "m": 1, "n": 4096, "k": 4096,
         "act": "silu", "bias": True, "residual": True, "pre": False},
        # one image's rows, widths that no tile divides, in binary16
        {"name": "linear_odd", "kind": "linear", "dtype": "f16", "m": 257, "n": 1040, "k": 1312,
         "act": "gelu_tanh", "bias": True, "residual": True, "pre": False},
        # the first feed-forward product of 64 images in training
        {"name": "linear_large", "kind": "linear", "dtype": "bf16", "m": 16448, "n": 5120, "k": 1280,
         "act": "gelu", "bias": True, "residual": False, "pre": True},
        # the gradients of a small batch of ragged sizes
        {"name": "linear_backward_odd", "kind": "linear_backward", "dtype": "f16", "m": 257, "n": 1040,
         "k": 1312, "act": "silu", "bias": True},
        # the gradients of the first feed-forward product of 64 images
        {"name": "linear_backward_large", "kind": "linear_backward", "dtype": "bf16", "m": 16448, "n": 5120,
         "k": 1280, "act": "gelu", "bias": True},
        # 16 sequences decoding through a W8A8 layer that adds to the residual stream
        {"name": "w8a8_decode", "kind": "w8a8", "m": 16, "n": 4096, "k": 4096, "act": "none", "bias": True,
         "residual": True},
        # a prompt of 2048 tokens through a W8A8 layer
        {"name": "w8a8_prefill", "kind": "w8a8", "m": 2048, "n": 4096, "k": 4096, "act": "gelu_tanh",
         "bias": True, "residual": True},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v / step + 0.5) * step)


def draw(rng):
    kind = rng.choice(["norm", "norm_backward", "linear", "linear_backward", "w8a8"])
    while True:
        if kind.startswith("norm"):
            c = {"kind": kind, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "rows": _log(rng, 1, 38400),
                 "width": _log(rng, 64, 8192), "post": rng.random() < 0.5,
                 "gate": rng.choice(["none", "channel", "token"])}
            if kind == "norm":
                c["out"] = rng.choice(["same", "int8", "mxfp4"])
                if c["out"] != "same":  # rows that a quantized product takes
                    c["width"] = max(32, c["width"] // 32 * 32)
            fits = work(c)["bytes"] <= work(listed()[4])["bytes"]
        elif kind == "w8a8":
            c = {"kind": kind, "m": _log(rng, 1, 16448), "n": _log(rng, 128, 8192, 16), "k": _log(rng, 128, 8192, 16),
                 "act": rng.choice(ACTIVATIONS), "bias": rng.random() < 0.7, "residual": rng.random() < 0.5}
            fits = work(c)["flops"] <= work(listed()[7])["flops"] and c["m"] * c["n"] <= 16448 * 5120
        else:
            c = {"kind": kind, "dtype": rng.choice(["bf16", "f16"]), "m": _log(rng, 1, 16448),
                 "n": _log(rng, 64, 8192, 8), "k": _log(rng, 64, 8192, 8), "act": rng.choice(ACTIVATIONS),
                 "bias": rng.random() < 0.7}
            if kind == "linear":
                c.update(residual=rng.random() < 0.5, pre=rng.random() < 0.3)
            fits = (c["m"] * c["n"] * c["k"] <= 16448 * 5120 * 1280
                    and max(c["m"] * c["n"], c["m"] * c["k"]) <= 16448 * 5120)
        if fits:
            return c


def work(case):
    kind = case["kind"]
    if kind.startswith("norm"):
        t, h, e = case["rows"], case["width"], BYTES[case["dtype"]]
        gate = 1 if case["gate"] == "token" else 0
        if kind == "norm":
            # y, r, the gate; r' and the rows for the next block
            out = {"same": e, "int8": 1, "mxfp4": 17 / 32}[case["out"]]
            return {"bytes": int(t * h * (e * (3 + gate) + out)) + 12 * h, "flops": (10 + 4 * case["post"]) * t * h}
        # the gradients of out and r', r', y, the gate; the gradients of r, y and the gate
        return {"bytes": t * h * e * (6 + 2 * gate) + 24 * h, "flops": (16 + 8 * case["post"]) * t * h}
    m, n, k = case["m"], case["n"], case["k"]
    if kind == "w8a8":
        return {"bytes": m * k + n * k + 2 * m * n * (1 + case["residual"]) + 4 * (m + 2 * n), "flops": 2 * m * n * k}
    if kind == "linear":
        return {"bytes": 2 * (m * k + n * k + m * n * (1 + case["residual"] + case["pre"])) + 4 * n,
                "flops": 2 * m * n * k}
    # x, w, d_out, pre; d_x, d_w, d_pre
    act = case["act"] != "none"
    return {"bytes": 2 * (2 * m * k + 2 * n * k + m * n * (1 + 2 * act)) + 4 * n, "flops": 4 * m * n * k}


# ---------------------------------------------------------------- inputs

def _rows(g, m, k):
    """Normal activations with a hundredth of the channels 20 times larger, in 32 bits."""
    x = torch.randn((m, k), generator=g, device=DEV)
    x[:, torch.randperm(k, generator=g, device=DEV)[:max(1, k // 100)]] *= 20.0
    return x


def _normal(g, *shape, scale=1.0, shift=0.0):
    return torch.randn(shape, generator=g, device=DEV) * scale + shift


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kind = case["kind"]
    s = {"kind": kind}
    if kind.startswith("norm"):
        t, h, dtype = case["rows"], case["width"], TYPES[case["dtype"]]
        s.update(post=case["post"], out=case.get("out"), scale=0.7)
        s["y"] = _normal(g, t, h, scale=3.0).to(dtype)
        s["r"] = _rows(g, t, h).to(dtype)
        s["weight"] = _normal(g, h, scale=0.2, shift=1.0)
        s["post_weight"] = _normal(g, h, scale=0.2, shift=1.0) if case["post"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: _normal(g, h, scale=0.5),
                     "token": lambda: torch.sigmoid(_normal(g, t, h)).to(dtype)}[case["gate"]]()
        if kind == "norm_backward":
            s["d_out"] = _normal(g, t, h).to(dtype)
            s["d_r"] = _normal(g, t, h).to(dtype)
        return s
    m, n, k = case["m"], case["n"], case["k"]
    s["act"] = case["act"]
    s["bias"] = _normal(g, n, scale=0.5) if case["bias"] else None
    if kind == "w8a8":
        # activations and a weight as the row quantization leaves them
        x, w = _rows(g, m, k), _normal(g, n, k, scale=k ** -0.5)
        s["xs"], s["ws"] = (v.abs().amax(dim=1) / 127 for v in (x, w))
        s["xq"], s["wq"] = (torch.round(v / d.unsqueeze(1)).to(torch.int8) for v, d in ((x, s["xs"]), (w, s["ws"])))
        s["residual"] = _normal(g, m, n, scale=2.0).to(torch.bfloat16) if case["residual"] else None
        return s
    dtype = TYPES[case["dtype"]]
    s["x"] = _rows(g, m, k).to(dtype)
    s["w"] = _normal(g, n, k, scale=k ** -0.5).to(dtype)
    if kind == "linear":
        s["residual"] = _normal(g, m, n, scale=2.0).to(dtype) if case["residual"] else None
        s["pre"] = case["pre"]
    else:
        s["pre"] = _normal(g, m, n, scale=1.5).to(dtype)
        s["d_out"] = _normal(g, m, n).to(dtype)
    return s


# ---------------------------------------------------------------- the plain form

def _activation(v, act):
    if act == "relu":
        return torch.where(v < 0, 0.0, v)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _slope(v, act):
    """The activation's derivative."""
    if act == "relu":
        return (v > 0).to(v.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * math.sqrt(2 / math.pi) * (1.0 + 3 * 0.044715 * v * v)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-v))
        return p * (1.0 + v * (1.0 - p))
    return torch.ones_like(v)


def _scaled(v, weight):
    return v if weight is None else v * weight


def _plain_norm(s):
    # values that go to 8 or 4 bits lie next to their borders: 64 bits there
    wide = torch.float32 if s["out"] == "same" else torch.float64
    y, r, dtype = s["y"].to(wide), s["r"].to(wide), s["r"].dtype
    if s["post"]:
        y = _scaled(y * torch.rsqrt((y * y).mean(dim=1, keepdim=True) + EPS), s["post_weight"])
    if s["gate"] is not None:
        y = y * s["gate"].to(wide)
    r = r + s["scale"] * y
    o = r * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + EPS) * s["weight"]
    if s["out"] == "int8":
        step = (o.abs().amax(dim=1, keepdim=True) / 127).float()
        o = torch.round(o / step).clamp(-127, 127) * step
    elif s["out"] == "mxfp4":
        o = _mx_values(o)
    return {"residual": r.to(dtype), "out": o.to(dtype if s["out"] == "same" else torch.bfloat16)}


def _mx_values(o):
    """The values that blocks of 32 take in MXFP4: a power-of-two step from the largest, 4-bit elements."""
    v = o.reshape(o.shape[0], -1, 32)
    top = v.abs().amax(dim=2, keepdim=True)
    scale = torch.exp2((torch.floor(torch.log2(top)) - 2).clamp_min(-127))
    a = v.abs() / scale
    q = 0.5 * ((a > 0.25).to(o.dtype) + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5.0)
    return (torch.sign(v) * q * scale).reshape(o.shape)


def _plain_norm_backward(s):
    y, r, dtype = s["y"].float(), s["r"].float(), s["r"].dtype
    d_out = s["d_out"].float()
    rstd = torch.rsqrt((r * r).mean(dim=1, keepdim=True) + EPS)
    rh = r * rstd
    dn = d_out * s["weight"]
    d_r = s["d_r"].float() + rstd * (dn - rh * (dn * rh).mean(dim=1, keepdim=True))
    found = {"d_residual": d_r.to(dtype), "d_weight": (d_out * rh).sum(dim=0)}
    g = s["scale"] * d_r
    if s["post"]:
        ystd = torch.rsqrt((y * y).mean(dim=1, keepdim=True) + EPS)
        yh = y * ystd
        u = yh * s["post_weight"]
    else:
        u = y
    gate = s["gate"]
    if gate is not None:
        found["d_gate"] = (g * u).sum(dim=0) if gate.dim() == 1 else (g * u).to(dtype)
        g = g * gate.float()
    if s["post"]:
        found["d_post_weight"] = (g * yh).sum(dim=0)
        dh = g * s["post_weight"]
        g = ystd * (dh - yh * (dh * yh).mean(dim=1, keepdim=True))
    found["d_y"] = g.to(dtype)
    return found


def _plain_linear(s):
    pre = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        pre = pre + s["bias"]
    out = _activation(pre, s["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    dtype = s["x"].dtype
    return {"out": out.to(dtype), "pre": pre.to(dtype)} if s["pre"] else out.to(dtype)


def _plain_linear_backward(s):
    d = s["d_out"].float() * _slope(s["pre"].float(), s["act"])
    d_pre, dtype = d.to(s["x"].dtype), s["x"].dtype
    found = {"d_x": (d_pre.float() @ s["w"].float()).to(dtype), "d_w": (d_pre.float().t() @ s["x"].float()).to(dtype)}
    if s["act"] != "none":
        found["d_pre"] = d_pre
    if s["bias"] is not None:
        found["d_bias"] = d.sum(dim=0)
    return found


def _plain_w8a8(s):
    out = (s["xq"].float() @ s["wq"].float().t()) * s["xs"].unsqueeze(1) * s["ws"]
    if s["bias"] is not None:
        out = out + s["bias"]
    out = _activation(out, s["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(torch.bfloat16)


def _own(s):
    from quantized_gemm_quantize_amd import binding as b
    kind = s["kind"]
    if kind == "norm":
        kw = dict(y=s["y"], post_norm=s["post"], post_weight=s["post_weight"], gate=s["gate"], scale=s["scale"], eps=EPS)
        if s["out"] == "same":
            residual, out = b.block_norm(s["r"], s["weight"], **kw)
        elif s["out"] == "int8":
            residual, xq, xs = b.block_norm_w8a8(s["r"], s["weight"], **kw)
            out = (xq * xs.unsqueeze(1)).to(torch.bfloat16)
        else:
            residual, codes, scales = b.block_norm_mxfp4(s["r"], s["weight"], **kw)
            out = b.mxfp4_dequantize_rows(codes, scales)
        return {"residual": residual, "out": out}
    if kind == "norm_backward":
        d_residual, d_weight, d_y, d_post_weight, d_gate = b.block_norm_backward(
            s["d_out"], s["r"], s["weight"], d_residual=s["d_r"], y=s["y"], post_norm=s["post"],
            post_weight=s["post_weight"], gate=s["gate"], scale=s["scale"], eps=EPS)
        found = {"d_residual": d_residual, "d_weight": d_weight}
        if s["gate"] is not None:
            found["d_gate"] = d_gate
        if s["post"]:
            found["d_post_weight"] = d_post_weight
        found["d_y"] = d_y
        return found
    if kind == "linear":
        if s["pre"]:
            out, pre = b.w16a16_linear(s["x"], s["w"], bias=s["bias"], activation=s["act"], residual=s["residual"],
                                       pre=True)
            return {"out": out, "pre": pre}
        return b.w16a16_linear(s["x"], s["w"], bias=s["bias"], activation=s["act"], residual=s["residual"])
    if kind == "linear_backward":
        d_x, d_w, d_bias, d_pre = b.w16a16_linear_backward(
            s["d_out"], s["x"], s["w"], pre=s["pre"] if s["act"] != "none" else None, activation=s["act"],
            d_bias=s["bias"] is not None)
        found = {"d_x": d_x, "d_w": d_w}
        if s["act"] != "none":
            found["d_pre"] = d_pre
        if s["bias"] is not None:
            found["d_bias"] = d_bias
        return found
    return b.w8a8_gemm_act(s["xq"], s["xs"], s["wq"], s["ws"], bias=s["bias"], activation=s["act"],
                           residual=s["residual"])


PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "linear": _plain_linear,
         "linear_backward": _plain_linear_backward, "w8a8": _plain_w8a8}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["kind"]](state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_act(v, act):
    """(act(v), act'(v))"""
    if act == "relu":
        return v.clamp_min(0), torch.where(v > 0, 1.0, 0.0).double()
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-v / math.sqrt(2))
        return v * cdf, cdf + v * torch.exp(-v.square() / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        # (1 + tanh(z)) / 2 = sigmoid(2 z)
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (v + 0.044715 * v ** 3))
        return v * p, p + v * p * (1 - p) * c * (1 + 3 * 0.044715 * v.square())
    if act == "silu":
        p = torch.sigmoid(v)
        return v * p, p + v * p * (1 - p)
    return v, torch.ones_like(v)


def _exact_grid(o):
    """MXFP4 values: per block of 32 a step of 2^(floor(log2 max) - 2), elements rounded half to even on
    the grid of one fraction bit above 1 and of halves below, at most 6."""
    v = o.reshape(o.shape[0], -1, 32)
    _, e = torch.frexp(v.abs().amax(dim=2, keepdim=True))
    a = torch.ldexp(v.abs(), 3 - e)
    _, ea = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (ea - 1).clamp(0, 2) - 1)
    return (torch.sign(v) * torch.ldexp((torch.round(a / step) * step).clamp_max(6.0), e - 3)).reshape(o.shape)


def _direction(v):
    """v over its root mean square, and that root's inverse."""
    inv = 1.0 / torch.sqrt(v.square().sum(dim=1, keepdim=True) / v.shape[1] + EPS)
    return v * inv, inv


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind.startswith("norm"):
        y, r = s["y"].double(), s["r"].double()
        post_weight = s["post_weight"].double() if s["post"] else None
        gate = 1.0 if s["gate"] is None else s["gate"].double()
        yh, yinv = _direction(y)
        u = yh * post_weight if s["post"] else y
        if kind == "norm":
            r = r + u * gate * s["scale"]
            o = _direction(r)[0] * s["weight"].double()
            if s["out"] == "int8":
                step = o.abs().amax(dim=1, keepdim=True).div(127)
                o = torch.round(o / step) * step
            elif s["out"] == "mxfp4":
                o = _exact_grid(o)
            return {"residual": r, "out": o}
        rh, rinv = _direction(r)
        d_out = s["d_out"].double()
        d = d_out * s["weight"].double()
        d_r = s["d_r"].double() + rinv * d - rinv * rh * (d * rh).sum(dim=1, keepdim=True) / r.shape[1]
        found = {"d_residual": d_r, "d_weight": torch.einsum("th,th->h", d_out, rh)}
        d_u = s["scale"] * d_r * gate
        if s["gate"] is not None:
            d_gate = s["scale"] * d_r * u
            found["d_gate"] = d_gate.sum(dim=0) if s["gate"].dim() == 1 else d_gate
        if s["post"]:
            found["d_post_weight"] = torch.einsum("th,th->h", d_u, yh)
            d_h = d_u * post_weight
            d_u = yinv * d_h - yinv * yh * (d_h * yh).sum(dim=1, keepdim=True) / y.shape[1]
        found["d_y"] = d_u
        return found
    bias = 0.0 if s["bias"] is None else s["bias"].double()
    if kind == "linear_backward":
        x, w = s["x"].double(), s["w"].double()
        d = s["d_out"].double() * _exact_act(s["pre"].double(), s["act"])[1]
        d_pre = d.to(s["x"].dtype).double()   # an output of its own, which the products take
        found = {"d_x": d_pre.mm(w), "d_w": d_pre.t().contiguous().mm(x)}
        if s["act"] != "none":
            found["d_pre"] = d
        if s["bias"] is not None:
            found["d_bias"] = d.sum(dim=0)
        return found
    if kind == "linear":
        pre = torch.addmm(torch.zeros((), dtype=torch.float64, device=DEV), s["x"].double(),
                          s["w"].double().t().contiguous()) + bias
    else:
        pre = s["xq"].double().mm(s["wq"].double().t().contiguous())
        pre = pre * s["xs"].double().unsqueeze(1) * s["ws"].double() + bias
    out = _exact_act(pre, s["act"])[0]
    if s["residual"] is not None:
        out = out + s["residual"].double()
    return {"out": out, "pre": pre} if kind == "linear" and s["pre"] else out
