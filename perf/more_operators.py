"""The feed-forward half of a decoder block with microscaled weights, and its gradient: the cases that are timed.

Five kinds of case:

* ``norm``: a block's output joins the residual stream (normalised, gated, scaled) and the stream is normalised for
  the next block.
* ``norm_grad``: its gradient, for the stream, the block's output and the vectors.
* ``gated``: activations times two 4-bit microscaled matrices, one's products through an activation function and
  times the other's.
* ``gated_grad``: its gradient for the activations, through the frozen weights.
* ``product_grad``: the gradient of a plain product with such weights for its activations.

The plain form of each is elementary torch arithmetic in float32, rounded once at the end; with ``own`` set the
same data goes through the package's entry points.

Microscaled format: blocks of 32 consecutive values of a row share a power of two 2^(byte - 127); elements are e2m1
(two to a byte, the even one low) or e4m3.  Rows are padded with zeros to 128 columns.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GRID4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------------------------

def _pow2(e):
    """2^e in float32 for whole e of -126 .. 127."""
    return torch.exp2(e.float())


def plain_quantize(x, fmt):
    """(codes, scale bytes) of x's rows: finite values."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % 128))
    b = x.reshape(x.shape[0], -1, 32)
    a = b.abs().amax(-1)
    e = torch.where(a == 0, -127, (torch.frexp(a).exponent - 1 - (2 if fmt == "fp4" else 8)).clamp(min=-127))
    y = (b * _pow2(-torch.div(e, 2, rounding_mode="floor"))[..., None]) * _pow2(-(e - torch.div(e, 2, rounding_mode="floor")))[..., None]
    m = y.abs()
    if fmt == "fp4":
        c = sum((m > t).int() for t in (0.25, 1.25, 2.5, 5.0)) + sum((m >= t).int() for t in (0.75, 1.75, 3.5))
        c = (c + torch.signbit(y).int() * 8).reshape(x.shape[0], -1)
        codes = (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8)
    else:
        k = (torch.frexp(m).exponent - 1).clamp(min=-6)
        c = ((k + 7) * 8 + torch.round(m * _pow2(3 - k)).int() - 8).clamp(max=0x7E) + torch.signbit(y).int() * 128
        codes = c.to(torch.uint8).reshape(x.shape[0], -1)
    return codes, (e + 127).to(torch.uint8)


def plain_values(codes, scales, fmt, cols):
    """The float32 values of codes and scale bytes."""
    if fmt == "fp4":
        grid = torch.tensor(GRID4 + tuple(-g for g in GRID4), device=codes.device)
        v = grid[torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1).int()]
    else:
        c = codes.int()
        k, q = (c >> 3) & 15, c & 7
        v = torch.where(k == 0, q.float() * 2.0 ** -9, (8 + q).float() * _pow2(k - 10))
        v = torch.where(c >= 128, -v, v)
    return (v.reshape(v.shape[0], -1, 32) * torch.exp2(scales.float() - 127)[..., None]).reshape(v.shape[0], -1)[:, :cols]


def _normed(v, layer, eps):
    """(normalised rows, reciprocal deviations)."""
    if layer:
        v = v - v.mean(-1, keepdim=True)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    return v * r, r


def _through_norm(t, n, r, layer):
    """The gradient for a normalised row's input, t that for its output n."""
    d = t - n * (t * n).mean(-1, keepdim=True)
    if layer:
        d = d - t.mean(-1, keepdim=True)
    return d * r


def plain_norm(s):
    h = s["x"].float() * s["scale"]
    if s["b"] is not None:
        p = s["b"].float()
        if s["post_weight"] is not None:
            p = _normed(p, s["layer"], s["eps"])[0] * s["post_weight"].float()
        if s["gate"] is not None:
            p = p * s["gate"].float()
        h = h + p
    y = _normed(h, s["layer"], s["eps"])[0] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return [h.to(s["x"].dtype), y.to(s["y_type"])]


def plain_norm_grad(s):
    out = {}
    dy, h, layer = s["dy"].float(), s["h"].float(), s["layer"]
    n, r = _normed(h, layer, s["eps"])
    d = _through_norm(dy * s["weight"].float(), n, r, layer) + s["dh"].float()
    out["weight"] = (dy * n).sum(0)
    if s["bias"] is not None:
        out["bias"] = dy.sum(0)
    out["x"] = (d * s["scale"]).to(s["h"].dtype)
    if s["b"] is not None:
        p, post = s["b"].float(), s["post_weight"] is not None
        if post:
            n, r = _normed(p, layer, s["eps"])
            p = n * s["post_weight"].float()
        if s["gate"] is not None:
            each = d * p
            out["gate"] = each.to(s["gate"].dtype) if s["gate"].dim() == 2 else each.sum(0)
            d = d * s["gate"].float()
        if post:
            out["post_weight"] = (d * n).sum(0)
            d = _through_norm(d * s["post_weight"].float(), n, r, layer)
        out["b"] = d.to(s["b"].dtype)
    return out


def _act(g, act):
    """(value, slope) of the activation function."""
    if act == "silu":
        e = torch.sigmoid(g)
        return g * e, e * (1 + g * (1 - e))
    if act == "gelu":
        e = 0.5 * torch.erfc(g * -(0.5 ** 0.5))
        return g * e, e + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        e = torch.sigmoid(2 * c * (g + 0.044715 * g ** 3))
        return g * e, e + g * e * (1 - e) * 2 * c * (1 + 3 * 0.044715 * g * g)
    return g.clamp(min=0), (g > 0).float()


def _weights(s, name):
    return plain_values(*s[name], "fp4", s["d_in"])


def plain_gated(s):
    x = s["x"].float() if s["x_scales"] is None else plain_values(s["x"], s["x_scales"], s["x_type"], s["d_in"])
    g, u = torch.matmul(x, _weights(s, "gate").t()), torch.matmul(x, _weights(s, "up").t())
    y = (_act(g, s["act"])[0] * u).to(s["dtype"])
    return [y, g.to(s["dtype"]), u.to(s["dtype"])] if s["pre"] else y


def plain_gated_grad(s):
    a, slope = _act(s["g"].float(), s["act"])
    dy = s["dy"].float()
    d = torch.matmul(dy * s["u"].float() * slope, _weights(s, "gate")) + torch.matmul(dy * a, _weights(s, "up"))
    return d.to(s["dtype"])


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        import post_weight_quantization_accum_amd as P
        kind = s["kind"]
        if kind == "norm":
            return list(P.residual_norm(s["x"], s["b"], weight=s["weight"], bias=s["bias"], post_weight=s["post_weight"],
                                        gate=s["gate"], kind="layer" if s["layer"] else "rms", eps=s["eps"],
                                        residual_scale=s["scale"], dtype=s["y_type"]))
        if kind == "norm_grad":
            return P.residual_norm_backward(s["dy"], s["h"], s["b"], dH=s["dh"], weight=s["weight"], bias=s["bias"],
                                            post_weight=s["post_weight"], gate=s["gate"],
                                            kind="layer" if s["layer"] else "rms", eps=s["eps"],
                                            residual_scale=s["scale"])
        if kind == "gated":
            if s["x_scales"] is None:
                out = P.mx_gated(s["x"], s["gate"], s["up"], act=s["act"], pre=s["pre"])
            else:
                out = P.mx_gated_quantized(s["x"], s["x_scales"], s["gate"], s["up"], act=s["act"], x_fmt=s["x_type"],
                                           dtype=s["dtype"], pre=s["pre"])
            return list(out) if s["pre"] else out
        if kind == "gated_grad":
            return P.mx_gated_backward(s["dy"], s["g"], s["u"], s["gate"], s["up"], s["d_in"], act=s["act"])
        return P.mx_matmul_backward(s["dy"], *s["w"], s["d_in"])
    if s["kind"] == "norm":
        return plain_norm(s)
    if s["kind"] == "norm_grad":
        return plain_norm_grad(s)
    if s["kind"] == "gated":
        return plain_gated(s)
    if s["kind"] == "gated_grad":
        return plain_gated_grad(s)
    return torch.matmul(s["dy"].float(), _weights(s, "w")).to(s["dtype"])


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    norm = dict(kind="norm", layer=False, post=False, gate="", bias=False, scale=1.0)
    grad = dict(norm, kind="norm_grad")
    return [
        # between the halves of a block for one decoded token, the product of attention's output in float32: latency
        dict(norm, name="norm one token", rows=1, cols=4096, type="bf16", x="bf16", b="f32"),
        # prompts of a batch, the block's output normalised and gated by channel before it joins: bytes
        dict(norm, name="norm prompts", rows=8000, cols=5120, type="bf16", x="bf16", b="bf16", post=True, gate="channel"),
        # tuning a small layer-normed model on short texts, gates of their own for every token: latency and sums
        dict(grad, name="norm gradient small", rows=500, cols=768, type="f16", x="f16", b="f16", layer=True, bias=True,
             gate="token", scale=0.5),
        # tuning norms and gates after quantization, on whole sequences: bytes and the sums over tokens
        dict(grad, name="norm gradient sequences", rows=8192, cols=4096, type="bf16", x="f32", b="bf16", post=True,
             gate="channel"),
        # one decoded token: the weights' bytes
        dict(name="gated one token", kind="gated", tokens=1, d_in=4096, d_ff=11008, type="bf16", act="silu", pre=False),
        # some sequences decoded together through a larger model's layer: the weights' bytes
        dict(name="gated decode batch", kind="gated", tokens=13, d_in=5120, d_ff=13824, type="f16", act="silu", pre=False),
        # a sequence of training, its products kept for the gradient: the 16-bit matrix rate
        dict(name="gated sequence", kind="gated", tokens=2048, d_in=4096, d_ff=11008, type="bf16", act="silu", pre=True),
        # a prompt, both sides in 4 bits, an odd width: the 4-bit matrix rate
        dict(name="gated prompt fp4", kind="gated", tokens=1500, d_in=4096, d_ff=11000, type="fp4", act="gelu_tanh", pre=False),
        # tuning on short texts through a small layer, nothing a multiple of a tile
        dict(name="gated gradient ragged", kind="gated_grad", tokens=300, d_in=768, d_ff=2050, type="f16", act="gelu"),
        # the gradient of a training sequence: the 16-bit matrix rate
        dict(name="gated gradient sequence", kind="gated_grad", tokens=2048, d_in=4096, d_ff=11008, type="bf16", act="silu"),
        # a few tokens' gradient through a square projection: the weights' bytes
        dict(name="product gradient few", kind="product_grad", tokens=24, d_in=4096, d_out=4096, type="bf16"),
        # the gradient through a down projection for a training sequence: the 16-bit matrix rate
        dict(name="product gradient sequence", kind="product_grad", tokens=2048, d_in=11008, d_out=4096, type="bf16"),
    ]


def _log(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49))))))


def draw(rng):
    kind = rng.choice(("norm", "norm_grad", "gated", "gated", "gated_grad", "product_grad"))
    if kind in ("norm", "norm_grad"):
        cols = _log(rng, 8, 16384)
        t = rng.choice(("bf16", "f16", "f32"))
        case = dict(kind=kind, rows=_log(rng, 1, min(16384, 33554432 // cols)), cols=cols, type=t, x=rng.choice((t, "f32")),
                    b=rng.choice(("", t, t, "f32")), layer=rng.random() < 0.4, bias=rng.random() < 0.4,
                    scale=rng.choice((1.0, 1.0, 0.5, 2.5)))
        return dict(case, post=bool(case["b"]) and rng.random() < 0.5,
                    gate=rng.choice(("", "channel", "token")) if case["b"] else "")
    case = dict(kind=kind, tokens=_log(rng, 1, 2048), d_in=_log(rng, 40, 5120),
                act=rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu")))
    if kind == "gated":
        return dict(case, d_ff=_log(rng, 40, 8192), type=rng.choice(("bf16", "bf16", "f16", "f32", "fp4", "fp4", "fp8")),
                    pre=rng.random() < 0.3)
    if kind == "gated_grad":
        return dict(case, d_ff=_log(rng, 40, 8192), type=rng.choice(("bf16", "bf16", "f16", "f32")))
    return dict(kind=kind, tokens=case["tokens"], d_in=_log(rng, 40, 11008), d_out=_log(rng, 40, 5120),
                type=rng.choice(("bf16", "bf16", "f16", "f32")))


def _activations(g, rows, cols, dtype):
    """Normal values whose channels have scales of their own, a few of them large."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    s = torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV))
    s = torch.where(torch.rand(cols, generator=g, device=DEV) < 0.005, s * 30, s)
    return (x * s).to(dtype)


def _gradients(g, rows, cols, dtype):
    """Small normal values, tokens of different weight."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    return (x * 2e-3 * torch.exp(torch.randn(rows, 1, generator=g, device=DEV))).to(dtype)


def _quantized(g, rows, cols):
    return plain_quantize(torch.randn(rows, cols, generator=g, device=DEV) * cols ** -0.5, "fp4")


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kind = case["kind"]
    s = dict(kind=kind)
    if kind in ("norm", "norm_grad"):
        n, d, t = case["rows"], case["cols"], TYPES[case["type"]]
        s.update(layer=case["layer"], eps=1e-5 if case["layer"] else 1e-6, scale=case["scale"], bias=None,
                 post_weight=None, gate=None, b=None)
        s["h" if kind == "norm_grad" else "x"] = _activations(g, n, d, TYPES[case["x"]])
        if case["b"]:
            s["b"] = _activations(g, n, d, TYPES[case["b"]])
        s["weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(t)
        if case["bias"]:
            s["bias"] = (0.1 * torch.randn(d, generator=g, device=DEV)).to(t)
        if case["post"]:
            s["post_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(t)
        if case["gate"]:
            s["gate"] = (0.5 * torch.randn(*((n,) if case["gate"] == "token" else ()), d, generator=g, device=DEV)).to(t)
        if kind == "norm":
            return dict(s, y_type=t)
        return dict(s, dy=_gradients(g, n, d, t), dh=_gradients(g, n, d, TYPES[case["x"]]))
    n, d_in = case["tokens"], case["d_in"]
    mx = case["type"] in ("fp4", "fp8")
    s.update(d_in=d_in, dtype=torch.bfloat16 if mx else TYPES[case["type"]])
    if kind == "product_grad":
        return dict(s, w=_quantized(g, case["d_out"], d_in), dy=_gradients(g, n, case["d_out"], s["dtype"]))
    d_ff = case["d_ff"]
    s.update(act=case["act"], gate=_quantized(g, d_ff, d_in), up=_quantized(g, d_ff, d_in))
    if kind == "gated":
        x = _activations(g, n, d_in, torch.float32)
        x = (x / x.square().mean(-1, keepdim=True).sqrt()).to(s["dtype"])       # behind a norm
        s.update(x=x, x_scales=None, x_type=case["type"], pre=case["pre"])
        if mx:
            s["x"], s["x_scales"] = plain_quantize(x, case["type"])
        return s
    for name in ("g", "u"):
        s[name] = torch.randn(n, d_ff, generator=g, device=DEV).to(s["dtype"])
    return dict(s, dy=_gradients(g, n, d_ff, s["dtype"]))


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1 + 1 / 32, "fp4": 0.5 + 1 / 32, "": 0}
    if case["kind"] in ("norm", "norm_grad"):
        n, d, t = case["rows"], case["cols"], size[case["type"]]
        x, b = size[case["x"]], size[case["b"]]
        gate = t if case["gate"] == "token" else 0
        if case["kind"] == "norm":
            return {"bytes": n * d * (2 * x + b + t + gate), "flops": 0}
        # h, dy, dh, dx; b and its gradient (b itself is needed for a norm's or a gate's gradient only)
        needs = b if case["post"] or case["gate"] else 0
        return {"bytes": n * d * (3 * x + t + needs + b + 2 * gate), "flops": 0}
    n, k, t = case["tokens"], case["d_in"], case["type"]
    y = 2 if t in ("fp4", "fp8") else size[t]
    if case["kind"] == "product_grad":
        m = case["d_out"]
        return {"bytes": n * m * size[t] + m * k * size["fp4"] + n * k * y, "flops": 2 * n * m * k}
    m = case["d_ff"]
    if case["kind"] == "gated":
        return {"bytes": n * k * size[t] + 2 * m * k * size["fp4"] + n * m * y * (3 if case["pre"] else 1), "flops": 4 * n * m * k}
    return {"bytes": 3 * n * m * size[t] + 2 * m * k * size["fp4"] + n * k * y, "flops": 4 * n * m * k}


# ---------------------------------------------------------------------------------------------------------------
# From the definition, in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _held64(codes, scales, fmt, cols):
    """float64 values of codes and scale bytes, from the list of every element."""
    if fmt == "fp4":
        grid = [m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1) for e in range(4) for m in range(2)]
    else:
        grid = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)]
    grid = torch.tensor(grid, dtype=torch.float64, device=codes.device)
    c = codes.long()
    if fmt == "fp4":
        c = torch.cat(((c % 16)[..., None], (c // 16)[..., None]), -1).flatten(-2)
    v = torch.cat((grid, -grid))[c]
    return (v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1))[:, :cols]


def _act64(g, act):
    if act == "relu":
        return torch.relu(g)
    return torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(
        g, approximate="tanh" if act == "gelu_tanh" else "none")


def _norm64(v, layer, eps):
    if layer:
        return torch.nn.functional.layer_norm(v, v.shape[-1:], eps=eps)
    return v / (v.square().mean(-1, keepdim=True) + eps).sqrt()


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "product_grad":
        return s["dy"].double() @ _held64(*s["w"], "fp4", s["d_in"])
    if kind == "gated":
        x = s["x"].double() if s["x_scales"] is None else _held64(s["x"], s["x_scales"], s["x_type"], s["d_in"])
        g, u = (x @ _held64(*s[n], "fp4", s["d_in"]).t() for n in ("gate", "up"))
        y = _act64(g, s["act"]) * u
        return [y, g, u] if s["pre"] else y
    if kind == "gated_grad":
        g, u = (s[n].double().requires_grad_() for n in ("g", "u"))
        (_act64(g, s["act"]) * u).backward(s["dy"].double())
        return g.grad @ _held64(*s["gate"], "fp4", s["d_in"]) + u.grad @ _held64(*s["up"], "fp4", s["d_in"])
    back = kind == "norm_grad"
    v = {k: s[k].double() for k in ("b", "weight", "bias", "post_weight", "gate") if s[k] is not None}
    v["x"] = s["h"].double() if back else s["x"].double()
    if back:
        # through the formula by differentiation, the stream's value set to the one at hand
        v = {k: t.requires_grad_() for k, t in v.items()}
    h = v["x"] * s["scale"]
    if "b" in v:
        p = v["b"]
        if "post_weight" in v:
            p = _norm64(p, s["layer"], s["eps"]) * v["post_weight"]
        h = h + p * v.get("gate", 1.0)
    if back:
        h = s["h"].double() + (h - h.detach())
    y = _norm64(h, s["layer"], s["eps"]) * v["weight"] + v.get("bias", 0.0)
    if not back:
        return [h, y]
    torch.autograd.backward([y, h], [s["dy"].double(), s["dh"].double()])
    return {k: t.grad for k, t in v.items()}
