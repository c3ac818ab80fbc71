"""Norms around a block and their gradient against float64 (needs an MI355X).

Bounds, with u = 2^-24 and all magnitudes taken in float64.  A normalised value
n = (v - m) r carries at most four roundings of N = r (|v| + |m|): of m, r, the
difference and the product (the sums behind m and r are float64).  Then

  h:  s x + g p has at most eight roundings of |s x| + |g| (|b| or N_b |w_post|);
  y:  the error dh of h passes through the norm as |w| r (dh + mean dh + N rms dh), and w n + c
      adds at most eight of |w| N + |c|;
  D:  t = dy w (one rounding), n (four of N), mean(t n) (those five), three products and three
      sums: at most sixteen of r (|t| + mean |t| + N mean(|t| N)) + |dH|;
  dB: the error of q = D g w passes through the norm like a value (r_b (dq + mean dq + N_b mean(dq N_b))),
      which adds sixteen roundings of its own magnitudes;
  sums over tokens: each term's error, and one rounding for each of a part's rows and two more.

A result of type t is then rounded once: half a step, eps / 2 of the value, or half of the smallest number.
"""
import pytest
import torch

import post_weight_quantization_accum_amd as P

pytestmark = pytest.mark.gpu

DEV = "cuda"
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24
SMALL = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def half_step(v, dtype):
    return torch.clamp(v.abs() * (torch.finfo(dtype).eps / 2), min=SMALL[dtype] / 2)


def mean(v):
    return v.mean(-1, keepdim=True)


class Ref:
    """float64 values and magnitudes of one normalisation."""

    def __init__(self, v, layer, eps):
        self.layer = layer
        self.m = mean(v) if layer else torch.zeros_like(v[:, :1])
        self.r = 1 / (mean((v - self.m) ** 2) + eps).sqrt()
        self.n = (v - self.m) * self.r
        self.N = self.r * (v.abs() + self.m.abs())

    def back(self, t):
        return self.r * (t - self.n * mean(t * self.n) - (mean(t) if self.layer else 0))

    def back_error(self, t):
        return self.r * (t.abs() + mean(t.abs()) + self.N * mean(t.abs() * self.N))

    def pass_error(self, dt):
        return self.r * (dt + mean(dt) + self.N * mean(dt * self.N))


def case(n, d, x="bf16", b=None, t="bf16", layer=False, post=False, gate=None, bias=False, scale=1.0, seed=0, ld=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)

    def rows(dtype):
        wide = rnd(n, d + ld) * torch.exp(rnd(d + ld) * 0.5)
        return wide.to(T[dtype])[:, ld // 2: ld // 2 + d] if ld else wide.to(T[dtype])

    c = dict(X=rows(x), B=rows(b) if b else None, dY=rows(t), dH=rows(x),
             kw=dict(weight=(1 + 0.2 * rnd(d)).to(T[t]), kind="layer" if layer else "rms", eps=1e-5, residual_scale=scale))
    if bias:
        c["kw"]["bias"] = rnd(d).to(T[t])
    if post:
        c["kw"]["post_weight"] = (1 + 0.2 * rnd(d)).to(T[t])
    if gate:
        c["kw"]["gate"] = (rnd(n, d) if gate == "token" else rnd(d)).to(T[t])
    return c


def doubles(c):
    kw = {k: v.double() if torch.is_tensor(v) else v for k, v in c["kw"].items()}
    return kw, c["X"].double(), None if c["B"] is None else c["B"].double()


def check_forward(c, h, y):
    kw, x, b = doubles(c)
    layer, eps, s = kw["kind"] == "layer", kw["eps"], kw["residual_scale"]
    want, size = s * x, (s * x).abs()
    if b is not None:
        p, ps = b, b.abs()
        if kw.get("post_weight") is not None:
            ref = Ref(b, layer, eps)
            p, ps = ref.n * kw["post_weight"], ref.N * kw["post_weight"].abs()
        gate = kw.get("gate")
        gate = torch.ones_like(x) if gate is None else gate
        want, size = want + gate * p, size + gate.abs() * ps
    dh = 8 * U * size
    if h is not None:
        assert bool(((h.double() - want).abs() <= dh + half_step(want, h.dtype)).all())
    if y is None:
        return
    ref = Ref(want, layer, eps)
    w, bias = kw.get("weight"), kw.get("bias")
    w = torch.ones_like(x[0]) if w is None else w
    bias = torch.zeros_like(x[0]) if bias is None else bias
    wy = ref.n * w + bias
    err = w.abs() * ref.r * (dh + mean(dh) + ref.N * mean(dh ** 2).sqrt()) + 8 * U * (w.abs() * ref.N + bias.abs())
    assert bool(((y.double() - wy).abs() <= err + half_step(wy, y.dtype)).all())


def check_backward(c, got, dh=True):
    kw, h, b = doubles(c)
    layer, eps, s = kw["kind"] == "layer", kw["eps"], kw["residual_scale"]
    dy, dH = c["dY"].double(), c["dH"].double() * (1 if dh else 0)
    n, d = h.shape
    # a part's rows: a wave's of at most 4096 waves, or a workgroup's of at most 512
    k = 2 + -(-n // (4096 if d <= 1024 else 512))
    w = kw.get("weight")
    w = torch.ones_like(h[0]) if w is None else w
    ref = Ref(h, layer, eps)
    t = dy * w
    D = ref.back(t) + dH
    eD = 16 * U * (ref.back_error(t) + dH.abs())

    def near(name, want, err, dtype):
        g = got[name]
        assert g.dtype == dtype and g.shape == want.shape, name
        bad = (g.double() - want).abs() > err + half_step(want, dtype)
        assert not bool(bad.any()), (name, int(bad.sum()))

    near("x", s * D, abs(s) * eD + U * (s * D).abs(), c["X"].dtype)
    names = {"x"}
    if kw.get("weight") is not None:
        near("weight", (dy * ref.n).sum(0), (k + 5) * U * (dy.abs() * ref.N).sum(0), torch.float32)
        names.add("weight")
    if kw.get("bias") is not None:
        near("bias", dy.sum(0), k * U * dy.abs().sum(0), torch.float32)
        names.add("bias")
    if b is not None:
        names.add("b")
        post, gate = kw.get("post_weight"), kw.get("gate")
        p, ps, q, eq = b, b.abs(), D, eD
        if post is not None:
            rb = Ref(b, layer, eps)
            p, ps = rb.n * post, rb.N * post.abs()
        if gate is not None:
            each, err = D * p, eD * ps + 8 * U * D.abs() * ps
            if gate.dim() == 2:
                near("gate", each, err, c["kw"]["gate"].dtype)
            else:
                near("gate", each.sum(0), (err + k * U * D.abs() * ps).sum(0), torch.float32)
            names.add("gate")
            q, eq = D * gate, eD * gate.abs() + U * (D * gate).abs()
        if post is not None:
            near("post_weight", (q * rb.n).sum(0), (eq * rb.N + (k + 6) * U * q.abs() * rb.N).sum(0), torch.float32)
            names.add("post_weight")
            q, eq = q * post, eq * post.abs() + U * (q * post).abs()
            eq = rb.pass_error(eq) + 16 * U * rb.back_error(q)
            q = rb.back(q)
        near("b", q, eq, c["B"].dtype)
    assert set(got) == names


SHAPES = [(1, 1), (3, 7), (5, 64), (2, 200), (9, 512), (4, 513), (3, 768), (2, 1000), (3, 1024), (7, 1025), (2, 4096),
          (3, 4097), (2, 5120), (2, 8192), (2, 8200), (1, 12288), (2, 16384), (2, 16385), (1, 33000)]
FORMS = [dict(), dict(b="bf16"), dict(b="f32", post=True, gate="channel", scale=0.5),
         dict(b="bf16", post=True, gate="token", layer=True, bias=True), dict(b="bf16", gate="token", scale=-2.0),
         dict(x="f32", b="bf16", gate="channel", layer=True), dict(x="f16", b="f16", t="f16", post=True),
         dict(x="f32", b="f32", t="f32", post=True, gate="token", layer=True, bias=True), dict(x="f32", b="f16", t="f16", layer=True)]


@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_forward_and_backward(n, d, form):
    f = FORMS[form]
    c = case(n, d, seed=n * 7 + d + form, **f)
    h, y = P.residual_norm(c["X"], c["B"], dtype=T[f.get("t", "bf16")], **c["kw"])
    check_forward(c, h, y)
    if not f.get("b"):
        assert h is c["X"]
    check_backward(c, P.residual_norm_backward(c["dY"], c["X"], c["B"], dH=c["dH"], **c["kw"]))


@pytest.mark.parametrize("n,d", [(700, 96), (5000, 40), (17000, 16), (700, 1500), (1300, 5000), (520, 9000), (515, 17000)])
def test_many_tokens(n, d):
    """Parts of more than one row, and more rows than parts of a wave."""
    c = case(n, d, x="f32", b="bf16", post=True, gate="channel", bias=True, layer=d % 3 == 0, seed=d)
    h, y = P.residual_norm(c["X"], c["B"], dtype=torch.bfloat16, **c["kw"])
    check_forward(c, h, y)
    got = P.residual_norm_backward(c["dY"], c["X"], c["B"], **c["kw"])
    check_backward(c, got, dh=False)
    again = P.residual_norm_backward(c["dY"], c["X"], c["B"], **c["kw"])
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("d", [96, 4096, 17000])
def test_strides_and_places(d):
    """Rows off 16 bytes, a gate's rows with a stride, h written over x, one of the outputs alone; what lies between rows stays."""
    c = case(6, d, x="f16", b="f16", t="f16", post=True, layer=True, bias=True, gate="token", seed=d, ld=10)
    wide = torch.zeros(6, d + 13, dtype=torch.float16, device=DEV)
    wide[:, 5: 5 + d] = c["kw"]["gate"]
    c["kw"]["gate"] = wide[:, 5: 5 + d]
    out = torch.full((2, 6, d + 9), 7.0, dtype=torch.float16, device=DEV)
    h, y = out[0, :, 3: 3 + d], out[1, :, 4: 4 + d]
    P.residual_norm(c["X"], c["B"], out=(h, y), **c["kw"])
    check_forward(c, h, y)
    assert bool((out[0, :, :3] == 7).all()) and bool((out[0, :, 3 + d:] == 7).all())
    assert bool((out[1, :, :4] == 7).all()) and bool((out[1, :, 4 + d:] == 7).all())
    check_backward(c, P.residual_norm_backward(c["dY"], c["X"], c["B"], dH=c["dH"], **c["kw"]))
    x = c["X"].clone()
    y2 = torch.empty_like(x)
    P.residual_norm(x, c["B"], out=(x, y2), **c["kw"])
    assert torch.equal(x, h) and torch.equal(y2, y)
    alone = torch.empty_like(x)
    assert P.residual_norm(c["X"], c["B"], out=(alone, None), **c["kw"])[1] is None and torch.equal(alone, h)
    P.residual_norm(c["X"], c["B"], out=(None, alone), **c["kw"])
    assert torch.equal(alone, y)


def test_without_vectors_and_without_tokens():
    c = case(5, 300, b="f32")
    kw = dict(eps=1e-5)
    c["kw"] = dict(weight=None, kind="rms", residual_scale=1.0, **kw)
    h, y = P.residual_norm(c["X"], c["B"], h_dtype=torch.float32, **kw)
    assert h.dtype == torch.float32 and y.dtype == torch.bfloat16
    check_forward(c, h, y)
    check_backward(c, P.residual_norm_backward(c["dY"], c["X"], c["B"], dH=c["dH"], **kw))
    w = torch.ones(300, device=DEV)
    h, y = P.residual_norm(c["X"][:0], weight=w)
    assert h.shape == y.shape == (0, 300)
    got = P.residual_norm_backward(c["dY"][:0], c["X"][:0], c["B"][:0], weight=w, gate=w, post_weight=w, bias=w)
    assert all(got[k].shape == (300,) and not got[k].any() for k in ("weight", "gate", "post_weight", "bias"))


@pytest.mark.parametrize("d", [600, 5000, 20000])
def test_values_far_out(d):
    """Squares that leave float32's range, rows of zeros, a mean far above its deviation; rows with an infinity or NaN
    spoil their own outputs alone."""
    c = case(6, d, x="f32", b="f32", t="f32", post=True, layer=True, seed=1)
    c["X"][0] *= 1e25
    c["B"][1] *= 1e-25
    c["B"][2] = c["B"][2] * 0.5 + 1000.0
    c["X"][3] = 0
    c["B"][3] = 0
    h, y = P.residual_norm(c["X"], c["B"], **c["kw"])
    check_forward(c, h, y)
    clean = [t[[0, 1, 3]].clone() for t in (h, y)]
    c["X"][2, d // 2] = float("inf")
    c["X"][4, 0] = float("nan")
    c["B"][5, d - 1] = float("-inf")
    h, y = P.residual_norm(c["X"], c["B"], **c["kw"])
    assert all(torch.equal(t[[0, 1, 3]], w) for t, w in zip((h, y), clean))
    assert not y[[2, 4, 5]].isfinite().any()
    got = P.residual_norm_backward(c["dY"], c["X"], c["B"], **c["kw"])
    assert got["x"][[0, 1, 3]].isfinite().all() and not got["x"][[2, 4]].isfinite().any()


def test_gradient_against_differences():
    """The gradients' products with a direction against the change of the formula's sum along it, in float64."""
    c = case(4, 50, x="f32", b="f32", t="f32", post=True, gate="channel", layer=True, bias=True, scale=0.7)
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    names = ("weight", "bias", "post_weight", "gate")
    at = [c["X"].double(), c["B"].double()] + [c["kw"][k].double() for k in names]
    way = [torch.randn(t.shape, generator=g, device=DEV, dtype=torch.float64) for t in at]

    def value(s):
        x, b, w, bias, post, gate = [a + s * v for a, v in zip(at, way)]
        h = 0.7 * x + gate * (Ref(b, True, 1e-5).n * post)
        return ((Ref(h, True, 1e-5).n * w + bias) * c["dY"].double()).sum() + (h * c["dH"].double()).sum()

    h, _ = P.residual_norm(c["X"], c["B"], **c["kw"])
    got = P.residual_norm_backward(c["dY"], h, c["B"], dH=c["dH"], **c["kw"])
    slope = sum((got[k].double() * v).sum() for k, v in zip(("x", "b") + names, way))
    step = 1e-5
    want = (value(step) - value(-step)) / (2 * step)
    size = sum((got[k].double() * v).abs().sum() for k, v in zip(("x", "b") + names, way))
    # float32 gradients of a rounded h (some 50 roundings of each term at most), differences to step^2
    assert abs(float(slope - want)) <= float(size) * (50 * U + 1e-8)


def test_other_stream_and_graph():
    """Calls on a stream of their own, captured and replayed with new values, workspaces given and made."""
    c = case(300, 2000, x="f32", b="bf16", post=True, gate="channel")
    ws = torch.empty(P.load().gptq_residual_norm_backward_workspace(300, 2000), dtype=torch.uint8, device=DEV)

    def both(**kw):
        h, y = P.residual_norm(c["X"], c["B"], dtype=torch.bfloat16, **c["kw"], **kw)
        return [h, y, *P.residual_norm_backward(c["dY"], h, c["B"], dH=c["dH"], workspace=ws, **c["kw"], **kw).values()]

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both()
    for turn in range(3):
        c["X"].mul_(-1.5)
        c["dY"].add_(0.25)
        g.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(kept, both()))


@pytest.mark.parametrize("n,d", [(3, 5), (40, 89), (700, 1003), (600, 5117), (300, 8191), (600, 9001), (600, 16386)])
@pytest.mark.parametrize("post", [False, True])
def test_stream_in_place_of_any_width(n, d, post):
    """h over X, whose last values two lanes read."""
    c = case(n, d, b="bf16", post=post, seed=d)
    h, y = P.residual_norm(c["X"], c["B"], **c["kw"])
    X = c["X"].clone()
    y2 = torch.empty_like(y)
    P.residual_norm(X, c["B"], out=(X, y2), **c["kw"])
    assert torch.equal(X, h) and torch.equal(y2, y)
    X = c["X"].clone()
    P.residual_norm(X, c["B"], out=(X, None), **c["kw"])
    assert torch.equal(X, h)
