"""Norms, gated products and their gradients used together, as a block's feed-forward half and as the sequential
driver use them (needs an MI355X).

Every step is checked against float64 of the tensors it was given, by the bounds stated in test_gpu_norm.py and
test_gpu_gated.py, and products by those of test_gpu_mx.py.
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_accum_amd as P
from post_weight_quantization_accum_amd import sequential as S

import test_gpu_gated as G
import test_gpu_norm as N
from test_gpu_mx import _check as check_product

pytestmark = pytest.mark.gpu

DEV = "cuda"
T = N.T


class FeedForward:
    """norm -> gated product -> product down -> normed, gated by channel, into the stream -> the next block's norm."""

    def __init__(self, seed, d, ff, dtype, act, layer=False, scale=1.0):
        rnd = self.rnd = G.gen(seed)
        self.d, self.ff, self.act, self.dtype = d, ff, act, dtype
        self.gate, self.up, self.down = G.weights(rnd, ff, d), G.weights(rnd, ff, d), G.weights(rnd, d, ff)
        vec = lambda m, s: (m + s * rnd(d)).to(dtype)
        self.norm1 = dict(weight=vec(1, 0.2), kind="layer" if layer else "rms", eps=1e-5)
        self.norm2 = dict(weight=vec(1, 0.2), post_weight=vec(1, 0.2), gate=vec(0, 0.5), kind=self.norm1["kind"], eps=1e-5,
                          residual_scale=scale)
        if layer:
            self.norm1["bias"] = vec(0, 0.1)

    def forward(self, X, **kw):
        h, self.n = P.residual_norm(X, dtype=self.dtype, **self.norm1, **kw)
        self.x = h
        self.y, self.g, self.u = P.mx_gated(self.n, self.gate, self.up, act=self.act, pre=True, **kw)
        self.b = P.mx_matmul(self.y, *self.down, **kw)
        self.h, self.out = P.residual_norm(X, self.b, dtype=self.dtype, **self.norm2, **kw)
        return self.h, self.out

    def backward(self, dh, dout, **kw):
        self.g2 = P.residual_norm_backward(dout, self.h, self.b, dH=dh, **self.norm2, **kw)
        self.db = self.g2["b"].to(self.dtype)
        self.dy = P.mx_matmul_backward(self.db, *self.down, self.ff, **kw)
        self.dn = P.mx_gated_backward(self.dy, self.g, self.u, self.gate, self.up, self.d, act=self.act, **kw)
        self.g1 = P.residual_norm_backward(self.dn, self.x, dH=self.g2["x"], **self.norm1, **kw)
        return [self.g1["x"], self.g1["weight"], self.g2["weight"], self.g2["gate"], self.g2["post_weight"]]


@pytest.mark.parametrize("dtype,act,layer,x,n,d,ff", [("bf16", "silu", False, "f32", 300, 512, 1300), ("f16", "gelu", True, "f16", 1, 640, 900),
                                                       ("f32", "gelu_tanh", False, "f32", 45, 200, 333), ("bf16", "relu", True, "bf16", 1100, 320, 700)])
def test_feed_forward_and_its_gradient(dtype, act, layer, x, n, d, ff):
    f = FeedForward(n, d, ff, T[dtype], act, layer, scale=0.75)
    X = (f.rnd(n, d) * 2).to(T[x])
    dout, dh = (f.rnd(n, d) * 1e-2).to(T[dtype]), (f.rnd(n, d) * 1e-2).to(T[x])
    f.forward(X)
    wg, wu, wd = G.values(f.gate, d), G.values(f.up, d), G.values(f.down, ff)
    one = dict(X=X, B=None, kw=dict(residual_scale=1.0, **f.norm1))
    N.check_forward(one, None, f.n)
    G.check((f.y, f.g, f.u), f.n.double(), wg, wu, act, True)
    check_product(f.b, f.y.double().cpu().numpy(), wd.cpu().numpy())
    two = dict(X=X, B=f.b, kw=f.norm2)
    N.check_forward(two, f.h, f.out)
    got = f.backward(dh, dout)
    two.update(X=f.h, dY=dout, dH=dh)
    N.check_backward(two, f.g2)
    G.check_back(f.dy, f.db.double(), wd)
    dG, dU = G.gated_gradients(f.dy, f.g, f.u, act)
    eG = 64 * G.U * (f.dy.double() * f.u.double()).abs() * (1 + f.g.double().abs())
    eU = f.dy.double().abs() * G.act_error(f.g.double(), act) + G.U * dU.abs()
    if dtype != "f32":
        eG, eU = G.rounded_error(eG, eU, dG, dU, dtype)
    G.check_back(f.dn, torch.cat((dG, dU), 1), torch.cat((wg, wu)), eG @ wg.abs() + eU @ wu.abs())
    N.check_backward(dict(X=X, B=None, dY=f.dn, dH=f.g2["x"], kw=dict(residual_scale=1.0, **f.norm1)), f.g1)
    # and the whole chain by differentiation in float64, to the types' roundings along the way: about 12 of at most 2^-8
    # (0.23 % in the mean), which add like their squares' sum, to 0.8 % and a norm's amplification of it.  The slope of
    # relu is no number near what a rounding changes: it jumps by 1 where G's sign does, for 0.3 % of the products and so
    # for sqrt(0.003) of the result's size; it is taken, as the call does, at the G that the forward call gave.
    v = {k: t.double().requires_grad_() for k, t in (("x", X), ("w1", f.norm1["weight"]), ("w2", f.norm2["weight"]),
                                                     ("gate", f.norm2["gate"]), ("post", f.norm2["post_weight"]))}
    norm = lambda t: torch.nn.functional.layer_norm(t, (d,), eps=1e-5) if layer else t / (t.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    m = norm(v["x"]) * v["w1"] + (f.norm1["bias"].double() if layer else 0)
    a = (m @ wg.t()) * (f.g > 0) if act == "relu" else G.act64(m @ wg.t(), act)
    b = (a * (m @ wu.t())) @ wd.t()
    h = 0.75 * v["x"] + v["gate"] * (norm(b) * v["post"])
    torch.autograd.backward([h, norm(h) * v["w2"]], [dh.double(), dout.double()])
    for t, w in zip(got, v.values()):
        off, size = float((t.double() - w.grad).norm()), float(w.grad.norm())
        assert off <= 0.02 * size


def test_feed_forward_captured_and_on_two_streams():
    """The chain in a graph, replayed with new tokens among eager calls; two chains on streams of their own."""
    f = [FeedForward(i, 384, 1000, torch.bfloat16, "silu") for i in range(2)]
    X = [c.rnd(200 + 70 * i, 384).bfloat16() for i, c in enumerate(f)]
    grads = [[(c.rnd(*x.shape) * 1e-2).bfloat16() for _ in range(2)] for c, x in zip(f, X)]
    run = lambda i, **kw: [*f[i].forward(X[i], **kw), *f[i].backward(*grads[i], **kw)]
    alone = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in f]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[run(i, stream=streams[i]) for i in range(2)] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for turn in got for i in range(2) for a, b in zip(turn[i], alone[i]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(0)
    for turn in range(3):
        X[0].mul_(-1.125)
        grads[0][1].add_(0.01)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, run(0)))


@pytest.mark.parametrize("kind,post,bias,scale,attention,dtype", [("rms", True, False, 1.0, None, "bf16"),
                                                                   ("layer", False, True, 0.5, (4, 2), "f16")])
def test_block_quantized_with_norms(kind, post, bias, scale, attention, dtype):
    """The sequential driver: layers calibrated on what the norms make of the stream, step by step."""
    rng = np.random.default_rng(7)
    n, hidden, ffn, dt = 512, 256, 512, T[dtype]
    kv = hidden if attention is None else hidden // attention[0] * attention[1]
    cfg = P.make_config(bits=4, group_size=128, act_order=False, block=128, damp=0.01)
    arr = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(DEV)
    rows = dict(q=(hidden, hidden), k=(kv, hidden), v=(kv, hidden), out=(hidden, hidden), fc1=(ffn, hidden), fc2=(hidden, ffn))
    vec = lambda: (1 + 0.2 * arr(hidden)).to(dt)
    names = ["norm1", "norm2"] + ["post1", "post2"] * post + ["bias1", "bias2"] * bias
    block = S.Block(**{m: (0.05 * arr(*s)).to(dt) for m, s in rows.items()}, **{m: vec() for m in names})
    X = (3 * arr(n, hidden)).to(dt)
    norms = S.Norms(kind, 1e-5, scale)
    att = None if attention is None else S.Attention(*attention)
    res, inputs, out = S.quantize_block(block, X, cfg, norms=norms, attention=att)
    kw = dict(kind=kind, eps=1e-5, residual_scale=scale)
    N.check_forward(dict(X=X, B=None, kw=dict(weight=block.norm1, bias=block.bias1, **{**kw, "residual_scale": 1.0})), None, inputs["q"])
    assert inputs["q"] is inputs["k"] is inputs["v"] and torch.equal(
        S._quantize_shared({"v": block.v}, inputs["v"], cfg, None)["v"]["codes"], res["v"]["codes"])
    if att is None:
        assert torch.equal(inputs["out"], S._product(inputs["q"], res["v"], cfg, None).to(dt))
    b1 = S._product(inputs["out"], res["out"], cfg, None)
    first = dict(X=X, B=b1, kw=dict(weight=block.norm2, bias=block.bias2, post_weight=block.post1, **kw))
    N.check_forward(first, None, inputs["fc1"])
    h1 = P.residual_norm(X, b1, post_weight=block.post1, h_dtype=torch.float32, **kw)[0]
    b2 = S._product(inputs["fc2"], res["fc2"], cfg, None)
    N.check_forward(dict(X=h1, B=b2, kw=dict(post_weight=block.post2, **kw)), out, None)
    stack, last = S.quantize_stack([block, block], X, cfg, norms=norms, attention=att)
    assert torch.equal(stack[0][1]["fc2"], inputs["fc2"]) and torch.equal(last, S.quantize_block(block, out, cfg, norms=norms, attention=att)[2])
