"""Gated products with e2m1 weights and the gradients of products, against float64 (needs an MI355X).

Bounds, with u = 2^-24.  Products: as in test_gpu_mx.py, a sum of K products is off by at most
(4 K + 64) 2^-23 sum |x w| (no product is rounded; more additions where parts of a sum are joined are inside that).

Activations in float32: with at most sixteen roundings of a value, and what the argument of an exponential
or of erfc adds to it (its rounding times the function's relative slope: v^2 for GELU, the argument itself for
GELU_TANH), act(v) is off by at most R(v) u |act(v)|, R = 16 + 4 v^2 + 8 (|v| + 0.05 |v|^3), and its slope by at
most 64 u (1 + |v|); |act'| < 1.2.

Gradients: D = dG or dU of 16-bit types is rounded for the matrix instructions: bfloat16 to itself (half a step: 2^-8
of the value), float16 to 11 bits (2^-11, or half of float16's smallest number, 2^-25, after the token's largest
has been brought to 2^14: 2^-39 of it); float32 ones are not.  Results of type t are rounded once: half a step.
"""
import math

import pytest
import torch

import post_weight_quantization_accum_amd as P

pytestmark = pytest.mark.gpu

DEV = "cuda"
T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24
SMALL = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def half_step(v, dtype):
    return torch.clamp(v.abs() * (torch.finfo(dtype).eps / 2), min=SMALL[dtype] / 2)


def act64(v, act):
    """From the definitions, without the difference of near numbers that 1 + tanh and 1 + erf are far below 0."""
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return v * 0.5 * torch.erfc(v * -math.sqrt(0.5))
    return v * torch.sigmoid(v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))


def act_error(v, act):
    a = v.abs()
    return (16 + 4 * a ** 2 + 8 * (a + 0.05 * a ** 3)) * U * act64(v, act).abs() + 1e-37


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device=DEV)


def values(pair, cols, fmt="fp4"):
    return P.mx_dequantize(*pair, cols, fmt=fmt).double()


def weights(rnd, rows, cols, scale=None):
    return P.mx_quantize(rnd(rows, cols) * (cols ** -0.5 if scale is None else scale))


def activations(rnd, kind, n, d, off=0):
    """(arguments for the call, float64 values); off: rows that do not start on 16 bytes."""
    x = rnd(n, d + off)
    if kind in T:
        x = x.to(T[kind])[:, off // 2: off // 2 + d]
        return (x,), x.double()
    pair = P.mx_quantize(x, fmt=kind)
    return pair, values(pair, d, kind)


def call(args, kind, gate, up, **kw):
    if kind in T:
        return P.mx_gated(*args, gate, up, **kw)
    return P.mx_gated_quantized(*args, gate, up, x_fmt=kind, **kw)


def sums_error(x, w):
    return (4 * x.shape[1] + 64) * 2.0 ** -23 * (x.abs() @ w.abs().t())


def check(got, x, gate, up, act, pre):
    y, g, u = got if pre else (got, None, None)
    wg, wu = x @ gate.t(), x @ up.t()
    eg, eu = sums_error(x, gate), sums_error(x, up)
    if pre:
        assert bool(((g.double() - wg).abs() <= eg + half_step(wg, g.dtype)).all())
        assert bool(((u.double() - wu).abs() <= eu + half_step(wu, u.dtype)).all())
    a = act64(wg, act)
    ea = 1.2 * eg + act_error(wg, act)
    want = a * wu
    assert y.shape == want.shape
    assert bool(((y.double() - want).abs() <= ea * (wu.abs() + eu) + a.abs() * eu + 2 * U * want.abs() + half_step(want, y.dtype)).all())


SIZES = [(1, 1, 1), (1, 40, 33), (2, 129, 70), (5, 300, 17), (16, 128, 64), (17, 384, 1100), (33, 200, 300), (70, 328, 500),
         (1, 4096, 11008), (13, 1280, 13824), (130, 328, 8300), (600, 512, 2050), (257, 256, 16500), (2048, 640, 1000)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32", "fp8", "fp4"])
@pytest.mark.parametrize("n,d,ff", SIZES)
def test_gated(n, d, ff, kind):
    rnd = gen(n + d + ff)
    gate, up = weights(rnd, ff, d), weights(rnd, ff, d)
    wg, wu = values(gate, d), values(up, d)
    for i, off in enumerate((0, 6)):
        if off and kind not in T:
            continue
        act, pre = ACTS[(n + d + i) % 4], (n + ff + i) % 2 == 0
        args, x = activations(rnd, kind, n, d, off)
        dtype = T[("bf16", "f16", "f32")[(n + i) % 3]]
        got = call(args, kind, gate, up, act=act, pre=pre, dtype=dtype)
        check(got, x, wg, wu, act, pre)
        again = call(args, kind, gate, up, act=act, pre=pre, dtype=dtype)
        assert all(torch.equal(a, b) for a, b in zip(got if pre else [got], again if pre else [again]))


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32", "fp8", "fp4"])
@pytest.mark.parametrize("n,ff", [(1, 100), (20, 1100), (40, 2000), (300, 2050), (140, 8300), (260, 16500)])
def test_products_are_exact_where_they_can_be(n, ff, kind):
    """Small integers times powers of two that differ from block to block: a wrong row, column, block or matrix shows."""
    rnd = gen(ff)
    d = 328
    def ints(rows):
        t = (rnd(rows, d) * 2).round().clamp(-4, 4)
        t[:, ::32] = 4.0
        e = (rnd(rows, -(-d // 32)).abs() * 1.5).floor().clamp(max=2).repeat_interleave(32, 1)[:, :d]
        return t * 2 ** e
    x = ints(n)
    gate, up = P.mx_quantize(ints(ff)), P.mx_quantize(ints(ff))
    args = (x.to(T[kind]),) if kind in T else P.mx_quantize(x, fmt=kind)
    xv = x.double() if kind in T else values(args, d, kind)
    y, g, u = call(args, kind, gate, up, act="relu", pre=True, dtype=torch.float32)
    wg, wu = xv @ values(gate, d).t(), xv @ values(up, d).t()
    assert torch.equal(g.double(), wg) and torch.equal(u.double(), wu)
    assert bool(((y.double() - wg.clamp(min=0) * wu).abs() <= 2 * U * (wg * wu).abs()).all())


def test_gated_odd_values_and_places():
    """Weights of scales that float16 lacks, NaN blocks, infinities and NaN among the activations; outputs with strides."""
    rnd = gen(3)
    n, d, ff = 40, 300, 220
    e = (rnd(ff, 10) * 25).round().clamp(-60, 40).repeat_interleave(32, 1)[:, :d]
    e[::3] = -5
    w = rnd(ff, d).clamp(-1.9, 1.9) * 2.0 ** e
    gate, up = P.mx_quantize(w), weights(rnd, ff, d)
    for kind in ("bf16", "f16", "f32"):
        x = rnd(n, d).to(T[kind])
        check(P.mx_gated(x, gate, up, act="relu", pre=True, dtype=torch.float32), x.double(), values(gate, d), values(up, d),
              "relu", True)
        up[1][7, 1] = 255
        x[3, 5], x[n - 1, d - 1] = float("inf"), float("nan")
        wide = torch.full((3, n, ff + 7), 7.0, device=DEV)
        out = [t[:, 3: 3 + ff] for t in wide]
        P.mx_gated(x, gate, up, act="relu", pre=True, out=out)
        assert bool((wide[..., :3] == 7).all()) and bool((wide[..., 3 + ff:] == 7).all())
        y, g, u = out
        assert u[:, 7].isnan().all() and u[n - 1].isnan().all() and not g[3][values(gate, d)[:, 5] != 0].isfinite().any()
        keep = [t for t in range(n) if t not in (3, n - 1)]
        assert u[keep][:, :7].isfinite().all() and u[keep][:, 8:].isfinite().all()
        up = weights(gen(4), ff, d)


def back_error(D, w):
    return (4 * D.shape[1] + 64) * 2.0 ** -23 * (D.abs() @ w.abs())


def check_back(dx, D, w, extra=0):
    want = D @ w
    bad = (dx.double() - want).abs() > back_error(D, w) + extra + half_step(want, dx.dtype)
    assert dx.shape == want.shape and not bool(bad.any()), int(bad.sum())


BACK = [(1, 1, 1), (1, 40, 33), (2, 129, 70), (5, 17, 300), (16, 64, 128), (24, 4096, 4096), (33, 300, 200), (70, 500, 328),
        (128, 256, 640), (130, 8300, 328), (300, 768, 2050), (600, 2050, 512), (1000, 128, 11000), (2048, 640, 1000), (2100, 2100, 96)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d,out", BACK)
def test_product_gradient(n, d, out, kind):
    rnd = gen(n + d + out)
    pair = weights(rnd, out, d)
    w = values(pair, d)
    for i, off in enumerate((0, 6)):
        (dy,), D = activations(rnd, kind, n, out, off)
        dx = P.mx_matmul_backward(dy, *pair, d, dtype=T[("bf16", "f16", "f32")[(n + i) % 3]])
        check_back(dx, D, w)
        assert torch.equal(dx, P.mx_matmul_backward(dy, *pair, d, dtype=dx.dtype))


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d,out", [(3, 100, 50), (20, 1000, 700), (200, 328, 2050), (700, 640, 328), (2048, 512, 1100)])
def test_product_gradient_is_exact_where_it_can_be(n, d, out, kind):
    rnd = gen(out)
    e = (rnd(out, -(-d // 32)).abs() * 1.5).floor().clamp(max=2).repeat_interleave(32, 1)[:, :d]
    w = (rnd(out, d) * 2).round().clamp(-4, 4)
    w[:, ::32] = 4.0
    pair = P.mx_quantize(w * 2 ** e)
    dy = (rnd(n, out) * 4).round().clamp(-15, 15).to(T[kind])
    dx = P.mx_matmul_backward(dy, *pair, d, dtype=torch.float32)
    assert torch.equal(dx.double(), dy.double() @ values(pair, d))


def test_product_gradient_odd_values_and_places():
    """Scales that float16 lacks, a NaN block, infinities and NaN in a token's gradient, results with a stride, no rows at all."""
    rnd = gen(8)
    n, d, out = 140, 300, 210
    e = (rnd(out, 10) * 25).round().clamp(-60, 40).repeat_interleave(32, 1)[:, :d]
    pair = P.mx_quantize(rnd(out, d).clamp(-1.9, 1.9) * 2.0 ** e)
    for kind in T:
        dy = rnd(n, out).to(T[kind])
        check_back(P.mx_matmul_backward(dy, *pair, d, dtype=torch.float32), dy.double(), values(pair, d))
        codes, scales = (t.clone() for t in pair)
        scales[11, 2] = 255
        dy[3, 5], dy[n - 1, out - 1] = float("inf"), float("nan")
        wide = torch.full((n, d + 9), 7.0, device=DEV, dtype=T[kind])
        dx = wide[:, 4: 4 + d]
        P.mx_matmul_backward(dy, codes, scales, d, out=dx)
        assert bool((wide[:, :4] == 7).all()) and bool((wide[:, 4 + d:] == 7).all())
        assert dx[:, 64:96].isnan().all() and dx[n - 1].isnan().all()
        assert not dx[3, :64][values(pair, d)[5, :64] != 0].isfinite().any()
        keep = torch.tensor([t for t in range(n) if t not in (3, n - 1)], device=DEV)
        if kind != "f16":                                  # float16 sums may pass its range
            assert dx[keep][:, :64].isfinite().all() and dx[keep][:, 96:].isfinite().all()
        empty = P.mx_matmul_backward(dy[:, :0], codes[:0], scales[:0], d)
        assert empty.shape == (n, d) and not empty.any()
        assert P.mx_matmul_backward(dy[:0], codes, scales, d).shape == (0, d)


def rounded_error(eG, eU, dG, dU, kind):
    """With the rounding of dG and dU for the matrix instructions."""
    top = torch.maximum(dG.abs().amax(1), dU.abs().amax(1))[:, None] * 2.0 ** -39
    step, low = (2.0 ** -8, 2.0 ** -134) if kind == "bf16" else (2.0 ** -11, top)
    return eG + dG.abs() * step + low, eU + dU.abs() * step + low


def gated_gradients(dy, g, u, act):
    g = g.double().requires_grad_()
    a = act64(g, act)
    a.backward(dy.double() * u.double())
    return g.grad, dy.double() * a.detach()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d,ff", [(1, 1, 1), (1, 40, 33), (5, 130, 70), (24, 1024, 2000), (33, 300, 200), (130, 328, 1100),
                                    (300, 768, 2050), (1000, 128, 5000), (2048, 640, 500), (600, 2050, 512)])
def test_gated_gradient(n, d, ff, kind):
    rnd = gen(n + d + ff)
    gate, up = weights(rnd, ff, d), weights(rnd, ff, d)
    wg, wu = values(gate, d), values(up, d)
    for i, off in enumerate((0, 6)):
        act = ACTS[(n + d + i) % 4]
        dy, g, u = ((rnd(n, ff + off) * s).to(T[kind])[:, off // 2: off // 2 + ff] for s in (2e-3, 1.5, 1.0))
        dG, dU = gated_gradients(dy, g, u, act)
        dx, gg, gu = P.mx_gated_backward(dy, g, u, gate, up, d, act=act, pre=True)
        v = g.double()
        eG = 64 * U * (dy.double() * u.double()).abs() * (1 + v.abs())
        eU = dy.double().abs() * act_error(v, act) + U * dU.abs()
        assert bool(((gg.double() - dG).abs() <= eG + half_step(dG, gg.dtype)).all())
        assert bool(((gu.double() - dU).abs() <= eU + half_step(dU, gu.dtype)).all())
        if kind != "f32":
            eG, eU = rounded_error(eG, eU, dG, dU, kind)
        check_back(dx, torch.cat((dG, dU), 1), torch.cat((wg, wu)), eG @ wg.abs() + eU @ wu.abs())
        assert torch.equal(dx, P.mx_gated_backward(dy, g, u, gate, up, d, act=act))


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_gated_gradient_ranges(kind):
    """Gradients from the type's smallest to large ones, tokens of zeros, saturated gates, an infinity in one token."""
    rnd = gen(5)
    n, d, ff = 12, 200, 150
    gate, up = weights(rnd, ff, d, 2.0 ** -20), weights(rnd, ff, d)
    dy = rnd(n, ff)
    dy *= (2.0 ** torch.tensor([-14.0, -20, 0, 5, -30, -100, -120, 0, 0, 0, 0, 0], device=DEV))[:, None]
    dy[7] = 0
    dy, g, u = dy.to(T[kind]), (rnd(n, ff) * 20).to(T[kind]), rnd(n, ff).to(T[kind])
    for act in ACTS:
        dG, dU = gated_gradients(dy, g, u, act)
        dx = P.mx_gated_backward(dy, g, u, gate, up, d, act=act, dtype=torch.float32)
        v = g.double()
        eG = 64 * U * (dy.double() * u.double()).abs() * (1 + v.abs()) + 1e-44
        eU = dy.double().abs() * act_error(v, act) + U * dU.abs() + 1e-44
        if kind != "f32":
            eG, eU = rounded_error(eG, eU, dG, dU, kind)
        else:                                              # parts below bfloat16's smallest step
            eG, eU = eG + 2.0 ** -133, eU + 2.0 ** -133
        wg, wu = values(gate, d), values(up, d)
        check_back(dx, torch.cat((dG, dU), 1), torch.cat((wg, wu)), eG @ wg.abs() + eU @ wu.abs() + 1e-44)
        assert not dx[7].any()
        bad = dy.clone()
        bad[2, 3] = float("inf")
        bad[4, 0] = float("nan")
        got = P.mx_gated_backward(bad, g, u, gate, up, d, act=act, dtype=torch.float32)
        rest = [t for t in range(n) if t not in (2, 4)]
        assert torch.equal(got[rest], dx[rest]) and got[4].isnan().all()
        assert (not got[2].isfinite().all()) or not (dG[2, 3] or dU[2, 3])


def test_gradient_against_differences():
    """The gradient's product with a direction against the change of the formula's sum along it, in float64."""
    rnd = gen(11)
    n, d, ff = 6, 96, 80
    gate, up, down = weights(rnd, ff, d), weights(rnd, ff, d), weights(rnd, 50, ff)
    wg, wu, wd = values(gate, d), values(up, d), values(down, ff)
    x, dz = rnd(n, d), rnd(n, 50)
    for act in ("silu", "gelu", "gelu_tanh"):
        y, g, u = P.mx_gated(x, gate, up, act=act, pre=True)
        dx = P.mx_gated_backward(P.mx_matmul_backward(dz, *down, ff), g, u, gate, up, d, act=act)
        way = rnd(n, d).double()
        value = lambda s: ((act64((x.double() + s * way) @ wg.t(), act) * ((x.double() + s * way) @ wu.t())) @ wd.t() * dz.double()).sum()
        want = (value(1e-5) - value(-1e-5)) / 2e-5
        # float32 throughout: some (4 K + 64) roundings of K = 2 ff + d + 50 terms, differences to step^2
        scale = (dx.double() * way).abs().sum() + (dz.double().abs() @ wd.abs() @ (wg.abs() + wu.abs()) * way.abs()).sum()
        assert abs(float((dx.double() * way).sum() - want)) <= float(scale) * (4 * 300 * 2 * U + 1e-8)


def test_streams_graphs_and_workspaces():
    rnd = gen(2)
    n, d, ff = 300, 512, 700
    gate, up = weights(rnd, ff, d), weights(rnd, ff, d)
    x, dy = rnd(n, d).bfloat16(), rnd(n, ff).bfloat16()
    lib = P.load()
    ws = torch.empty(max(1, lib.gptq_mx_gated_backward_workspace(2, n, d, ff)), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(max(1, lib.gptq_mx_matmul_backward_workspace(2, n, d, ff)), dtype=torch.uint8, device=DEV)

    def run(**kw):
        y, g, u = P.mx_gated(x, gate, up, pre=True, **kw)
        return [y, g, u, P.mx_gated_backward(dy, g, u, gate, up, d, workspace=ws, **kw),
                P.mx_matmul_backward(dy, *gate, d, workspace=ws2, **kw)]

    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for turn in range(3):
        x.mul_(-1.25)
        dy.add_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(kept, run()))
    with pytest.raises(P.WorkspaceError):
        P.mx_gated_backward(dy, got[1], got[2], gate, up, d, workspace=ws[:1024])
