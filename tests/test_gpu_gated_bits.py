"""How many bits of a gated product's gradients reach the result (needs an MI355X).

dG and dU are rounded for the matrix instructions: of bfloat16 to 11 bits, of float16 to 22 (two float16 values), both
after the token's largest has been brought to 2^14 .. 2^15, so that what float16 loses below its smallest number is
2^-25 there and 2^-39 of the largest at most; of float32 not at all.  That is at least three bits more than the type
of the inputs has.  Sums of K products: as in test_gpu_gated.py.
"""
import pytest
import torch

import post_weight_quantization_accum_amd as P

import test_gpu_gated as G

pytestmark = pytest.mark.gpu

DEV, T, U = G.DEV, G.T, G.U
STEP = {"bf16": 2.0 ** -11, "f16": 2.0 ** -22, "f32": 0.0}


def arithmetic_error(dy, g, u, dU, act):
    """Of dG and dU as the kernels compute them in float32."""
    v = g.double()
    return (64 * U * (dy.double() * u.double()).abs() * (1 + v.abs()),
            dy.double().abs() * G.act_error(v, act) + U * dU.abs())


def rounded(kind, dG, dU):
    """What the matrix instructions' operands lose."""
    low = 0.0 if kind == "f32" else torch.maximum(dG.abs().amax(1), dU.abs().amax(1))[:, None] * 2.0 ** -39
    return dG.abs() * STEP[kind] + low, dU.abs() * STEP[kind] + low


@pytest.mark.parametrize("kind", list(T))
@pytest.mark.parametrize("n,d,ff", [(7, 130, 7), (300, 300, 300), (700, 200, 2050), (900, 64, 9000), (1500, 40, 17000)])
def test_each_gradient_alone(n, d, ff, kind):
    """One value of dY a token, another place for each: the result is dG gate + dU up of that place, two terms in all."""
    rnd = G.gen(ff)
    gate, up = G.weights(rnd, ff, d), G.weights(rnd, ff, d)
    wg, wu = G.values(gate, d), G.values(up, d)
    at = torch.arange(n, device=DEV) * ff // n
    dy, g, u = torch.zeros(n, ff, device=DEV), rnd(n, ff) * 1.5, rnd(n, ff)
    dy[torch.arange(n, device=DEV), at] = rnd(n)
    dy, g, u = (t.to(T[kind]) for t in (dy, g, u))
    for act in ("silu", "relu"):
        dG, dU = G.gated_gradients(dy, g, u, act)
        dx = P.mx_gated_backward(dy, g, u, gate, up, d, act=act, dtype=torch.float32).double()
        pick = lambda t: t.gather(1, at[:, None])
        dg, du, (eG, eU), (rG, rU) = pick(dG), pick(dU), arithmetic_error(dy, g, u, dU, act), rounded(kind, dG, dU)
        wgt, wut = wg[at], wu[at]
        # two terms of up to three parts: six sums of products that are exact
        terms = (dg * wgt).abs() + (du * wut).abs()
        bound = (pick(eG) + pick(rG)) * wgt.abs() + (pick(eU) + pick(rU)) * wut.abs() + 16 * U * terms + 1e-40
        bad = (dx - (dg * wgt + du * wut)).abs() > bound
        assert not bool(bad.any()), (act, int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("kind", list(T))
@pytest.mark.parametrize("n,d,ff", [(64, 512, 700), (300, 768, 2050), (200, 1024, 8200), (130, 512, 16400)])
def test_error_of_all_together(n, d, ff, kind):
    """The roundings of dG and dU are independent: their errors' norm is that of step * D w at most, where every one is at
    its worst, and float32 sums add 1e-5 of the result (as the products' tests allow them)."""
    rnd = G.gen(n + ff)
    gate, up = G.weights(rnd, ff, d), G.weights(rnd, ff, d)
    w = torch.cat((G.values(gate, d), G.values(up, d)))
    for act in ("silu", "gelu"):
        dy, g, u = ((rnd(n, ff) * s).to(T[kind]) for s in (2e-3, 1.5, 1.0))
        D = torch.cat(G.gated_gradients(dy, g, u, act), 1)
        want = D @ w
        err = P.mx_gated_backward(dy, g, u, gate, up, d, act=act, dtype=torch.float32).double() - want
        allowed = STEP[kind] * float(((D ** 2) @ (w ** 2)).sum().sqrt()) + 1e-5 * float(want.norm())
        assert float(err.norm()) <= allowed, (act, float(err.norm()) / allowed)


@pytest.mark.parametrize("kind", list(T))
@pytest.mark.parametrize("ff", [8192, 8200, 11008, 13824, 16384, 16392, 20001])
def test_wide_rows(ff, kind):
    """Rows that a thread takes once, twice, or that are computed twice; all that the call gives."""
    rnd = G.gen(ff)
    n, d = 6, 150
    gate, up = G.weights(rnd, ff, d), G.weights(rnd, ff, d)
    wg, wu = G.values(gate, d), G.values(up, d)
    for act in G.ACTS:
        # the largest of a token is anywhere, also among what the last thread has
        dy, g, u = ((rnd(n, ff) * s).to(T[kind]) for s in (2e-3, 1.5, 1.0))
        dy[1, ff - 1], dy[2, 0], dy[3, 8191], dy[4] = 50.0, -50.0, 20.0, 0.0
        dG, dU = G.gated_gradients(dy, g, u, act)
        dx, gg, gu = P.mx_gated_backward(dy, g, u, gate, up, d, act=act, pre=True)
        eG, eU = arithmetic_error(dy, g, u, dU, act)
        assert bool(((gg.double() - dG).abs() <= eG + G.half_step(dG, gg.dtype)).all())
        assert bool(((gu.double() - dU).abs() <= eU + G.half_step(dU, gu.dtype)).all())
        rG, rU = rounded(kind, dG, dU)
        G.check_back(dx, torch.cat((dG, dU), 1), torch.cat((wg, wu)), (eG + rG) @ wg.abs() + (eU + rU) @ wu.abs())
        assert not dx[4].any()


def full(t):
    """float32 values of 22 bits, all of them used: times an e2m1 value they are float32 values still."""
    m = 1 + ((t.double() * 1e6).round().long() * 2 + 1).remainder(2 ** 21).double() * 2.0 ** -21
    return (torch.where(t < 0, -m, m) * 2.0 ** (t.double() * 3).round().clamp(-9, 9)).float()


@pytest.mark.parametrize("n,d,out", [(3, 100, 50), (300, 1000, 700), (200, 328, 2050), (700, 640, 328), (2048, 300, 1100), (130, 2050, 8000)])
def test_float32_products_keep_every_bit(n, d, out):
    """One value a token: its three parts' products with a weight sum to a float32 value, in any order."""
    rnd = G.gen(out)
    pair, other = G.weights(rnd, out, d), G.weights(rnd, out, d)
    w, w2 = G.values(pair, d), G.values(other, d)
    at = torch.arange(n, device=DEV) * out // n
    dy = torch.zeros(n, out, device=DEV)
    dy[torch.arange(n, device=DEV), at] = full(rnd(n))
    value = dy.gather(1, at[:, None]).double()
    assert torch.equal(P.mx_matmul_backward(dy, *pair, d).double(), value * w[at])
    # relu at G = 1: dG = dY U, dU = dY; with U = 2^-30 the sum keeps dG's bits only where up's weight is 0, with U = 0 dU's
    ones = torch.ones(n, out, device=DEV)
    got = P.mx_gated_backward(dy, ones, 0 * ones, pair, other, d, act="relu").double()
    assert torch.equal(got, value * w2[at])
    got = P.mx_gated_backward(dy, -0.5 * ones, ones, pair, other, d, act="relu").double()
    assert not got.any()
    got = P.mx_gated_backward(dy, ones, ones * 2.0 ** 60, pair, other, d, act="relu").double()
    far = (w[at] != 0)
    assert torch.equal(got[far], (value * w[at] * 2.0 ** 60)[far]) and torch.equal(got[~far], (value * w2[at])[~far])
    x = torch.zeros(n, d, device=DEV)
    at = torch.arange(n, device=DEV) * d // n
    x[torch.arange(n, device=DEV), at] = full(rnd(n))
    y, g, u = P.mx_gated(x, pair, other, act="relu", pre=True)
    value = x.gather(1, at[:, None]).double()
    assert torch.equal(g.double(), value * w[:, at].t()) and torch.equal(u.double(), value * w2[:, at].t())


@pytest.mark.parametrize("kind", list(T))
@pytest.mark.parametrize("n,d,out", [(24, 4096, 4096), (300, 768, 2050), (600, 2050, 512), (130, 2050, 8000), (1000, 128, 11000), (17, 384, 1100)])
def test_products_are_far_inside_their_bound(n, d, out, kind):
    """An error of every addition at its worst does not happen: 1e-5 of the norm at most in float32, as plain products have."""
    rnd = G.gen(n + out)
    pair, other = G.weights(rnd, out, d), G.weights(rnd, out, d)
    w, w2 = G.values(pair, d), G.values(other, d)
    dy = (rnd(n, out) * torch.exp(rnd(out))).to(T[kind])
    want = dy.double() @ w
    assert float((P.mx_matmul_backward(dy, *pair, d, dtype=torch.float32).double() - want).norm()) <= 1e-5 * float(want.norm())
    x = (rnd(n, d) * torch.exp(rnd(d))).to(T[kind])
    y, g, u = P.mx_gated(x, pair, other, act="silu", pre=True, dtype=torch.float32)
    wg, wu = x.double() @ w.t(), x.double() @ w2.t()
    for got, want in ((g, wg), (u, wu), (y, G.act64(wg, "silu") * wu)):
        assert float((got.double() - want).norm()) <= 1e-5 * float(want.norm())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("n,d,ff", [(1, 300, 2050), (20, 140000, 300), (32, 1000, 700), (33, 1000, 700), (64, 600, 4100), (65, 300, 1000),
                                    (130, 140000, 130)])
def test_second_values_beside_the_tokens(n, d, ff, kind):
    """Few tokens, whose second values may share a tile with them; one part and several, weights near and far from float16."""
    rnd = G.gen(n + ff)
    dy, g, u = ((rnd(n, ff) * s).to(T[kind]) for s in (2e-3, 1.5, 1.0))
    dy[0] *= 2.0 ** -10                                    # another power of two
    dG, dU = G.gated_gradients(dy, g, u, "silu")
    eG, eU = (a + b + 2.0 ** -133 for a, b in zip(arithmetic_error(dy, g, u, dU, "silu"), rounded(kind, dG, dU)))
    for scale in (None, 2.0 ** -30):
        gate, up = G.weights(rnd, ff, d), G.weights(rnd, ff, d, scale)
        w = torch.cat((G.values(gate, d), G.values(up, d)))
        for dtype in (torch.float32, T[kind]):
            wide = torch.full((n, d + 5), 7.0, device=DEV, dtype=dtype)
            dx = wide[:, 2: 2 + d]
            P.mx_gated_backward(dy, g, u, gate, up, d, out=dx)
            G.check_back(dx, torch.cat((dG, dU), 1), w, torch.cat((eG, eU), 1) @ w.abs())
            assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 2 + d:] == 7).all())
