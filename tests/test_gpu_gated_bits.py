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
