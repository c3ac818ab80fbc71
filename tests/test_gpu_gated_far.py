"""Gradients of gated products through weights whose scales float16 lacks (needs an MI355X).

Bounds: as in test_gpu_gated.py; parts of a gradient below bfloat16's smallest step are off by 2^-133 at most.
"""
import pytest
import torch

import post_weight_quantization_accum_amd as P

import test_gated_refusals as R
import test_gpu_gated as G

pytestmark = pytest.mark.gpu

DEV, T, U = G.DEV, G.T, G.U


def check(dy, g, u, gate, up, d, act, kind):
    """dX in float32 against float64."""
    dG, dU = G.gated_gradients(dy, g, u, act)
    dx = P.mx_gated_backward(dy, g, u, gate, up, d, act=act, dtype=torch.float32)
    assert bool(dx.isfinite().all())
    v = g.double()
    eG = 64 * U * (dy.double() * u.double()).abs() * (1 + v.abs()) + 2.0 ** -133
    eU = dy.double().abs() * G.act_error(v, act) + U * dU.abs() + 2.0 ** -133
    if kind != "f32":
        eG, eU = G.rounded_error(eG, eU, dG, dU, kind)
    wg, wu = G.values(gate, d), G.values(up, d)
    G.check_back(dx, torch.cat((dG, dU), 1), torch.cat((wg, wu)), eG @ wg.abs() + eU @ wu.abs())


@pytest.mark.parametrize("kind", list(T))
@pytest.mark.parametrize("n,d,ff", [(12, 200, 150), (70, 300, 700)])
def test_large_weights_and_small_gradients(n, d, ff, kind):
    """Weights of 2^114 beside gradients of 2^-24: results of 2^90, far inside float32."""
    rnd = G.gen(n)
    gate, up = G.weights(rnd, ff, d, 2.0 ** 114), G.weights(rnd, ff, d, 2.0 ** 112)
    dy = rnd(n, ff) * (2.0 ** torch.tensor([-12.0, -20, -8, -24], device=DEV))[torch.arange(n, device=DEV) % 4, None]
    dy, g, u = dy.to(T[kind]), rnd(n, ff).to(T[kind]), rnd(n, ff).to(T[kind])
    check(dy, g, u, gate, up, d, "silu", kind)


def far(rnd, rows, cols):
    """Weights whose blocks' scales go from 2^-60 to 2^40: most are not float16's."""
    e = (rnd(rows, -(-cols // 32)) * 20).round().clamp(-60, 40).repeat_interleave(32, 1)[:, :cols]
    return P.mx_quantize(rnd(rows, cols).clamp(-1.9, 1.9) * 2.0 ** e)


def near(rnd, rows, cols):
    return G.weights(rnd, rows, cols)


# (tokens, columns, d_ff): every tile, with one part and with several
PLANS = [(20, 40000, 60), (20, 600, 700), (200, 20000, 60), (1000, 130, 8000), (400, 20000, 60), (130, 2050, 8000), (700, 20000, 60),
         (200, 10000, 8000)]


@pytest.mark.parametrize("kind", list(T))
def test_far_weights_in_one_matrix_of_two(kind):
    """Every tile, one part and several: which matrix and which rows a second pass takes shows, since the other's are near."""
    seen = set()
    for n, d, ff in PLANS:
        tokens, parts = R.plan(R.KINDS[kind][0], 2, n, d, ff)[1]
        seen.add((tokens, parts > 1))
        rnd = G.gen(n + d)
        dy, g, u = ((rnd(n, ff) * s).to(T[kind]) for s in (2e-3, 1.5, 1.0))
        for a, b in ((far, near), (near, far), (far, far)):
            check(dy, g, u, a(rnd, ff, d), b(rnd, ff, d), d, "silu", kind)
    assert seen == {(t, p) for t in (64, 128, 192, 256) for p in (False, True)}


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_far_weights_in_one_matrix_of_a_product(kind):
    """The same forward, at sizes that reach each kernel."""
    for aligned in (1, 0):
        for k, (n, ff) in R.SIZES[kind, aligned].items():
            rnd = G.gen(k + ff)
            d = 328 + (not aligned)
            assert R.kernel(kind, n, d, ff, aligned) == k
            (x,), xv = G.activations(rnd, kind, n, d, 0 if aligned else 6)
            for a, b in ((far, near), (near, far)):
                gate, up = a(rnd, ff, d), b(rnd, ff, d)
                G.check(P.mx_gated(x, gate, up, act="relu", pre=True, dtype=torch.float32), xv, G.values(gate, d), G.values(up, d), "relu", True)
