"""Gradients of gated products through weights whose scales float16 lacks (needs an MI355X).

Bounds: as in test_gpu_gated.py; parts of a gradient below bfloat16's smallest step are off by 2^-133 at most.
"""
import pytest
import torch

import post_weight_quantization_accum_amd as P

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
