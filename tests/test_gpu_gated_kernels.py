"""Each kernel of the gated products and each tile and split of the gradients, at sizes that reach it (needs an MI355X).

test_gated_refusals.py asks the library on the CPU which sizes reach which kernel.
"""
import pytest
import torch

import post_weight_quantization_accum_amd as P

import test_gated_refusals as R
import test_gpu_gated as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,aligned", list(R.SIZES))
def test_gated_kernels(kind, aligned):
    rnd = G.gen(aligned)
    for k, (n, ff) in R.SIZES[kind, aligned].items():
        d = 328 + (not aligned)
        assert R.kernel(kind, n, d, ff, aligned) == k
        gate, up = G.weights(rnd, ff, d), G.weights(rnd, ff, d)
        args, x = G.activations(rnd, kind, n, d, 0 if aligned else 6)
        for pre in (False, True):
            got = G.call(args, kind, gate, up, act="silu", pre=pre, dtype=torch.float32)
            G.check(got, x, G.values(gate, d), G.values(up, d), "silu", pre)


# (tokens, columns, rows of W): every tile, with one part and with several
PLANS = [(20, 1000, 700), (20, 130000, 40), (200, 20000, 40), (500, 40, 8000), (2048, 40, 8000), (400, 20000, 40), (3000, 40, 8000),
         (700, 20000, 40), (2048, 300, 8000), (200, 10000, 8000)]


@pytest.mark.parametrize("kind", list(G.T))
def test_gradient_tiles(kind):
    code, seen = R.KINDS[kind][0], set()
    for n, d, out in PLANS:
        tokens, parts = R.plan(code, 1, n, d, out)[1]
        seen.add((tokens, parts > 1))
        rnd = G.gen(n + d)
        pair = G.weights(rnd, out, d)
        (dy,), D = G.activations(rnd, kind, n, out)
        G.check_back(P.mx_matmul_backward(dy, *pair, d, dtype=torch.float32), D, G.values(pair, d))
    assert seen == {(t, p) for t in (64, 128, 192, 256) for p in (False, True)}
