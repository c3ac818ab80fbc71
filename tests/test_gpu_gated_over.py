"""Gradients of a gated product's two products, written over those (needs an MI355X)."""
import pytest
import torch

import post_weight_quantization_accum_amd as P

import test_gpu_gated as G

pytestmark = pytest.mark.gpu

DEV, T = G.DEV, G.T


@pytest.mark.parametrize("kind", list(T))
@pytest.mark.parametrize("ff", [70, 4096, 8200, 16384, 16392, 20001])
def test_written_over_the_products(ff, kind):
    """dG where G lies and dU where U does: the same bits as apart."""
    rnd = G.gen(ff)
    n, d = 5, 200
    gate, up = G.weights(rnd, ff, d), G.weights(rnd, ff, d)
    dy, g, u = ((rnd(n, ff + 3)).to(T[kind])[:, :ff] for _ in range(3))
    want = P.mx_gated_backward(dy, g, u, gate, up, d, pre=True)
    lib, code = P.load(), {"f32": 0, "f16": 1, "bf16": 2}[kind]
    need = lib.gptq_mx_gated_backward_workspace(code, n, d, ff)
    ws, dx = torch.empty(need, dtype=torch.uint8, device=DEV), torch.empty(n, d, dtype=T[kind], device=DEV)
    st = lib.gptq_mx_gated_backward(dy.data_ptr(), code, n, ff, ff + 3, g.data_ptr(), u.data_ptr(), ff + 3, gate[0].data_ptr(),
                                    gate[1].data_ptr(), up[0].data_ptr(), up[1].data_ptr(), d, 0, dx.data_ptr(), code, d,
                                    g.data_ptr(), u.data_ptr(), ff + 3, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for a, b in zip((dx, g, u), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", list(T))
@pytest.mark.parametrize("n,d,ff", [(1, 40, 33), (20, 600, 700), (24, 4096, 2000), (20, 140000, 70), (200, 300, 4100), (700, 2050, 300)])
def test_workspaces_are_as_large_as_they_say(n, d, ff, kind):
    """Nothing behind the bytes that the size's entry names is written, and nothing in them is read before it is."""
    rnd = G.gen(n + d)
    gate, up = G.weights(rnd, ff, d), G.weights(rnd, ff, d)
    dy, g, u = (rnd(n, ff).to(T[kind]) for _ in range(3))
    lib, code = P.load(), {"f32": 0, "f16": 1, "bf16": 2}[kind]
    for need, call in ((lib.gptq_mx_gated_backward_workspace(code, n, d, ff), lambda **kw: P.mx_gated_backward(dy, g, u, gate, up, d, **kw)),
                       (lib.gptq_mx_matmul_backward_workspace(code, n, d, ff), lambda **kw: P.mx_matmul_backward(dy, *gate, d, **kw))):
        ws = torch.full((need + (1 << 20),), 255, dtype=torch.uint8, device=DEV)      # NaN in every type
        assert torch.equal(call(workspace=ws), call())
        assert bool((ws[need:] == 255).all())
