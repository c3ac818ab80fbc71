"""Gated products and gradients: refusals, and which kernel and tile a call takes (CPU: no call here reaches a launch)."""
import ctypes

import pytest
import torch

import post_weight_quantization_accum_amd as P
from post_weight_quantization_accum_amd import _lib
from post_weight_quantization_accum_amd import sequential as S

FAKE = 0x1000          # never dereferenced
BAD = _lib.ERR_INVALID_ARG


def _gated(X=FAKE, xt=2, n=4, d=64, ldx=64, gc=FAKE, gs=FAKE, uc=FAKE, us=FAKE, ff=32, act=0, Y=FAKE, yt=2, ldy=32, G=None, U=None,
           ldgu=32):
    return P.load().gptq_mx_gated(X, xt, n, d, ldx, gc, gs, uc, us, ff, act, Y, yt, ldy, G, U, ldgu, None)


def _quantized(xc=FAKE, xs=FAKE, f=2, n=4, d=64, gc=FAKE, gs=FAKE, uc=FAKE, us=FAKE, ff=32, act=0, Y=FAKE, yt=0, ldy=32, G=None,
               U=None, ldgu=32):
    return P.load().gptq_mx_gated_quantized(xc, xs, f, n, d, gc, gs, uc, us, ff, act, Y, yt, ldy, G, U, ldgu, None)


def _back(dY=FAKE, dt=2, n=4, out=64, ldy=64, c=FAKE, s=FAKE, d=128, dX=FAKE, xt=2, ldx=128, ws=None, nws=0):
    return P.load().gptq_mx_matmul_backward(dY, dt, n, out, ldy, c, s, d, dX, xt, ldx, ws, nws, None)


def _gated_back(dY=FAKE, dt=2, n=4, ff=64, ldy=64, G=FAKE, U=FAKE, ldgu=64, gc=FAKE, gs=FAKE, uc=FAKE, us=FAKE, d=128, act=0, dX=FAKE,
                xt=2, ldx=128, dG=None, dU=None, lddgu=64, ws=None, nws=0):
    return P.load().gptq_mx_gated_backward(dY, dt, n, ff, ldy, G, U, ldgu, gc, gs, uc, us, d, act, dX, xt, ldx, dG, dU, lddgu, ws, nws,
                                           None)


def test_gated_refusals():
    shared = (dict(n=-1), dict(n=(1 << 20) + 1), dict(d=0), dict(ff=-1), dict(ff=(1 << 20) + 1), dict(act=4), dict(act=-1), dict(yt=3),
              dict(ldy=31), dict(gc=None), dict(gs=None), dict(uc=FAKE + 8), dict(us=FAKE + 2), dict(Y=None), dict(Y=FAKE + 1),
              dict(G=FAKE), dict(U=FAKE), dict(G=FAKE, U=FAKE, ldgu=31), dict(G=FAKE, U=FAKE + 1))
    for kw in shared + (dict(xt=3), dict(ldx=63), dict(X=None), dict(X=FAKE + 1)):
        assert _gated(**kw) == BAD, kw
    for kw in shared + (dict(f=0), dict(f=3), dict(xc=None), dict(xc=FAKE + 4), dict(xs=FAKE + 1)):
        assert _quantized(**kw) == BAD, kw
    for call in (_gated, _quantized):
        assert call(n=0) == call(ff=0, ldy=0) == call(n=0, Y=None) == _lib.OK


def test_gradient_refusals():
    for kw in (dict(dt=3), dict(xt=-1), dict(n=-1), dict(d=0), dict(out=-1), dict(ldy=63), dict(ldx=127), dict(dY=None), dict(dX=None),
               dict(c=None), dict(s=FAKE + 1), dict(c=FAKE + 8), dict(dY=FAKE + 1), dict(dX=FAKE + 1)):
        assert _back(**kw) == BAD, kw
    for kw in (dict(dt=3), dict(xt=5), dict(n=-1), dict(d=0), dict(ff=-1), dict(ldy=63), dict(ldgu=63), dict(ldx=127), dict(act=4),
               dict(dY=None), dict(G=None), dict(U=FAKE + 1), dict(gc=None), dict(us=None), dict(dX=None), dict(dG=FAKE),
               dict(dG=FAKE, dU=FAKE, lddgu=63), dict(dG=FAKE, dU=FAKE + 1)):
        assert _gated_back(**kw) == BAD, kw
    lib = P.load()
    need = lib.gptq_mx_matmul_backward_workspace(2, 4, 128, 64)
    assert need > 0
    for kw in (dict(), dict(ws=FAKE, nws=need - 1), dict(ws=FAKE + 8, nws=need)):
        assert _back(**kw) == _lib.ERR_WORKSPACE, kw
    need = lib.gptq_mx_gated_backward_workspace(2, 4, 128, 64)
    assert need >= 4 * 2 * 64 * 2
    for kw in (dict(), dict(ws=FAKE, nws=need - 1), dict(ws=FAKE + 8, nws=need)):
        assert _gated_back(**kw) == _lib.ERR_WORKSPACE, kw
    assert _back(n=0) == _gated_back(n=0) == _lib.OK
    for f in (lib.gptq_mx_matmul_backward_workspace, lib.gptq_mx_gated_backward_workspace):
        assert f(3, 4, 128, 64) == f(2, 0, 128, 64) == f(2, 4, 0, 64) == f(2, 4, 128, 0) == f(2, (1 << 20) + 1, 128, 64) == 0


# kernel -> (tokens, d_ff); columns: 328 where rows are to start on 16 bytes, else 329
FEW = {1: (3, 100), 3: (1, 4200), 10: (1, 8250), 11: (7, 12300)}
HALF = {**FEW, 4: (17, 2100), 5: (4200, 20)}
SIXTEEN = {**HALF, 7: (17, 8250), 8: (18, 16500)}
ODD = {1: (3, 100), 3: (2, 4200), 4: (17, 2100), 5: (18, 4200), 9: (33, 8250)}
SIZES = {("f32", 1): {**FEW, 9: (33, 12300)}, ("f32", 0): {1: (3, 100), 3: (2, 4200), 9: (33, 10950)}, ("f16", 1): SIXTEEN,
         ("bf16", 1): SIXTEEN, ("f16", 0): ODD, ("bf16", 0): ODD, ("fp8", 1): {**HALF, 9: (33, 10950)}, ("fp4", 1): SIXTEEN}
KINDS = {"f32": (_lib.F32, 0), "f16": (_lib.F16, 0), "bf16": (_lib.BF16, 0), "fp8": (0, _lib.MX_FP8), "fp4": (0, _lib.MX_FP4)}


def kernel(kind, n, d, ff, aligned=1):
    return P.load().gptq_mx_gated_kernel(*KINDS[kind], n, d, ff, aligned)


def test_sizes_reach_their_kernels():
    for (kind, aligned), sizes in SIZES.items():
        for k, (n, ff) in sizes.items():
            assert kernel(kind, n, 328 + (not aligned), ff, aligned) == k, (kind, aligned, k)
    # the rule knows no other kernel for the kind, whatever the sizes
    ffs = [*range(8, 600, 16), *range(600, 17000, 150), 1 << 16, 1 << 20]
    for (kind, aligned), sizes in SIZES.items():
        for n in (1, 7, 16, 17, 33, 48, 64, 65, 100, 128, 129, 256, 300, 600, 1024, 2048, 4200, 1 << 14, 1 << 20):
            found = {kernel(kind, n, 4096, f, aligned) for f in ffs}
            assert found <= set(sizes), (kind, aligned, n, found)
    assert kernel("bf16", 0, 128, 16) == kernel("bf16", 1, 0, 16) == kernel("bf16", 1, 128, 0) == -1
    assert P.load().gptq_mx_gated_kernel(7, 0, 1, 128, 16, 1) == P.load().gptq_mx_gated_kernel(0, 3, 1, 128, 16, 1) == -1


def plan(dt, m, n, d, out):
    p = (ctypes.c_int64 * 2)(-1, -1)
    return P.load().gptq_mx_backward_plan(dt, m, n, d, out, p), tuple(p)


def test_plans_of_gradients():
    assert plan(3, 1, 4, 4, 4)[0] == plan(2, 3, 4, 4, 4)[0] == plan(2, 1, 0, 4, 4)[0] == plan(2, 1, 4, 4, (1 << 20) + 1)[0] == BAD
    assert P.load().gptq_mx_backward_plan(2, 1, 4, 4, 4, None) == BAD
    for dt in (0, 1, 2):
        for m in (1, 2):
            for n in (1, 5, 64, 65, 200, 500, 2048, 1 << 20):
                for d in (1, 300, 4096, 11008, 1 << 20):
                    for out in (1, 64, 65, 4096, 1 << 20):
                        st, (tokens, parts) = plan(dt, m, n, d, out)
                        stages = -(-out // 64) * m * (3 if dt == 0 else 1)
                        assert st == _lib.OK and tokens in (64, 128, 192, 256) and 1 <= parts <= stages
                        # parts are for calls whose tiles leave compute units idle: their sums stay bounded
                        tiles = -(-d // 256) * -(-n // tokens)
                        assert parts == 1 or tiles * parts <= 512


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    pair = torch.zeros(32, 64, dtype=torch.uint8), torch.zeros(32, 4, dtype=torch.uint8)
    for call in (lambda: P.mx_gated(x, pair, pair), lambda: P.mx_gated_quantized(*pair, pair, pair),
                 lambda: P.mx_matmul_backward(x[:, :32], *pair, 100), lambda: P.mx_gated_backward(x[:, :32], x[:, :32], x[:, :32], pair, pair, 100)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="act"):
        P.mx_gated(x, pair, pair, act="swish")
    with pytest.raises(ValueError, match="act"):
        P.mx_gated_backward(x, x, x, pair, pair, 100, act="")
    from post_weight_quantization_accum_amd import mx
    with pytest.raises(ValueError, match="shape"):
        mx._weights(pair, (pair[0][:16].clone(), pair[1][:16].clone()))
    with pytest.raises(TypeError, match="out"):
        mx._gated_out(x, 4, 32, None, True, x)
    with pytest.raises(TypeError, match="out"):
        mx._rows_like(x, "out", 4, 63)


def test_driver_refuses_norms_before_any_work():
    w = lambda r, c=256: torch.zeros(r, c)
    v = torch.ones(256)
    args = [w(256) for _ in range(4)] + [w(512), w(256, 512)]
    X = torch.zeros(10, 256)
    for block, norms, what in ((S.Block(*args), S.Norms(), "no norm1"), (S.Block(*args, norm1=v), None, "norm1 and norm2"),
                               (S.Block(*args, norm1=v, norm2=v[:128]), None, "norm2"),
                               (S.Block(*args, norm1=v, norm2=v, post1=v.half()), None, "post1"),
                               (S.Block(*args, norm1=v, norm2=v), S.Norms("batch"), "kind"),
                               (S.Block(*args, norm1=v, norm2=v), S.Norms(eps=-1.0), "eps"),
                               (S.Block(*args, norm1=v, norm2=v), S.Norms(residual_scale=float("nan")), "finite")):
        with pytest.raises(ValueError, match=what):
            S.quantize_block(block, X, None, norms=norms)
