"""Refusals of the norms around a block (CPU: no call here reaches a launch)."""
import ctypes

import pytest
import torch

import post_weight_quantization_accum_amd as P
from post_weight_quantization_accum_amd import _lib

FAKE = 0x1000          # never dereferenced
BAD = _lib.ERR_INVALID_ARG


def _norm(kind=0, eps=1e-6, scale=1.0, dt=0, w=FAKE, bias=None, post=None, gate=None, ld=0):
    return _lib.Norm(kind, eps, scale, dt, w, bias, post, gate, ld)


def _forward(c=None, n=4, d=64, X=FAKE, xt=0, ldx=64, B=FAKE, bt=0, ldb=64, H=FAKE, ht=0, ldh=64, Y=FAKE, yt=0, ldy=64):
    return P.load().gptq_residual_norm(None if c == 0 else ctypes.byref(c or _norm()), n, d, X, xt, ldx, B, bt, ldb, H, ht, ldh,
                                       Y, yt, ldy, None)


def _backward(c=None, n=4, d=64, dY=FAKE, yt=0, ldy=64, H=FAKE, ht=0, ldh=64, B=FAKE, bt=0, ldb=64, dH=None, lddh=64, dX=FAKE,
              lddx=64, dB=FAKE, lddb=64, dw=None, dbias=None, dpost=None, dgate=None, ldg=64, ws=None, nws=0):
    return P.load().gptq_residual_norm_backward(ctypes.byref(c or _norm()), n, d, dY, yt, ldy, H, ht, ldh, B, bt, ldb, dH, lddh,
                                                dX, lddx, dB, lddb, dw, dbias, dpost, dgate, ldg, ws, nws, None)


def test_forward_refusals():
    assert _forward(c=0) == BAD
    for kw in (dict(kind=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(dt=3), dict(w=FAKE + 2), dict(gate=FAKE, ld=63), dict(ld=64),
               dict(dt=1, bias=FAKE + 1), dict(gate=FAKE, ld=-64)):
        assert _forward(_norm(**kw)) == BAD, kw
    for kw in (dict(n=-1), dict(n=(1 << 20) + 1), dict(d=0), dict(d=(1 << 20) + 1), dict(xt=3), dict(bt=-1), dict(ht=9), dict(yt=4),
               dict(ldx=63), dict(ldb=63), dict(ldh=63), dict(ldy=0), dict(X=None), dict(X=FAKE + 1), dict(B=FAKE + 2),
               dict(H=FAKE + 2), dict(Y=FAKE + 1)):
        assert _forward(**kw) == BAD, kw
    assert _forward(_norm(post=FAKE), B=None) == BAD and _forward(_norm(gate=FAKE), B=None) == BAD
    assert _forward(n=0) == _lib.OK and _forward(n=0, X=None, H=None) == _lib.OK and _forward(H=None, Y=None) == _lib.OK


def test_backward_refusals():
    for kw in (dict(n=-1), dict(d=0), dict(yt=3), dict(ht=3), dict(bt=3), dict(ldy=63), dict(ldh=63), dict(ldb=63),
               dict(dH=FAKE, lddh=63), dict(lddx=63), dict(lddb=63), dict(dY=None), dict(H=None), dict(dX=FAKE + 2),
               dict(dB=FAKE + 1), dict(dH=FAKE + 2), dict(dgate=FAKE), dict(dpost=FAKE), dict(dw=FAKE + 2)):
        assert _backward(**kw) == BAD, kw
    assert _backward(_norm(gate=FAKE, ld=64), dgate=FAKE, ldg=63) == BAD
    assert _backward(_norm(gate=FAKE, ld=64), B=None) == _backward(_norm(post=FAKE), B=None) == BAD
    need = P.load().gptq_residual_norm_backward_workspace(4, 64)
    assert need >= 4 * 4 * 64 * 4
    for kw in (dict(dw=FAKE), dict(dbias=FAKE)):
        assert _backward(**kw) == _backward(ws=FAKE, nws=need - 1, **kw) == _backward(ws=FAKE + 8, nws=need, **kw) == \
            _lib.ERR_WORKSPACE
    assert _backward(_norm(gate=FAKE), dgate=FAKE) == _lib.ERR_WORKSPACE
    assert _backward(n=0) == _lib.OK
    ws = P.load().gptq_residual_norm_backward_workspace
    assert ws(0, 64) == ws(4, 0) == ws(-1, 64) == ws(4, (1 << 20) + 1) == 0


def test_binding_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="GPU"):
        P.residual_norm(x, weight=w)
    with pytest.raises(ValueError, match="GPU"):
        P.residual_norm_backward(x, x, weight=w)
    from post_weight_quantization_accum_amd.norm import _norm as make
    for kw, what in ((dict(kind="batch"), "kind"), (dict(eps=-1.0), "eps"), (dict(residual_scale=float("inf")), "finite"),
                     (dict(weight=torch.zeros(7)), "weight"), (dict(bias=torch.zeros(4, 8)), "bias"),
                     (dict(gate=torch.zeros(3, 8)), "gate"), (dict(gate=torch.zeros(8).expand(4, 8)), "gate"),
                     (dict(post_weight=torch.zeros(16)[::2]), "post_weight")):
        args = dict(kind="rms", eps=1e-6, residual_scale=1.0, weight=None, bias=None, post_weight=None, gate=None)
        with pytest.raises(ValueError, match=what):
            make(4, 8, **{**args, **kw})
    args.update(weight=w, bias=w.bfloat16())
    with pytest.raises(TypeError, match="one dtype"):
        make(4, 8, **args)
    args.update(weight=w.double(), bias=None)
    with pytest.raises(TypeError, match="float64"):
        make(4, 8, **args)
