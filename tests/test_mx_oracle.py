"""The microscaled oracle's pins and the refusals of the microscaled and cache
entry points (CPU: no call here reaches a launch)."""
import ctypes

import numpy as np
import pytest
import torch

import post_weight_quantization_accum_amd as P
from oracle import mx_oracle as M
from post_weight_quantization_accum_amd import _lib

FAKE = ctypes.c_void_p(0x1000)      # never dereferenced: validation fails first
BAD = _lib.ERR_INVALID_ARG


def test_grids():
    assert M.GRID["fp4"].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    g = M.GRID["fp8"]
    assert len(g) == 127 and g[-1] == 448 and g[1] == 2.0 ** -9 and g[8] == 2.0 ** -6 and (np.diff(g) > 0).all()


def test_hand_worked_blocks():
    # largest 6: floor(log2 6) = 2, so e = 0; ties go to the even code
    row = np.zeros((1, 128))
    row[0, :8] = [6, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    codes, scales = M.mx_quantize(row, "fp4")
    assert scales[0].tolist() == [127, 0, 0, 0]
    assert M.mx_values(codes, scales, "fp4")[0, :8].tolist() == [6, 0, 1, 1, 2, 2, 4, 4]
    assert codes[0, 0] >> 4 == 8            # -0.25 rounds to -0
    # largest 7.9 has the same scale and clamps to 6; 3 halves of everything halve
    row[0, 0] = 7.9
    assert M.mx_values(*M.mx_quantize(row, "fp4"), "fp4")[0, 0] == 6
    assert M.mx_values(*M.mx_quantize(row / 2, "fp4"), "fp4")[0, 0] == 3
    # e4m3: 500 has e = 0 and clamps to 448; 1 / 3 rounds to 0.34375
    row[0, :2] = [500, 1 / 3]
    v = M.mx_values(*M.mx_quantize(row, "fp8"), "fp8")[0]
    assert v[0] == 448 and v[1] == 0.34375
    # a NaN or infinity takes its block
    row[0, 40] = np.inf
    v = M.mx_values(*M.mx_quantize(row, "fp8"), "fp8")[0]
    assert np.isnan(v[32:64]).all() and v[0] == 448 and (v[64:] == 0).all()


def test_scale_stays_at_its_least():
    tiny = np.full((1, 32), 2.0 ** -140)
    codes, scales = M.mx_quantize(tiny, "fp4")
    assert scales[0, 0] == 0 and (M.mx_values(codes, scales, "fp4") == 0).all()


def test_attention_rows():
    rng = np.random.default_rng(0)
    Q, K, V = rng.standard_normal((3, 2, 4)), rng.standard_normal((5, 1, 4)), rng.standard_normal((5, 1, 4))
    o, _, _ = M.attention(Q, K, V, 1, 0.5)       # tokens at -2, -1, 0: two of them see nothing
    assert (o[:2] == 0).all() and np.allclose(o[2], V[0])
    o, _, _ = M.attention(Q, K, V, 5, 0.5, window=1)
    assert np.allclose(o, V[2:5])                # a window of one: the token's own value
    s = 0.5 * K[:, 0] @ Q[2, 1]
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(M.attention(Q, K, V, 5, 0.5)[0][2, 1], w @ V[:, 0])


def test_row_sizes():
    lib = P.load()
    assert [lib.gptq_mx_codes_per_row(n, _lib.MX_FP4) for n in (0, 1, 128, 129)] == [0, 64, 64, 128]
    assert [lib.gptq_mx_codes_per_row(n, _lib.MX_FP8) for n in (0, 1, 128, 129)] == [0, 128, 128, 256]
    assert [lib.gptq_mx_scales_per_row(n) for n in (0, 1, 128, 129)] == [0, 4, 4, 8]
    assert lib.gptq_mx_codes_per_row(-1, _lib.MX_FP4) == lib.gptq_mx_codes_per_row(4, 0) == -1
    assert lib.gptq_mx_scales_per_row(-1) == -1


def _quant(**kw):
    a = dict(X=FAKE, dt=2, n=4, d=64, ld=64, f=2, c=FAKE, s=FAKE)
    a.update(kw)
    return P.load().gptq_mx_quantize(a["X"], a["dt"], a["n"], a["d"], a["ld"], a["f"], a["c"], a["s"], None)


def _dequant(**kw):
    a = dict(c=FAKE, s=FAKE, f=2, n=4, d=64, Y=FAKE, dt=2, ld=64)
    a.update(kw)
    return P.load().gptq_mx_dequantize(a["c"], a["s"], a["f"], a["n"], a["d"], a["Y"], a["dt"], a["ld"], None)


@pytest.mark.parametrize("call", [_quant, _dequant])
def test_quantize_refusals(call):
    for kw in (dict(dt=7), dict(f=0), dict(f=3), dict(n=-1), dict(d=0), dict(ld=63), dict(n=(1 << 20) + 1),
               dict(d=(1 << 20) + 1, ld=1 << 21), dict(c=None), dict(s=None), dict(c=ctypes.c_void_p(0x1008)),
               dict(s=ctypes.c_void_p(0x1002))):
        assert call(**kw) == BAD, kw
    assert call(**({"X": ctypes.c_void_p(0x1001)} if call is _quant else {"Y": ctypes.c_void_p(0x1001)})) == BAD
    assert call(n=0) == _lib.OK


def _mm(**kw):
    a = dict(X=FAKE, dt=2, n=4, d=64, ld=64, c=FAKE, s=FAKE, o=32, Y=FAKE, ly=32)
    a.update(kw)
    return P.load().gptq_mx_matmul(a["X"], a["dt"], a["n"], a["d"], a["ld"], a["c"], a["s"], a["o"], a["Y"], a["ly"],
                                   None)


def _mmq(**kw):
    a = dict(X=FAKE, xs=FAKE, f=2, n=4, d=64, c=FAKE, s=FAKE, o=32, Y=FAKE, ly=32)
    a.update(kw)
    return P.load().gptq_mx_matmul_quantized(a["X"], a["xs"], a["f"], a["n"], a["d"], a["c"], a["s"], a["o"], a["Y"],
                                             a["ly"], None)


def test_product_refusals():
    for kw in (dict(n=-1), dict(d=0), dict(o=-1), dict(ly=31), dict(c=None), dict(s=None), dict(Y=None), dict(X=None),
               dict(o=(1 << 20) + 1, ly=1 << 21), dict(c=ctypes.c_void_p(0x1008))):
        assert _mm(**kw) == BAD, kw
        assert _mmq(**kw) == BAD, kw
    assert _mm(dt=5) == _mm(ld=63) == _mm(X=ctypes.c_void_p(0x1001)) == BAD
    assert _mmq(f=0) == _mmq(xs=None) == _mmq(X=ctypes.c_void_p(0x1008)) == BAD
    for call in (_mm, _mmq):
        assert call(n=0) == call(o=0, ly=0) == _lib.OK


def _c(**kw):
    a = dict(k=0x1000, v=0x1000, ks=0x1000, vs=0x1000, n_pages=8, page_size=16, n_kv=2, d=64, f=_lib.MX_FP8, dt=0)
    a.update(kw)
    return _lib.Cache(*a.values())


BAD_CACHES = [dict(k=None), dict(v=0x1008), dict(ks=None), dict(vs=None), dict(n_pages=0), dict(page_size=0),
              dict(n_kv=0), dict(d=0), dict(f=3), dict(f=0, dt=0), dict(n_pages=1 << 31),
              dict(n_pages=1 << 20, page_size=1 << 10, n_kv=2)]


def _write(c, **kw):
    a = dict(K=FAKE, V=FAKE, dt=2, n=4, lk=128, lv=128, s=FAKE)
    a.update(kw)
    return P.load().gptq_cache_write(ctypes.byref(c), *a.values(), None)


def _read(c, **kw):
    a = dict(t=FAKE, mp=4, ns=2, rs=FAKE, n=4, K=FAKE, V=FAKE, dt=2, lk=128, lv=128)
    a.update(kw)
    return P.load().gptq_cache_read(ctypes.byref(c), *a.values(), None)


def _attend(c, **kw):
    a = dict(Q=FAKE, dt=2, n=4, h=8, lq=512, qs=FAKE, kl=FAKE, t=FAKE, mp=4, ns=2, mq=4, sc=1.0, w=0, O=FAKE, lo=512,
             ws=None, nb=0)
    a.update(kw)
    return P.load().gptq_cache_attention(ctypes.byref(c), *a.values(), None)


def test_cache_refusals():
    for call in (_write, _read, _attend):
        for kw in BAD_CACHES:
            assert call(_c(**kw)) == BAD, (call, kw)
        for d in (16, 48, 160, 256):
            assert call(_c(d=d)) == _lib.ERR_UNSUPPORTED
        assert call(_c(), n=0) == _lib.OK
        assert call(_c(), n=-1) == call(_c(), dt=9) == BAD
    for kw in (dict(lk=127), dict(lv=127), dict(K=None), dict(V=ctypes.c_void_p(0x1001)), dict(s=None),
               dict(s=ctypes.c_void_p(0x1004))):
        assert _write(_c(), **kw) == BAD, kw
    half = _c(f=0, dt=_lib.BF16, ks=None, vs=None)
    assert _write(half, dt=_lib.F16) == _write(half, dt=_lib.F32) == _attend(half, dt=_lib.F16) == BAD
    for kw in (dict(lk=127), dict(K=None), dict(rs=None), dict(t=None), dict(mp=-1), dict(ns=-1)):
        assert _read(_c(), **kw) == BAD, kw
    for kw in (dict(h=7), dict(h=0), dict(lq=511), dict(lo=511), dict(Q=None), dict(O=None), dict(qs=None),
               dict(kl=None), dict(t=None), dict(w=-1), dict(w=(1 << 30) + 1), dict(mq=-1), dict(dt=0), dict(sc=0.0), dict(sc=-1.0), dict(sc=float("nan")), dict(sc=float("inf"))):
        assert _attend(_c(), **kw) == BAD, kw
    # a long table makes parts, which need a workspace
    c = _c()
    need = P.load().gptq_cache_attention_workspace(ctypes.byref(c), 4, 8, 2, 4096, 4, 0)
    assert need > 0
    assert _attend(c, mp=4096) == _lib.ERR_WORKSPACE
    assert _attend(c, mp=4096, ws=FAKE, nb=need - 1) == _lib.ERR_WORKSPACE
    assert _attend(c, mp=4096, ws=ctypes.c_void_p(0x1004), nb=need) == _lib.ERR_WORKSPACE
    assert P.load().gptq_cache_attention_workspace(ctypes.byref(_c(d=48)), 4, 8, 2, 4096, 4, 0) == 0


def test_python_refuses_cpu_tensors_and_bad_formats():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        P.mx_quantize(x)
    with pytest.raises(ValueError):
        P.mx_quantize(x, fmt="fp6")
    with pytest.raises(ValueError):
        P.mx_matmul(x, x, x)
    with pytest.raises(ValueError):
        P.new_cache(4, 16, 2, 64, fmt="int8", device="cpu")
    with pytest.raises(ValueError):
        P.new_cache(4, 16, 2, 40, device="cpu")
    c = P.new_cache(4, 16, 2, 64, fmt="fp4", device="cpu")
    assert (c.page_size, c.n_kv_heads, c.head_dim) == (16, 2, 64)
    with pytest.raises(ValueError):
        P.cache_write(c, x, x, x)
    c.k = c.k[..., :16]
    with pytest.raises(TypeError):
        P.cache_write(c, x, x, x)


def test_sequential_attention_refusals():
    """Shapes that do not fit are refused before any work on the GPU."""
    from post_weight_quantization_accum_amd import sequential as S
    w = lambda r: torch.zeros(r, 256)
    X = torch.zeros(10, 256, dtype=torch.bfloat16)
    block = S.Block(w(256), w(128), w(128), w(256), w(512), torch.zeros(256, 512))
    for bad in (S.Attention(4, 2, [5, 4]), S.Attention(4, 2, [11, -1]), S.Attention(3, 3), S.Attention(4, 3),
                S.Attention(4), S.Attention(16, 8), S.Attention(0), S.Attention(4, 2, page_size=0),
                S.Attention(4, 2, window=-1)):
        with pytest.raises(ValueError):
            S.quantize_block(block, X, None, attention=bad)
