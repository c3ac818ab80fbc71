"""Microscaled quantisation and products on the GPU against float64 (needs an MI355X).

Quantisation is exact: codes, scales and values equal the oracle's.

Products: every product of a weight and an activation part is exact in
float32, so only additions round.  One output adds fewer than 4 d_in + 64
numbers (at most three parts, one addition per wave or step on top), each
addition being off by at most 2^-23 of a partial sum of at most
A = sum_k |x_k w_k| (a matrix instruction may cut instead of rounding), hence
|Y - exact| <= (4 d_in + 64) 2^-23 A; integer inputs with power-of-two scales
whose sums stay below 2^24 have to come out exactly, which pins the indexing.
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_accum_amd as P
from oracle import mx_oracle as M

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _values(rng, rows, cols, spread=3.0):
    x = rng.standard_normal((rows, cols)) * np.exp(spread * rng.standard_normal((rows, 1)))
    x[rng.random(x.shape) < 0.1] = 0.0
    x[rng.random(x.shape) < 0.05] *= -0.0
    return x


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 128), (7, 333), (64, 1000)])
def test_quantize_equals_the_oracle(rows, cols, dtype, fmt):
    rng = np.random.default_rng(rows * 1000 + cols)
    X = torch.from_numpy(_values(rng, rows, cols)).to(TYPES[dtype])
    want = M.mx_quantize(X.double().numpy(), fmt)
    codes, scales = P.mx_quantize(X.to(DEV), fmt=fmt)
    assert np.array_equal(scales.cpu().numpy(), want[1])
    assert np.array_equal(codes.cpu().numpy(), want[0])
    for back in TYPES.values():
        got = P.mx_dequantize(codes, scales, cols, fmt=fmt, dtype=back).cpu()
        assert torch.equal(got, torch.from_numpy(M.mx_values(*want, fmt, cols)).to(back))


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_quantize_rounds_every_tie_and_clamps(fmt):
    """Every multiple of a sixteenth of the finest step around the grid, in blocks whose largest value fixes the scale."""
    g = M.GRID[fmt]
    mids = (g[1:] + g[:-1]) / 2
    eps = 2.0 ** -12
    v = np.concatenate([mids, mids * (1 + eps), mids * (1 - eps), g, [g[-1] * 1.1]])
    v = np.concatenate([v, -v])
    v = np.pad(v, (0, -len(v) % 31)).reshape(-1, 31)
    for e in (-100, -20, 0, 30, 100):
        x = np.concatenate([np.full((len(v), 1), g[-1] * 1.05), v], 1) * 2.0 ** e
        X = torch.from_numpy(x).float()
        want = M.mx_quantize(X.double().numpy(), fmt)
        codes, scales = P.mx_quantize(X.to(DEV), fmt=fmt)
        assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_quantize_extremes(fmt):
    x = np.zeros((12, 64), dtype=np.float32)
    x[0, :3] = [np.inf, 1, -2]
    x[1, 40] = np.nan
    x[2, 5] = -np.inf
    x[3, :] = 2.0 ** -149 * np.arange(64)
    x[4, :] = 2.0 ** -127 * np.arange(64)
    x[5, :] = 2.0 ** -126 * (np.arange(64) - 30)
    x[6, :] = 3.4e38 * np.linspace(-1, 1, 64)
    x[7, :] = -0.0
    x[8, 0] = 2.0 ** -149
    x[9, :] = 2.0 ** -119 * np.linspace(-1, 1, 64)
    x[10, 0], x[10, 1] = 2.0 ** 127, 2.0 ** 100
    want = M.mx_quantize(x, fmt)
    codes, scales = P.mx_quantize(torch.from_numpy(x).to(DEV), fmt=fmt)
    assert np.array_equal(scales.cpu().numpy(), want[1])
    assert np.array_equal(codes.cpu().numpy(), want[0])
    got = P.mx_dequantize(codes, scales, 64, fmt=fmt).cpu().numpy()
    assert np.array_equal(got, M.mx_values(*want, fmt, 64).astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_dequantize_every_code_and_scale(fmt):
    n = 16 if fmt == "fp4" else 256
    c = np.resize(np.arange(n), (256, 256)).astype(np.uint8)
    codes = (c[:, 0::2] | c[:, 1::2] << 4) if fmt == "fp4" else c
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
    want = M.mx_values(codes, scales, fmt)
    with np.errstate(over="ignore"):
        want = want.astype(np.float32)
    got = P.mx_dequantize(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), 256, fmt=fmt)
    assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)


def test_quantize_strides_and_alignment():
    rng = np.random.default_rng(5)
    base = torch.from_numpy(_values(rng, 9, 403)).to(torch.bfloat16).to(DEV)
    for part in (base[:, 1:300], base[::2, 3:131], base[:, 8:264]):
        want = M.mx_quantize(part.double().cpu().numpy(), "fp4")
        codes, scales = P.mx_quantize(part)
        assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])
        room = torch.full((9, 403), 7.0, device=DEV)
        view = room[: part.shape[0], 5: 5 + part.shape[1]]
        P.mx_dequantize(codes, scales, part.shape[1], out=view)
        assert np.array_equal(view.cpu().numpy(), M.mx_values(*want, "fp4", part.shape[1]))
        view.fill_(7.0)
        assert (room == 7.0).all()


def _weights(rng, d_out, d_in):
    return M.mx_quantize(0.02 * rng.standard_normal((d_out, d_in)), "fp4")


def _check(Y, x, w):
    exact = x @ w.T
    bound = (4 * x.shape[1] + 64) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    err = np.abs(Y.double().cpu().numpy() - exact)
    assert (err <= bound).all(), f"off by {np.max(err / np.maximum(bound, 1e-300)):.3g} of the bound"
    # and far inside it: an error of every addition at its worst does not happen
    assert np.linalg.norm(err) <= 1e-5 * np.linalg.norm(exact)


SHAPES = [(1, 1, 1), (1, 40, 17), (2, 128, 16), (5, 129, 33), (16, 1000, 64), (17, 384, 100), (33, 256, 128),
          (64, 2049, 48), (65, 160, 200), (128, 128, 128), (129, 500, 131), (200, 1111, 300), (300, 64, 257)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_product(n, d_in, d_out, dtype):
    rng = np.random.default_rng(n + d_in + d_out)
    w, ws = _weights(rng, d_out, d_in)
    X = torch.from_numpy(rng.standard_normal((n, d_in)) * np.exp(2 * rng.standard_normal(d_in))).to(TYPES[dtype])
    Y = P.mx_matmul(X.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV))
    _check(Y, X.double().numpy(), M.mx_values(w, ws, "fp4", d_in))


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_product_of_quantized(n, d_in, d_out, fmt):
    rng = np.random.default_rng(n + d_in + d_out)
    w, ws = _weights(rng, d_out, d_in)
    x, xs = M.mx_quantize(rng.standard_normal((n, d_in)) * np.exp(2 * rng.standard_normal(d_in)), fmt)
    t = [torch.from_numpy(a).to(DEV) for a in (x, xs, w, ws)]
    Y = P.mx_matmul_quantized(*t, x_fmt=fmt)
    _check(Y, M.mx_values(x, xs, fmt, d_in), M.mx_values(w, ws, "fp4", d_in))


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32", "fp4", "fp8"])
@pytest.mark.parametrize("n,d_in,d_out", [(1, 999, 50), (13, 1300, 70), (40, 256, 33), (150, 700, 140), (257, 96, 260)])
def test_integers_come_out_exactly(n, d_in, d_out, kind):
    """Weights and activations of small integers and scales that differ from block to block: a wrong column, block or scale shows."""
    rng = np.random.default_rng(d_in)
    w = rng.integers(-4, 5, (d_out, d_in)).astype(np.float64)
    w[:, ::32] = 4.0                                        # every block's scale is 2^0 before the factor
    w *= 2.0 ** np.repeat(rng.integers(0, 3, (d_out, -(-d_in // 32))), 32, 1)[:, :d_in]
    codes, scales = M.mx_quantize(w, "fp4")
    w = M.mx_values(codes, scales, "fp4", d_in)
    x = rng.integers(-4, 5, (n, d_in)).astype(np.float64)
    x[:, ::32] = -4.0
    x *= 2.0 ** np.repeat(rng.integers(0, 3, (n, -(-d_in // 32))), 32, 1)[:, :d_in]
    wt = torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)
    if kind in TYPES:
        Y = P.mx_matmul(torch.from_numpy(x).to(TYPES[kind]).to(DEV), *wt)
    else:
        xc, xs = M.mx_quantize(x, kind)
        x = M.mx_values(xc, xs, kind, d_in)
        Y = P.mx_matmul_quantized(torch.from_numpy(xc).to(DEV), torch.from_numpy(xs).to(DEV), *wt, x_fmt=kind)
    assert np.abs(x) .max() * np.abs(w).max() * d_in < 2 ** 24
    assert np.array_equal(Y.double().cpu().numpy(), x @ w.T)


@pytest.mark.parametrize("n", [1, 20, 140])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_product_strides_and_outside(n, dtype):
    """Unaligned and strided activations and outputs; nothing outside the output is touched."""
    rng = np.random.default_rng(n)
    d_in, d_out = 300, 77
    w, ws = _weights(rng, d_out, d_in)
    base = torch.from_numpy(rng.standard_normal((n, 517))).to(TYPES[dtype]).to(DEV)
    room = torch.full((n + 2, 99), 5.0, device=DEV)
    for at in (0, 1, 8):
        X = base[:, at: at + d_in]
        out = room[1: n + 1, 3: 3 + d_out]
        Y = P.mx_matmul(X, torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV), out=out)
        assert Y is out
        _check(Y, X.double().cpu().numpy(), M.mx_values(w, ws, "fp4", d_in))
        out.fill_(5.0)
        assert (room == 5.0).all()


@pytest.mark.parametrize("n", [3, 150])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_infinities_stay_in_their_token(n, dtype):
    rng = np.random.default_rng(n)
    d_in, d_out = 200, 40
    w, ws = _weights(rng, d_out, d_in)
    wv = M.mx_values(w, ws, "fp4", d_in)
    x = rng.standard_normal((n, d_in))
    x[1, 7], x[2, 150] = np.inf, np.nan
    X = torch.from_numpy(x).to(TYPES[dtype])
    Y = P.mx_matmul(X.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV)).cpu().numpy()
    assert np.isnan(Y[2]).all()
    with np.errstate(invalid="ignore"):
        assert np.array_equal(Y[1], np.inf * wv[:, 7], equal_nan=True)
    keep = np.delete(np.arange(n), [1, 2])
    _check(torch.from_numpy(Y[keep]), X.double().numpy()[keep], wv)
    # a weight block that is NaN reaches every token of its rows and no other row
    ws = ws.copy()
    ws[5, 1] = 255
    Y = P.mx_matmul(X[keep].to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV)).cpu().numpy()
    assert np.isnan(Y[:, 5]).all() and np.isfinite(np.delete(Y, 5, 1)).all()


def test_empty_products_and_quantisation():
    w = torch.zeros(8, 64, dtype=torch.uint8, device=DEV), torch.zeros(8, 4, dtype=torch.uint8, device=DEV)
    assert P.mx_matmul(torch.zeros(0, 100, device=DEV), *w).shape == (0, 8)
    assert P.mx_matmul(torch.zeros(3, 100, device=DEV), w[0][:0], w[1][:0]).shape == (3, 0)
    codes, scales = P.mx_quantize(torch.zeros(0, 100, device=DEV))
    assert codes.shape == (0, 64) and P.mx_dequantize(codes, scales, 100).shape == (0, 100)
    for bad in (lambda: P.mx_matmul(torch.zeros(3, 200, device=DEV), *w),
                lambda: P.mx_dequantize(*w, 129), lambda: P.mx_dequantize(*w, 0),
                lambda: P.mx_matmul_quantized(*w, *w, x_fmt="fp8")):
        with pytest.raises(ValueError):
            bad()


def test_quantize_and_product_on_another_stream_and_replayed():
    rng = np.random.default_rng(1)
    d_in, d_out, n = 640, 96, 9
    W = torch.from_numpy(0.02 * rng.standard_normal((d_out, d_in))).float().to(DEV)
    w = P.mx_quantize(W)
    X = torch.from_numpy(rng.standard_normal((n, d_in))).to(torch.bfloat16).to(DEV)

    def step():
        return P.mx_matmul(X, *w), P.mx_matmul_quantized(*P.mx_quantize(X, fmt="fp4"), *w)

    eager = [y.clone() for y in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y = P.mx_matmul(X, *w, stream=s)
    s.synchronize()
    assert torch.equal(Y, eager[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for k in range(4):
        X.copy_(torch.from_numpy(rng.standard_normal((n, d_in))))
        want = [y.clone() for y in step()]
        for y in out:
            y.fill_(-1.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k


def test_rows_past_4_gib():
    """Codes past 2^32 bytes: the last rows of a matrix of 2^20 outputs."""
    d_in, d_out = 8400, 1 << 20
    w = torch.zeros(d_out, P.mx_codes_per_row(d_in), dtype=torch.uint8, device=DEV)
    ws = torch.zeros(d_out, P.mx_scales_per_row(d_in), dtype=torch.uint8, device=DEV)
    assert w.numel() > 1 << 32
    rng = np.random.default_rng(2)
    c, s = _weights(rng, 64, d_in)
    w[-64:].copy_(torch.from_numpy(c))
    ws[-64:].copy_(torch.from_numpy(s))
    for n in (1, 70):
        X = torch.from_numpy(rng.standard_normal((n, d_in))).to(torch.bfloat16)
        Y = P.mx_matmul(X.to(DEV), w, ws)
        _check(Y[:, -64:].contiguous(), X.double().numpy(), M.mx_values(c, s, "fp4", d_in))
        assert (Y[:, :-64] == 0).all()
        q = P.mx_quantize(X.to(DEV))
        Y = P.mx_matmul_quantized(*q, w, ws)
        xq = M.mx_values(q[0].cpu().numpy(), q[1].cpu().numpy(), "fp4", d_in)
        _check(Y[:, -64:].contiguous(), xq, M.mx_values(c, s, "fp4", d_in))
        assert (Y[:, :-64] == 0).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,d_in,d_out", [(1, 300, 20), (13, 1100, 40), (40, 260, 200), (300, 200, 300), (600, 130, 70)])
def test_weights_of_every_size(n, d_in, d_out, dtype):
    """Blocks of weights from 2^-60 to 2^40, among them scales just inside and outside float16's range."""
    rng = np.random.default_rng(d_in)
    e = np.repeat(rng.integers(-60, 40, (d_out, -(-d_in // 32))), 32, 1)[:, :d_in].astype(np.float64)
    e[0], e[1, :64], e[2], e[3] = -24.0 + 2, 15.0, -23.0 + 2, 13.0 + 2
    e[4::3] = -5.0
    w, ws = M.mx_quantize(np.clip(rng.standard_normal((d_out, d_in)), -1.9, 1.9) * 2.0 ** e, "fp4")
    X = torch.from_numpy(rng.standard_normal((n, d_in))).to(TYPES[dtype])
    Y = P.mx_matmul(X.to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV)).double().cpu().numpy()
    x, wv = X.double().numpy(), M.mx_values(w, ws, "fp4", d_in)
    bound = (4 * d_in + 64) * 2.0 ** -23 * (np.abs(x) @ np.abs(wv).T)
    assert (np.abs(Y - x @ wv.T) <= bound).all()


# Enough rows and tokens for every matrix-core tile; d_in ends inside a step, so the last columns take another path.
LARGE = [(1100, 200, 1100), (2100, 328, 2100), (1500, 120, 1500), (4200, 392, 1030)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32", "fp4", "fp8"])
@pytest.mark.parametrize("n,d_in,d_out", LARGE)
def test_large_products(n, d_in, d_out, kind):
    """Aligned and unaligned activations, an output inside a larger one, an infinity, a NaN and a NaN weight block."""
    rng = np.random.default_rng(n + d_in)
    w, ws = _weights(rng, d_out, d_in)
    wt = torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV)
    wv = M.mx_values(w, ws, "fp4", d_in)
    x = rng.standard_normal((n, d_in)) * np.exp(2 * rng.standard_normal(d_in))
    room = torch.full((n + 2, d_out + 7), 5.0, device=DEV)
    out = room[1: n + 1, 3: 3 + d_out]
    if kind in TYPES:
        base = torch.zeros(n, d_in + 24, dtype=TYPES[kind], device=DEV)
        for at in (0, 8, 1):
            X = base[:, at: at + d_in]
            X.copy_(torch.from_numpy(x))
            P.mx_matmul(X, *wt, out=out)
            _check(out, X.double().cpu().numpy(), wv)
            out.fill_(5.0)
            assert (room == 5.0).all()
            bad = X.clone() if at == 0 else X
            bad[n - 1, 7], bad[130, d_in - 1] = np.inf, np.nan
            ws_nan = wt[1].clone()
            ws_nan[d_out - 2, 1] = 255
            Y = P.mx_matmul(bad, wt[0], ws_nan).cpu().numpy()
            keep = np.delete(np.arange(n), [130, n - 1])
            assert np.isnan(Y[130]).all() and np.isnan(Y[:, d_out - 2]).all()
            assert np.isfinite(np.delete(Y[keep], d_out - 2, 1)).all()
            with np.errstate(invalid="ignore"):
                assert np.array_equal(np.delete(Y[n - 1], d_out - 2), np.delete(np.inf * wv[:, 7], d_out - 2), equal_nan=True)
    else:
        xc, xs = M.mx_quantize(x, kind)
        xt = torch.from_numpy(xc).to(DEV), torch.from_numpy(xs).to(DEV)
        P.mx_matmul_quantized(*xt, *wt, x_fmt=kind, out=out)
        _check(out, M.mx_values(xc, xs, kind, d_in), wv)
        out.fill_(5.0)
        assert (room == 5.0).all()
        xt[1][130, 1] = 255
        ws_nan = wt[1].clone()
        ws_nan[d_out - 2, 1] = 255
        Y = P.mx_matmul_quantized(*xt, wt[0], ws_nan, x_fmt=kind).cpu().numpy()
        assert np.isnan(Y[130]).all() and np.isnan(Y[:, d_out - 2]).all()
        assert np.isfinite(np.delete(np.delete(Y, 130, 0), d_out - 2, 1)).all()


@pytest.mark.parametrize("n,d_in,d_out", LARGE[:2])
def test_large_products_of_weights_of_every_size(n, d_in, d_out):
    """Float16 activations by weight blocks inside and outside float16's range, in tiles of many tokens."""
    test_weights_of_every_size(n, d_in, d_out, "f16")


def test_tokens_far_apart():
    """A row stride whose tile passes 32-bit offsets."""
    rng = np.random.default_rng(3)
    n, d_in, d_out, ld = 600, 128, 1300, 1 << 24
    w, ws = _weights(rng, d_out, d_in)
    base = torch.zeros((n - 1) * ld + d_in, dtype=torch.bfloat16, device=DEV)
    X = torch.as_strided(base, (n, d_in), (ld, 1))
    X.copy_(torch.from_numpy(rng.standard_normal((n, d_in))))
    Y = P.mx_matmul(X, torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV))
    _check(Y, X.double().cpu().numpy(), M.mx_values(w, ws, "fp4", d_in))


@pytest.mark.parametrize("n,d_out", [(3, 40), (300, 300), (1100, 1100)])
def test_infinite_float16_by_weights_outside_its_range(n, d_out):
    """An infinity meets weights inside and outside float16's range in one sum: no zero stands in for either."""
    rng = np.random.default_rng(n)
    d_in = 1224
    e = np.repeat(rng.choice([-40.0, -5.0, 25.0], (d_out, -(-d_in // 32)), p=[0.05, 0.9, 0.05]), 32, 1)[:, :d_in]
    w, ws = M.mx_quantize(rng.uniform(1.0, 1.9, (d_out, d_in)) * rng.choice([-1.0, 1.0], (d_out, d_in)) * 2.0 ** e, "fp4")
    wv = M.mx_values(w, ws, "fp4", d_in)
    assert (wv != 0).all()
    x = rng.standard_normal((n, d_in))
    at = rng.integers(0, d_in, n)
    x[np.arange(n), at] = np.inf
    Y = P.mx_matmul(torch.from_numpy(x).half().to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV))
    assert np.array_equal(Y.cpu().numpy(), np.inf * wv[:, at].T)


@pytest.mark.parametrize("n", [3, 40, 1500])
def test_float32_of_every_size(n):
    """Float32 activations from 2^-100 to 2^100, and infinities and NaN of small payloads among them."""
    rng = np.random.default_rng(n)
    d_in, d_out = 400, 1500
    w, ws = _weights(rng, d_out, d_in)
    wv = M.mx_values(w, ws, "fp4", d_in)
    wt = torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV)
    x = rng.standard_normal((n, d_in)) * 2.0 ** rng.integers(-100, 100, (n, 1))
    X = torch.from_numpy(x).float()
    Y = P.mx_matmul(X.to(DEV), *wt).double().cpu().numpy()
    x = X.double().numpy()
    bound = (4 * d_in + 64) * 2.0 ** -23 * (np.abs(x) @ np.abs(wv).T)
    assert (np.abs(Y - x @ wv.T) <= bound).all()
    bits = X.numpy().view(np.uint32).copy()
    bits[0, 5], bits[1, 150], bits[2, 399] = 0x7F800000, 0x7F800001, 0xFF80FFFF      # an infinity, NaN with low payloads
    Y2 = P.mx_matmul(torch.from_numpy(bits.view(np.float32)).to(DEV), *wt).double().cpu().numpy()
    assert np.isnan(Y2[1:3]).all() and np.array_equal(Y2[3:], Y[3:])
    with np.errstate(invalid="ignore"):
        assert np.array_equal(Y2[0], np.inf * wv[:, 5], equal_nan=True)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32", "fp4", "fp8"])
@pytest.mark.parametrize("n,d_in,d_out", [(1, 520, 11000), (16, 1024, 12288 - 5), (30, 640, 9000), (5, 384, 6000), (33, 256, 17000)])
def test_few_tokens_by_many_rows(n, d_in, d_out, kind):
    """One round of every few-token tile, with rows past the end of the last."""
    test_integers_come_out_exactly(n, d_in, d_out, kind)
