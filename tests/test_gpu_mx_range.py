"""Microscaled values at the ends of their range: every code and scale byte
through the products and the attention, activations near the bottom of
float32, the largest number of tokens (needs an MI355X).
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_accum_amd as P
from oracle import mx_oracle as M
from test_mx_kernels import DEV, SIZES, TYPES, _multiply, kernel

pytestmark = pytest.mark.gpu

# a scale byte of 253 or 254 takes the largest elements out of float32's range; 255 is NaN
BYTES = np.array([b for b in range(256) if b not in (253, 254)], dtype=np.uint8)


def _weights_of_every_byte(rows, bytes_):
    """Row r has scale byte bytes_[r mod len] and all sixteen codes in each of four blocks."""
    c = np.resize(np.arange(16, dtype=np.uint8), (rows, 128))
    s = np.repeat(np.resize(bytes_, rows)[:, None], 4, 1)
    return c[:, 0::2] | c[:, 1::2] << 4, s


@pytest.mark.parametrize("kind,k", [(kind, k) for (kind, aligned), sizes in SIZES.items() if aligned for k in sizes])
def test_every_weight_code_and_scale(kind, k):
    """Tokens with one activation, a power of two: outputs are the weights times it, subnormal ones too."""
    n, d_out = SIZES[kind, 1][k]
    w, ws = _weights_of_every_byte(d_out, BYTES)
    wv = M.mx_values(w, ws, "fp4")
    assert kernel(kind, n, 128, d_out) == k
    for power in ((0, 14) if kind == "f16" else (0, 100)):
        x = np.zeros((n, 128))
        x[np.arange(n), np.arange(n) * 5 % 128] = 2.0 ** power
        Y, x = _multiply(kind, x, w, ws)
        with np.errstate(over="ignore", invalid="ignore"):
            want = (wv[:, np.arange(n) * 5 % 128].T * 2.0 ** power).astype(np.float32)
        assert np.array_equal(Y.astype(np.float32), want, equal_nan=True)


@pytest.mark.parametrize("k", [0, 5, 7, 8])
def test_float16_weights_inside_their_range(k):
    """Only scales that float16 holds, so that every wave takes them as they are."""
    n, d_out = SIZES["f16", 1][k]
    w, ws = _weights_of_every_byte(d_out, np.arange(104, 141, dtype=np.uint8))
    x = np.zeros((n, 128))
    x[np.arange(n), np.arange(n) * 5 % 128] = 1.0
    Y, x = _multiply("f16", x, w, ws)
    assert np.array_equal(Y, x @ M.mx_values(w, ws, "fp4").T)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("many", [0, 1])
def test_every_activation_code_and_scale(kind, many):
    """All codes by one weight of 2 or of 2^100; with e4m3, scale bytes below 3 put small elements under bfloat16's
    smallest step, 2^-133, and those are off by at most half of it."""
    d_out = 2048 if many else 40
    codes = 256 if kind == "fp8" else 16
    n = 4096 if many else 256 * max(1, codes // 128)
    c = (np.arange(n)[:, None] // 256 * 128 + np.arange(128)).astype(np.int64) % codes
    if kind == "fp8":
        c = np.where(c % 128 == 127, 0, c)                   # e4m3's NaN
    c = c.astype(np.uint8)
    b = np.resize(np.arange(253 if kind == "fp4" else 247, dtype=np.uint8), n)
    xs = np.repeat(b[:, None], 4, 1)
    xv = M.mx_values(c[:, 0::2] | c[:, 1::2] << 4 if kind == "fp4" else c, xs, kind)
    xc = c[:, 0::2] | c[:, 1::2] << 4 if kind == "fp4" else c
    for value in (2.0, 2.0 ** 100):
        wv = np.zeros((d_out, 128))
        wv[np.arange(d_out), np.arange(d_out) * 3 % 128] = value
        w, ws = M.mx_quantize(wv, "fp4")
        Y = P.mx_matmul_quantized(*[torch.from_numpy(t).to(DEV) for t in (xc, xs, w, ws)], x_fmt=kind).double().cpu().numpy()
        with np.errstate(over="ignore"):
            want = (xv[:, np.arange(d_out) * 3 % 128] * value).astype(np.float32).astype(np.float64)
        room = np.where((b < 3)[:, None], 2.0 ** -134 * value, 0.0) if kind == "fp8" else 0.0
        with np.errstate(invalid="ignore"):
            assert ((Y == want) | (np.abs(Y - want) <= room)).all()


@pytest.mark.parametrize("n", [3, 40, 1500])
def test_float32_near_the_bottom(n):
    """Activations from 2^-105 to 2^-148: their parts end at bfloat16's smallest step, 2^-133, so beside the bound of
    all products (4 d_in + 64) 2^-23 sum |x w| each is off by less than 2^-133 |w|."""
    rng = np.random.default_rng(n)
    d_in, d_out = 400, 2048
    w, ws = M.mx_quantize(rng.standard_normal((d_out, d_in)) * 2.0 ** 30, "fp4")
    wv = M.mx_values(w, ws, "fp4", d_in)
    x = rng.standard_normal((n, d_in)) * 2.0 ** rng.integers(-148, -105, (n, 1))
    Y, x = _multiply("f32", x, w, ws)
    bound = (4 * d_in + 64) * 2.0 ** -23 * (np.abs(x) @ np.abs(wv).T) + 2.0 ** -133 * np.abs(wv).sum(1)
    assert (np.abs(Y - x @ wv.T) <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("group", [1, 80])
def test_every_cached_code_and_scale(group, fmt, dtype):
    """One position a sequence: the output is its value, rounded to the queries' type, by both kernels."""
    d, n_kv = 128, 2 if fmt == "fp8" else 1
    codes = 256 if fmt == "fp8" else 16
    b = np.arange(253 if fmt == "fp4" else 247)
    c = (np.arange(n_kv)[:, None] * d + np.arange(d)) % codes
    if fmt == "fp8":
        c = np.where(c % 128 == 127, 0, c)
    c = np.broadcast_to(c, (len(b), n_kv, d)).astype(np.uint8)
    s = np.broadcast_to(b[:, None, None], (len(b), n_kv, d // 32)).astype(np.uint8)
    held = c[..., 0::2] | c[..., 1::2] << 4 if fmt == "fp4" else c
    cache = P.new_cache(len(b), 1, n_kv, d, fmt=fmt, device=DEV)
    cache.v.copy_(torch.from_numpy(np.ascontiguousarray(held))[:, :, None])
    cache.v_scales.copy_(torch.from_numpy(np.ascontiguousarray(s))[:, :, None])
    table = torch.arange(len(b), dtype=torch.int32, device=DEV)[:, None].contiguous()
    start = torch.arange(len(b) + 1, dtype=torch.int32, device=DEV)
    Q = torch.ones(len(b), n_kv * group, d, dtype=TYPES[dtype], device=DEV)
    out = P.cache_attention(Q, cache, start, torch.ones(len(b), dtype=torch.int32, device=DEV), table, max_q=1).cpu()
    want = torch.from_numpy(M.mx_values(held, s, fmt)).to(TYPES[dtype]).repeat_interleave(group, 1)
    ok = (out == want) | (want.isinf() & ~out.isfinite())        # an infinite value is not finite, whatever else
    assert ok.all(), (out[~ok][:8], want[~ok][:8], [int(i) for i in (~ok).any(-1).any(-1).nonzero()[:8]])


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
def test_a_million_tokens(kind):
    """2^20 tokens, the most that a product takes, by a few outputs."""
    rng = np.random.default_rng(1)
    n, d_in, d_out = 1 << 20, 32, 5
    x = rng.integers(-4, 5, (n, d_in)).astype(np.float64)
    x[:, 0] = 4.0
    b = rng.integers(-4, 5, (d_out, d_in)).astype(np.float64)
    b[:, 0] = 4.0
    w, ws = M.mx_quantize(b, "fp4")
    if kind == "fp8":
        q = P.mx_quantize(torch.from_numpy(x).float().to(DEV), fmt="fp8")
        Y = P.mx_matmul_quantized(*q, torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV), x_fmt="fp8")
    else:
        Y = P.mx_matmul(torch.from_numpy(x).to(TYPES[kind]).to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV))
    assert np.array_equal(Y.double().cpu().numpy(), x @ b.T)
