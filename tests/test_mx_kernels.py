"""Which kernel a product takes (CPU), and every one of them against float64 (needs an MI355X).

SIZES names, for each kind of activations and each kernel that the rule can
choose for it, sizes that reach it; the bounds are those of test_gpu_mx.py.
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_accum_amd as P
from oracle import mx_oracle as M
from post_weight_quantization_accum_amd import _lib

DEV = "cuda"
KINDS = {"f32": (_lib.F32, 0), "f16": (_lib.F16, 0), "bf16": (_lib.BF16, 0), "fp8": (0, _lib.MX_FP8), "fp4": (0, _lib.MX_FP4)}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# kernel -> (tokens, outputs); columns: 328 where rows are to start on 16 bytes, else 329
FEW = {0: (3, 100), 1: (2, 4200), 2: (7, 8300), 3: (16, 12400)}
HALF = {**FEW, 4: (30, 6300), 5: (25, 8300)}
SIZES = {("f32", 1): {**FEW, 4: (96, 2700), 9: (1500, 2048)}, ("f32", 0): {**FEW, 4: (4100, 20), 9: (1500, 2048)},
         ("f16", 1): {**HALF, 7: (140, 8300), 8: (260, 16500)}, ("bf16", 1): {**HALF, 7: (140, 8300), 8: (260, 16500)},
         ("f16", 0): {**FEW, 9: (2048, 2048)}, ("bf16", 0): {**FEW, 9: (2048, 2048)},
         ("fp8", 1): {**HALF, 6: (60, 11000), 9: (4096, 2048)},
         ("fp4", 1): {**HALF, 7: (140, 8300), 8: (100, 33000)}}
CASES = [(kind, aligned, k) for (kind, aligned), sizes in SIZES.items() for k in sizes]


def kernel(kind, n, d_in, d_out, aligned=1):
    dt, f = KINDS[kind]
    return P.load().gptq_mx_matmul_kernel(dt, f, n, d_in, d_out, aligned)


def test_sizes_reach_their_kernels():
    for kind, aligned, k in CASES:
        n, d_out = SIZES[kind, aligned][k]
        assert kernel(kind, n, 328 + (not aligned), d_out, aligned) == k, (kind, aligned, k)
    # the rule knows no other kernel for the kind, whatever the sizes
    outs = [*range(16, 1100, 32), *range(1100, 34000, 300), 1 << 16, 1 << 20]
    for (kind, aligned), sizes in SIZES.items():
        for n in (1, 7, 16, 17, 33, 48, 64, 65, 100, 128, 129, 256, 300, 600, 1024, 2048, 4200, 1 << 14, 1 << 20):
            assert {kernel(kind, n, 4096, o, aligned) for o in outs} <= set(sizes), (kind, aligned, n)


def test_refused_sizes():
    assert kernel("bf16", 0, 128, 16) == kernel("bf16", 1, 0, 16) == kernel("bf16", 1, 128, 0) == -1
    assert P.load().gptq_mx_matmul_kernel(7, 0, 1, 128, 16, 1) == P.load().gptq_mx_matmul_kernel(0, 3, 1, 128, 16, 1) == -1


def _multiply(kind, x, w, ws):
    """(product, the activations as held) of float64 x by the weights."""
    wt = torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV)
    if kind in TYPES:
        X = torch.from_numpy(x).to(TYPES[kind])
        return P.mx_matmul(X.to(DEV), *wt).double().cpu().numpy(), X.double().numpy()
    xc, xs = M.mx_quantize(x, kind)
    Y = P.mx_matmul_quantized(torch.from_numpy(xc).to(DEV), torch.from_numpy(xs).to(DEV), *wt, x_fmt=kind)
    return Y.double().cpu().numpy(), M.mx_values(xc, xs, kind, x.shape[1])


def _within(Y, x, w):
    bound = (4 * x.shape[1] + 64) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    return (np.abs(Y - x @ w.T) <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind,aligned,k", CASES)
def test_every_kernel(kind, aligned, k):
    n, d_out = SIZES[kind, aligned][k]
    d_in = 328 + (not aligned)
    rng = np.random.default_rng(k)
    # small integers and scales that differ from block to block: a wrong column, block or scale shows
    blocks = -(-d_in // 32)
    a, b = (rng.integers(-4, 5, (m, d_in)).astype(np.float64) for m in (n, d_out))
    for t in (a, b):
        t[:, ::32] = 4.0
        t *= 2.0 ** np.repeat(rng.integers(0, 3, (len(t), blocks)), 32, 1)[:, :d_in]
    w, ws = M.mx_quantize(b, "fp4")
    Y, x = _multiply(kind, a, w, ws)
    assert np.array_equal(Y, x @ M.mx_values(w, ws, "fp4", d_in).T)
    # weights from 2^-60 to 2^40 (float16's range of scales is inside), a NaN block, an infinity and a NaN among the activations
    e = np.repeat(rng.integers(-60, 40, (d_out, blocks)), 32, 1)[:, :d_in]
    e[::3] = -5
    w, ws = M.mx_quantize(np.clip(rng.standard_normal((d_out, d_in)), -1.9, 1.9) * 2.0 ** e, "fp4")
    wv = M.mx_values(w, ws, "fp4", d_in)
    a = rng.standard_normal((n, d_in))
    Y, x = _multiply(kind, a, w, ws)
    assert _within(Y, x, wv)
    a[0, 7], a[n - 1, d_in - 1] = np.inf, np.nan
    ws[d_out - 2, 1] = 255
    Y, _ = _multiply(kind, a, w, ws)
    assert np.isnan(Y[n - 1]).all() and np.isnan(Y[:, d_out - 2]).all()
    keep = np.delete(np.arange(d_out), d_out - 2)
    if n > 2:
        assert _within(Y[1:-1][:, keep], x[1:-1], wv[keep])
    if kind in TYPES and n > 1:
        with np.errstate(invalid="ignore"):
            assert np.array_equal(Y[0, keep], np.inf * wv[keep, 7], equal_nan=True)
