"""Microscaled values (blocks of 32 e2m1 or e4m3 elements with a shared power
of two) and products with e2m1 weights, over the gptq_mx_* entry points of
``include/gptq.h``; that header states the format and the storage.

A call's checks cost more than its launch for small inputs, so they are
written for few Python operations: plain integers go to the library, and a
device is made current only where it is not.
"""
from __future__ import annotations

import contextlib

from . import _lib
from ._lib import load

FORMATS = {"fp8": _lib.MX_FP8, "fp4": _lib.MX_FP4}

_t = None            # torch and the dtype codes, on first use
_codes: dict = {}


def _torch():
    global _t
    if _t is None:
        import torch
        _codes.update({torch.float32: _lib.F32, torch.float16: _lib.F16, torch.bfloat16: _lib.BF16})
        _t = torch
    return _t


def _dtype_code(t) -> int:
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _format(fmt: str) -> int:
    f = FORMATS.get(fmt)
    if f is None:
        raise ValueError(f"fmt must be one of {', '.join(FORMATS)}")
    return f


def _gpu(t, *ts) -> int:
    """The index of the one GPU that holds all the tensors."""
    dev = t.get_device()
    for x in ts:
        if x.get_device() != dev:
            raise ValueError("tensors must live on the GPU" if dev < 0 or x.get_device() < 0 else
                             "tensors must live on one GPU")
    if dev < 0:
        raise ValueError("tensors must live on the GPU")
    return dev


_HERE = contextlib.nullcontext()


def _on(dev: int, stream=None):
    """Context in which the library's calls and new tensors belong to GPU dev
    and to stream (the caching allocator then never hands their memory to
    other work before the stream's queued kernels are done with it)."""
    torch = _torch()
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("stream belongs to another GPU than the tensors")
        return torch.cuda.stream(stream)
    return _HERE if torch.cuda.current_device() == dev else torch.cuda.device(dev)


def _current(dev: int) -> int:
    """hipStream_t of the current stream, as an integer."""
    return _t._C._cuda_getCurrentRawStream(dev)


def _rows(X, name="X"):
    if X.dim() != 2:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    n, d = X.shape
    ld, one = X.stride()
    if one != 1 and d > 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return n, d, ld if n > 1 else max(d, 1)


def _mx_pair(codes, scales, fmt: str, name="codes"):
    """(rows, padded columns) of a pair of code and scale tensors."""
    u8 = _torch().uint8
    if codes.dtype != u8 or codes.dim() != 2 or not codes.is_contiguous():
        raise TypeError(f"{name} must be a contiguous 2-D uint8 tensor")
    if scales.dtype != u8 or scales.dim() != 2 or not scales.is_contiguous():
        raise TypeError("scales must be a contiguous 2-D uint8 tensor")
    n, c = codes.shape
    m, s = scales.shape
    per = 16 if fmt == "fp4" else 32               # bytes of codes to a scale byte
    if c == 0 or m != n or s * per != c or s % 4:
        raise ValueError(f"{name} and scales do not have the padded widths of one {fmt} matrix")
    return n, 32 * s


def mx_codes_per_row(n_cols: int, fmt: str = "fp4") -> int:
    return int(load().gptq_mx_codes_per_row(n_cols, _format(fmt)))


def mx_scales_per_row(n_cols: int) -> int:
    return int(load().gptq_mx_scales_per_row(n_cols))


def mx_quantize(X, fmt: str = "fp4", out=None, stream=None):
    """(codes, scales) of X (rows x columns, bf16 / f16 / f32) as uint8 tensors, rows padded to 128 columns."""
    lib, torch, f = load(), _torch(), _format(fmt)
    dev = _gpu(X)
    n, d, ld = _rows(X)
    dt = _dtype_code(X)
    if d < 1:
        raise ValueError("X must have at least one column")
    units = -(-d // 128)
    wide = units * (64 if f == _lib.MX_FP4 else 128), units * 4
    with _on(dev, stream):
        if out is None:
            codes = X.new_empty((n, wide[0]), dtype=torch.uint8)
            scales = codes.new_empty((n, wide[1]))
        else:
            codes, scales = out
            _gpu(X, codes, scales)
            for t, w in zip((codes, scales), wide):
                if t.dtype != torch.uint8 or tuple(t.shape) != (n, w) or not t.is_contiguous():
                    raise TypeError(f"out must be contiguous uint8 tensors of shapes {(n, wide[0])} and {(n, wide[1])}")
        st = lib.gptq_mx_quantize(X.data_ptr(), dt, n, d, ld, f, codes.data_ptr(), scales.data_ptr(), _current(dev))
    if st:
        _lib.check(st, "gptq_mx_quantize")
    return codes, scales


def mx_dequantize(codes, scales, n_cols: int, fmt: str = "fp4", dtype=None, out=None, stream=None):
    """The rows x n_cols values of codes and scales (float32 unless dtype or out says otherwise)."""
    lib, torch, f = load(), _torch(), _format(fmt)
    dev = _gpu(codes, scales)
    n, padded = _mx_pair(codes, scales, fmt)
    if not padded - 128 < n_cols <= padded:
        raise ValueError("n_cols does not match the width of codes")
    with _on(dev, stream):
        if out is None:
            out = codes.new_empty((n, n_cols), dtype=dtype or torch.float32)
            ld = n_cols
        else:
            _gpu(codes, out)
            if tuple(out.shape) != (n, n_cols) or (dtype is not None and out.dtype != dtype):
                raise TypeError("out must be rows x n_cols of dtype")
            _, _, ld = _rows(out, "out")
        st = lib.gptq_mx_dequantize(codes.data_ptr(), scales.data_ptr(), f, n, n_cols, out.data_ptr(), _dtype_code(out),
                                    ld, _current(dev))
    if st:
        _lib.check(st, "gptq_mx_dequantize")
    return out


def _product_out(out, n_tok, d_out, like):
    torch = _torch()
    if out is None:
        return like.new_empty((n_tok, d_out), dtype=torch.float32), max(d_out, 1)
    if out.get_device() != like.get_device() or out.dtype != torch.float32 or tuple(out.shape) != (n_tok, d_out) or \
            (d_out > 1 and out.stride(1) != 1):
        raise TypeError("out must be float32 tokens x d_out with unit column stride, on the inputs' GPU")
    return out, out.stride(0) if n_tok > 1 else max(d_out, 1)


def mx_matmul(X, codes, scales, out=None, stream=None):
    """Y = X W^T (float32, tokens x d_out), W the e2m1 values of (codes, scales); X bf16 / f16 / f32."""
    lib = load()
    dev = _gpu(X, codes, scales)
    n, d, ld = _rows(X)
    d_out, padded = _mx_pair(codes, scales, "fp4")
    dt = _dtype_code(X)
    if not padded - 128 < d <= padded:
        raise ValueError("X and codes differ in columns")
    with _on(dev, stream):
        out, ld_y = _product_out(out, n, d_out, X)
        st = lib.gptq_mx_matmul(X.data_ptr(), dt, n, d, ld, codes.data_ptr(), scales.data_ptr(), d_out, out.data_ptr(),
                                ld_y, _current(dev))
    if st:
        _lib.check(st, "gptq_mx_matmul")
    return out


def mx_matmul_quantized(x_codes, x_scales, codes, scales, x_fmt: str = "fp4", out=None, stream=None):
    """Y = X W^T (float32) with microscaled activations (x_codes, x_scales of x_fmt) and e2m1 weights."""
    lib, f = load(), _format(x_fmt)
    dev = _gpu(x_codes, x_scales, codes, scales)
    n, d = _mx_pair(x_codes, x_scales, x_fmt, "x_codes")
    d_out, padded = _mx_pair(codes, scales, "fp4")
    if d != padded:
        raise ValueError("x_codes and codes differ in columns")
    with _on(dev, stream):
        out, ld_y = _product_out(out, n, d_out, x_codes)
        st = lib.gptq_mx_matmul_quantized(x_codes.data_ptr(), x_scales.data_ptr(), f, n, d, codes.data_ptr(),
                                          scales.data_ptr(), d_out, out.data_ptr(), ld_y, _current(dev))
    if st:
        _lib.check(st, "gptq_mx_matmul_quantized")
    return out


__all__ = ["mx_quantize", "mx_dequantize", "mx_matmul", "mx_matmul_quantized", "mx_codes_per_row", "mx_scales_per_row"]
