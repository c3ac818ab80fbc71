"""Norms around a block, fused with the residual stream, and their gradient: the
gptq_residual_norm* entry points of ``include/gptq.h``, which state the formulas.
"""
from __future__ import annotations

import math

from . import _lib
from ._lib import load
from .mx import _codes, _current, _dtype_code, _gpu, _on, _rows, _torch

KINDS = {"rms": _lib.NORM_RMS, "layer": _lib.NORM_LAYER}


def _norm(n, d, kind, eps, residual_scale, weight, bias, post_weight, gate):
    """gptq_norm of the call, its vectors checked (one dtype; gate d or tokens x d values)."""
    k = KINDS.get(kind)
    if k is None:
        raise ValueError(f"kind must be one of {', '.join(KINDS)}")
    if not (eps >= 0 and math.isfinite(eps) and math.isfinite(residual_scale)):
        raise ValueError("eps must be 0 or more, and eps and residual_scale finite")
    dt, ld_gate, ptr = None, 0, []
    for name, t in (("weight", weight), ("bias", bias), ("post_weight", post_weight), ("gate", gate)):
        if t is None:
            ptr.append(None)
            continue
        if t.dim() == 2 and name == "gate":
            n_g, d_g, ld_gate = _rows(t, "gate")
            if (n_g, d_g) != (n, d) or ld_gate < d:
                raise ValueError("gate must have d values, or d for each token")
        elif t.shape != (d,) or (d > 1 and t.stride(0) != 1):
            raise ValueError(f"{name} must have d values in a row")
        if dt is not None and t.dtype != dt:
            raise TypeError("weight, bias, post_weight and gate must have one dtype")
        dt = t.dtype
        ptr.append(t.data_ptr())
    code = _lib.F32
    if dt is not None:
        code = _codes.get(dt)
        if code is None:
            raise TypeError(f"unsupported dtype {dt}")
    return _lib.Norm(k, eps, residual_scale, code, *ptr, ld_gate)


def _given(*ts):
    return [t for t in ts if t is not None]


def _like(t, name, n, d, dtype=None):
    """Row stride of a tokens x d tensor."""
    n_t, d_t, ld = _rows(t, name)
    if (n_t, d_t) != (n, d) or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must match in tokens, width and dtype")
    return ld


def residual_norm(X, B=None, *, weight=None, bias=None, post_weight=None, gate=None, kind="rms", eps=1e-6,
                  residual_scale=1.0, h_dtype=None, dtype=None, out=None, stream=None):
    """(h, y): h = residual_scale * X + gate * p, p = B or norm(B) * post_weight, and y = norm(h) * weight + bias.

    X, B: tokens x d (B, a block's output, may be left out); weight, bias,
    post_weight: d values; gate: d values, or tokens x d.  kind: "rms" or
    "layer".  h has X's dtype unless h_dtype says otherwise (h is X itself where
    neither B nor a scale nor a dtype changes it), y X's unless dtype does.
    out: (h, y) to write to; either may be None, and is then not computed.  h
    may be X.
    """
    lib, _ = load(), _torch()
    dev = _gpu(X, *_given(B, weight, bias, post_weight, gate))
    n, d, ld_x = _rows(X)
    if d < 1:
        raise ValueError("X must have at least one column")
    c = _norm(n, d, kind, eps, residual_scale, weight, bias, post_weight, gate)
    b, b_dt, ld_b = None, 0, d
    if B is not None:
        b, b_dt, ld_b = B.data_ptr(), _dtype_code(B), _like(B, "B", n, d)
    elif post_weight is not None or gate is not None:
        raise ValueError("post_weight and gate act on B")
    with _on(dev, stream):
        if out is None:
            same = B is None and residual_scale == 1.0 and h_dtype in (None, X.dtype)
            h = None if same else X.new_empty((n, d), dtype=h_dtype)
            y = X.new_empty((n, d), dtype=dtype)
            out = (X if same else h), y
            ld_h = ld_y = d
        else:
            h, y = out
            _gpu(X, *_given(h, y))
            ld_h = d if h is None else _like(h, "out", n, d, h_dtype)
            ld_y = d if y is None else _like(y, "out", n, d, dtype)
        st = lib.gptq_residual_norm(c, n, d, X.data_ptr(), _dtype_code(X), ld_x, b, b_dt, ld_b,
                                    None if h is None else h.data_ptr(), 0 if h is None else _dtype_code(h), ld_h,
                                    None if y is None else y.data_ptr(), 0 if y is None else _dtype_code(y), ld_y,
                                    _current(dev))
    if st:
        _lib.check(st, "gptq_residual_norm")
    return out


def residual_norm_backward(dY, H, B=None, *, dH=None, weight=None, bias=None, post_weight=None, gate=None, kind="rms",
                           eps=1e-6, residual_scale=1.0, workspace=None, stream=None):
    """The gradients of residual_norm's inputs as a dict: "x" (of H's dtype),
    "b" where B is given (of its dtype), and "weight", "bias", "post_weight",
    "gate" where those are (float32; a gate for each token: of its dtype).

    dY, dH: the gradients for y and, if any, for h (of H's dtype); H, B: as the
    forward call gave and had them.  workspace: at least
    gptq_residual_norm_backward_workspace bytes, made by the call otherwise.
    """
    lib, torch = load(), _torch()
    dev = _gpu(dY, H, *_given(B, dH, weight, bias, post_weight, gate))
    n, d, ld_h = _rows(H, "H")
    if d < 1:
        raise ValueError("H must have at least one column")
    c = _norm(n, d, kind, eps, residual_scale, weight, bias, post_weight, gate)
    ld_dy = _like(dY, "dY", n, d)
    if B is None and (post_weight is not None or gate is not None):
        raise ValueError("post_weight and gate act on B")
    ld_b = d if B is None else _like(B, "B", n, d)
    ld_dh = d if dH is None else _like(dH, "dH", n, d, H.dtype)
    with _on(dev, stream):
        out = {"x": H.new_empty((n, d))}
        if B is not None:
            out["b"] = B.new_empty((n, d))
        for name, t in (("weight", weight), ("bias", bias), ("post_weight", post_weight)):
            if t is not None:
                out[name] = t.new_empty(d, dtype=torch.float32)
        if gate is not None:
            out["gate"] = gate.new_empty((n, d)) if gate.dim() == 2 else gate.new_empty(d, dtype=torch.float32)
        nws = 0
        if workspace is not None:
            _gpu(H, workspace)
            if not workspace.is_contiguous():
                raise TypeError("workspace must be contiguous")
            nws = workspace.numel() * workspace.element_size()
        elif any(t is not None for t in (weight, bias, post_weight)) or (gate is not None and gate.dim() == 1):
            nws = lib.gptq_residual_norm_backward_workspace(n, d)
            workspace = H.new_empty(nws, dtype=torch.uint8)

        def at(name):
            t = out.get(name)
            return None if t is None else t.data_ptr()

        st = lib.gptq_residual_norm_backward(c, n, d, dY.data_ptr(), _dtype_code(dY), ld_dy, H.data_ptr(), _dtype_code(H),
                                             ld_h, None if B is None else B.data_ptr(), 0 if B is None else _dtype_code(B),
                                             ld_b, None if dH is None else dH.data_ptr(), ld_dh, at("x"), d, at("b"), d,
                                             at("weight"), at("bias"), at("post_weight"), at("gate"), d,
                                             None if workspace is None else workspace.data_ptr(), nws, _current(dev))
    if st:
        _lib.check(st, "gptq_residual_norm_backward")
    return out


__all__ = ["residual_norm", "residual_norm_backward"]
