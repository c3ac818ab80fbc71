"""A paged cache of keys and values in 16 bits or microscaled, and attention
over it: the gptq_cache_* entry points of ``include/gptq.h``, which state the
layout, the masks and what happens at bad pages.
"""
from __future__ import annotations

import ctypes
import dataclasses

from . import _lib
from ._lib import load
from .mx import _base, _same_device

FORMATS = {"16bit": _lib.MX_NONE, "fp8": _lib.MX_FP8, "fp4": _lib.MX_FP4}


@dataclasses.dataclass
class KVCache:
    """Pages [page][kv head][offset][...]: k, v hold 16-bit values ("16bit")
    or uint8 codes of fmt ("fp8": head_dim bytes, "fp4": head_dim / 2), and
    k_scales, v_scales head_dim / 32 uint8 scale bytes per row (None for
    "16bit").  See new_cache."""
    k: object
    v: object
    k_scales: object = None
    v_scales: object = None
    fmt: str = "fp8"

    @property
    def page_size(self) -> int:
        return self.k.shape[2]

    @property
    def n_kv_heads(self) -> int:
        return self.k.shape[1]

    @property
    def head_dim(self) -> int:
        return self.k.shape[3] * (2 if self.fmt == "fp4" else 1)


def new_cache(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, fmt: str = "fp8", dtype=None,
              device="cuda") -> KVCache:
    """An empty cache (all zeros); dtype: of a "16bit" cache's values (bfloat16)."""
    torch = _base()._torch()
    if fmt not in FORMATS:
        raise ValueError(f"fmt must be one of {', '.join(FORMATS)}")
    if head_dim % 32:
        raise ValueError("head_dim must be a multiple of 32")
    rows = (n_pages, n_kv_heads, page_size)
    if fmt == "16bit":
        return KVCache(*(torch.zeros((*rows, head_dim), dtype=dtype or torch.bfloat16, device=device)
                         for _ in range(2)), fmt=fmt)
    width = head_dim // 2 if fmt == "fp4" else head_dim
    k, v = (torch.zeros((*rows, width), dtype=torch.uint8, device=device) for _ in range(2))
    ks, vs = (torch.zeros((*rows, head_dim // 32), dtype=torch.uint8, device=device) for _ in range(2))
    return KVCache(k, v, ks, vs, fmt)


def _cache(c: KVCache):
    """(gptq_kv_cache, device) of c, with its tensors checked."""
    base = _base()
    torch = base._torch()
    if c.fmt not in FORMATS:
        raise ValueError(f"cache.fmt must be one of {', '.join(FORMATS)}")
    mx = c.fmt != "16bit"
    for name, t in (("k", c.k), ("v", c.v)):
        if t.dim() != 4 or not t.is_contiguous() or t.shape != c.k.shape:
            raise TypeError(f"cache.{name} must be a contiguous [page][kv head][offset][...] tensor, k and v alike")
        if t.dtype not in ((torch.uint8,) if mx else (torch.bfloat16, torch.float16)) or t.dtype != c.k.dtype:
            raise TypeError(f"cache.{name} has the wrong dtype for a {c.fmt} cache")
    if c.head_dim % 32:
        raise ValueError("the cache's head_dim must be a multiple of 32")
    if mx:
        want = (*c.k.shape[:3], c.head_dim // 32)
        for name, t in (("k_scales", c.k_scales), ("v_scales", c.v_scales)):
            if t is None or t.dtype != torch.uint8 or tuple(t.shape) != want or not t.is_contiguous():
                raise TypeError(f"cache.{name} must be a contiguous uint8 tensor of shape {want}")
    dev = _same_device(c.k, c.v, *((c.k_scales, c.v_scales) if mx else ()))
    p = lambda t: t.data_ptr() if t is not None and mx else None  # noqa: E731
    return _lib.Cache(c.k.data_ptr(), c.v.data_ptr(), p(c.k_scales), p(c.v_scales), c.k.shape[0], c.page_size,
                      c.n_kv_heads, c.head_dim, FORMATS[c.fmt], 0 if mx else base._dtype_code(c.k)), dev


def _heads(X, name, n_heads, head_dim):
    """(tokens, token stride) of a tokens x heads x head_dim tensor whose tokens are contiguous."""
    if X.dim() != 3 or (n_heads is not None and X.shape[1] != n_heads) or X.shape[2] != head_dim:
        raise ValueError(f"{name} must be tokens x heads x head_dim of the cache")
    if X.stride(2) != 1 or (X.shape[1] > 1 and X.stride(1) != head_dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return X.shape[0], X.stride(0) if X.shape[0] > 1 else X.shape[1] * head_dim


def _int32(name, t, shape):
    torch = _base()._torch()
    if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor of shape {shape}")


def cache_write(cache: KVCache, K, V, slots, stream=None):
    """Token t's keys and values (tokens x kv heads x head_dim) to slot
    slots[t] (int64: page * page_size + offset; outside the cache: skipped)."""
    lib, base = load(), _base()
    torch = base._torch()
    c, dev = _cache(cache)
    _same_device(cache.k, K, V, slots)
    n, ld_k = _heads(K, "K", cache.n_kv_heads, cache.head_dim)
    n_v, ld_v = _heads(V, "V", cache.n_kv_heads, cache.head_dim)
    if n != n_v or K.dtype != V.dtype:
        raise ValueError("K and V must match in tokens and dtype")
    if slots.dtype != torch.int64 or tuple(slots.shape) != (n,) or not slots.is_contiguous():
        raise TypeError("slots must be contiguous int64, one per token")
    with torch.cuda.device(dev):
        st = lib.gptq_cache_write(ctypes.byref(c), base._ptr(K), base._ptr(V), base._dtype_code(K), n, ld_k, ld_v,
                                  base._ptr(slots), base._stream(stream))
    _lib.check(st, "gptq_cache_write")
    return cache


def cache_read(cache: KVCache, table, row_start, n_rows: int, dtype=None, out=None, stream=None):
    """(K, V), n_rows x kv heads x head_dim: row row_start[s] + j is position j
    of sequence s (int32 row_start[n_seq + 1], table[n_seq][max_pages]); rows
    outside row_start[0] .. row_start[n_seq] - 1 are not written.  dtype:
    bfloat16 unless given (a "16bit" cache's own)."""
    lib, base = load(), _base()
    torch = base._torch()
    c, dev = _cache(cache)
    _same_device(cache.k, table, row_start)
    if table.dim() != 2:
        raise TypeError("table must be 2-D")
    n_seq, max_pages = table.shape
    _int32("table", table, (n_seq, max_pages))
    _int32("row_start", row_start, (n_seq + 1,))
    if dtype is None:
        dtype = out[0].dtype if out is not None else cache.k.dtype if cache.fmt == "16bit" else torch.bfloat16
    with torch.cuda.device(dev):
        if out is None:
            with base._alloc_on(stream):
                out = tuple(torch.empty((n_rows, cache.n_kv_heads, cache.head_dim), dtype=dtype, device=dev)
                            for _ in range(2))
        K, V = out
        _same_device(cache.k, K, V)
        n_k, ld_k = _heads(K, "out", cache.n_kv_heads, cache.head_dim)
        n_v, ld_v = _heads(V, "out", cache.n_kv_heads, cache.head_dim)
        if n_k != n_rows or n_v != n_rows or K.dtype != dtype or V.dtype != dtype:
            raise TypeError("out must be two tensors of n_rows rows and dtype")
        st = lib.gptq_cache_read(ctypes.byref(c), base._ptr(table), max_pages, n_seq, base._ptr(row_start), n_rows,
                                 base._ptr(K), base._ptr(V), base._dtype_code(K), ld_k, ld_v, base._stream(stream))
    _lib.check(st, "gptq_cache_read")
    return K, V


def cache_attention(Q, cache: KVCache, q_start, kv_len, table, *, max_q: int | None = None, scale: float | None = None,
                    window: int = 0, out=None, workspace=None, stream=None):
    """Attention of the new tokens Q (tokens x heads x head_dim, bf16 / f16)
    over their sequences' pages; the new tokens' keys and values are in the
    cache already.

    Sequence s has tokens q_start[s] .. q_start[s + 1] - 1 and kv_len[s]
    positions in all (int32 tensors on the GPU); its newest token stands last.
    max_q: the largest number of new tokens of a sequence, if known (decoding:
    1); it only chooses between kernels.  scale: head_dim ** -0.5 unless
    given.  window > 0: only the last `window` positions.
    """
    lib, base = load(), _base()
    torch = base._torch()
    c, dev = _cache(cache)
    _same_device(cache.k, Q, q_start, kv_len, table)
    n, ld_q = _heads(Q, "Q", None, cache.head_dim)
    n_heads = Q.shape[1]
    if table.dim() != 2:
        raise TypeError("table must be 2-D")
    n_seq, max_pages = table.shape
    _int32("table", table, (n_seq, max_pages))
    _int32("q_start", q_start, (n_seq + 1,))
    _int32("kv_len", kv_len, (n_seq,))
    most = n if max_q is None else int(max_q)
    scale = cache.head_dim ** -0.5 if scale is None else float(scale)
    with torch.cuda.device(dev):
        nws = lib.gptq_cache_attention_workspace(ctypes.byref(c), n, n_heads, n_seq, max_pages, most, int(window))
        with base._alloc_on(stream):
            if out is None:
                out = torch.empty((n, n_heads, cache.head_dim), dtype=Q.dtype, device=dev)
            ws = workspace if workspace is not None else base._workspace(nws, dev)
        _same_device(cache.k, out, ws)
        n_o, ld_o = _heads(out, "out", n_heads, cache.head_dim)
        if n_o != n or out.dtype != Q.dtype:
            raise TypeError("out must match Q in tokens and dtype")
        st = lib.gptq_cache_attention(ctypes.byref(c), base._ptr(Q), base._dtype_code(Q), n, n_heads, ld_q,
                                      base._ptr(q_start), base._ptr(kv_len), base._ptr(table), max_pages, n_seq, most,
                                      scale, int(window), base._ptr(out), ld_o, base._ptr(ws),
                                      ws.numel() * ws.element_size() if ws is not None else 0, base._stream(stream))
    _lib.check(st, "gptq_cache_attention")
    return out


__all__ = ["KVCache", "new_cache", "cache_write", "cache_read", "cache_attention"]
