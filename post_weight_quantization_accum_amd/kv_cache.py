"""A paged cache of keys and values in 16 bits or microscaled, and attention
over it: the gptq_cache_* entry points of ``include/gptq.h``, which state the
layout, the masks and what happens at bad pages.
"""
from __future__ import annotations

import ctypes
import dataclasses

from . import _lib
from ._lib import load
from .mx import _codes, _current, _dtype_code, _gpu, _on, _torch

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
    torch = _torch()
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
    """(gptq_kv_cache, GPU, kv heads, head_dim) of c, with its tensors checked."""
    torch = _torch()
    f = FORMATS.get(c.fmt)
    if f is None:
        raise ValueError(f"cache.fmt must be one of {', '.join(FORMATS)}")
    k, v = c.k, c.v
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or not k.is_contiguous() or not v.is_contiguous():
        raise TypeError("cache.k and cache.v must be contiguous [page][kv head][offset][...] tensors, both alike")
    n_pages, heads, page, d = shape
    dt = k.dtype
    if v.dtype != dt or (dt != torch.uint8 if f else dt != torch.bfloat16 and dt != torch.float16):
        raise TypeError(f"cache.k and cache.v have the wrong dtype for a {c.fmt} cache")
    if f == _lib.MX_FP4:
        d *= 2
    if d % 32:
        raise ValueError("the cache's head_dim must be a multiple of 32")
    if not f:
        return _lib.Cache(k.data_ptr(), v.data_ptr(), None, None, n_pages, page, heads, d, f, _codes[dt]), \
            _gpu(k, v), heads, d
    ks, vs = c.k_scales, c.v_scales
    want = (n_pages, heads, page, d // 32)
    for t in (ks, vs):
        if t is None or t.dtype != torch.uint8 or t.shape != want or not t.is_contiguous():
            raise TypeError(f"cache.k_scales and cache.v_scales must be contiguous uint8 tensors of shape {want}")
    return _lib.Cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), n_pages, page, heads, d, f, 0), \
        _gpu(k, v, ks, vs), heads, d


def _heads(X, name, n_heads, head_dim):
    """(tokens, token stride, heads) of a tokens x heads x head_dim tensor whose tokens are contiguous."""
    shape = X.shape
    if len(shape) != 3 or (n_heads is not None and shape[1] != n_heads) or shape[2] != head_dim:
        raise ValueError(f"{name} must be tokens x heads x head_dim of the cache")
    n, h, _ = shape
    ld, by, one = X.stride()
    if one != 1 or (h > 1 and by != head_dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return n, ld if n > 1 else h * head_dim, h


def _int32(name, t, shape):
    if t.dtype != _torch().int32 or t.shape != shape or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor of shape {shape}")


def _table(table):
    if table.dim() != 2 or table.dtype != _torch().int32 or not table.is_contiguous():
        raise TypeError("table must be a contiguous 2-D int32 tensor")
    return table.shape


def cache_write(cache: KVCache, K, V, slots, stream=None):
    """Token t's keys and values (tokens x kv heads x head_dim) to slot
    slots[t] (int64: page * page_size + offset; outside the cache: skipped)."""
    lib, torch = load(), _torch()
    c, dev, heads, d = _cache(cache)
    _gpu(cache.k, K, V, slots)
    n, ld_k, _ = _heads(K, "K", heads, d)
    n_v, ld_v, _ = _heads(V, "V", heads, d)
    if n != n_v or K.dtype != V.dtype:
        raise ValueError("K and V must match in tokens and dtype")
    if slots.dtype != torch.int64 or slots.shape != (n,) or not slots.is_contiguous():
        raise TypeError("slots must be contiguous int64, one per token")
    with _on(dev, stream):
        st = lib.gptq_cache_write(c, K.data_ptr(), V.data_ptr(), _dtype_code(K), n, ld_k, ld_v, slots.data_ptr(),
                                  _current(dev))
    if st:
        _lib.check(st, "gptq_cache_write")
    return cache


def cache_read(cache: KVCache, table, row_start, n_rows: int, dtype=None, out=None, stream=None):
    """(K, V), n_rows x kv heads x head_dim: row row_start[s] + j is position j
    of sequence s (int32 row_start[n_seq + 1], table[n_seq][max_pages]); rows
    outside row_start[0] .. row_start[n_seq] - 1 are not written.  dtype:
    bfloat16 unless given (a "16bit" cache's own)."""
    lib, torch = load(), _torch()
    c, dev, heads, d = _cache(cache)
    _gpu(cache.k, table, row_start)
    n_seq, max_pages = _table(table)
    _int32("row_start", row_start, (n_seq + 1,))
    if dtype is None:
        dtype = out[0].dtype if out is not None else cache.k.dtype if cache.fmt == "16bit" else torch.bfloat16
    with _on(dev, stream):
        if out is None:
            K = table.new_empty((n_rows, heads, d), dtype=dtype)
            V = torch.empty_like(K)
            ld_k = ld_v = heads * d
        else:
            K, V = out
            _gpu(table, K, V)
            n_k, ld_k, _ = _heads(K, "out", heads, d)
            n_v, ld_v, _ = _heads(V, "out", heads, d)
            if n_k != n_rows or n_v != n_rows or K.dtype != dtype or V.dtype != dtype:
                raise TypeError("out must be two tensors of n_rows rows and dtype")
        st = lib.gptq_cache_read(c, table.data_ptr(), max_pages, n_seq, row_start.data_ptr(), n_rows, K.data_ptr(),
                                 V.data_ptr(), _dtype_code(K), ld_k, ld_v, _current(dev))
    if st:
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
    given (2^-100 .. 2^100).  window > 0: only the last `window` positions.
    """
    lib, torch = load(), _torch()
    c, dev, _, d = _cache(cache)
    _gpu(cache.k, Q, q_start, kv_len, table)
    n, ld_q, n_heads = _heads(Q, "Q", None, d)
    n_seq, max_pages = _table(table)
    _int32("q_start", q_start, (n_seq + 1,))
    _int32("kv_len", kv_len, (n_seq,))
    max_q = n if max_q is None else int(max_q)
    with _on(dev, stream):
        nws = lib.gptq_cache_attention_workspace(c, n, n_heads, n_seq, max_pages, max_q, window)
        if out is None:
            out, ld_o = Q.new_empty((n, n_heads, d)), n_heads * d
        else:
            _gpu(Q, out)
            n_o, ld_o, _ = _heads(out, "out", n_heads, d)
            if n_o != n or out.dtype != Q.dtype:
                raise TypeError("out must match Q in tokens and dtype")
        if workspace is not None:
            _gpu(Q, workspace)
            if not workspace.is_contiguous():
                raise TypeError("workspace must be contiguous")
            nws = workspace.numel() * workspace.element_size()
        elif nws:
            workspace = Q.new_empty(nws, dtype=torch.uint8)
        st = lib.gptq_cache_attention(c, Q.data_ptr(), _dtype_code(Q), n, n_heads, ld_q, q_start.data_ptr(),
                                      kv_len.data_ptr(), table.data_ptr(), max_pages, n_seq, max_q,
                                      d ** -0.5 if scale is None else scale, window, out.data_ptr(), ld_o,
                                      workspace.data_ptr() if workspace is not None else None, nws, _current(dev))
    if st:
        _lib.check(st, "gptq_cache_attention")
    return out


__all__ = ["KVCache", "new_cache", "cache_write", "cache_read", "cache_attention"]
