"""Quantize a stack of decoder blocks in sequence (true-sequential).

"GPTQ量化算法深度解析" §3.1: layers are quantized one after another, each
from calibration activations; "GPTQ论文复现指南" §3.2: --true-sequential
quantizes inside a transformer block in order, so that every layer sees
the outputs of the layers before it already quantized.

The pages give no attention or normalisation details, so a block is the
plainest chain those passages support (identity attention, residuals, no
layer norm, ReLU as in OPT):

    q, k, v  <- H(X)                      (one Hessian, one factorisation)
    A  = X  W_v^T                         out <- H(A)
    h1 = X  + A W_out^T                   fc1 <- H(h1)
    r  = relu(h1 W_fc1^T)                 fc2 <- H(r)
    X' = h1 + r W_fc2^T                   (the next block's input)

With attention=Attention(...) the tokens are sequences and A is their causal
attention instead, as a serving program computes it: keys and values, products
of the quantized k and v, are written into the pages of a cache (16 bits or
microscaled, so that the layers behind see that rounding too) and read by
cache_attention from there.

    A  = attention(X W_q^T, cache of X W_k^T and X W_v^T)

Every product uses the already-quantized weights, computed by
gptq_dequant_matmul from the packed words (with act-order: packed in
quantization order, activations gathered into that order first).  Products come out
in float32; residual sums are taken in float32 and every activation that
feeds a Hessian or a product is rounded to the stack's dtype.  All steps of
the method run in the library; this module only sequences the calls and
does the elementwise glue (residual, ReLU, dtype rounding).
"""
from __future__ import annotations

import dataclasses

from . import (cache_attention, cache_write, dequant_matmul, factored_supported, gather_columns, hessian_accumulate,
               load, new_cache, pack, pack_permuted, prepare_hinv, prepare_hinv_factored, quantize_layer,
               quantize_layer_factored)
from .kv_cache import FORMATS

LAYERS = ("q", "k", "v", "out", "fc1", "fc2")


@dataclasses.dataclass
class Block:
    """Weights of one block (device tensors, d_out x d_in, fp16/bf16/fp32):
    q, k, v, out: hidden x hidden; fc1: ffn x hidden; fc2: hidden x ffn.
    With attention of fewer kv heads, k and v have kv_heads * head_dim rows."""
    q: object
    k: object
    v: object
    out: object
    fc1: object
    fc2: object


@dataclasses.dataclass
class Attention:
    """Attention inside a block: heads of q; kv_heads of k and v (heads unless
    given); lengths: tokens of each sequence, in the order of X's rows (one
    sequence of all of them unless given); fmt, page_size: the cache's, as in
    new_cache; window: as in cache_attention."""
    heads: int
    kv_heads: int | None = None
    lengths: object = None
    fmt: str = "16bit"
    page_size: int = 64
    window: int = 0


def _torch():
    import torch
    return torch


def _hessian(X):
    torch = _torch()
    d = X.shape[1]
    H = torch.zeros((d, d), dtype=torch.float64, device=X.device)
    hessian_accumulate(H, X)
    return H


def _quantize_shared(Ws: dict, X, cfg, stats: dict | None, want_w_hat: bool = True):
    """Quantize the layers of Ws (all reading X) from one Hessian of X."""
    torch = _torch()
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)] if stats is not None else None
    if ev:
        ev[0].record()
    H = _hessian(X)
    if ev:
        ev[1].record()
    d_in = H.shape[0]
    factored = all(factored_supported(W.shape[0], d_in, cfg) for W in Ws.values())
    perm = (prepare_hinv_factored if factored else prepare_hinv)(H, cfg)
    res = {}
    for name, W in Ws.items():
        out = (quantize_layer_factored if factored else quantize_layer)(W, H, perm, cfg, want_w_hat=want_w_hat)
        out["perm"] = perm
        if cfg.act_order:
            out["packed"] = pack_permuted(out["codes"], cfg.bits, perm)
        else:
            out["packed"] = pack(out["codes"], cfg.bits)
        res[name] = out
    if ev:
        ev[2].record()
        torch.cuda.synchronize()
        stats["hessian_ms"] += ev[0].elapsed_time(ev[1])
        stats["solver_ms"] += ev[1].elapsed_time(ev[2])
    return res


def _product(X, q, cfg, stats: dict | None):
    """X W_hat^T (float32) from the packed layer."""
    torch = _torch()
    if stats is not None:
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
    if cfg.act_order and X.shape[0] >= 128:
        # many tokens: gather once into quantization order, then the matrix-core route
        Y = dequant_matmul(gather_columns(X, q["perm"]), q["packed"], cfg.bits, q["scales"], q["zeros"],
                           group_size=cfg.group_size)
    elif cfg.act_order:
        Y = dequant_matmul(X, q["packed"], cfg.bits, q["scales"], q["zeros"], perm=q["perm"],
                           group_size=cfg.group_size)
    else:
        Y = dequant_matmul(X, q["packed"], cfg.bits, q["scales"], q["zeros"], group_size=cfg.group_size)
    if stats is not None:
        e1.record()
        torch.cuda.synchronize()
        stats["product_ms"] += e0.elapsed_time(e1)
    return Y


def _attention_shape(block: Block, X, attention: Attention):
    """(lengths, kv heads, head_dim), checked against the block and its tokens."""
    n, heads, kv_heads = X.shape[0], attention.heads, attention.kv_heads or attention.heads
    lengths = [n] if attention.lengths is None else [int(k) for k in attention.lengths]
    if sum(lengths) != n or min(lengths, default=0) < 0:
        raise ValueError("attention.lengths must add up to the tokens")
    if heads < 1 or kv_heads < 1 or heads % kv_heads or block.q.shape[0] % heads:
        raise ValueError("attention.heads must divide q's rows, and attention.kv_heads the heads")
    d = block.q.shape[0] // heads
    if d not in (32, 64, 96, 128):
        raise ValueError("head_dim must be 32, 64, 96 or 128")
    if block.k.shape[0] != kv_heads * d or block.v.shape[0] != kv_heads * d:
        raise ValueError("k and v must have kv_heads * head_dim rows")
    if attention.page_size < 1 or not 0 <= attention.window <= 1 << 30:
        raise ValueError("attention.page_size must be positive and attention.window within 0 .. 2^30")
    if attention.fmt not in FORMATS:
        raise ValueError(f"attention.fmt must be one of {', '.join(FORMATS)}")
    if X.dtype not in (_torch().float16, _torch().bfloat16):
        raise ValueError("attention takes tokens of float16 or bfloat16")
    return lengths, kv_heads, d


def _attend(X, res, cfg, attention: Attention, shape, stats: dict | None):
    """Causal attention of the sequences in X by the quantized q, k, v."""
    torch = _torch()
    (lengths, kv_heads, d), n, dt, dev = shape, X.shape[0], X.dtype, X.device
    Q, K, V = (_product(X, res[name], cfg, stats).to(dt) for name in ("q", "k", "v"))
    page = attention.page_size
    pages = [-(-k // page) for k in lengths]
    cache = new_cache(sum(pages), page, kv_heads, d, fmt=attention.fmt, dtype=dt, device=dev)
    # sequence after sequence: its pages in a row, its tokens from the first one's start
    table = torch.zeros((len(lengths), max(pages, default=0)), dtype=torch.int32)
    slots = torch.empty(n, dtype=torch.int64)
    at = first = 0
    for s, (k, m) in enumerate(zip(lengths, pages)):
        table[s, :m] = torch.arange(first, first + m, dtype=torch.int32)
        slots[at: at + k] = torch.arange(first * page, first * page + k)
        at, first = at + k, first + m
    length = torch.tensor(lengths, dtype=torch.int32)
    start = torch.cat([torch.zeros(1, dtype=torch.int32), length.cumsum(0, dtype=torch.int32)])
    if stats is not None:
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
    cache_write(cache, K.unflatten(1, (kv_heads, d)), V.unflatten(1, (kv_heads, d)), slots.to(dev))
    A = cache_attention(Q.unflatten(1, (attention.heads, d)), cache, start.to(dev), length.to(dev), table.to(dev),
                        max_q=max(lengths, default=0), window=attention.window).flatten(1)
    if stats is not None:
        e1.record()
        torch.cuda.synchronize()
        stats["attention_ms"] = stats.get("attention_ms", 0.0) + e0.elapsed_time(e1)
    return A


def quantize_block(block: Block, X, cfg, stats: dict | None = None, want_w_hat: bool = True,
                   attention: Attention | None = None):
    """Quantize one block from its input activations X (tokens x hidden,
    device, fp16/bf16).  Returns (per-layer outputs of quantize_layer plus
    perm and packed, the activations each layer was quantized on, the next
    block's input X').  want_w_hat=False skips the float32 reconstructions
    (4 bytes per weight).  attention: identity unless given (stats then gets
    attention_ms)."""
    dt = X.dtype
    shape = None if attention is None else _attention_shape(block, X, attention)
    res, inputs = {}, {}
    res.update(_quantize_shared({"q": block.q, "k": block.k, "v": block.v}, X, cfg, stats, want_w_hat))
    for n in ("q", "k", "v"):
        inputs[n] = X
    A = _product(X, res["v"], cfg, stats).to(dt) if attention is None else _attend(X, res, cfg, attention, shape, stats)
    inputs["out"] = A
    res.update(_quantize_shared({"out": block.out}, A, cfg, stats, want_w_hat))
    h1f = X.float() + _product(A, res["out"], cfg, stats)
    h1 = h1f.to(dt)
    inputs["fc1"] = h1
    res.update(_quantize_shared({"fc1": block.fc1}, h1, cfg, stats, want_w_hat))
    r = _torch().relu(_product(h1, res["fc1"], cfg, stats)).to(dt)
    inputs["fc2"] = r
    res.update(_quantize_shared({"fc2": block.fc2}, r, cfg, stats, want_w_hat))
    X_next = (h1f + _product(r, res["fc2"], cfg, stats)).to(dt)
    return res, inputs, X_next


def quantize_stack(blocks, X0, cfg, stats: dict | None = None, want_w_hat: bool = True,
                   attention: Attention | None = None):
    """Quantize the blocks in order; block b+1 is calibrated on the output of
    the already-quantized block b.  Returns a list of (outputs, inputs) per
    block and the stack's output activations."""
    load()
    out = []
    X = X0
    for b in blocks:
        res, inputs, X = quantize_block(b, X, cfg, stats, want_w_hat, attention)
        out.append((res, inputs))
    return out, X


def new_stats() -> dict:
    return {"hessian_ms": 0.0, "solver_ms": 0.0, "product_ms": 0.0}


__all__ = ["Attention", "Block", "LAYERS", "quantize_block", "quantize_stack", "new_stats"]
