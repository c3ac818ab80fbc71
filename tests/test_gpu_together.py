"""The microscaled products, the cache and its attention used together, as a
serving program and as the sequential driver use them (needs an MI355X).

Every step is checked against float64 of the tensors it was given, by the
bounds stated in test_gpu_mx.py (products) and test_gpu_cache.py (attention).
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_accum_amd as P
from post_weight_quantization_accum_amd import sequential as S

from test_gpu_cache import Paged, check as check_attention
from test_gpu_mx import _check as check_product

pytestmark = pytest.mark.gpu

DEV = "cuda"


class Layer:
    """Attention of one layer with e2m1 weights over a paged cache."""

    def __init__(self, rng, hidden, heads, kv_heads, d):
        self.heads, self.kv_heads, self.d = heads, kv_heads, d
        self.w = {}
        for name, rows, cols in (("qkv", (heads + 2 * kv_heads) * d, hidden), ("out", hidden, heads * d)):
            W = torch.from_numpy(rng.standard_normal((rows, cols)) * cols ** -0.5).float().to(DEV)
            self.w[name] = P.mx_quantize(W)
            self.w[name + "64"] = P.mx_dequantize(*self.w[name], cols).double().cpu().numpy()

    def __call__(self, X, cache, slots, q_start, kv_len, table, max_q, window=0):
        """New tokens' keys and values into the cache, their attention, the product with out."""
        h, kv, d = self.heads, self.kv_heads, self.d
        self.y = P.mx_matmul(X, *self.w["qkv"])
        qkv = self.y.to(X.dtype)
        self.q = qkv[:, : h * d].unflatten(1, (h, d))
        self.k = qkv[:, h * d: (h + kv) * d].unflatten(1, (kv, d))
        self.v = qkv[:, (h + kv) * d:].unflatten(1, (kv, d))
        P.cache_write(cache, self.k, self.v, slots)
        self.a = P.cache_attention(self.q, cache, q_start, kv_len, table, max_q=max_q, window=window)
        return P.mx_matmul(self.a.flatten(1), *self.w["out"])


@pytest.mark.parametrize("fmt,dtype,window", [("fp4", "bf16", 0), ("fp8", "f16", 0), ("16bit", "bf16", 40)])
def test_prompts_then_decoding(fmt, dtype, window):
    """Prompts of a ragged batch at once, then single tokens, with rows of the batch that hold no sequence."""
    rng = np.random.default_rng(5)
    hidden, heads, kv_heads, d, page, steps = 384, 6, 2, 64, 16, 4
    prompts = [37, 1, 0, 150]
    p = Paged(6, [n + steps if n else 0 for n in prompts], kv_heads, d, page, fmt, dtype, garbage=True)
    layer = Layer(rng, hidden, heads, kv_heads, d)
    table = torch.from_numpy(p.table).to(DEV)
    done = [0] * len(prompts)
    for step in range(1 + steps):
        new = prompts if step == 0 else [int(n > 0) for n in prompts]
        pad = 3                                          # tokens of no sequence behind the batch
        X = torch.from_numpy(rng.standard_normal((sum(new) + pad, hidden))).to(p.dtype).to(DEV)
        rows = np.concatenate([p.start[s] + done[s] + np.arange(n) for s, n in enumerate(new)]).astype(int)
        slots = np.concatenate([p.slots[rows], np.full(pad, -1)])
        done = [a + b for a, b in zip(done, new)]
        start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        kv_len = torch.tensor(done, dtype=torch.int32, device=DEV)
        Y = layer(X, p.cache, torch.from_numpy(slots).to(DEV), start, kv_len, table, max(new), window)
        n = sum(new)
        check_product(layer.y, X.double().cpu().numpy(), layer.w["qkv64"])
        for w, t in ((0, layer.k), (1, layer.v)):
            p.new[w][rows] = t[:n].cpu()
        whole, p.kv = p.kv, done
        now = Paged.__new__(Paged)                       # the positions there so far
        now.__dict__.update(p.__dict__, last=[None, None], known={}, start=np.concatenate([[0], np.cumsum(done)]).astype(int))
        now.new = [torch.cat([t[p.start[s]: p.start[s] + m] for s, m in enumerate(done)]) for t in p.new]
        check_attention(layer.a, layer.q, now, new, d ** -0.5, window)
        got = P.cache_read(p.cache, table, torch.from_numpy(now.start.astype(np.int32)).to(DEV), now.start[-1], dtype=p.dtype)
        assert all(np.array_equal(got[w].double().cpu().numpy(), now.held(w)) for w in (0, 1))
        p.kv = whole
        check_product(Y[:n], layer.a[:n].flatten(1).double().cpu().numpy(), layer.w["out64"])


def test_decoding_captured_and_replayed():
    """One graph for the step: lengths, slots and tokens change in place; each replay equals the eager step."""
    rng = np.random.default_rng(8)
    hidden, heads, kv_heads, d, page, n_seq = 256, 4, 2, 64, 16, 5
    layer = Layer(rng, hidden, heads, kv_heads, d)
    caches = [P.new_cache(n_seq * 4, page, kv_heads, d, fmt="fp8", device=DEV) for _ in range(2)]
    table = torch.from_numpy(rng.permutation(n_seq * 4).reshape(n_seq, 4).astype(np.int32)).to(DEV)
    start = torch.arange(n_seq + 1, dtype=torch.int32, device=DEV)
    kv_len = torch.ones(n_seq, dtype=torch.int32, device=DEV)
    slots = torch.full((n_seq,), -1, dtype=torch.int64, device=DEV)
    X = torch.zeros(n_seq, hidden, dtype=torch.bfloat16, device=DEV)
    layer(X, caches[0], slots, start, kv_len, table, 1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(X, caches[0], slots, start, kv_len, table, 1)
    at = np.array([0, 3, 15, 31, 58])
    for k in range(5):
        kv_len.copy_(torch.from_numpy((at + 1).astype(np.int32)))
        slots.copy_(torch.from_numpy(table.cpu().numpy()[np.arange(n_seq), at // page].astype(np.int64) * page + at % page))
        X.copy_(torch.from_numpy(rng.standard_normal((n_seq, hidden))))
        want = layer(X, caches[1], slots, start, kv_len, table, 1)
        out.fill_(-1.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.isfinite(out).all(), k
        assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v_scales, caches[1].v_scales)
        at = at + 1


@pytest.mark.parametrize("fmt,kv_heads,lengths,window", [("16bit", 2, [300, 1, 0, 211], 0), ("fp8", 4, None, 0),
                                                         ("fp4", 1, [256, 256], 100)])
def test_block_quantized_with_attention(fmt, kv_heads, lengths, window):
    """The sequential driver: out is calibrated on the attention of the quantized q, k, v; the rest as without."""
    rng = np.random.default_rng(9)
    n, hidden, ffn, heads = 512, 256, 512, 4
    d = hidden // heads
    cfg = P.make_config(bits=4, group_size=128, act_order=False, block=128, damp=0.01)
    X = torch.from_numpy(rng.standard_normal((n, hidden))).to(torch.bfloat16).to(DEV)
    rows = dict(q=hidden, k=kv_heads * d, v=kv_heads * d, out=hidden, fc1=ffn, fc2=hidden)
    cols = dict(q=hidden, k=hidden, v=hidden, out=hidden, fc1=hidden, fc2=ffn)
    block = S.Block(**{m: torch.from_numpy(0.05 * rng.standard_normal((rows[m], cols[m]))).to(torch.bfloat16).to(DEV)
                       for m in S.LAYERS})
    att = S.Attention(heads, kv_heads, lengths, fmt=fmt, page_size=48, window=window)
    stats = S.new_stats()
    res, inputs, out = S.quantize_block(block, X, cfg, stats, attention=att)
    assert stats["attention_ms"] > 0
    q, k, v = (S._product(X, res[m], cfg, None).to(torch.bfloat16) for m in "qkv")
    p = Paged(1, lengths or [n], kv_heads, d, 48, fmt, "bf16")
    p.new = [t.unflatten(1, (kv_heads, d)).cpu() for t in (k, v)]
    check_attention(inputs["out"].unflatten(1, (heads, d)), q.unflatten(1, (heads, d)), p, p.kv, d ** -0.5, window)
    # what the other layers see and become, by the same steps as without attention
    A = inputs["out"]
    again = S._quantize_shared({"out": block.out}, A, cfg, None)
    assert torch.equal(again["out"]["codes"], res["out"]["codes"])
    h1 = (X.float() + S._product(A, res["out"], cfg, None)).to(torch.bfloat16)
    assert torch.equal(h1, inputs["fc1"]) and torch.isfinite(out).all()
    stack, last = S.quantize_stack([block], X, cfg, attention=att)
    assert torch.equal(last, out)


def test_two_streams_at_once():
    """Calls that overlap on two streams, with workspaces and outputs of their own, give what they give alone."""
    rng = np.random.default_rng(12)
    work = []
    for i, (fmt, dtype) in enumerate((("fp8", "bf16"), ("fp4", "f16"))):
        p = Paged(20 + i, [9000, 500, 4000], 2, 128, 64, fmt, dtype).write()
        Q = torch.from_numpy(rng.standard_normal((3, 8, 128))).to(p.dtype).to(DEV)
        w = P.mx_quantize(torch.from_numpy(rng.standard_normal((700, 640))).float().to(DEV))
        X = torch.from_numpy(rng.standard_normal((40 + 600 * i, 640))).to(p.dtype).to(DEV)
        work.append((p, Q, p.tensors([1, 1, 1]), w, X))

    def run(item, stream=None):
        p, Q, (start, kv, table), w, X = item
        return (P.cache_attention(Q, p.cache, start, kv, table, max_q=1, stream=stream), P.mx_matmul(X, *w, stream=stream),
                P.mx_matmul_quantized(*P.mx_quantize(X, stream=stream), *w, stream=stream))

    alone = [run(item) for item in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [[] for _ in work]
    for _ in range(5):
        for i, item in enumerate(work):
            got[i].append(run(item, streams[i]))
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, alone[i]))
