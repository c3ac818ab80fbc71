"""Attention where both kernels run in one call (needs an MI355X); bounds as in test_gpu_cache.py."""
import ctypes

import numpy as np
import pytest
import torch

import post_weight_quantization_accum_amd as P
from post_weight_quantization_accum_amd import _lib
from post_weight_quantization_accum_amd.kv_cache import _cache
from oracle import mx_oracle as M
from test_gpu_cache import Paged, attend

pytestmark = pytest.mark.gpu


def plan(p, q, heads, max_q, window=0):
    out = (ctypes.c_int64 * 3)()
    st = P.load().gptq_cache_attention_plan(_cache(p.cache)[0], sum(q), heads, len(q), p.table.shape[1], max_q, window, out)
    assert st == _lib.OK
    return list(out)


def check_tokens(out, Q, p, q, scale, which):
    """The tokens which[s] of sequence s, each by itself, against float64."""
    eps = torch.finfo(p.dtype).eps
    K, V = p.held(0), p.held(1)
    at = 0
    for s, n in enumerate(q):
        for i in which[s]:
            keys = p.kv[s] - n + i + 1
            k, v = (x[p.start[s]: p.start[s] + keys] for x in (K, V))
            o, mag, dot = M.attention(Q[at + i: at + i + 1].double().cpu().numpy(), k, v, keys, scale)
            fact = 2 * (p.d + 8) * 2.0 ** -23 * (scale * dot + 8)
            bound = (fact + eps / 2 + keys * 2.0 ** -32 + (keys + 64) * 2.0 ** -23) * mag + eps / 2 * np.abs(o) * (1 + fact) + 2.0 ** -25
            err = np.abs(out[at + i: at + i + 1].double().cpu().numpy() - o)
            assert (err <= bound).all(), (s, i, np.max(err / bound))
        at += n


@pytest.mark.parametrize("fmt,dtype,long", [("16bit", "bf16", 12000), ("16bit", "f16", 12000), ("fp4", "bf16", 5000), ("fp8", "f16", 5000)])
def test_a_chunk_beside_decoded_tokens_in_parts(fmt, dtype, long):
    kv, q = [long, 2100], [1, 2048]
    p = Paged(3, kv, 8, 128, 64, fmt, dtype, garbage=True).write()
    p.table = np.concatenate((p.table, np.full((2, 1024 - p.table.shape[1]), -1, np.int32)), 1)
    few, many, rows = plan(p, q, 32, 2048)
    assert few > 1 and many == 1 and rows < sum(q) * 32
    for order in ([0, 1], [1, 0]):
        p.kv, p.table, q = [p.kv[i] for i in order], np.ascontiguousarray(p.table[order]), [q[i] for i in order]
        old = p.start
        p.start = np.concatenate(([0], np.cumsum(p.kv))).astype(int)
        if order[0]:
            p.new = [torch.cat([x[old[i]: old[i + 1]] for i in order]) for x in p.new]
            p.last = [None, None]
        out, Q, scale = attend(p, q, 32, max_q=2048)
        check_tokens(out, Q, p, q, scale, [[0, n // 2, n - 2, n - 1] if n > 1 else [0] for n in q])
        again, _, _ = attend(p, q, 32, max_q=2048, Q=Q)
        assert torch.equal(out, again)


def test_workspace_that_is_not_as_large_as_it_says():
    """A tensor that repeats its elements has fewer bytes than its shape tells."""
    p = Paged(1, [20], 2, 64, 16, "fp8", "bf16").write()
    start, kv, table = p.tensors([1])
    table = table.repeat(1, 3000).contiguous()
    Q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    need = P.load().gptq_cache_attention_workspace(_cache(p.cache)[0], 1, 4, 1, table.shape[1], 1, 0)
    assert need > 0
    for bad in (torch.zeros(1, dtype=torch.uint8, device="cuda").expand(need), torch.zeros(2, need, dtype=torch.uint8, device="cuda")[:, ::2]):
        with pytest.raises(TypeError):
            P.cache_attention(Q, p.cache, start, kv, table, max_q=1, workspace=bad)
    good = torch.zeros(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(P.cache_attention(Q, p.cache, start, kv, table, max_q=1, workspace=good), P.cache_attention(Q, p.cache, start, kv, table, max_q=1))


@pytest.mark.parametrize("starts", [[0, 200, 50, 250], [250, 0, 240, 10], [0, 150, 0, 0], [-5, 300, 100, 1 << 30]])
def test_starts_that_do_not_ascend_touch_nothing_else(starts):
    """Tiles are found by searching the starts: whatever is found, rows stay within the call's tokens."""
    p = Paged(4, [300, 280, 260], 2, 64, 16, "fp8", "bf16").write()
    n, heads = 250, 8
    room = torch.full((n + 40, heads, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    Q = torch.randn(n, heads, 64, device="cuda").to(torch.bfloat16)
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    _, kv, table = p.tensors([1, 1, 1])
    for wide in (table, torch.cat((table, torch.full((3, 900), -1, dtype=torch.int32, device="cuda")), 1).contiguous()):
        for max_q in (1, 200):
            P.cache_attention(Q, p.cache, start, kv, wide, max_q=max_q, out=room[20: 20 + n])
            torch.cuda.synchronize()
            assert (room[:20] == 9.0).all() and (room[20 + n:] == 9.0).all()


@pytest.mark.parametrize("fmt", ["16bit", "fp8", "fp4"])
@pytest.mark.parametrize("q", [4, 5, 8, 9, 16, 17])
def test_rows_at_each_limit(q, fmt):
    """16, 32 and 64 rows and a token more: the last of the few-row kernel and the first of the other, whole and in parts."""
    for kv in ([q + 3, 70, q], [2500, 40, q]):
        p = Paged(q, kv, 1, 64, 16, fmt, "f16", garbage=True).write()
        qs = [q, 3, q]
        few, many, _ = plan(p, qs, 4, q)
        assert (many > 0) == (4 * q > {"16bit": 16, "fp8": 32, "fp4": 64}[fmt])
        out, Q, scale = attend(p, qs, 4, max_q=q)
        check_tokens(out, Q, p, qs, scale, [range(n) for n in qs])
