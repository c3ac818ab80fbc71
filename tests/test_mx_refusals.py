"""Further refusals of the cache and attention entry points (CPU: no call here reaches a launch)."""
import ctypes

import pytest
import torch

import post_weight_quantization_accum_amd as P
from post_weight_quantization_accum_amd import _lib
from test_mx_oracle import BAD, _attend, _c


def test_scales_outside_their_range():
    """8 / scale and scale * log2(e) are held in float32: neither may overflow."""
    for scale in (2.0 ** -101, 1e-38, 1e-45, 2.0 ** 101, 3e38, -1.0):
        assert _attend(_c(), sc=scale) == BAD, scale
    for scale in (2.0 ** -100, 2.0 ** 100):
        assert _attend(_c(), sc=scale, n=0) == _lib.OK and _attend(_c(), sc=scale, mp=4096) == _lib.ERR_WORKSPACE


def _plan(c, n=4, h=8, ns=2, mp=4, mq=4, w=0):
    plan = (ctypes.c_int64 * 3)(-1, -1, -1)
    st = P.load().gptq_cache_attention_plan(ctypes.byref(c), n, h, ns, mp, mq, w, plan)
    return st, list(plan), P.load().gptq_cache_attention_workspace(ctypes.byref(c), n, h, ns, mp, mq, w)


def test_plan_of_attention():
    assert _plan(_c()) == (_lib.OK, [1, 0, 0], 0)
    assert _plan(_c(), n=0)[1] == _plan(_c(), ns=0)[1] == [0, 0, 0]
    assert _plan(_c(), h=7)[0] == _plan(_c(), mq=-1)[0] == _plan(_c(k=None))[0] == BAD
    assert _plan(_c(d=48))[0] == _lib.ERR_UNSUPPORTED
    assert P.load().gptq_cache_attention_plan(ctypes.byref(_c()), 4, 8, 2, 4, 4, 0, None) == BAD
    st, (few, many, rows), ws = _plan(_c(), mp=4096)               # one launch in parts: every row has room for them
    assert st == _lib.OK and few > 1 and many == 0 and rows == 4 * 8 and ws == few * rows * (64 + 2) * 4


@pytest.mark.parametrize("f,most", [(_lib.MX_NONE, 16), (_lib.MX_FP8, 32), (_lib.MX_FP4, 64)])
def test_parts_beside_a_chunk_need_room_for_few_rows_only(f, most):
    """A decoded token in parts beside a chunk that is whole: the workspace holds what sequences of few rows can have."""
    c = _c(f=f, dt=_lib.BF16, n_pages=2048, page_size=64, n_kv=8, d=128)
    st, (few, many, rows), ws = _plan(c, n=2049, h=32, ns=2, mp=1024, mq=2048)
    assert st == _lib.OK and few > 1 and many == 1
    assert rows == 2 * 8 * most and ws == few * rows * (128 + 2) * 4
    # a million tokens of 32 heads: their rows are no reason to refuse the call
    c = _c(f=f, dt=_lib.BF16, n_pages=1 << 16, page_size=64, n_kv=8, d=32)
    st, (few, many, rows), ws = _plan(c, n=1 << 20, h=32, ns=2, mp=1 << 14, mq=(1 << 20) - 1)
    assert st == _lib.OK and few > 1 and many == 1 and rows == 2 * 8 * most


def test_sequential_attention_refused_before_any_work():
    """A format, type or window that the cache or its attention would refuse after q, k and v are quantized."""
    from post_weight_quantization_accum_amd import sequential as S
    w = lambda r: torch.zeros(r, 256)
    block = S.Block(w(256), w(128), w(128), w(256), w(512), torch.zeros(256, 512))
    for X, kw in ((torch.bfloat16, dict(fmt="int8")), (torch.bfloat16, dict(fmt=None)), (torch.float32, {}),
                  (torch.float32, dict(fmt="fp8")), (torch.float16, dict(window=(1 << 30) + 1))):
        with pytest.raises(ValueError, match="fmt|float16|window"):
            S.quantize_block(block, torch.zeros(10, 256, dtype=X), None, attention=S.Attention(4, 2, **kw))
