"""Attention at scores far from zero (needs an MI355X).

The scores here are sums of products that float32 holds exactly, so that a
weight's exponent, (score - largest) * scale, is all that is computed: off by
at most 3 * 2^-24 of its size (two factors, one product), which is at most
10 where a weight counts, and 2^-22 for the power of two: together less than
2^-19 of the weight.  With eps / 2 half a step of the 16-bit type, and
M = sum_j p_j |v_j|, an output is off by at most
  (2 * 2^-19 + eps / 2 + (n_keys + 64) 2^-23) M + (eps / 2) |o| + 2^-25
(weights rounded to the type, sums in float32, the output's rounding).
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_accum_amd as P
from oracle import mx_oracle as M
from test_gpu_cache import TYPES, Paged, attend

pytestmark = pytest.mark.gpu

# kv lengths, new tokens, heads per kv head: few rows, whole and in parts; many rows, whole and in parts
FORMS = [([300, 70], [1, 3], 4), ([9000, 200], [1, 1], 4), ([300, 64], [150, 64], 2), ([9000], [200], 2)]


def _compare(out, Q, p, q, scale):
    eps = torch.finfo(p.dtype).eps
    at = 0
    for s, n in enumerate(q):
        k, v = (p.held(w)[p.start[s]: p.start[s + 1]] for w in (0, 1))
        o, mag, _ = M.attention(Q[at: at + n].double().cpu().numpy(), k, v, p.kv[s], scale)
        bound = (2.0 ** -18 + eps / 2 + (p.kv[s] + 64) * 2.0 ** -23) * mag + eps / 2 * np.abs(o) + 2.0 ** -25
        got = out[at: at + n].double().cpu().numpy()
        assert np.isfinite(got).all()
        assert (np.abs(got - o) <= bound).all(), (s, np.max(np.abs(got - o) / bound))
        at += n


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kv,q,group", FORMS)
def test_scores_of_billions(kv, q, group, dtype):
    """All scores equal, and one key above the others: means, and that key's value."""
    d, unit = 128, 64.0 if dtype == "f16" else 4096.0
    for a in (129, 131, 135, 141):
        p = Paged(a, kv, 1, d, 64, "16bit", dtype)
        K = torch.full((sum(kv), 1, d), a * unit)
        for s in range(len(kv)):
            K[p.start[s] + kv[s] - 20] = (a + 1) * unit      # some of the tokens of a chunk see it
        Q = torch.full((sum(q), group, d), a * unit, dtype=p.dtype, device="cuda")
        for keys in (torch.full_like(K, a * unit), K):
            p.new[0] = keys.to(p.dtype)
            p.write()
            out, Q, scale = attend(p, q, group, Q=Q)
            _compare(out, Q, p, q, scale)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kv,q,group", FORMS)
def test_close_scores_far_from_zero(kv, q, group, dtype):
    """Scores of 127 * 2^16 + r, r from -8 to 8 along the keys, negative ones too: the weights are those of r alone."""
    d = 128
    for sign in (1.0, -1.0):
        p = Paged(len(kv), kv, 1, d, 64, "16bit", dtype)
        K = torch.full((sum(kv), 1, d), 2.0 ** 7)
        K[..., -1] = torch.cat([torch.linspace(-8, 8, m).round() for m in kv])[:, None]
        p.new[0] = K.to(p.dtype)
        p.write()
        Q = torch.full((sum(q), group, d), sign * 2.0 ** 9, dtype=p.dtype, device="cuda")
        Q[..., -1] = 1.0
        out, Q, _ = attend(p, q, group, Q=Q, scale=0.125)
        _compare(out, Q, p, q, 0.125)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("seqs,new", [(64, 64), (1, 1), (1, 64), (40, 1)])
def test_one_key_and_a_long_tail(seqs, new, dtype):
    """131072 keys: the first outweighs each other one by 2^25 (2^21), all others together weigh 2^-8 (2^-4) of it.

    With w a tail key's weight, N their number and o = (N w - 1) / (1 + N w)
    (values 1 and -1), do <= 2 d(N w): a tail weight is off by half a step, or
    in float16 by half its smallest step, 2^-25 beside a largest weight of 2^7.
    A matrix instruction adds 16 keys to a sum of at most 1 (2^-23 each, it may
    cut), the weights' sum grows by a step of 64 keys at a time (2^-24).
    """
    page, d, kv, heads = 64, 32, 1 << 17, 16
    t = TYPES[dtype]
    eps = torch.finfo(t).eps
    cache = P.new_cache(kv // page, page, 1, d, fmt="16bit", dtype=t, device="cuda")
    cache.v.fill_(1.0)
    cache.v[0, 0, 0] = -1.0
    table = torch.arange(kv // page, dtype=torch.int32, device="cuda").repeat(seqs, 1).contiguous()
    start = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * new
    lens = torch.full((seqs,), kv, dtype=torch.int32, device="cuda")
    Q = torch.zeros(seqs * new, heads, d, dtype=t, device="cuda")
    Q[..., 0] = 1.0
    for top in (17.4375, 15.0):
        cache.k[0, 0, 0, 0] = top
        out = P.cache_attention(Q, cache, start, lens, table, max_q=new, scale=1.0).double().cpu().numpy()
        n = kv - new + np.arange(new, dtype=np.float64)
        w = np.exp(-float(torch.tensor(top).to(t)))
        o = (n * w - 1) / (1 + n * w)
        bound = 2 * n * w * max(eps / 2, 2.0 ** -32 / w if dtype == "f16" else 0.0) + (n / 16 + 64) * 2.0 ** -23 + \
            (n / 64 + 64) * 2.0 ** -24 + eps / 2 * np.abs(o)
        err = np.abs(out.reshape(seqs, new, -1) - o[:, None])
        assert (err <= bound[:, None]).all(), np.max(err / bound[:, None])


@pytest.mark.parametrize("new", [1, 64])
def test_sum_of_weights_beside_a_large_one(new):
    """The keys of the test above with values 1 and 0: o = 1 / (1 + N w), and only the weights' sum can lose any.

    do <= d(N w): n 2^-32 from the weights, (n / 64 + 64) 2^-24 from a sum that grows by a step of 64 keys at a time.
    """
    page, d, kv, heads, seqs = 64, 32, 1 << 17, 16, 64
    cache = P.new_cache(kv // page, page, 1, d, fmt="16bit", dtype=torch.float16, device="cuda")
    cache.v[0, 0, 0] = 1.0
    cache.k[0, 0, 0, 0] = 17.4375
    table = torch.arange(kv // page, dtype=torch.int32, device="cuda").repeat(seqs, 1).contiguous()
    start = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * new
    Q = torch.zeros(seqs * new, heads, d, dtype=torch.float16, device="cuda")
    Q[..., 0] = 1.0
    out = P.cache_attention(Q, cache, start, torch.full((seqs,), kv, dtype=torch.int32, device="cuda"), table, max_q=new, scale=1.0)
    n = kv - new + np.arange(new, dtype=np.float64)
    o = 1 / (1 + n * np.exp(-17.4375))
    bound = n * 2.0 ** -32 + (n / 64 + 64) * 2.0 ** -24 + 2.0 ** -11 * o
    err = np.abs(out.double().cpu().numpy().reshape(seqs, new, -1) - o[:, None])
    assert (err <= bound[:, None]).all(), np.max(err / bound[:, None])


@pytest.mark.parametrize("kv,q,group", FORMS)
@pytest.mark.parametrize("power", [-100, 100])
def test_scales_at_the_ends(kv, q, group, power):
    """Scores that the scale brings down to nothing (means) or up to 2^100 times their size."""
    p = Paged(3, kv, 1, 64, 64, "16bit", "bf16")
    p.new[0] = torch.zeros_like(p.new[0])
    p.new[0][..., 0] = torch.cat([torch.arange(m) % 7 for m in kv])[:, None].to(torch.bfloat16)
    p.write()
    Q = torch.zeros(sum(q), group, 64, dtype=torch.bfloat16, device="cuda")
    Q[..., 0] = 1.0 if power < 0 else 2.0 ** -100
    out, Q, scale = attend(p, q, group, Q=Q, scale=2.0 ** power)
    _compare(out, Q, p, q, scale)


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
@pytest.mark.parametrize("new", [2, 200])
def test_positions_near_two_to_the_31(new, fmt):
    """Two pages that a table repeats 16384 times, and a window: what stands at the last positions that count equals
    what stands a multiple of both pages before; tokens behind are NaN."""
    page, d, heads, last = 1 << 16, 64, 2, (1 << 31) - 4096
    cache = P.new_cache(2, page, 1, d, fmt=fmt, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(new)
    K, V = (torch.randn(2 * page, 1, d, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(2))
    P.cache_write(cache, K, V, torch.arange(2 * page, dtype=torch.int64, device="cuda"))
    table = torch.tensor([0, 1], dtype=torch.int32, device="cuda").repeat(16384)[None].contiguous()
    start = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    Q = torch.randn(new, heads, d, device="cuda", generator=gen).to(torch.bfloat16)

    def at(kv):
        return P.cache_attention(Q, cache, start, torch.tensor([kv], dtype=torch.int32, device="cuda"), table, max_q=new, window=700)

    assert last % (2 * page) > 1000
    near = at(last % (2 * page) + 2 * page)
    assert torch.isfinite(near).all() and torch.equal(at(last), near)
    past = at(last + 1)
    assert past[-1].isnan().all() and torch.isfinite(past[:-1]).all()
    assert at((1 << 31) - 1).isnan().all()
