"""The paged cache and the attention over it against float64 (needs an MI355X).

Writing and reading back are exact.  Attention, with eps / 2 half a step of
the 16-bit type (bf16 2^-8, fp16 2^-11 relative), and for one output channel
o = sum_j p_j v_j, M = sum_j p_j |v_j|:
  scores: d products and sums in float32, each off by at most 2^-23 of
    B = scale * max_j sum_c |q_c k_jc|, the scaling, and the base-2 exponent's
    argument and result: a weight is off by a factor of at most
    1 + 2 (d + 8) 2^-23 (B + 8);
  weights rounded to the 16-bit type for the product: (eps / 2) M, and for
    fp16 weights below 2^-14 2^-25 each, which a whole 2^-20 M covers (they
    are taken relative to a weight of at least 1);
  sums and rescalings in float32: (n_keys + 64) 2^-23 M;
  the output's rounding: (eps / 2) |o|, and fp16's smallest step 2^-25.
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_accum_amd as P
from oracle import mx_oracle as M

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Paged:
    """A batch of sequences with every page's content known in float64."""

    def __init__(self, seed, kv, n_kv, d, page, fmt, dtype, spare=2, garbage=False):
        rng = np.random.default_rng(seed)
        self.rng, self.kv, self.n_kv, self.d, self.page, self.fmt = rng, list(kv), n_kv, d, page, fmt
        self.dtype, self.last = TYPES[dtype], [None, None]
        need = [-(-m // page) for m in kv]
        n_pages = max(1, sum(need) + spare)
        self.cache = P.new_cache(n_pages, page, n_kv, d, fmt=fmt, dtype=self.dtype, device=DEV)
        order = rng.permutation(n_pages)
        self.table = np.full((len(kv), max(1, max(need, default=1))), -1, np.int32)
        at = 0
        for i, m in enumerate(need):
            self.table[i, :m] = order[at: at + m]
            at += m
        if garbage:                                      # NaN in every place that is not written
            for t in (self.cache.k, self.cache.v):
                t.fill_(float("nan") if fmt == "16bit" else 0xFF)
            for t in (self.cache.k_scales, self.cache.v_scales):
                if t is not None:
                    t.fill_(255)
        total = sum(kv)
        scale = np.exp(0.5 * rng.standard_normal((2, 1, n_kv, d)))
        x = rng.standard_normal((2, total, n_kv, d)) * scale
        self.new = [torch.from_numpy(a).to(self.dtype) for a in x]
        seq = np.repeat(np.arange(len(kv)), kv)
        pos = np.concatenate([np.arange(m) for m in kv]) if total else np.zeros(0, int)
        self.slots = self.table[seq, pos // page].astype(np.int64) * page + pos % page
        self.start = np.concatenate(([0], np.cumsum(kv))).astype(int)

    def write(self):
        P.cache_write(self.cache, self.new[0].to(DEV), self.new[1].to(DEV), torch.from_numpy(self.slots).to(DEV))
        return self

    def held(self, which):
        """What the cache should hold of all keys (0) or values (1), in float64, rounded to the dtype as attention reads it."""
        x = self.new[which].double().numpy()
        if self.fmt == "16bit" or x.size == 0:
            return x
        if self.last[which] is not None and np.array_equal(self.last[which][0], x, equal_nan=True):
            return self.last[which][1]
        flat = x.reshape(-1, self.d)
        v = M.mx_values(*M.mx_quantize(flat, self.fmt), self.fmt, self.d)
        self.last[which] = x, torch.from_numpy(v).to(self.dtype).double().numpy().reshape(x.shape)
        return self.last[which][1]

    def tensors(self, q):
        start = np.concatenate(([0], np.cumsum(q))).astype(np.int32)
        return [torch.from_numpy(a).to(DEV) for a in (start, np.array(self.kv, np.int32), self.table)]


def check(out, Q, p, q, scale, window=0):
    """Every sequence's output against float64 within the bound above."""
    eps = torch.finfo(p.dtype).eps
    K, V = p.held(0), p.held(1)
    known = p.__dict__.setdefault("known", {})           # one reference for several runs on the same data
    at = 0
    for s, n in enumerate(q):
        k, v = K[p.start[s]: p.start[s + 1]], V[p.start[s]: p.start[s + 1]]
        key = (id(Q), s, tuple(q), int(p.kv[s]), scale, window)
        if key not in known:
            known[key] = (Q, M.attention(Q[at: at + n].double().cpu().numpy(), k, v, p.kv[s], scale, window))
        o, mag, dot = known[key][1]
        got = out[at: at + n].double().cpu().numpy()
        keys = p.kv[s]
        fact = 2 * (p.d + 8) * 2.0 ** -23 * (scale * dot + 8)
        bound = (fact + eps / 2 + 2.0 ** -20 + (keys + 64) * 2.0 ** -23) * mag + eps / 2 * np.abs(o) * (1 + fact) + 2.0 ** -25
        err = np.abs(got - o)
        assert np.isfinite(got).all()
        assert (err <= bound).all(), f"sequence {s}: off by {np.max(err / np.maximum(bound, 1e-30)):.3g} of the bound"
        at += n


def attend(p, q, heads, window=0, max_q=None, scale=None, Q=None):
    if Q is None:
        Q = torch.from_numpy(p.rng.standard_normal((sum(q), heads, p.d))).to(p.dtype).to(DEV)
    scale = p.d ** -0.5 if scale is None else scale
    start, kv, table = p.tensors(q)
    out = P.cache_attention(Q, p.cache, start, kv, table, max_q=max_q, scale=scale, window=window)
    return out, Q, scale


@pytest.mark.parametrize("fmt", ["16bit", "fp8", "fp4"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("d,n_kv,page", [(32, 1, 1), (64, 3, 16), (96, 2, 7), (128, 2, 64)])
def test_written_and_read_back(d, n_kv, page, dtype, fmt):
    p = Paged(d + page, [1, 0, 45, 130], n_kv, d, page, fmt, dtype, garbage=True).write()
    rows = p.start[-1] + 3
    start = torch.from_numpy(p.start.astype(np.int32)).to(DEV)
    for dt in (p.dtype, torch.float32):
        out = tuple(torch.full((rows, n_kv, d), 7.0, dtype=dt, device=DEV) for _ in range(2))
        got = P.cache_read(p.cache, torch.from_numpy(p.table).to(DEV), start, rows, out=out)
        for w in range(2):
            assert np.array_equal(got[w][:-3].double().cpu().numpy(), p.held(w))
            assert (got[w][-3:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["16bit", "fp8", "fp4"])
def test_skipped_slots_and_strided_rows(fmt):
    """Slots outside the cache write nothing; keys and values may be slices of one fused, unaligned matrix."""
    n_kv, d, page, n = 2, 64, 8, 20
    cache = P.new_cache(4, page, n_kv, d, fmt=fmt, device=DEV)
    rng = np.random.default_rng(3)
    fused = torch.from_numpy(rng.standard_normal((n, 1 + 2 * n_kv * d + 5))).to(torch.bfloat16).to(DEV)
    K = fused[:, 1: 1 + n_kv * d].unflatten(1, (n_kv, d))
    V = fused[:, 1 + n_kv * d: 1 + 2 * n_kv * d].unflatten(1, (n_kv, d))
    slots = rng.permutation(32)[:n].astype(np.int64)
    slots[3], slots[7], slots[9] = -1, 32, 1 << 40
    P.cache_write(cache, K, V, torch.from_numpy(slots).to(DEV))
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    got = P.cache_read(cache, table, torch.tensor([0, 32], dtype=torch.int32, device=DEV), 32, dtype=torch.float32)
    for t, x in zip(got, (K, V)):
        want = np.zeros((32, n_kv, d))
        for i, s in enumerate(slots):
            if 0 <= s < 32:
                v = x[i].double().cpu().numpy()
                want[s] = v if fmt == "16bit" else M.mx_values(*M.mx_quantize(v, fmt), fmt, d)
        assert np.array_equal(t.double().cpu().numpy(), want)


def test_read_of_bad_pages_is_nan():
    p = Paged(1, [20], 1, 64, 8, "fp8", "bf16").write()
    table = torch.tensor([[int(p.table[0, 0]), 999, -5]], dtype=torch.int32, device=DEV)
    K, V = P.cache_read(p.cache, table, torch.tensor([0, 30], dtype=torch.int32, device=DEV), 30)
    for t, w in ((K, 0), (V, 1)):
        assert np.array_equal(t[:8].double().cpu().numpy(), p.held(w)[:8]) and t[8:].isnan().all()


KINDS = [  # kv lengths, new tokens, kv heads, group, head dim, page
    ([1], [1], 1, 1, 64, 16),
    ([33, 1, 100], [1, 1, 1], 2, 4, 128, 16),
    ([70, 5, 64, 31], [3, 5, 0, 31], 2, 2, 64, 7),
    ([200, 150], [40, 150], 1, 4, 128, 20),
    ([257, 64, 300], [100, 1, 129], 2, 3, 96, 1),
    ([90, 10], [2, 2], 1, 24, 32, 100),
    ([513], [513], 2, 1, 128, 64),
    ([400, 0, 2], [1, 0, 2], 4, 8, 64, 32),
]


@pytest.mark.parametrize("fmt", ["16bit", "fp8", "fp4"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(KINDS)))
def test_attention(case, dtype, fmt):
    kv, q, n_kv, group, d, page = KINDS[case]
    p = Paged(case, kv, n_kv, d, page, fmt, dtype, garbage=True).write()
    for window in (0, 1, 37):
        out, Q, scale = attend(p, q, n_kv * group, window)
        check(out, Q, p, q, scale, window)


@pytest.mark.parametrize("fmt", ["16bit", "fp8", "fp4"])
@pytest.mark.parametrize("q", [1, 4, 200])
def test_long_sequences_in_parts(q, fmt):
    """Tables wide enough that the keys are cut into parts, with sequences much shorter than the table as well."""
    kv = [9000, 40, 3000]
    p = Paged(q, kv, 2, 128, 64, fmt, "bf16", garbage=True).write()
    qs = [q, min(q, 40), q]
    out, Q, scale = attend(p, qs, 8, max_q=q)
    check(out, Q, p, qs, scale)
    # whatever the hint says, every sequence is computed
    for hint in (0, 1, 16, 17, 1000):
        other, _, _ = attend(p, qs, 8, max_q=hint, Q=Q)
        check(other, Q, p, qs, scale)
    out, Q, scale = attend(p, qs, 8, window=2500, Q=Q)
    check(out, Q, p, qs, scale, 2500)


@pytest.mark.parametrize("big", [0.0, 30.0])
def test_large_and_flat_scores(big):
    """Scores that grow along the keys (the maximum moves at every step), and all equal ones."""
    p = Paged(4, [700, 300], 1, 64, 16, "16bit", "f16")
    ramp = torch.linspace(0, 1, 1000)[:, None, None]
    p.new[0] = (ramp * big * torch.ones(1000, 1, 64) / 64 * 8).to(torch.float16)
    p.write()
    Q = torch.ones(2 + 150, 4, 64, dtype=torch.float16, device=DEV)
    out, Q, scale = attend(p, [2, 150], 4, scale=1.0, Q=Q)
    check(out, Q, p, [2, 150], 1.0)


@pytest.mark.parametrize("fmt", ["16bit", "fp8"])
@pytest.mark.parametrize("q", [4, 150])
@pytest.mark.parametrize("window", [0, 9])
def test_what_a_token_does_not_see_has_no_influence(q, fmt, window):
    """Infinities and NaN in keys and values of later tokens (and of those behind the window) reach only the tokens that see them."""
    kv, at = 200, 200 - q + q // 2
    p = Paged(q, [kv, 64], 2, 64, 16, fmt, "bf16", garbage=True)
    p.new[1][at, 0, 5] = float("inf")
    p.new[0][at, 1, 3] = float("nan")
    p.write()
    Q = torch.from_numpy(p.rng.standard_normal((q + 1, 4, 64))).to(p.dtype).to(DEV)
    out, Q, scale = attend(p, [q, 1], 4, window=window, Q=Q)
    pos = np.arange(kv - q, kv)
    sees = (pos >= at) & ((pos - at < window) if window else True)
    got = out[:q].double().cpu().numpy()
    hit = [5] if fmt == "16bit" else list(range(32))        # a microscaled block is lost as a whole
    assert not np.isfinite(got[sees][:, :2][:, :, hit]).any() and np.isnan(got[sees][:, 2:]).all()
    # the others equal what they are without the offending token
    p.new[1][at, 0, 5], p.new[0][at, 1, 3] = 0.0, 0.0
    p.write()
    clean, _, _ = attend(p, [q, 1], 4, window=window, Q=Q)
    keep = np.concatenate((~sees, [True]))
    assert torch.equal(out.cpu()[keep], clean.cpu()[keep])


def test_bad_pages_and_short_tables():
    q = [3, 100]
    p = Paged(9, [60, 160], 1, 64, 16, "fp8", "bf16").write()
    good, Q, scale = attend(p, q, 2)
    p.table[0, 0] = 1 << 20                                  # every token sees it
    p.table[1, 6] = -7                                       # positions 96 .. 111
    out, _, _ = attend(p, q, 2, Q=Q)
    assert out[:3].isnan().all()
    pos = torch.arange(60, 160)
    assert out[3:][pos >= 96].isnan().all() and torch.equal(out[3:][pos < 96], good[3:][pos < 96])
    p.table = p.table[:, :5]                                 # 80 positions: later tokens are past the table
    p.table[0, 0] = 0
    out, _, _ = attend(p, q, 2, Q=Q)
    assert out[3:][pos >= 80].isnan().all() and torch.equal(out[3:][pos < 80], good[3:][pos < 80])


@pytest.mark.parametrize("q", [[2, 0, 3], [40, 0, 60]])
def test_tokens_that_see_nothing_and_rows_behind_the_last_sequence(q):
    """More new tokens than positions: the first ones stand before position 0.  Rows outside the sequences stay as they were."""
    kv = [1, 0, q[2] - 1]
    p = Paged(2, kv, 1, 64, 16, "fp4", "bf16", garbage=True).write()
    n = sum(q)
    Q = torch.from_numpy(p.rng.standard_normal((n + 7, 2, 64))).to(p.dtype).to(DEV)
    start, kvl, table = p.tensors(q)
    out = torch.full((n + 7, 2, 64), 3.0, dtype=p.dtype, device=DEV)
    P.cache_attention(Q[:], p.cache, start + 2, kvl, table, out=out)
    assert (out[:2] == 3).all() and (out[n + 2:] == 3).all()
    check(out[2: n + 2], Q[2: n + 2], p, q, 64 ** -0.5)
    assert (out[2: 2 + q[0] - 1] == 0).all()


def test_strided_and_unaligned_queries_and_outputs():
    p = Paged(6, [100, 50], 2, 64, 16, "fp8", "f16").write()
    for q in ([1, 1], [70, 20]):
        n = sum(q)
        fused = torch.from_numpy(p.rng.standard_normal((n, 3 + 4 * 64 + 6))).to(p.dtype).to(DEV)
        room = torch.full((n, 5 + 4 * 64 + 2), 9.0, dtype=p.dtype, device=DEV)
        start, kv, table = p.tensors(q)
        for at in (3, 0):
            Q = fused[:, at: at + 256].unflatten(1, (4, 64))
            out = room[:, at: at + 256].unflatten(1, (4, 64))
            P.cache_attention(Q, p.cache, start, kv, table, out=out)
            check(out, Q, p, q, 64 ** -0.5)
            out.fill_(9.0)
            assert (room == 9.0).all()


def test_step_of_a_decoder_captured_and_replayed():
    """write, attend, on a stream of its own and in a graph, replayed with other lengths and a padded batch."""
    p = Paged(8, [300, 40, 77, 5], 2, 128, 16, "fp8", "bf16").write()
    heads, n = 8, 4
    start, kv, table = p.tensors([1, 1, 1, 1])
    wide = torch.cat((table, torch.full((4, 500), -1, dtype=torch.int32, device=DEV)), 1).contiguous()
    Q = torch.zeros(n, heads, 128, dtype=p.dtype, device=DEV)
    K, V = (torch.zeros(n, 2, 128, dtype=p.dtype, device=DEV) for _ in range(2))
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    lens = kv.clone()

    def step():
        P.cache_write(p.cache, K, V, slots)
        return P.cache_attention(Q, p.cache, start, lens, wide, max_q=1)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for k in range(4):
        new = np.array([[300 - k, 40, 77, 5], [12, 40, 1, 0]][k % 2])
        lens.copy_(torch.from_numpy(new.astype(np.int32)))
        s = np.where(new > 0, p.table[np.arange(4), np.maximum(new - 1, 0) // 16].astype(np.int64) * 16 + (new - 1) % 16, -1)
        slots.copy_(torch.from_numpy(s))
        for t in (Q, K, V):
            t.copy_(torch.from_numpy(p.rng.standard_normal(tuple(t.shape))))
        out.fill_(5.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            want = step()
        side.synchronize()
        assert torch.equal(got, want), k
        for i in range(4):
            if new[i]:
                at = p.start[i] + new[i] - 1
                p.new[0][at], p.new[1][at] = K[i].cpu(), V[i].cpu()
        q = Paged.__new__(Paged)
        q.__dict__.update(p.__dict__, known={})
        q.kv = list(new)
        check(got, Q, q, [1] * 4, 128 ** -0.5)
        assert (got[new == 0] == 0).all() if (new == 0).any() else True


def test_pages_past_4_gib():
    n_kv, d, page = 4, 128, 64
    n_pages = (1 << 25) // (n_kv * page) + 70               # 128 bytes a row: beyond 2^32
    cache = P.KVCache(*(torch.empty((n_pages, n_kv, page, d), dtype=torch.uint8, device=DEV) for _ in range(2)),
                      *(torch.empty((n_pages, n_kv, page, 4), dtype=torch.uint8, device=DEV) for _ in range(2)), "fp8")
    assert cache.k.numel() > 1 << 32
    p = Paged(11, [150, 100], n_kv, d, page, "fp8", "bf16")
    p.cache, p.table = cache, np.array([[n_pages - 1, 0, n_pages - 3], [n_pages - 2, 3, -1]], np.int32)
    seq, pos = np.repeat([0, 1], p.kv), np.concatenate([np.arange(m) for m in p.kv])
    p.slots = p.table[seq, pos // page].astype(np.int64) * page + pos % page
    p.write()
    for q in ([1, 1], [80, 60]):
        out, Q, scale = attend(p, q, 8)
        check(out, Q, p, q, scale)
    K, V = P.cache_read(cache, torch.from_numpy(p.table).to(DEV), torch.tensor([0, 150, 250], dtype=torch.int32, device=DEV), 250)
    assert np.array_equal(K.double().cpu().numpy(), p.held(0)) and np.array_equal(V.double().cpu().numpy(), p.held(1))


def test_python_refusals():
    p = Paged(1, [20], 2, 64, 16, "fp8", "bf16").write()
    start, kv, table = p.tensors([1])
    Q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    ok = dict(q_start=start, kv_len=kv, table=table)
    for exc, kw in ((TypeError, dict(q_start=start.long())), (TypeError, dict(kv_len=kv[:0])), (TypeError, dict(table=table[0])),
                    (P.InvalidArgument, dict(window=-1)), (TypeError, dict(out=torch.zeros(1, 4, 64, device=DEV)))):
        with pytest.raises(exc):
            P.cache_attention(Q, p.cache, **{**ok, **kw})
    with pytest.raises(ValueError):
        P.cache_attention(Q[..., :32], p.cache, **ok)
    with pytest.raises(P.InvalidArgument):
        P.cache_attention(Q[:, :3], p.cache, **ok)
    with pytest.raises(P.InvalidArgument):
        P.cache_attention(Q.float(), p.cache, **ok)
    with pytest.raises(ValueError):
        P.cache_attention(Q, p.cache, start.cpu(), kv, table)
    half = P.new_cache(4, 16, 2, 64, fmt="16bit", dtype=torch.float16, device=DEV)
    with pytest.raises(P.InvalidArgument):
        P.cache_attention(Q, half, **ok)
    with pytest.raises(P.WorkspaceError):
        P.cache_attention(Q, p.cache, start, kv, table.repeat(1, 3000).contiguous(), max_q=1,
                          workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        P.cache_write(p.cache, Q[:, :2], Q[:, :2], start)
    with pytest.raises(P.Unsupported):
        P.cache_write(P.new_cache(2, 16, 1, 160, device=DEV), torch.zeros(1, 1, 160, device=DEV),
                      torch.zeros(1, 1, 160, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV))


@pytest.mark.parametrize("n_seq", [1, 2, 62, 63, 64, 65, 300, 5000])
def test_read_of_many_sequences(n_seq):
    """Empty, short and long sequences in any number, rows before the first and behind the last left alone."""
    rng = np.random.default_rng(n_seq)
    n_kv, d, page = 1, 32, 4
    n = rng.choice([0, 1, 2, 9], n_seq, p=[0.5, 0.2, 0.2, 0.1])
    n[rng.integers(0, n_seq)] = 37
    start = 5 + np.concatenate([[0], np.cumsum(n)])
    pages = rng.permutation(n_seq * 10)
    cache = P.new_cache(n_seq * 10, page, n_kv, d, fmt="fp8", device=DEV)
    table = pages.reshape(n_seq, 10).astype(np.int32)
    X = torch.from_numpy(rng.standard_normal((start[-1] - 5, n_kv, d))).to(torch.bfloat16).to(DEV)
    slots = np.concatenate([table[i, np.arange(k) // page].astype(np.int64) * page + np.arange(k) % page for i, k in enumerate(n)])
    P.cache_write(cache, X, -X, torch.from_numpy(slots).to(DEV))
    out = tuple(torch.full((start[-1] + 6, n_kv, d), 7.0, device=DEV) for _ in range(2))
    K, V = P.cache_read(cache, torch.from_numpy(table).to(DEV), torch.from_numpy(start.astype(np.int32)).to(DEV), len(out[0]), out=out)
    want = M.mx_values(*M.mx_quantize(X[:, 0].double().cpu().numpy(), "fp8"), "fp8", d)[:, None]
    for t, w in ((K, want), (V, -want)):
        assert np.array_equal(t[5:-6].double().cpu().numpy(), w)
        assert (t[:5] == 7.0).all() and (t[-6:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["16bit", "fp8", "fp4"])
@pytest.mark.parametrize("q", [8, 9, 12, 13, 16, 17, 40])
def test_rows_around_the_kernels_limits(q, fmt):
    """32, 48 and 64 rows of a sequence and one more token, whole and in parts, with shorter sequences beside them."""
    for kv in ([q + 3, 70, q], [2500, 40, q]):
        p = Paged(q, kv, 1, 128, 16, fmt, "bf16", garbage=True).write()
        qs = [q, 3, q]
        out, Q, scale = attend(p, qs, 4, max_q=q)
        check(out, Q, p, qs, scale)


def test_long_sequences_captured_and_replayed():
    """Parts and their join in a graph: lengths change between replays, other work runs in between."""
    p = Paged(4, [6000, 100, 3000], 2, 128, 64, "fp8", "bf16").write()
    start, kv, table = p.tensors([1, 1, 1])
    Q = torch.from_numpy(p.rng.standard_normal((3, 8, 128))).to(torch.bfloat16).to(DEV)
    P.cache_attention(Q, p.cache, start, kv, table, max_q=1)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = P.cache_attention(Q, p.cache, start, kv, table, max_q=1)
        graphs.append((g, out))
    for lengths in ([6000, 100, 3000], [1, 0, 2999], [4097, 64, 65], [0, 0, 0]):
        kv.copy_(torch.tensor(lengths, dtype=torch.int32))
        want = P.cache_attention(Q, p.cache, start, kv, table, max_q=1)
        for _, out in graphs:
            out.fill_(9.0)
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out in graphs), lengths
