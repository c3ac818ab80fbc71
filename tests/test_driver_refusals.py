"""Norms and attention that the sequential driver refuses before it quantizes anything (CPU)."""
import pytest
import torch

from post_weight_quantization_accum_amd import sequential as S


def block(**kw):
    w = lambda r, c=256: torch.zeros(r, c)
    return S.Block(*[w(256) for _ in range(4)], w(512), w(256, 512), **kw)


@pytest.mark.parametrize("name", ["norm1", "bias1", "post1", "norm2", "bias2", "post2"])
def test_norms_elsewhere(name):
    """Norms on another device than the tokens: the later ones would be met after q, k and v are quantized."""
    v = dict(norm1=torch.ones(256), norm2=torch.ones(256))
    v[name] = torch.ones(256, device="meta")
    with pytest.raises(ValueError, match=f"{name} must live"):
        S.quantize_block(block(**v), torch.zeros(10, 256), None)


def test_later_blocks(monkeypatch):
    """A stack whose later block cannot be run: nothing of the earlier ones is quantized."""
    ran = []
    monkeypatch.setattr(S, "quantize_block", lambda b, X, *a: ran.append(b) or ({}, {}, X))
    v = torch.ones(256)
    X, normed = torch.zeros(10, 256).half(), dict(norm1=v, norm2=v)
    for kw, norms, attention, what in ((dict(), S.Norms(), None, "no norm1"), (dict(norm1=v), None, None, "norm1 and norm2"),
                                       (dict(normed, post2=v[:128]), None, None, "post2"),
                                       (dict(normed, k=torch.zeros(128, 256)), None, S.Attention(heads=4), "rows")):
        first, last = block(**normed), block(**{n: t for n, t in kw.items() if n != "k"})
        last.k = kw.get("k", last.k)
        for stack in ([first, last], (first, first, last)):
            with pytest.raises(ValueError, match=what):
                S.quantize_stack(stack, X, None, attention=attention, norms=norms)
    assert not ran
    # blocks that come one after the other are met one after the other
    assert len(S.quantize_stack((block() for _ in range(3)), X, None)[0]) == 3 and len(ran) == 3
