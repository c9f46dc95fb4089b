"""The example layer's own side of its calls, on the CPU: the library's entry
points are replaced by ones that write down their arguments and check every
address against the tensor it belongs to."""
import pytest
import torch

import blas_symmetric_mat_amd as X
from blas_symmetric_mat_amd import q8_layer

D, HEADS, F, TOKENS = 32, 2, 48, 8


def rows(n, k):
    w = q8_layer.Q8Weight.__new__(q8_layer.Q8Weight)
    w.n, w.k = n, k
    w.codes, w.scale = torch.zeros((n, k), dtype=torch.int8), torch.ones((n,))
    return w


@pytest.fixture
def layer():
    """A layer whose tensors are on the CPU."""
    v = q8_layer.Q8Layer.__new__(q8_layer.Q8Layer)
    v.d, v.heads, v.hd, v.f, v.tokens, v.eps, v.used = D, HEADS, D // HEADS, F, TOKENS, 1e-5, 0
    v.norm1 = v.norm2 = torch.ones((D,), dtype=torch.bfloat16)
    v.wqkv, v.wo, v.wgu, v.wd = rows(3 * D, D), rows(D, D), rows(2 * F, D), rows(D, F)
    v.kv = [(torch.zeros((TOKENS * HEADS, v.hd), dtype=torch.int8), torch.zeros((TOKENS * HEADS,)))
            for _ in range(2)]
    v.place = torch.randperm(TOKENS, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    return v


@pytest.fixture
def calls(monkeypatch):
    made = []

    def stand_in(name):
        def call(*a, **kw):
            made.append((name, a))
            if "q8store" in name or "q8read" in name:
                slot = a[4] if "store" in name else a[5]
                assert slot is None or slot.numel() >= a[0], f"{name}: {a[0]} rows, {slot.numel()} slots"
        return call

    for name in X.__all__:
        if name.startswith("xsymv_q8"):
            monkeypatch.setattr(X, name, stand_in(name))
    return made


def tokens(m):
    return torch.zeros((m, D), dtype=torch.bfloat16), torch.zeros((m, D), dtype=torch.bfloat16)


def test_a_full_cache_takes_no_more(layer, calls):
    """The last token that fits is taken; one more is refused before any call
    is made, and leaves the layer as it was."""
    layer(*tokens(5))
    layer(*tokens(3))
    assert layer.used == TOKENS
    made = len(calls)
    for m in (1, 5, TOKENS + 1):
        with pytest.raises(ValueError, match="8 tokens, 8 are there"):
            layer(*tokens(m))
        assert len(calls) == made and layer.used == TOKENS


def test_a_prompt_longer_than_the_cache(layer, calls):
    with pytest.raises(ValueError):
        layer(*tokens(TOKENS + 1))
    assert not calls and layer.used == 0
    layer(*tokens(TOKENS))
    assert layer.used == TOKENS


def test_a_call_that_fails_takes_no_room(layer, calls, monkeypatch):
    def fails(*a):
        raise X.XsymvError("xsymv_q8glu_b", 1002)

    monkeypatch.setattr(X, "xsymv_q8glu_b", fails)
    with pytest.raises(X.XsymvError):
        layer(*tokens(2))
    assert layer.used == 0


def test_rows_at_a_stride_are_read_there(layer, calls):
    """x the left half of wider rows, r every second row: the norm is given
    their strides, and a single row's own length."""
    wide = torch.zeros((3, 2 * D), dtype=torch.bfloat16)
    every = torch.zeros((6, D), dtype=torch.bfloat16)[::2]
    layer(wide[:, :D], every)
    layer(wide[:1, D:], every[:1].expand(1, D))
    norms = [a for name, a in calls if name == "xsymv_q8norm_b"]
    assert [(a[3], a[6], a[11]) for a in norms[0::2]] == [(2 * D, 2 * D, D), (D, D, D)]


@pytest.mark.parametrize("which", ["x", "r"])
def test_other_tensors_are_refused(layer, calls, which):
    good = torch.zeros((3, D), dtype=torch.bfloat16)
    for bad in (good.float(), good.half(), good[:, :D - 1], good[:2, None], good.flatten(),
                torch.zeros((D, 3), dtype=torch.bfloat16).t(), good[:1].expand(3, D),
                good.to("meta")):
        x, r = (bad, good) if which == "x" else (good, bad)
        with pytest.raises(ValueError):
            layer(x, r)
    with pytest.raises(ValueError):
        layer(*((good[:2], good) if which == "x" else (good, good[:2])))
    assert not calls and layer.used == 0
