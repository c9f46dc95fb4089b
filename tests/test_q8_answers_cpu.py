"""The example layer for several answers, its own side of its calls, on the CPU:
the entry points are replaced by ones that keep their arguments."""
import pytest
import torch

import blas_symmetric_mat_amd as X
from blas_symmetric_mat_amd import q8_layer
from tests.pages_model import Model
from tests.test_q8_layer_cpu import D, F, HEADS, TOKENS, calls, rows  # noqa: F401

ANSWERS, PAGE = 3, 2


def make(tokens=TOKENS, answers=ANSWERS, page=PAGE):
    v = q8_layer.Q8Answers.__new__(q8_layer.Q8Answers)
    v.d, v.heads, v.hd, v.f, v.tokens, v.eps = D, HEADS, D // HEADS, F, tokens, 1e-5
    v.norm1 = v.norm2 = torch.ones((D,), dtype=torch.bfloat16)
    v.wqkv, v.wo, v.wgu, v.wd = rows(3 * D, D), rows(D, D), rows(2 * F, D), rows(D, F)
    v.kv = [(torch.zeros((tokens * HEADS, v.hd), dtype=torch.int8), torch.zeros((tokens * HEADS,)))
            for _ in range(2)]
    v.place = torch.zeros((tokens,), dtype=torch.int32)
    v._pages(answers, page)
    return v


def tokens(m):
    return torch.zeros((m, D), dtype=torch.bfloat16), torch.zeros((m, D), dtype=torch.bfloat16)


def names(made):
    return [name for name, _ in made]


def test_a_step_is_these_calls(calls):  # noqa: F811
    layer = make(tokens=32)
    layer.prompt(*tokens(5))
    layer.fork()
    del calls[:]
    layer.step(*tokens(ANSWERS))
    assert names(calls) == ["xsymv_q8pages_grow", "xsymv_q8norm_b", "xsymv_q8gemm_b", "xsymv_q8pages_slots",
                            "xsymv_q8store_b", "xsymv_q8store_b", "xsymv_q8attn_b", "xsymv_q8store_b",
                            "xsymv_q8gemm_b", "xsymv_q8norm_b", "xsymv_q8gemm_b", "xsymv_q8glu_b", "xsymv_q8gemm_b"]
    attn = dict(calls)["xsymv_q8attn_b"]
    rows_, seqs, start, groups, first, shared = attn[0], attn[6], attn[7], attn[11], attn[12], attn[13]
    assert (rows_, seqs, groups) == (ANSWERS, ANSWERS + 1, 1)
    assert start.tolist() == [0, 0, 1, 2, 3] and first.tolist() == [0, 4]
    assert shared.tolist() == [4]  # the prompt's whole pages of 2 tokens


def test_room(calls):  # noqa: F811
    """4 pages of 2 tokens: a prompt of 3 takes 2, each of 3 answers another for its last token."""
    layer = make()
    layer.prompt(*tokens(3))
    made = len(calls)
    with pytest.raises(ValueError, match="4 pages of 2 tokens: 3 of a prompt and 0 of 3 answers"):
        layer.fork()
    with pytest.raises(ValueError, match="9 of a prompt do not fit"):
        layer.prompt(*tokens(6))
    assert len(calls) == made and not layer.forked
    layer = make(tokens=10)
    layer.prompt(*tokens(3))
    layer.fork()
    layer.step(*tokens(3))  # (fills the last pages)
    made = len(calls)
    with pytest.raises(ValueError, match="2 of 3 answers"):
        layer.step(*tokens(3))
    assert len(calls) == made and layer.more == 1
    layer.free()
    layer.prompt(*tokens(5))
    assert layer.used == 8
    layer = make(tokens=10)  # whole pages: nothing of its own for an answer without tokens
    layer.prompt(*tokens(10))
    layer.fork()
    with pytest.raises(ValueError):
        layer.step(*tokens(3))


def test_order_of_calls(calls):  # noqa: F811
    layer = make(tokens=32)
    for call in (lambda: layer.step(*tokens(3)), layer.free):
        with pytest.raises(ValueError, match="no answers"):
            call()
    layer.prompt(*tokens(1))
    layer.fork()
    for call in (lambda: layer.prompt(*tokens(1)), layer.fork):
        with pytest.raises(ValueError, match="has answers"):
            call()
    for m in (1, 2, 4):
        with pytest.raises(ValueError):
            layer.step(*tokens(m))
    layer.free()
    layer.fork()
    for bad in (dict(answers=0), dict(page=0), dict(page=3)):
        with pytest.raises(ValueError):
            make(**bad)


def test_likely(calls, monkeypatch):  # noqa: F811
    monkeypatch.setattr(X, "xsymv_logp_b", lambda *a: calls.append(("xsymv_logp_b", a)))
    layer = make()
    index, value = layer.likely(*tokens(3), rows(50, D), 7)
    assert index.shape == value.shape == (3, 7)
    assert names(calls) == ["xsymv_q8norm_b", "xsymv_q8gemm_b", "xsymv_logp_b"]
    assert (calls[-1][1][0], calls[-1][1][1], calls[-1][1][3], calls[-1][1][8]) == (3, 50, 50, 7)


@pytest.fixture
def pages(monkeypatch, calls):  # noqa: F811
    """The calls that give and take pages do so, as the model does."""
    def on(cache, name, *lists):
        seqs, length, table, ldt, count, page, refs = cache
        m = Model(seqs, ldt, count, page)
        m.len, m.table, m.refs = length.tolist(), table.tolist(), refs.tolist()
        out = getattr(m, name)(*(v.tolist() for v in lists))
        length.copy_(torch.tensor(m.len)), table.copy_(torch.tensor(m.table)), refs.copy_(torch.tensor(m.refs))
        return out

    monkeypatch.setattr(X, "xsymv_q8pages_grow", lambda n, seq, add, *a: a[-1][:n].copy_(
        torch.tensor(on(a[:-1], "grow", seq[:n], add[:n]))))

    def fork(n, parent, child, *a):
        for to, v in zip(a[-2:], on(a[:-2], "fork", parent[:n], child[:n])):
            to[:n].copy_(torch.tensor(v))
    monkeypatch.setattr(X, "xsymv_q8pages_fork", fork)
    monkeypatch.setattr(X, "xsymv_q8pages_free", lambda n, seq, *a: on(a, "free", seq[:n]))


def test_a_call_that_fails_takes_no_room(pages, monkeypatch):
    """Where a later call cannot be made, pages, lengths and counts are what they were, and the same call works when it
    can: a prompt that ends in a page and between, the fork of it, a step that fills pages and one that begins them."""
    layer = make(tokens=32)

    def state():
        return layer.len.tolist(), layer.refs.tolist(), layer.used, layer.more, layer.forked

    def fails(name, call):
        before = state()
        with monkeypatch.context() as m:
            m.setattr(X, name, lambda *a: (_ for _ in ()).throw(X.XsymvError(name, 1002)))
            for _ in range(2):
                with pytest.raises(X.XsymvError):
                    call()
                assert state() == before
        call()
        assert state() != before

    fails("xsymv_q8attn_b", lambda: layer.prompt(*tokens(1)))
    fails("xsymv_q8glu_b", lambda: layer.prompt(*tokens(4)))
    assert layer.len.tolist()[0] == layer.used == 5 and layer.refs.tolist() == [1] * 3 + [0] * 13
    fails("xsymv_q8pages_copy", layer.fork)
    assert layer.refs.tolist() == [4, 4] + [1] * 4 + [0] * 10
    for name in ("xsymv_q8pages_slots", "xsymv_q8gemm_b", "xsymv_q8norm_b"):
        fails(name, lambda: layer.step(*tokens(ANSWERS)))
    assert layer.more == 3 and layer.len.tolist() == [5, 8, 8, 8] and layer.refs.tolist() == [4, 4] + [1] * 7 + [0] * 7
    layer.free()
    assert layer.refs.tolist() == [1] * 3 + [0] * 13 and layer.len.tolist() == [5, 0, 0, 0]
