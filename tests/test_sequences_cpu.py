"""Attention over pages, calls on pages and log probabilities: refusals, in the order of the arguments and
before any device work, through both ways of calling; workspaces; and the pages' model on cases by hand."""
import pytest

import blas_symmetric_mat_amd as X
from tests.pages_model import Model

P = 4096  # an address

GOOD = {
    "attn": dict(rows=3, heads=8, kvheads=2, hd=64, q=P, ldq=512, seqs=3, start=None, len=P, table=P, ldt=4, groups=1,
                 first=P, shared=P, k=P, ldk=64, ks=P, v=P, ldv=64, vs=P, pages=10, ps=16, scale=0.125, out=P, ldo=512,
                 lse=P),
    "logp": dict(m=2, n=100, x=P, ldx=100, token=P, logp=P, entropy=P, lse=P, top=5, index=P, value=P, ldt=5),
    "grow": dict(n=2, seq=P, add=P, seqs=3, len=P, table=P, ldt=4, pages=10, ps=16, refs=P, got=P),
    "slots": dict(rows=3, kvheads=2, start=P, seqs=3, len=P, table=P, ldt=4, pages=10, ps=16, slot=P),
    "fork": dict(n=2, parent=P, child=P, seqs=3, len=P, table=P, ldt=4, pages=10, ps=16, refs=P, src=P, dst=P),
    "free": dict(n=2, seq=P, seqs=3, len=P, table=P, ldt=4, pages=10, ps=16, refs=P),
    "compact": dict(seqs=3, table=P, ldt=4, out=2 * P, ldo=4, pages=10, refs=P, rout=P, src=P, dst=P, live=P),
    "copy": dict(n=2, src=P, dst=P, pages=10, rows=32, hd=64, k=P, ldk=64, ks=P, v=P, ldv=64, vs=P, layers=2, stride=320),
}
BIG = 2147483647
BAD = {
    "attn": [("rows", -1, -1), ("heads", 0, -2), ("heads", 7, -2), ("heads", 1 << 26, -2), ("kvheads", 0, -3),
             ("hd", 15, -4), ("hd", 257, -4), ("rows", 1 << 29, -1), ("q", None, -5), ("ldq", 511, -6), ("seqs", -1, -7), ("seqs", 2, -7),
             ("len", None, -9), ("table", None, -10), ("ldt", -1, -11), ("groups", -1, -12), ("first", None, -13),
             ("shared", None, -14), ("k", None, -15), ("ldk", 63, -16), ("ks", None, -17), ("v", None, -18),
             ("ldv", 63, -19), ("vs", None, -20), ("pages", -1, -21), ("pages", BIG // 30, -21), ("ps", 0, -22),
             ("ps", BIG, -21), ("scale", float("nan"), -23), ("scale", float("inf"), -23), ("out", None, -24),
             ("ldo", 511, -25)],
    "logp": [("m", -1, -1), ("n", -1, -2), ("n", 2 ** 31 - 4095, -2), ("x", None, -3), ("ldx", 99, -4), ("logp", None, -6), ("top", -1, -9),
             ("top", 101, -9), ("index", None, -10), ("ldt", 4, -12)],
    "grow": [("n", -1, -1), ("n", 8193, -1), ("seq", None, -2), ("add", None, -3), ("seqs", -1, -4), ("len", None, -5),
             ("table", None, -6), ("ldt", -1, -7), ("pages", -1, -8), ("ps", 0, -9), ("refs", None, -10),
             ("got", None, -11)],
    "slots": [("rows", -1, -1), ("kvheads", 0, -2), ("seqs", -1, -4), ("len", None, -5), ("table", None, -6),
              ("ldt", -1, -7), ("pages", -1, -8), ("pages", BIG // 30, -8), ("ps", 0, -9), ("slot", None, -10)],
    "fork": [("n", -1, -1), ("n", 8193, -1), ("parent", None, -2), ("child", None, -3), ("seqs", -1, -4),
             ("len", None, -5), ("table", None, -6), ("ldt", -1, -7), ("pages", -1, -8), ("ps", 0, -9),
             ("refs", None, -10), ("src", None, -11), ("dst", None, -12)],
    "free": [("n", -1, -1), ("seq", None, -2), ("seqs", -1, -3), ("len", None, -4), ("table", None, -5), ("ldt", -1, -6),
             ("pages", -1, -7), ("ps", 0, -8), ("refs", None, -9)],
    "compact": [("seqs", -1, -1), ("table", None, -2), ("ldt", -1, -3), ("out", None, -4), ("ldo", 3, -5),
                ("pages", -1, -6), ("refs", None, -7), ("rout", None, -8), ("src", None, -9), ("dst", None, -10),
                ("live", None, -11)],
    "copy": [("n", -1, -1), ("src", None, -2), ("dst", None, -3), ("pages", -1, -4), ("pages", 1 << 27, -4),
             ("rows", -1, -5), ("hd", -1, -6), ("k", None, -7), ("ldk", 63, -8), ("ks", None, -9), ("ldv", 63, -11),
             ("vs", None, -12), ("layers", -1, -13), ("stride", 319, -14)],
}
EMPTY = {"attn": dict(rows=0, seqs=0), "logp": dict(m=0), "grow": dict(n=0), "slots": dict(rows=0, seqs=0), "fork": dict(n=0),
         "free": dict(n=0), "copy": dict(n=0)}


def entries(op):
    if op == "attn":
        return [f"xsymv_q8attn_{t}" for t in "shb"]
    return [f"xsymv_logp_{t}" for t in "shb"] if op == "logp" else [f"xsymv_q8pages_{op}"]


def call(entry, op, **change):
    getattr(X, entry)(*{**GOOD[op], **change}.values(), stream=0)


@pytest.fixture(params=["compiled", "ctypes"])
def way(request, monkeypatch):
    monkeypatch.setattr(X, "_q8_calls", None)
    X._q8()
    if request.param == "ctypes":
        monkeypatch.setattr(X, "_q8_calls", X._Q8Ctypes())


@pytest.mark.parametrize("op", sorted(BAD))
def test_refusals(way, op):
    for entry in entries(op):
        for name, value, code in BAD[op]:
            with pytest.raises(X.XsymvError) as e:
                call(entry, op, **{name: value})
            assert e.value.code == code and entry in str(e.value), (name, value)


@pytest.mark.parametrize("op", sorted(EMPTY))
def test_nothing_to_do(way, op):
    """No pointer is needed where there is nothing to do."""
    for entry in entries(op):
        call(entry, op, **{**{k: None for k, v in GOOD[op].items() if v in (P, 2 * P)}, **EMPTY[op]})


def test_places_that_may_not_be_one(way):
    with pytest.raises(X.XsymvError) as e:
        call("xsymv_q8pages_compact", "compact", out=P, ldo=5)
    assert e.value.code == -5
    with pytest.raises(X.XsymvError) as e:
        call("xsymv_logp_b", "logp", top=129, n=1000, ldx=1000, ldt=129)
    assert e.value.code == -9


def test_arguments(way):
    for entry, op in (("xsymv_q8attn_b", "attn"), ("xsymv_q8pages_fork", "fork"), ("xsymv_logp_s", "logp")):
        first = next(iter(GOOD[op]))
        with pytest.raises(TypeError):
            call(entry, op, **{first: 1.5})
        with pytest.raises(OverflowError):
            call(entry, op, **{first: 1 << 40})
    with pytest.raises((TypeError, ValueError)):
        call("xsymv_q8attn_s", "attn", scale="s")


def test_workspaces():
    for bad in ((-1, 100, 1), (1, 0, 1), (1, 100, 129), (1, 100, -1)):
        assert X.logp_workspace_bytes(*bad) == 0
    assert X.logp_workspace_bytes(1, 128000, 20) > 0
    assert X.logp_workspace_bytes(2000, 128000, 20) == 0


def test_the_model_by_hand():
    m = Model(seqs=4, ldt=3, pages=6, ps=4)
    assert m.grow([0, 1, 0, 9], [6, 4, 1, 1]) == [6, 4, 0, 0]
    assert m.table[0][:2] == [0, 1] and m.table[1][0] == 2 and m.refs == [1, 1, 1, 0, 0, 0]
    assert m.slots([0, 2, 3, 3, 3], 2) == [2 * 0 * 4 + 4 * 0 + 4 * 2 + 0, 12, 9, 13, 2 * 2 * 4 + 3, 2 * 2 * 4 + 4 + 3]
    assert m.fork([0, 1, 0, 0], [2, 3, 2, 1]) == ([1, -1, -2, -2], [3, -1, -2, -2])
    assert m.table[2][:2] == [0, 3] and m.table[3][0] == 2 and m.refs == [2, 1, 2, 1, 0, 0]
    assert m.grow([0, 1, 2, 3], [3, 9, 2, 5]) == [3, 0, 2, 0]
    assert m.refs == [2, 1, 2, 1, 1, 0]
    m.free([0, 0, 7])
    assert m.refs == [1, 0, 2, 1, 0, 0] and m.len == [0, 4, 8, 4]
    table, refs, src, dst, live = m.compact()
    assert (src, dst, live) == ([3, -1, -1], [1, -1, -1], 3) and refs == [1, 1, 2, 0, 0, 0]
    assert table[2][:2] == [0, 1]


def test_rows_without_logits(way):
    """They have outputs like others, and no alternatives."""
    for entry in entries("logp"):
        for change, code in ((dict(top=1), -9), (dict(top=0, logp=None), -6), (dict(top=0, ldx=0), -4)):
            with pytest.raises(X.XsymvError) as e:
                call(entry, "logp", **{"n": 0, "ldx": 1, "x": None, **change})
            assert e.value.code == code
        call(entry, "logp", m=0, n=0, ldx=1, x=None, token=None, logp=None, entropy=None, lse=None, index=None, value=None)
