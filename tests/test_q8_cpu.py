"""The operators on rows in 8 bits on the CPU: every refusal of an argument,
with its position, before any device work, and the calls that have nothing to
do.  Addresses are numbers that nothing may follow."""
import math

import pytest

import blas_symmetric_mat_amd as X

# A valid call of each operator (m = 3, n = 40, k = 24), argument by argument.
GOOD = {
    "norm": dict(m=3, n=40, x=64, ldx=40, rtype=None, r=64, ldr=40, wtype=None, w=64, eps=1e-5,
                 h=64, ldh=40, q=64, ldq=40, scale=64),
    "glu": dict(m=3, n=40, g=64, ldg=80, u=104, ldu=80, q=64, ldq=40, scale=64),
    "store": dict(m=3, n=40, x=64, ldx=40, slot=64, cap=9, q=64, ldq=40, scale=64),
    "read": dict(m=3, n=40, q=64, ldq=40, scale=64, slot=64, cap=9, out=64, ldo=40),
    "gemm": dict(m=3, n=40, k=24, a=64, lda=24, sa=64, w=64, ldw=24, sw=64, bias=None, c=64,
                 ldc=40),
}

BAD = {
    "norm": [("m", -1, -1), ("n", -1, -2), ("x", None, -3), ("ldx", 39, -4), ("rtype", "d", -5),
             ("ldr", 39, -7), ("wtype", "?", -8), ("w", None, -9), ("eps", -1e-9, -10),
             ("eps", math.inf, -10), ("eps", math.nan, -10), ("ldh", 39, -12),
             ("ldh", 41, -12), ("q", None, -13), ("ldq", 0, -14), ("scale", None, -15)],
    "glu": [("m", -1, -1), ("n", -7, -2), ("g", None, -3), ("ldg", 39, -4), ("u", None, -5),
            ("ldu", 39, -6), ("q", None, -7), ("ldq", 39, -8), ("scale", None, -9)],
    "store": [("m", -1, -1), ("n", -1, -2), ("x", None, -3), ("ldx", 39, -4), ("cap", -1, -6),
              ("q", None, -7), ("ldq", 39, -8), ("scale", None, -9)],
    "read": [("m", -1, -1), ("n", -1, -2), ("q", None, -3), ("ldq", 39, -4), ("scale", None, -5),
             ("cap", -1, -7), ("out", None, -8), ("ldo", 39, -9)],
    "gemm": [("m", -1, -1), ("n", -1, -2), ("k", -1, -3), ("k", 131072, -3), ("a", None, -4),
             ("lda", 23, -5), ("sa", None, -6), ("w", None, -7), ("ldw", 23, -8),
             ("sw", None, -9), ("c", None, -11), ("ldc", 39, -12)],
}


def call(op, t, **change):
    args = dict(GOOD[op])
    for k in ("rtype", "wtype"):
        if k in args:
            args[k] = t
    args.update(change)
    getattr(X, f"xsymv_q8{op}_{t}")(*args.values(), stream=0)


@pytest.mark.parametrize("t", ["s", "h", "b"])
@pytest.mark.parametrize("op", sorted(BAD))
def test_refusals(op, t):
    for name, value, code in BAD[op]:
        with pytest.raises(X.XsymvError) as e:
            call(op, t, **{name: value})
        assert e.value.code == code, (op, name, value)


@pytest.mark.parametrize("t", ["s", "h", "b"])
def test_types_beside_the_calls_own(t):
    """A residual or weight of the other 16-bit type is refused; capitals are
    letters too (the refusal that follows is a later argument's)."""
    for other in {"h", "b"} - {t}:
        for name, code in (("rtype", -5), ("wtype", -8)):
            with pytest.raises(X.XsymvError) as e:
                call("norm", t, **{name: other})
            assert e.value.code == code
    for letter in (t, t.upper(), "s", "S"):
        with pytest.raises(X.XsymvError) as e:
            call("norm", t, rtype=letter, wtype=letter, scale=None)
        assert e.value.code == -15


@pytest.mark.parametrize("op,code", [("store", -6), ("read", -7)])
def test_rows_without_slots_need_room(op, code):
    with pytest.raises(X.XsymvError) as e:
        call(op, "b", slot=None, cap=2)
    assert e.value.code == code


@pytest.mark.parametrize("t", ["s", "h", "b"])
@pytest.mark.parametrize("op", sorted(GOOD))
def test_nothing_to_do(op, t):
    for name in ("m", "n"):
        change = {k: None for k, v in GOOD[op].items() if v in (64, 104)}
        change[name] = 0
        if op in ("store", "read"):
            change["cap"] = 3
        call(op, t, **change)
    if op == "store":  # a cache without rows takes none
        call(op, t, cap=0, q=None, scale=None)


def test_strides_of_empty_rows_are_checked():
    with pytest.raises(X.XsymvError) as e:
        call("glu", "s", m=0, ldg=0)
    assert e.value.code == -4
