"""The two ways of calling the 8-bit row operators from Python, compiled and
through ctypes, refuse and convert alike; and what a build without a C compiler
or Python's headers makes."""
import os
import sysconfig

import pytest

import blas_symmetric_mat_amd as X
from blas_symmetric_mat_amd import build as B
from tests.test_q8_cpu import BAD, GOOD, call

COMPILED = "_q8_bind" + sysconfig.get_config_var("EXT_SUFFIX")


@pytest.fixture(params=["compiled", "ctypes"])
def way(request, monkeypatch):
    monkeypatch.setattr(X, "_q8_calls", None)
    X._q8()
    if request.param == "ctypes":
        monkeypatch.setattr(X, "_q8_calls", X._Q8Ctypes())
    else:
        assert os.path.basename(X._q8_calls.__file__) == COMPILED  # this interpreter's own
    return request.param


@pytest.mark.parametrize("t", ["s", "h", "b"])
@pytest.mark.parametrize("op", sorted(BAD))
def test_refusals(way, op, t):
    for name, value, code in BAD[op]:
        with pytest.raises(X.XsymvError) as e:
            call(op, t, **{name: value})
        assert e.value.code == code and f"xsymv_q8{op}_{t}" in str(e.value)
    change = {k: None for k, v in GOOD[op].items() if v in (64, 104)}
    call(op, t, **{**change, "m": 0})


def test_arguments_that_cannot_be_converted(way):
    class Tensor:
        def data_ptr(self):
            return 64

    class Number:
        def __index__(self):
            return -5

    with pytest.raises(X.XsymvError) as e:
        call("glu", "s", g=Tensor(), u=Tensor(), m=Number())
    assert e.value.code == -1
    for change, error in ((dict(m=1.5), TypeError), (dict(m="3"), TypeError), (dict(m=1 << 40), OverflowError),
                          (dict(m=-(1 << 31) - 1), OverflowError), (dict(x="x"), AttributeError),
                          (dict(eps="e"), (TypeError, ValueError)), (dict(rtype=3), TypeError)):
        with pytest.raises(error):
            call("norm", "b", **change)
    with pytest.raises(X.XsymvError) as e:
        call("norm", "b", rtype="")
    assert e.value.code == -5
    assert X._q8_calls is not None
    with pytest.raises(TypeError):
        X._q8_calls.glu_s(1, 2, 3)


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """A build's folder that holds nothing but the library."""
    os.symlink(B.LIB, tmp_path / "libxsymv.so")
    monkeypatch.setattr(B, "HERE", str(tmp_path))
    return tmp_path


def test_the_compiled_file_is_this_interpreters(elsewhere):
    assert B.build_bind() == str(elsewhere / COMPILED)
    assert sorted(os.listdir(elsewhere)) == sorted(["libxsymv.so", COMPILED])


@pytest.mark.parametrize("lacks", ["compiler", "headers"])
def test_a_build_without_a_compiler_or_headers(elsewhere, monkeypatch, lacks, capsys):
    (elsewhere / COMPILED).write_bytes(b"an older library's")
    if lacks == "compiler":
        monkeypatch.setattr(B, "CC", "no-such-compiler")
    else:
        monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(elsewhere)})
    assert B.build_bind() is None
    assert "through ctypes" in capsys.readouterr().err
    assert os.listdir(elsewhere) == ["libxsymv.so"]
