"""The 8-bit product's host side, without a GPU: what it does where a stream's
workspace cannot be had, on a stand-in for the HIP runtime that writes kernels
down and counts device memory (tests/native/q8_host.cpp)."""
import os

import pytest

from tests import native

MiB = 1 << 20


@pytest.fixture(scope="module")
def program():
    exe = native.build_q8_host()
    yield exe
    os.remove(exe)


@pytest.fixture
def host(program):
    h = native.Q8Host(program)
    yield h
    h.close()


# products whose plan shares out k, copies the rows first, or both
SHARED = ("b", 256, 8192, 14336, 4096, 14336, 4096, 14336)
COPIED = ("s", 4096, 8192, 4099, 4096, 4099, 8192, 4099)
BOTH = ("h", 300, 2000, 16385, 4097, 16385, 8193, 16385)


def product(host, case):
    """(code, device memory held, kernels)"""
    w = host.ask("gemm", *case)
    return int(w[0]), int(w[1]), [k.split(":")[0] for k in w[2:]]


def kinds(kernels):
    return ["copy" if k == "?" else "join" if "q8_gemm_join" in k else "product" for k in kernels]


@pytest.mark.parametrize("case,want", [(SHARED, ["product", "join"]), (COPIED, ["copy", "product"]),
                                       (BOTH, ["copy", "product", "join"])])
def test_products_that_use_a_workspace(host, case, want):
    rc, held, kernels = product(host, case)
    assert (rc, kinds(kernels)) == (0, want) and held >= MiB
    assert product(host, case) == (rc, held, kernels)  # and keep it
    assert host.ask("state") == ["0", "0", "0"]


@pytest.mark.parametrize("case", [SHARED, COPIED, BOTH])
def test_without_device_memory(host, case):
    """No memory left for the workspace: the product is made without one, no
    error is left behind, and the memory is used as soon as it is there."""
    host.ask("room", MiB // 2)
    for attempt in (1, 2):
        rc, held, kernels = product(host, case)
        assert (rc, held, kinds(kernels)) == (0, 0, ["product"])
        assert host.ask("state") == ["0", str(attempt), "0"]
    host.ask("room", 1 << 40)
    rc, held, kernels = product(host, case)
    assert rc == 0 and held > 0 and len(kernels) > 1


@pytest.mark.parametrize("case", [SHARED, COPIED, BOTH])
def test_first_product_of_a_capture(host, case):
    """Nothing that a capture forbids is called, on a stream without a
    workspace and on one whose workspace is too small; one that is large enough
    is used."""
    host.ask("capture", 1)
    rc, held, kernels = product(host, case)
    assert (rc, held, kinds(kernels)) == (0, 0, ["product"])
    host.ask("capture", 0)
    assert product(host, ("b", 5, 33, 8200, 4096, 8208, 4096, 8208))[:2] == (0, MiB)
    host.ask("capture", 1)
    rc, held, kernels = product(host, case)
    assert (rc, held, kinds(kernels)) == (0, MiB, ["product"])
    host.ask("capture", 0)
    want = product(host, case)
    host.ask("capture", 1)
    assert product(host, case) == want and len(want[2]) > 1
    assert host.ask("state") == ["0", "0", "0"]


def test_an_installed_workspace_that_is_too_small(host):
    """The caller's choice is not passed over: refused before any work, whether
    or not the stream is being captured."""
    host.ask("workspace", 4096)
    for capture in (0, 1):
        host.ask("capture", capture)
        assert product(host, SHARED) == (2000, 0, [])
    assert host.ask("state") == ["0", "0", "0"]


def test_what_a_graph_holds_is_not_freed(host):
    """A workspace that a captured product uses is kept when a larger product
    outgrows it, and freed by the release."""
    small = ("b", 40, 300, 20000, 4096, 20000, 8192, 20000)
    assert product(host, small)[:2] == (0, MiB)
    host.ask("capture", 1)
    assert len(product(host, small)[2]) == 2
    host.ask("capture", 0)
    rc, held, kernels = product(host, SHARED)
    assert rc == 0 and len(kernels) == 2 and held > 32 * MiB
    assert held - MiB == 256 * 8192 * 4 * 4  # both buffers
    assert host.ask("release") == ["0"]
    assert product(host, ("b", 1, 16, 16, 4096, 16, 4096, 16))[1] == 0
