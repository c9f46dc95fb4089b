"""The 8-bit product's host side, without a GPU: what it does where a stream's
workspace cannot be had, and which kernels it chooses, on a stand-in for the HIP
runtime that writes kernels down and counts device memory
(tests/native/q8_host.cpp)."""
import collections
import json
import math
import os
import random
import re

import pytest

import blas_symmetric_mat_amd as X
from tests import native
from tests.test_gpu_q8 import KERNELS
from tests.test_gpu_q8_gemm import ENDS, MORE, operands

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


def chosen(host, sizes):
    """The kernel of each product (how, m, n, k), bfloat16, and whether k is
    shared out."""
    calls = []
    for how, m, n, k in sizes:
        pads, offs = operands(how, k)
        calls.append(("gemm", "b", m, n, k, 4096 + offs[0], k + pads[0], 8192 + offs[1], k + pads[1]))
    out = []
    for size, words in zip(sizes, host.many(calls)):
        assert words[0] == "0", size
        kernels = [w.split(":")[0] for w in words[2:]]
        product, = [w for w, kind in zip(kernels, kinds(kernels)) if kind == "product"]
        out.append((product, "join" in kinds(kernels)))
    return out


def test_every_kernel_is_tested(host):
    """Sizes over the whole range choose no kernel, whole or with k shared out,
    that the sizes of the GPU tests of kernels do not choose at a dozen ends of
    k or more."""
    tested = collections.Counter(chosen(host, [(how, m, n, k // 128 * 128 + end)
                                               for how, m, n, k in KERNELS + MORE for end in ENDS]))
    rng = random.Random(3)

    def log(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    reached = collections.Counter()
    for how in ("lines", "any", "odd"):
        sizes = []
        while len(sizes) < 20000:
            m, n, k = log(1, 8192), log(1, 32768), log(1, 32768)
            if m * n * k <= 1 << 40:
                sizes.append((how, m, n, k))
        reached.update(chosen(host, sizes))
    missing = {k: (n, tested[k]) for k, n in reached.items() if tested[k] < 12}
    assert not missing
    assert len(reached) > 30


def named(kernel, groups, m, n):
    """A launched kernel's name in the record, and its shares of k."""
    a = [int(v) for v in re.findall(r"Li(\d+)E", kernel)]
    if "stream" in kernel:
        name, tile = "stream", (16, 16)
    elif "ring" in kernel:
        name, tile = ("ring", "ring32")[a[0] - 1], (16 * a[0], 16 * a[0])
    else:
        bm, bn, _, _, q, buffers, how = a
        tile = bm, bn
        name = {(16, 64): "tile16", (32, 64): "tile32", (64, 64): "tile64", (128, 64): "tile128x64",
                (128, 128): "tile128", (256, 128): "tile256x128", (256, 256): "tile256"}[tile]
        if name in ("tile64", "tile128") and (q, buffers) == (1, 2) and how != 0:
            name += "_short"
    return name, groups // (-(-m // tile[0]) * -(-n // tile[1]))


@pytest.mark.parametrize("how,over", [("lines", 1.02), ("any", 1.03), ("odd", 1.02)])
def test_choices_against_the_record(host, how, over):
    """Over the sizes of the committed measurements the kernel and the shares
    of k that the cost model chooses are hardly slower on average than the
    fastest that was measured (products whose rows are copied first apart)."""
    path = os.path.join(os.path.dirname(X.__file__), "tuned", "mi355x_q8gemm.json")
    with open(path) as f:
        record = json.load(f)
    names, rows = record["kernels"], record[how]
    pad_a, pad_w, start = {"lines": (0, 0, 0), "any": (3, 5, 0), "odd": (3, 5, 1)}[how]
    calls = [("gemm", "b", m, n, k, 4096 + start, k + pad_a, 8192 + start, k + pad_w)
             for m, n, k, *_ in rows]
    ratios, unmeasured, copied = [], 0, 0
    for (m, n, k, *times), words in zip(rows, host.many(calls)):
        kernel, groups, _ = words[2].split(":")
        if kernel == "?":
            copied += 1
            continue
        measured = {(names[i], s): us for i, s, us in zip(times[::3], times[1::3], times[2::3])}
        us = measured.get(named(kernel, int(groups), m, n))
        if us is None:  # not measured, or slower than the record keeps
            unmeasured += 1
        else:
            ratios.append(us / min(measured.values()))
    assert math.exp(sum(map(math.log, ratios)) / len(ratios)) <= over
    assert unmeasured <= 0.1 * len(rows) and copied <= 0.4 * len(rows)
