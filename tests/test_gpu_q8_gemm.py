"""The 8-bit product where its stream's workspace cannot grow, and by the
kernels, whole and with k shared out, that few sizes take."""
import math

import pytest

from tests.gpu_util import log
from tests.test_gpu_q8 import gemm_case, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,pad", [(256, 2048, 9000, 8), (40, 300, 20000, 0), (600, 1100, 4099, 2)])
@pytest.mark.parametrize("before", [False, True])
def test_first_product_in_a_graph(m, n, k, pad, before):
    """Captured on a stream that has run no product (or a smaller one only, so
    that a workspace is there and too small): the graph is whole, and every
    replay gives the eager bytes."""
    import torch
    import blas_symmetric_mat_amd as X
    log(f"first product in a graph {m}x{n}x{k}, before: {before}")
    g = gen(m)
    ld = k + pad
    a = torch.randint(-127, 128, (m, ld), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (n, ld), generator=g, device="cuda", dtype=torch.int8)
    one = torch.ones((max(m, n),), device="cuda")
    c = torch.empty((m, n), device="cuda")

    def product(rows, stream=None):
        X.xsymv_q8gemm_s(rows, n, k, a, ld, one, w, ld, one, None, c, n, stream=stream)

    product(m)
    torch.cuda.synchronize()
    want = c.clone()
    assert X.q8gemm_workspace_bytes(m, n, k) > 0
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    X.set_workspace(None, stream=st)  # nothing is left of an earlier stream of this handle
    if before:
        product(3, st)
        st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        product(m, st)
    for i in range(4):
        c.fill_(math.nan)
        product(m)  # the program's own
        torch.cuda.synchronize()
        c.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want)
    c.fill_(math.nan)
    product(m, st)  # and eagerly on the same stream
    torch.cuda.synchronize()
    assert torch.equal(c, want)


# sizes at which the kernels that KERNELS reaches seldom or not at all are the
# ones chosen, at every end of k; test_q8_host_cpu.py checks that the two lists
# together reach every kernel
MORE = [("any", 7, 588, 6364), ("any", 6, 716, 6915), ("odd", 6, 34, 4774), ("odd", 7, 14676, 1672),
        ("any", 19, 1033, 7513), ("any", 21, 939, 9858), ("lines", 20, 1049, 10353),
        ("lines", 19, 724, 15893), ("odd", 2936, 66, 10168), ("odd", 2725, 70, 12175),
        ("any", 144, 18850, 3080), ("any", 136, 9506, 6660), ("any", 140, 2764, 8011),
        ("any", 2718, 141, 11727), ("lines", 69, 16498, 7412), ("lines", 37, 19025, 3581),
        ("lines", 41, 17876, 5219), ("lines", 5801, 76, 6610), ("any", 34, 177, 7319),
        ("lines", 19, 181, 12143), ("odd", 70, 8276, 4696), ("any", 4331, 43, 2144),
        ("lines", 1422, 42, 9808), ("any", 37, 4818, 3292)]
ENDS = (0, 4, 11, 12, 13, 28, 84, 85, 99, 100, 101, 115, 116, 211, 212, 213, 228)


def operands(how, k):
    """Gaps after the rows of A, W and C, and where their first rows start."""
    return {"lines": ((-k % 16, -k % 16 + 32, 0), (0, 16, 0)), "any": ((5, 3, 0), (0, 0, 0)),
            "odd": ((5, 3, 0), (3, 1, 0))}[how]


@pytest.mark.parametrize("how,m,n,k", MORE)
def test_seldom_kernels(how, m, n, k):
    for end in ENDS:
        kk = k // 128 * 128 + end
        log(f"gemm {how} {m}x{n}x{kk}")
        gemm_case("b", m, n, kk, *operands(how, kk), m + n + kk, bias=False)
