"""The 8-bit product where its stream's workspace cannot grow."""
import math

import pytest

from tests.gpu_util import log
from tests.test_gpu_q8 import gen

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
