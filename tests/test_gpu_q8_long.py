"""Rows in 8 bits longer than 2^27 elements: the read's workgroups along a row
reach the most that a grid holds there."""
import pytest

from tests.test_gpu_q8 import FLOOR, U, gen
from tests.gpu_util import log

pytestmark = pytest.mark.gpu


def test_one_row_of_more_than_2_27_elements():
    """Stored and read back, bfloat16: the scale, codes within half a step (in
    parts, for the memory's sake) and values to their rounding."""
    import torch
    import blas_symmetric_mat_amd as X
    n = (1 << 27) + 2051
    log(f"store/read b n={n}")
    x = torch.randn((1, n), generator=gen(1), device="cuda", dtype=torch.float32).bfloat16()
    q = torch.empty((1, n), dtype=torch.int8, device="cuda")
    sc = torch.empty((1,), device="cuda")
    out = torch.full((1, n), -3.0, dtype=torch.bfloat16, device="cuda")
    X.xsymv_q8store_b(1, n, x, n, None, 1, q, n, sc)
    X.xsymv_q8read_b(1, n, q, n, sc, None, 1, out, n)
    torch.cuda.synchronize()
    a = max(x.abs().max().double().item(), FLOOR)
    scale = sc.double().item()
    assert abs(scale - a / 127) <= U * 1.01 * a / 127
    for i in range(0, n, 1 << 25):
        s = slice(i, i + (1 << 25))
        t = x[0, s].double() * 127 / a
        c = q[0, s].double()
        # 127 / a and its product with x round once each
        assert bool(((c - t).abs() <= 0.5 + 127 * 2 * U * 1.01).all())
        exact = c * scale
        assert bool(((out[0, s].double() - exact).abs() <= exact.abs() * (U + 2.0 ** -8) * 1.01).all())
