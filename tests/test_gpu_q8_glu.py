"""The gated activation on rows in 8 bits where all gates of a row are far
below zero: exp(g) leaves the normal 32-bit numbers at g = -87.4, the results
of large other factors do not."""
import pytest

from tests.test_gpu_q8 import FLOOR, U, check_codes, dtype_of, gen
from tests.gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 7, 8, 100, 1031])
@pytest.mark.parametrize("t,low,size", [("h", -95.0, 6e4), ("b", -170.0, 1e38), ("s", -170.0, 1e38)])
def test_gates_far_below_zero(t, low, size, n):
    import torch
    import blas_symmetric_mat_amd as X
    log(f"glu {t} n={n}, gates {low} to -77")
    g = gen(n)
    m = 400

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    # each row's gates within 3 of one another
    gate = (low + 3 + (-83 - low) * uniform(m, 1) + 3 * uniform(m, n)).to(dtype_of(t))
    up = (size * (0.1 + 0.9 * uniform(m, n)) * torch.sign(uniform(m, n) - 0.5)).to(dtype_of(t))
    assert gate.max().item() <= -77 and bool(up.isfinite().all())
    q = torch.empty((m, n), dtype=torch.int8, device="cuda")
    sc = torch.empty((m,), device="cuda")
    getattr(X, f"xsymv_q8glu_{t}")(m, n, gate, n, up, n, q, n, sc)
    torch.cuda.synchronize()
    gd, ud = gate.double(), up.double()
    v = gd * torch.sigmoid(gd) * ud
    a = v.abs().amax(dim=1, keepdim=True).clamp_min(FLOOR)
    assert int((127 * v / a).abs().amax(dim=1).ge(1).sum()) > m // 12  # rows that have codes
    # the exponent: its constant and its product round (2 |g| u); the power is
    # good to one unit and squared (4u); 1 + z rounds (u), the reciprocal is
    # good to one unit (2u), four products (4u)
    rel = (2 * gd.abs() + 11) * U
    top = (v.abs() * rel).amax(dim=1, keepdim=True) / a
    check_codes(v, q, sc, rel + top, top.max().item() / U + 1.0, f"glu {t} n={n}")
