"""The norm on rows in 8 bits where its output replaces an input, and for rows
at the ends of the 32-bit range."""
import pytest

from tests.test_gpu_q8 import WIDTHS, Rows, dtype_of, gen, randn
from tests.gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("t", ["s", "h", "b"])
def test_h_in_xs_place(t, n):
    """h kept in x's place, with a residual, without one and with x itself as
    the residual: the bytes of a call that keeps it elsewhere."""
    import torch
    import blas_symmetric_mat_amd as X
    log(f"norm in place {t} n={n}")
    g = gen(n + 7)
    m = 9 if n <= 2048 else 3
    x0 = randn((m, n), g).to(dtype_of(t))
    r0 = randn((m, n), g, 3.0).to(dtype_of(t))
    w = (1.0 + randn((n,), g, 0.2)).to(dtype_of(t))
    f = getattr(X, f"xsymv_q8norm_{t}")

    def run(residual, in_place):
        x = Rows(m, n, dtype_of(t), pad=3, off=1, fill=8, data=x0)
        h = x if in_place else Rows(m, n, dtype_of(t), pad=3, off=1, fill=8)
        r = {"none": None, "other": r0, "x": x.t}[residual]
        ldr = {"none": 0, "other": n, "x": x.ld}[residual]
        q = Rows(m, n, torch.int8, pad=1, off=3, fill=55)
        sc = torch.empty((m,), device="cuda")
        f(m, n, x.t, x.ld, t, r, ldr, t, w, 1e-5, h.t, h.ld, q.t, q.ld, sc)
        torch.cuda.synchronize()
        assert h.intact() and q.intact()
        return h.t, q.t, sc

    for residual in ("none", "other", "x"):
        for a, b in zip(run(residual, False), run(residual, True)):
            assert torch.equal(a, b), residual
