"""The norm on rows in 8 bits where its output replaces an input, and for rows
at the ends of the 32-bit range."""
import pytest

from tests.test_gpu_q8 import U, WIDTHS, Rows, check_codes, dtype_of, gen, randn
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


@pytest.mark.parametrize("n", [1, 5, 8, 1000, 70001])
@pytest.mark.parametrize("t", ["s", "b"])
def test_rows_at_the_ends_of_the_range(t, n):
    """Rows of the smallest numbers there are (below 2^-126, eps = 0) and of the
    largest: 1 / sqrt(mean(h^2)) is outside the normal 32-bit numbers, the
    normalised rows are of ordinary size."""
    import torch
    import blas_symmetric_mat_amd as X
    log(f"norm of the ends {t} n={n}")
    g = gen(n + 31)
    m = 12
    x = randn((m, n), g).clamp_(-4, 4) + 0.01
    power = torch.tensor([-149, -146, -140, -133, -128, -126, -100, -99, 99, 101, 120, 125],
                         dtype=torch.float64, device="cuda")
    if t == "b":
        power.clamp_min_(-133.0)
    x = (x.double() * torch.exp2(power)[:, None]).to(dtype_of(t))
    x[x == 0] = 2.0 ** -149 if t == "s" else 2.0 ** -133  # no row of zeros
    w = (1.0 + randn((n,), g, 0.1)).to(dtype_of(t))
    q = torch.empty((m, n), dtype=torch.int8, device="cuda")
    sc = torch.empty((m,), device="cuda")
    getattr(X, f"xsymv_q8norm_{t}")(m, n, x, n, t, None, 0, t, w, 0.0, None, 0, q, n, sc)
    torch.cuda.synchronize()
    k = x.double()
    assert bool(k.isfinite().all()) and bool((k[:, 0] != 0).all())
    v = k / (k * k).mean(dim=1, keepdim=True).sqrt() * w.double()
    # as for ordinary rows: factor, product with h, product with w
    check_codes(v, q, sc, 6 * U, 4.0, f"norm of the ends {t} n={n}")
