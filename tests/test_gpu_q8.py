"""The operators on rows in 8 bits against their definition in 64 bits.

Bounds, with u = 2^-24 (half a step of 32-bit floating point, relative):
a code may differ from the exact quotient t = 127 v / a by half a step of the
code plus what the 32-bit arithmetic before the rounding moves t by; a scale
and a value by their roundings.  Each bound is derived where it is used."""
import math

import numpy as np
import pytest

from tests.gpu_util import log, torch_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FLOOR = 2.0 ** -100
LETTERS = ["s", "h", "b"]


def dtype_of(t):
    import torch
    return {"s": torch.float32, "h": torch.float16, "b": torch.bfloat16}[t]


def half_step(t):
    import torch
    return 0.0 if t == "s" else torch.finfo(dtype_of(t)).eps / 2


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, spread=1.0):
    import torch
    return torch.randn(shape, generator=g, device="cuda") * spread


class Rows:
    """An m x n matrix inside a larger buffer of `fill`, rows n + pad apart,
    starting `off` elements in; `intact` tells whether the rest still holds
    the fill."""

    def __init__(self, m, n, dtype, pad=0, off=0, fill=0, data=None):
        import torch
        self.ld = max(1, n + pad)
        self.buf = torch.full((off + m * self.ld + 64,), fill, dtype=dtype, device="cuda")
        self.t = torch.as_strided(self.buf, (m, n), (self.ld, 1), off)
        self.m, self.n, self.off, self.fill = m, n, off, fill
        if data is not None:
            self.t.copy_(data)

    def intact(self):
        import torch
        rest = self.buf.clone()
        torch.as_strided(rest, (self.m, self.n), (self.ld, 1), self.off).fill_(self.fill)
        return bool((rest == self.fill).all())


def check_codes(v, q, scale, moved, scale_steps, label):
    """v exact rows (64 bits); `moved`: relative error of an element of v and
    of the row's maximum before the quantisation, in units of 1.  Dividing
    127 by a and multiplying by v add two roundings."""
    import torch
    a = v.abs().amax(dim=1, keepdim=True).clamp_min(FLOOR)
    t = v * 127 / a
    off = (q.double() - t).abs()
    allowed = 0.5 + 127 * (moved + 2 * U) * 1.01
    worst = (off - allowed).max().item()
    assert worst <= 0, f"{label}: a code off by {off.max().item()}"
    step = (scale.double() - a[:, 0] / 127).abs() / (a[:, 0] / 127)
    assert step.max().item() <= scale_steps * U * 1.01, label
    assert q.min().item() >= -127


WIDTHS = [1, 7, 8, 9, 64, 65, 128, 129, 250, 256, 257, 512, 515, 1024, 1031, 2048, 2050, 4096,
          4099, 8192, 8200, 16384, 16391, 32768, 32771, 65536, 65543]


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("t", LETTERS)
def test_store_and_read(t, n):
    """Rows into slots of a cache and back: codes and scales against the
    definition, rows of other slots and the gaps untouched, slots outside the
    cache left out by the store and zeros from the read."""
    import torch
    import blas_symmetric_mat_amd as X
    log(f"store/read {t} n={n}")
    g = gen(n)
    m, cap = (37, 61) if n <= 2048 else (5, 9)
    x = Rows(m, n, dtype_of(t), pad=n % 5, off=3, data=randn((m, n), g))
    x.t[0] = 0.0
    x.t[1] *= 2.0 ** -9
    x.t[2, n // 2] = 40.0
    slot = torch.randperm(cap, generator=g, device="cuda")[:m].to(torch.int32)
    slot[3], slot[m - 1] = -1, cap
    kept = [i for i in range(m) if i not in (3, m - 1)]
    q = Rows(cap, n, torch.int8, pad=3, off=1, fill=99)
    sc = torch.full((cap,), 7.5, device="cuda")
    getattr(X, f"xsymv_q8store_{t}")(m, n, x.t, x.ld, slot, cap, q.t, q.ld, sc)
    torch.cuda.synchronize()
    at = slot[kept].long()
    check_codes(x.t[kept].double(), q.t[at], sc[at], 0.0, 1.0, f"store {t} n={n}")
    others = [i for i in range(cap) if i not in set(at.tolist())]
    assert bool((q.t[others] == 99).all()) and bool((sc[others] == 7.5).all())
    assert q.intact()

    out = Rows(m, n, dtype_of(t), pad=5, off=1, fill=-3)
    getattr(X, f"xsymv_q8read_{t}")(m, n, q.t, q.ld, sc, slot, cap, out.t, out.ld)
    torch.cuda.synchronize()
    exact = q.t[at].double() * sc[at].double()[:, None]
    # the product rounds once to 32 bits and, in 16 bits, once more; below the
    # smallest normal number of half precision by half its smallest step
    tiny = 2.0 ** -25 if t == "h" else 0.0
    bound = exact.abs() * (U + half_step(t)) * 1.01 + tiny
    assert bool(((out.t[kept].double() - exact).abs() <= bound).all())
    assert bool((out.t[[3, m - 1]] == 0).all()) and out.intact()


@pytest.mark.parametrize("t", LETTERS)
def test_rows_without_slots(t):
    """slot None: row i of x is row i of the codes, of the same bytes as with
    the slots 0, 1, ..."""
    import torch
    import blas_symmetric_mat_amd as X
    m, n = 19, 300
    x = randn((m, n), gen(5)).to(dtype_of(t))
    res = []
    for slot in (None, torch.arange(m, dtype=torch.int32, device="cuda")):
        q = torch.empty((m, n), dtype=torch.int8, device="cuda")
        sc = torch.empty((m,), device="cuda")
        out = torch.empty_like(x)
        getattr(X, f"xsymv_q8store_{t}")(m, n, x, n, slot, m, q, n, sc)
        getattr(X, f"xsymv_q8read_{t}")(m, n, q, n, sc, slot, m, out, n)
        res.append((q, sc, out))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*res))
    err = (res[0][2].double() - x.double()).abs()
    assert bool((err <= 0.51 * res[0][1].double()[:, None] + half_step(t) * x.double().abs()).all())


@pytest.mark.parametrize("t", LETTERS)
def test_rows_that_are_not_finite(t):
    """A NaN or an infinity makes its own row NaN and leaves the others."""
    import torch
    import blas_symmetric_mat_amd as X
    for n in (100, 6000, 66000):
        log(f"not finite {t} n={n}")
        x = randn((6, n), gen(n)).to(dtype_of(t))
        clean = x.clone()
        x[1, n - 1] = math.nan
        x[2, 3] = math.inf
        x[4, n // 2] = -math.inf
        w = torch.ones((n,), device="cuda").to(dtype_of(t))
        one = torch.ones_like(x)
        for op in ("store", "norm", "glu"):
            outs = []
            for v in (x, clean):
                q = torch.empty((6, n), dtype=torch.int8, device="cuda")
                sc = torch.empty((6,), device="cuda")
                if op == "store":
                    getattr(X, f"xsymv_q8store_{t}")(6, n, v, n, None, 6, q, n, sc)
                elif op == "glu":
                    getattr(X, f"xsymv_q8glu_{t}")(6, n, one, n, v, n, q, n, sc)
                else:
                    getattr(X, f"xsymv_q8norm_{t}")(6, n, v, n, t, None, 0, t, w, 1e-5, None, 0,
                                                    q, n, sc)
                out = torch.empty_like(x)
                getattr(X, f"xsymv_q8read_{t}")(6, n, q, n, sc, None, 6, out, n)
                outs.append(out)
            torch.cuda.synchronize()
            assert bool(outs[0][[1, 2, 4]].isnan().all()), op
            assert torch.equal(outs[0][[0, 3, 5]], outs[1][[0, 3, 5]]), op


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("t,rt,wt", [("s", "s", "s"), ("h", "h", "h"), ("h", "s", "h"),
                                     ("h", "h", "s"), ("h", "s", "s"), ("b", "b", "b"),
                                     ("b", "s", "b"), ("b", "b", "s"), ("b", "s", "s")])
def test_norm(t, rt, wt, n):
    import torch
    import blas_symmetric_mat_amd as X
    log(f"norm {t}{rt}{wt} n={n}")
    g = gen(n + 1)
    m = 9 if n <= 2048 else 3
    x = Rows(m, n, dtype_of(t), pad=n % 3, off=1, data=randn((m, n), g))
    r = Rows(m, n, dtype_of(rt), pad=2, off=5, fill=6, data=randn((m, n), g, 3.0))
    w = (1.0 + randn((n,), g, 0.2)).to(dtype_of(wt))
    x.t[0], r.t[0] = 0.0, 0.0  # a row of zeros: codes of zero
    x.t[1] *= 2.0 ** -6
    r.t[1] *= 2.0 ** -6
    r0 = r.t.clone()
    eps = 1e-5
    f = getattr(X, f"xsymv_q8norm_{t}")

    def run(res, h):
        q = Rows(m, n, torch.int8, pad=1, off=3, fill=55)
        sc = torch.empty((m,), device="cuda")
        f(m, n, x.t, x.ld, rt, None if res is None else res.t, 0 if res is None else res.ld, wt, w,
          eps, None if h is None else h.t, 0 if h is None else h.ld, q.t, q.ld, sc)
        torch.cuda.synchronize()
        assert q.intact()
        return q.t, sc

    h = Rows(m, n, dtype_of(rt), pad=4, off=7, fill=8)
    q, sc = run(r, h)
    whole = x.t.double() + r0.double()
    # the sum rounds to 32 bits and, where h is in 16, once more
    tiny = 2.0 ** -25 if rt == "h" else 0.0
    assert bool(((h.t.double() - whole).abs() <= whole.abs() * (U + half_step(rt)) * 1.01 + tiny).all())
    assert h.intact()

    def exact(k):
        k = k.double()
        return k / torch.sqrt((k * k).mean(dim=1, keepdim=True) + float(torch.tensor(eps))) \
            * w.double()

    # factor, product with h, product with w: three roundings of an element,
    # three of the maximum; the scale has the maximum's and one of its own
    check_codes(exact(h.t), q, sc, 6 * U, 4.0, f"norm {t}{rt}{wt} n={n}")
    assert bool((q[0] == 0).all())

    # h kept in r's place, h not kept: the same bytes; no residual: x itself
    q1, sc1 = run(r, None)
    q2, sc2 = run(r, r)
    assert torch.equal(q, q1) and torch.equal(sc, sc1)
    assert torch.equal(q, q2) and torch.equal(sc, sc2)
    assert torch.equal(r.t, h.t) and r.intact()
    alone = Rows(m, n, dtype_of(rt), pad=0, off=0)
    q3, sc3 = run(None, alone)
    assert torch.equal(alone.t, x.t.to(dtype_of(rt)))
    check_codes(exact(alone.t), q3, sc3, 6 * U, 4.0, f"norm {t}{rt}{wt} n={n} alone")


def test_norm_of_the_largest_numbers():
    """The sum of squares does not overflow where the rows are finite."""
    import torch
    import blas_symmetric_mat_amd as X
    n = 1000
    x = randn((3, n), gen(2)).clamp_(-3, 3)
    x *= torch.tensor([[1e30], [1e-30], [1e37]], device="cuda")
    w = torch.ones((n,), device="cuda")
    q = torch.empty((3, n), dtype=torch.int8, device="cuda")
    sc = torch.empty((3,), device="cuda")
    X.xsymv_q8norm_s(3, n, x, n, "s", None, 0, "s", w, 0.0, None, 0, q, n, sc)
    torch.cuda.synchronize()
    k = x.double()
    v = k / (k * k).mean(dim=1, keepdim=True).sqrt()
    # the third row's factor is near 1e-37, a normal number still
    check_codes(v, q, sc, 6 * U, 4.0, "norm of large and small rows")


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("t", LETTERS)
def test_glu(t, n):
    import torch
    import blas_symmetric_mat_amd as X
    log(f"glu {t} n={n}")
    g = gen(n + 2)
    m = 11 if n <= 2048 else 3
    both = Rows(m, 2 * n, dtype_of(t), pad=n % 4, off=1, data=randn((m, 2 * n), g, 2.5))
    gate, up = both.t[:, :n], both.t[:, n:]
    gate[0] = 0.0
    gate[1] = -gate[1].abs() - 3.0  # a row of small results
    gate[2, 0] = 30.0
    q = Rows(m, n, torch.int8, pad=2, off=1, fill=44)
    sc = torch.empty((m,), device="cuda")
    getattr(X, f"xsymv_q8glu_{t}")(m, n, gate, both.ld, up, both.ld, q.t, q.ld, sc)
    torch.cuda.synchronize()
    gd, ud = gate.double(), up.double()
    v = gd * torch.sigmoid(gd) * ud
    # z = 2^(-|g| log2 e): the constant and the product round (2 |g| u in z),
    # the power is good to one unit (2u); 1 + z and z's share in it 2u, the
    # reciprocal one unit (2u), three products 3u: (2 |g| + 10) u
    rel = (2 * gd.abs() + 10) * U
    a = v.abs().amax(dim=1, keepdim=True).clamp_min(FLOOR)
    top = (v.abs() * rel).amax(dim=1, keepdim=True) / a
    check_codes(v, q.t, sc, rel + top, top.max().item() / U + 1.0,
                f"glu {t} n={n}")
    assert q.intact()


GEMM = [(1, 1, 1), (1, 5, 16), (2, 16, 15), (3, 100, 63), (7, 33, 64), (16, 129, 65), (1, 515, 4099),
        (17, 64, 255), (31, 200, 256), (33, 250, 257), (48, 31, 1000), (64, 512, 512),
        (65, 130, 130), (100, 1003, 771), (128, 256, 1024), (129, 257, 129), (200, 96, 2050),
        (255, 640, 640), (256, 256, 256), (257, 300, 1111), (300, 1000, 128), (511, 777, 333),
        (513, 1025, 2048), (1024, 1024, 515), (1300, 700, 1300), (2049, 520, 260), (5, 9, 20000)]


def gemm_case(t, m, n, k, pads, offs, seed, bias):
    import torch
    import blas_symmetric_mat_amd as X
    g = gen(seed)

    def codes(rows):
        return torch.randint(-128, 128, (rows, k), generator=g, device="cuda", dtype=torch.int8)

    a = Rows(m, k, torch.int8, pads[0], offs[0], fill=77, data=codes(m))
    w = Rows(n, k, torch.int8, pads[1], offs[1], fill=77, data=codes(n))
    c = Rows(m, n, dtype_of(t), pads[2], offs[2], fill=-5)
    sa = 0.01 + torch.rand((m,), generator=g, device="cuda")
    sw = (0.01 + torch.rand((n,), generator=g, device="cuda")) / (100.0 * math.sqrt(max(1, k)))
    b = randn((n,), g, 10.0) if bias else None
    outs = []
    for _ in range(2):
        c.t.fill_(math.nan)
        getattr(X, f"xsymv_q8gemm_{t}")(m, n, k, a.t, a.ld, sa, w.t, w.ld, sw, b, c.t, c.ld)
        torch.cuda.synchronize()
        outs.append(c.t.clone())
    assert torch.equal(outs[0], outs[1])
    # whole numbers below 2^53: the sums in 64 bits are exact
    p = a.t.double() @ w.t.double().t().contiguous() * sa.double()[:, None] * sw.double()
    exact = p if b is None else p + b.double()
    # sum, two scales: three roundings of the product, the bias one of the sum
    bound = (3 * U * p.abs() + (U if bias else 0.0) * exact.abs()) * 1.01
    bound = bound + (exact.abs() + bound) * half_step(t) + (2.0 ** -25 if t == "h" else 0.0)
    bad = ~((outs[0].double() - exact).abs() <= bound)
    assert not bool(bad.any()), (f"gemm {t} {m}x{n}x{k}: {int(bad.sum())} elements off, first "
                                 f"{bad.nonzero()[0].tolist()}")
    assert c.intact()


@pytest.mark.parametrize("m,n,k", GEMM)
@pytest.mark.parametrize("t", LETTERS)
def test_gemm_aligned(t, m, n, k):
    log(f"gemm {t} {m}x{n}x{k}, rows at multiples of 16 bytes")
    up = -k % 16
    gemm_case(t, m, n, k, (up, up + 16, -n % 8), (0, 16, 0), m + n + k, bias=False)


@pytest.mark.parametrize("m,n,k", GEMM)
@pytest.mark.parametrize("t", LETTERS)
def test_gemm_odd(t, m, n, k):
    log(f"gemm {t} {m}x{n}x{k}, rows anywhere, with a bias")
    gemm_case(t, m, n, k, (3, 1, 5), (1, 7, 3), m + n + k + 1, bias=True)


@pytest.mark.parametrize("m,n,k", [c for c in GEMM if c[2] >= 16])
@pytest.mark.parametrize("t", LETTERS)
def test_gemm_any_stride(t, m, n, k):
    log(f"gemm {t} {m}x{n}x{k}, the first row at a multiple of 16 bytes, the others anywhere")
    gemm_case(t, m, n, k, (3 + m % 2, 5, 3), (16, 0, 1), m + n + k + 2, bias=False)


# ends of k around the 16-byte pieces and the steps of 128 and 256 bytes, in
# tiles of every height, with the operands' last rows in and out of a tile
ENDS = [16, 17, 31, 32, 47, 100, 127, 128, 129, 143, 144, 145, 160, 255, 256, 257, 271, 272, 273,
        383, 384, 400, 511, 512, 513, 528, 640, 641, 777, 1040]


@pytest.mark.parametrize("k", ENDS)
@pytest.mark.parametrize("m,n", [(1, 1), (2, 67), (16, 128), (20, 33), (33, 130), (70, 64),
                                 (129, 129), (257, 300), (600, 1100)])
def test_gemm_ends(m, n, k):
    log(f"gemm {m}x{n}x{k}: ends")
    gemm_case("s", m, n, k, (-k % 16, -k % 16 + 16, 0), (0, 0, 0), m + n + k, bias=False)
    for pad in (1, 2, 4, 8):
        gemm_case("s", m, n, k, (pad, pad + 6, 0), (0, 16, 0), m + n + k + pad, bias=False)
    gemm_case("s", m, n, k, (0, 0, 0), (0, 0, 0), m + n + k + 9, bias=False)


@pytest.mark.parametrize("m,n,k", [(3, 200, 40000), (16, 2048, 28000), (30, 300, 30000),
                                   (60, 1000, 20000), (130, 2000, 16384), (256, 2048, 9000),
                                   (300, 4096, 20000), (1024, 8192, 1024), (2048, 4096, 515)])
@pytest.mark.parametrize("pad", ["lines", "any", "odd"])
def test_gemm_large(m, n, k, pad):
    """Sizes at which k is shared out between workgroups, and the largest tiles."""
    log(f"gemm {m}x{n}x{k} {pad}")
    pads, offs = {"lines": ((-k % 16, -k % 16, 0), (0, 0, 0)), "any": ((7, 9, 1), (0, 0, 3)),
                  "odd": ((7, 9, 1), (5, 1, 3))}[pad]
    gemm_case("b", m, n, k, pads, offs, m + n + k, bias=True)


# sizes at which each kernel of the product is the one chosen, k whole and shared out
KERNELS = [("lines", 5, 33, 300), ("lines", 5, 33, 8200), ("lines", 5, 4100, 300),
           ("lines", 16, 4100, 16400), ("lines", 40, 33, 2060), ("lines", 100, 33, 2060),
           ("lines", 100, 8200, 780), ("lines", 2050, 33, 8200), ("lines", 100, 16400, 780),
           ("lines", 100, 4100, 8200), ("lines", 200, 16400, 300), ("lines", 4100, 33, 16400),
           ("lines", 260, 30000, 520), ("lines", 130, 4100, 16400), ("lines", 5, 1000, 8200),
           ("lines", 40, 16400, 300), ("lines", 200, 16400, 520), ("lines", 130, 8200, 8200),
           ("any", 5, 16400, 300), ("any", 5, 33, 4110), ("any", 40, 33, 2060),
           ("any", 5, 33, 300), ("any", 16, 130, 2060), ("any", 5, 33, 8200),
           ("any", 5, 500, 8200),
           ("any", 100, 33, 300), ("any", 100, 33, 8200), ("any", 100, 16400, 780),
           ("any", 100, 4100, 4110), ("any", 100, 30000, 2060), ("any", 2050, 130, 8200),
           ("any", 200, 16400, 300), ("any", 200, 4100, 4110), ("any", 260, 30000, 300),
           ("any", 100, 4100, 16400), ("any", 600, 1000, 8200), ("any", 1000, 16400, 300),
           ("any", 1030, 1000, 1040), ("any", 4100, 2000, 300),
           ("lines", 130, 500, 300), ("lines", 200, 33, 8200), ("lines", 4100, 33, 300),
           ("lines", 1030, 33, 16400), ("lines", 130, 2000, 16400), ("lines", 5, 16400, 520),
           ("lines", 5, 4100, 4110), ("lines", 130, 16400, 8200), ("lines", 257, 1000, 140),
           ("any", 130, 500, 300), ("any", 100, 130, 8200), ("any", 40, 4100, 300),
           ("any", 4100, 33, 520), ("any", 1000, 33, 16400), ("any", 4100, 33, 2060),
           ("any", 4100, 33, 300), ("any", 100, 4100, 8200), ("any", 130, 2000, 2060),
           ("any", 2050, 500, 8200), ("any", 257, 1000, 140),
           ("odd", 5, 16400, 300), ("odd", 5, 33, 4110), ("odd", 40, 33, 300),
           ("odd", 40, 33, 2060), ("odd", 200, 16400, 300), ("odd", 130, 2000, 8200),
           ("odd", 1030, 500, 8200), ("odd", 2050, 2000, 520)]


@pytest.mark.parametrize("how,m,n,k", KERNELS)
def test_gemm_kernels(how, m, n, k):
    for end in (0, 4, 11, 12, 13, 28, 84, 85, 99, 100, 101, 115, 116, 211, 212, 213, 228):
        kk = k // 128 * 128 + end
        log(f"gemm {how} {m}x{n}x{kk}")
        pads, offs = {"lines": ((-kk % 16, -kk % 16 + 32, 0), (0, 16, 0)),
                      "any": ((5, 3, 0), (0, 0, 0)), "odd": ((5, 3, 0), (3, 1, 0))}[how]
        gemm_case("b", m, n, kk, pads, offs, m + n + kk, bias=False)


@pytest.mark.parametrize("t", LETTERS)
def test_gemm_workspace(t):
    """A caller's workspace: large enough it is used, too small it is refused
    before any work; the query covers every alignment."""
    import torch
    import blas_symmetric_mat_amd as X
    m, n, k = 40, 256, 20000
    need = X.q8gemm_workspace_bytes(m, n, k)
    assert need > 0 and X.q8gemm_workspace_bytes(1, 1, 16) == 0
    g = gen(11)
    a = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    one = torch.ones((n,), device="cuda")
    f = getattr(X, f"xsymv_q8gemm_{t}")
    want = torch.empty((m, n), device="cuda", dtype=dtype_of(t))
    f(m, n, k, a, k, one, w, k, one, None, want, n)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws = torch.empty((need,), dtype=torch.uint8, device="cuda")
    for nbytes in (need, 64):
        X.set_workspace(ws, nbytes, stream=st)
        c = torch.full((m, n), math.nan, device="cuda", dtype=dtype_of(t))
        torch.cuda.synchronize()
        if nbytes == need:
            f(m, n, k, a, k, one, w, k, one, None, c, n, stream=st)
            st.synchronize()
            assert torch.equal(c, want)
        else:
            with pytest.raises(X.XsymvError) as e:
                f(m, n, k, a, k, one, w, k, one, None, c, n, stream=st)
            assert e.value.code == 2000
            st.synchronize()
            assert bool(c.isnan().all())
        X.set_workspace(None, stream=st)


@pytest.mark.parametrize("t", LETTERS)
def test_gemm_of_empty_rows(t):
    """k = 0: the bias, or zeros."""
    import torch
    import blas_symmetric_mat_amd as X
    m, n = 5, 70
    one = torch.ones((max(m, n),), device="cuda")
    b = randn((n,), gen(1))
    for bias, want in ((b, b.to(dtype_of(t)).expand(m, n)), (None, torch.zeros((m, n)))):
        c = torch.full((m, n), math.nan, device="cuda", dtype=dtype_of(t))
        getattr(X, f"xsymv_q8gemm_{t}")(m, n, 0, None, 1, one, None, 1, one, bias, c, n)
        torch.cuda.synchronize()
        assert torch.equal(c, want.to("cuda", dtype_of(t)))


@pytest.mark.parametrize("m", [1, 20, 300])
def test_gemm_of_the_longest_rows(m):
    """k = 131071, all codes -128 or 127: the largest sums 32 bits can hold."""
    import torch
    import blas_symmetric_mat_amd as X
    k, n = 131071, 40
    a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one = torch.ones((max(m, n),), device="cuda")
    c = torch.empty((m, n), device="cuda")
    X.xsymv_q8gemm_s(m, n, k, a, k, one, w, k, one, None, c, n)
    torch.cuda.synchronize()
    want = torch.tensor([float(128 * 128 * k), float(-128 * 127 * k)], device="cuda").repeat(n // 2)
    assert torch.equal(c, want.expand(m, n))


def test_gemm_scale_that_is_not_finite():
    """A row whose scale is not finite (a row of zeros' codes beside it) is
    NaN throughout; the others are as without it."""
    import torch
    import blas_symmetric_mat_amd as X
    m, n, k = 40, 50, 64
    x = randn((m, k), gen(3))
    x[7, 9] = math.nan
    x[8, 1] = math.inf
    w = torch.randint(-127, 128, (n, k), generator=gen(4), device="cuda", dtype=torch.int8)
    q = torch.empty((m, k), dtype=torch.int8, device="cuda")
    sc = torch.empty((m,), device="cuda")
    X.xsymv_q8store_s(m, k, x, k, None, m, q, k, sc)
    c = torch.empty((m, n), device="cuda")
    X.xsymv_q8gemm_s(m, n, k, q, k, sc, w, k, torch.ones((n,), device="cuda"), None, c, n)
    torch.cuda.synchronize()
    assert bool(c[7].isnan().all()) and bool(c[8].isnan().all())
    rest = [i for i in range(m) if i not in (7, 8)]
    assert bool(c[rest].isfinite().all())


def test_offsets_past_32_bits():
    """Rows of a cache, of weights and of the output beyond 2^31 elements."""
    import torch
    import blas_symmetric_mat_amd as X
    n, cap = 128, (1 << 24) + 1000  # 2.1e9 codes
    q = torch.zeros((cap, n), dtype=torch.int8, device="cuda")
    sc = torch.zeros((cap,), device="cuda")
    slot = torch.tensor([0, cap - 1, (1 << 24) + 3], dtype=torch.int32, device="cuda")
    x = randn((3, n), gen(8))
    out = torch.empty_like(x)
    X.xsymv_q8store_s(3, n, x, n, slot, cap, q, n, sc)
    X.xsymv_q8read_s(3, n, q, n, sc, slot, cap, out, n)
    torch.cuda.synchronize()
    check_codes(x.double(), q[slot.long()], sc[slot.long()], 0.0, 1.0, "far rows")
    assert bool(((out - x).abs() <= 0.51 * sc[slot.long()][:, None]).all())
    assert int((sc != 0).sum()) == 3
    # the same codes as weights: a product with the cache's rows, few and many
    # rows of A, the last columns against the definition
    for m in (2, 70):
        a = torch.randint(-127, 128, (m, n), generator=gen(9), device="cuda", dtype=torch.int8)
        one = torch.ones((m,), device="cuda")
        c = torch.empty((m, cap), dtype=torch.float16, device="cuda")
        X.xsymv_q8gemm_h(m, cap, n, a, n, one, q, n, sc, None, c, cap)
        torch.cuda.synchronize()
        for s in slot.tolist():
            want = (a.double() @ q[s].double()) * sc[s].double()
            assert bool(((c[:, s].double() - want).abs()
                         <= want.abs() * (3 * U + 2.0 ** -11) * 1.01 + 2.0 ** -25).all())
        del c


def block(X, t, s, stream):
    """Norm, product with the gate and up weights, activation, product."""
    m, d, f = s["m"], s["d"], s["f"]
    getattr(X, f"xsymv_q8norm_{t}")(m, d, s["x"], d, t, s["r"], d, t, s["w"], 1e-5, s["h"], d,
                                    s["q"], d, s["sc"], stream=stream)
    getattr(X, f"xsymv_q8gemm_{t}")(m, 2 * f, d, s["q"], d, s["sc"], s["w1"], d, s["s1"], None,
                                    s["gu"], 2 * f, stream=stream)
    gu = s["gu"]
    getattr(X, f"xsymv_q8glu_{t}")(m, f, gu, 2 * f, gu[:, f:], 2 * f, s["q2"], f, s["sc2"],
                                   stream=stream)
    getattr(X, f"xsymv_q8gemm_{t}")(m, d, f, s["q2"], f, s["sc2"], s["w2"], f, s["s2"], None,
                                    s["y"], d, stream=stream)


def block_state(t, m, d, f, seed):
    import torch
    g = gen(seed)
    dt = dtype_of(t)

    def codes(a, b):
        return torch.randint(-127, 128, (a, b), generator=g, device="cuda", dtype=torch.int8)

    e = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    f32, i8 = torch.float32, torch.int8
    return dict(m=m, d=d, f=f, x=randn((m, d), g).to(dt), r=randn((m, d), g).to(dt),
                w=(1 + randn((d,), g, 0.1)).to(dt), h=e(m, d), q=e(m, d, dtype=i8),
                sc=e(m, dtype=f32), w1=codes(2 * f, d), s1=1e-3 * torch.rand((2 * f,), generator=g, device="cuda"),
                gu=e(m, 2 * f), q2=e(m, f, dtype=i8), sc2=e(m, dtype=f32), w2=codes(d, f),
                s2=1e-3 * torch.rand((d,), generator=g, device="cuda"), y=e(m, d))


@pytest.mark.parametrize("t,m,d,f", [("b", 1, 1024, 2816), ("h", 37, 520, 1100), ("s", 300, 768, 1500)])
def test_replayed_from_a_graph(t, m, d, f):
    """A feed-forward block captured into a graph: every replay, with eager
    work between, gives the eager bytes."""
    import torch
    import blas_symmetric_mat_amd as X
    log(f"graph {t} m={m}")
    s = block_state(t, m, d, f, seed=m)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    block(X, t, s, st)
    st.synchronize()
    eager = [s[k].clone() for k in ("h", "q", "sc", "gu", "q2", "sc2", "y")]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        block(X, t, s, st)
    for i in range(4):
        for k in ("h", "sc", "gu", "sc2", "y"):
            s[k].fill_(math.nan)
        s["q"].fill_(i)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, s[k]) for a, k in
                   zip(eager, ("h", "q", "sc", "gu", "q2", "sc2", "y")))


def test_graph_keeps_its_workspace():
    """A captured product whose stream's workspace a later, larger product
    outgrows, and one whose workspace the caller then replaces: every replay
    still gives the eager bytes."""
    import torch
    import blas_symmetric_mat_amd as X
    g = gen(21)
    n, k = 300, 20000
    w = torch.randint(-127, 128, (2048, k), generator=g, device="cuda", dtype=torch.int8)
    a = torch.randint(-127, 128, (300, k), generator=g, device="cuda", dtype=torch.int8)
    one = torch.ones((2048,), device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    small, large = X.q8gemm_workspace_bytes(40, n, k), X.q8gemm_workspace_bytes(300, 2048, k)
    assert large > max(small, 1 << 20)
    c = torch.empty((40, n), device="cuda")
    big = torch.empty((300, 2048), device="cuda")

    def product(m, cols, out, first=0):
        X.xsymv_q8gemm_s(m, cols, k, a[first:], k, one, w, k, one, None, out, cols, stream=st)

    product(40, n, c)
    st.synchronize()
    want = c.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        product(40, n, c)
    ws = torch.empty((large,), dtype=torch.uint8, device="cuda")
    for i in range(4):
        if i == 1:
            product(300, 2048, big)
        if i == 2:
            X.set_workspace(ws, large, stream=st)
            product(300, 2048, big)
        if i == 3:
            X.set_workspace(None, stream=st)
            product(20, n, big, first=100)
        st.synchronize()
        c.fill_(math.nan)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        st.synchronize()
        assert torch.equal(c, want)
    del graph
    torch.cuda.synchronize()


@pytest.mark.parametrize("n", [1, 8, 13])
def test_codes_to_the_bit(n):
    """Scales and codes are the definition's in 32 bits: a / 127, 127 / a and
    its products with the elements round once each, the products then half to
    even.  Rows of every magnitude down to the floor."""
    import torch
    import blas_symmetric_mat_amd as X
    m = 1 << 17
    r = np.random.default_rng(n)
    x = r.uniform(-1.0, 1.0, (m, n)).astype(np.float32)
    x = np.ldexp(x, r.integers(-110, 127, (m, 1))).astype(np.float32)
    q = torch.empty((m, n), device="cuda", dtype=torch.int8)
    s = torch.empty((m,), device="cuda")
    X.xsymv_q8store_s(m, n, torch.from_numpy(x).cuda(), n, None, m, q, n, s)
    a = np.maximum(np.abs(x).max(axis=1), np.float32(2.0 ** -100))
    assert np.array_equal(s.cpu().numpy(), a / np.float32(127.0))
    inv = (np.float32(127.0) / a)[:, None]
    assert np.array_equal(q.cpu().numpy(), np.rint(x * inv).astype(np.int8))


@pytest.mark.parametrize("m,n", [(70001, 128), (40003, 500), (9001, 2100), (4500, 9000),
                                 (2300, 16000), (1100, 66000)])
def test_many_rows_in_turn(m, n):
    """More rows than workgroups: each takes several in turn, with the bytes
    of calls on a few rows at a time.  One row in a hundred is not finite."""
    import torch
    import blas_symmetric_mat_amd as X
    log(f"rows in turn {m}x{n}")
    g = gen(m)
    x = torch.randn((m, n), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    x[::100, n // 2] = math.nan
    w = torch.randn((n,), generator=g, device="cuda").to(torch.bfloat16)
    u = x.flip(0).contiguous()

    def run(lo, hi):
        c = hi - lo
        out = []
        for f in (lambda q, s: X.xsymv_q8norm_b(c, n, x[lo:hi], n, "b", None, n, "b", w, 1e-5,
                                                None, n, q, n, s),
                  lambda q, s: X.xsymv_q8glu_b(c, n, x[lo:hi], n, u[lo:hi], n, q, n, s),
                  lambda q, s: X.xsymv_q8store_b(c, n, x[lo:hi], n, None, c, q, n, s)):
            q = torch.empty((c, n), device="cuda", dtype=torch.int8)
            s = torch.empty((c,), device="cuda")
            f(q, s)
            out += [q, s.view(torch.int32)]
        return out

    full = run(0, m)
    step = m // 3 if n < 9000 else 300
    for lo in range(0, m, step):
        hi = min(lo + step, m)
        for a, b in zip(full, run(lo, hi)):
            assert torch.equal(a[lo:hi], b), lo


def test_streams_of_their_own():
    """Two streams at once, each with its own buffers, give the bytes of one
    after the other."""
    import torch
    import blas_symmetric_mat_amd as X
    states = [block_state("b", 130, 1024, 2000, seed=i) for i in range(2)]
    want = []
    for s in states:
        block(X, "b", s, None)
        torch.cuda.synchronize()
        want.append(s["y"].clone())
        s["y"].fill_(math.nan)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, st in zip(states, streams):
            block(X, "b", s, st)
    torch.cuda.synchronize()
    assert all(torch.equal(s["y"], w) for s, w in zip(states, want))


def test_timing_records_each_call():
    import torch
    import blas_symmetric_mat_amd as X
    s = block_state("h", 4, 512, 700, seed=1)
    block(X, "h", s, None)
    torch.cuda.synchronize()
    X.timing_read()
    X.timing_enable(1)
    try:
        block(X, "h", s, None)
    finally:
        rec = X.timing_read()
        X.timing_enable(0)
    assert len(rec) == 4 and all(a > 0 for a, _ in rec)


def test_refusals_leave_no_trace():
    torch = torch_dev()
    import blas_symmetric_mat_amd as X
    q = torch.full((4, 8), 3, dtype=torch.int8, device="cuda")
    sc = torch.full((4,), 2.0, device="cuda")
    x = torch.ones((4, 8), device="cuda")
    with pytest.raises(X.XsymvError):
        X.xsymv_q8store_s(4, 8, x, 7, None, 4, q, 8, sc)
    torch.cuda.synchronize()
    assert bool((q == 3).all()) and bool((sc == 2.0).all())


def test_layer_of_prompt_and_tokens():
    """The example layer: a prompt at once and the same tokens one by one give
    the same bytes (rows do not depend on the rows beside them, the products'
    sums are exact, and the attention between them runs in 64 bits), and both
    are what the layer is in 64 bits up to the 8-bit rows' steps."""
    import torch
    from blas_symmetric_mat_amd import q8_layer
    g = gen(21)
    x = randn((23, 512), g).bfloat16()
    r = randn((23, 512), g).bfloat16()
    whole = q8_layer.Q8Layer(d=512, heads=4, f=1100, tokens=64, seed=3)
    single = q8_layer.Q8Layer(d=512, heads=4, f=1100, tokens=64, seed=3)
    y, h = whole(x, r)
    parts = [single(x[i:j], r[i:j]) for i, j in ((0, 7), (7, 8), (8, 9), (9, 20), (20, 23))]
    torch.cuda.synchronize()
    assert torch.equal(y, torch.cat([p[0] for p in parts]))
    assert torch.equal(h, torch.cat([p[1] for p in parts]))
    for (a, b), (c, d) in zip(whole.kv, single.kv):
        assert torch.equal(a, c) and torch.equal(b, d)
    want, want_h = q8_layer.plain(whole, x, r)
    # A code is off by at most half a step, evenly over it: its variance is
    # step^2 / 12, and a row's largest of some 500 numbers is about 3.5 times
    # their size, so a step is 3.5 / 127 and a row is off by 0.8 % of its size;
    # bfloat16 adds 0.17 % a rounding.  Eight such rows one after the other,
    # added as independent errors, stay under 2.5 %; the bound is twice that.
    assert ((y - want).norm() / want.norm()).item() < 0.05
    assert ((h - want_h).norm() / want_h.norm()).item() < 0.05
