"""Log probabilities, entropy and alternatives against their definition in 64 bits.

Bounds, with u = 2^-24: a power e^z (z = x - c, c within 20 of the row's largest logit where it counts)
is off by 3 u |z| (its argument's rounding in units of log 2, and the constant's on x) plus 2 u; sums of n
add n u relative to the sum; log l is off by that, relative errors becoming absolute; results round once more.
"""
import math

import pytest

from tests.test_gpu_q8 import LETTERS, U, Rows, dtype_of, gen

pytestmark = pytest.mark.gpu


def logits(m, n, t, seed=0, spread=3.0, pad=0, off=0):
    import torch
    return Rows(m, n, dtype_of(t), pad, off, data=torch.randn((m, n), generator=gen(seed), device="cuda") * spread)


def call(x, t, token, top, ldt=None, stream=None, skip=()):
    """logp, entropy, lse, index, value of rows x; what is in `skip` is not asked for."""
    import torch
    import blas_symmetric_mat_amd as X
    ldt = top if ldt is None else ldt
    f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    out = {"logp": f(x.m), "entropy": f(x.m), "lse": f(x.m),
           "index": torch.full((x.m, ldt), -7, dtype=torch.int32, device="cuda"), "value": f(x.m, ldt)}
    give = {k: None if k in skip else v for k, v in out.items()}
    getattr(X, "xsymv_logp_" + t)(x.m, x.n, x.t, x.ld, token, give["logp"], give["entropy"], give["lse"], top,
                                  give["index"], give["value"], ldt, stream=stream)
    torch.cuda.synchronize()
    return out


def check(x, token, got, top):
    """Against 64 bits, row by row in one go; the alternatives exactly."""
    import torch
    v = x.t.double()
    n = x.n
    m = v.amax(1)
    z = v - m[:, None]
    e = z.exp()
    l = e.sum(1)
    lse = m + l.log()
    size = torch.where(e > 0, z, 0.0).abs()
    rel = (3 * U * size + 2 * U)
    # the reference may lie up to 20 below the largest, and is itself up to |m| + 20 in size
    err_l = (e * rel).sum(1) / l + n * U + 6 * U * (m.abs() + 25)
    tol = err_l + 4 * U * lse.abs() + 4 * U
    assert bool(((got["lse"].double() - lse).abs() <= tol).all())
    if token is not None:
        ok = (token >= 0) & (token < n)
        want = torch.where(ok, v.gather(1, token.long().clamp(0, n - 1)[:, None])[:, 0] - lse, 0.0)
        same = got["logp"].double() == want
        assert bool((same | ((got["logp"].double() - want).abs() <= tol + 2 * U * want.abs())).all())
    p = e / l[:, None]
    ent = l.log() - torch.where(e > 0, p * z, 0.0).sum(1)
    # s / l: each term off by e's error and n roundings of sums of terms up to z in size (taken from the reference)
    err_e = tol + (p * (size + 25) * (2 * rel + 2 * n * U)).sum(1) + err_l * (l.log() + 25)
    assert bool(((got["entropy"].double() - ent).abs() <= err_e).all())
    if top:
        val, idx = torch.sort(x.t, dim=1, descending=True, stable=True)
        assert torch.equal(got["index"][:, :top].long(), idx[:, :top])
        want = val[:, :top].double() - lse[:, None]
        some = want > -math.inf
        assert bool((got["value"][:, :top][~some] == -math.inf).all())
        off = (got["value"][:, :top].double() - want).abs() <= tol[:, None] + 2 * U * want.abs()
        assert bool(off[some].all())


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("m,n", [(1, 1), (3, 7), (2, 8), (1, 255), (5, 256), (2, 2047), (3, 2049), (1, 4097),
                                 (1, 32000), (37, 50021), (300, 1003), (1500, 2500), (1, 262147), (9, 131072)])
def test_sizes(t, m, n):
    """Rows alone and many, lengths around a load's, a workgroup's and a part's ends, odd strides."""
    import torch
    for pad, off in ((0, 0), (3, 1)):
        x = logits(m, n, t, seed=n, pad=pad, off=off)
        token = torch.randint(0, n, (m,), generator=gen(m), device="cuda").to(torch.int32)
        for top in sorted({min(n, k) for k in (0, 1, 5, 20, 128)}):
            check(x, token, call(x, t, token, top, ldt=top + 2), top)
        assert x.intact()


@pytest.mark.parametrize("t", LETTERS)
def test_order(t):
    """Rows in ascending and descending order, equal throughout, of few values, with all large logits in
    one stretch, in one thread's places: the alternatives are the largest, the lowest index first."""
    import torch
    for n in (3000, 40000, 100001):
        up = torch.linspace(-8, 8, n, device="cuda")
        few = torch.randint(0, 3, (n,), generator=gen(n), device="cuda").float()
        block = torch.where((torch.arange(n, device="cuda") - n // 2).abs() < 900, 5.0 + up, up / 16)
        comb = torch.where(torch.arange(n, device="cuda") % 2048 < 8, 9.0 + up / 8, up / 16)
        zeros = torch.where(torch.arange(n, device="cuda") % 3 == 0, -0.0, 0.0)
        rows = torch.stack([up, up.flip(0), torch.zeros_like(up), few, block, comb, comb.flip(0), zeros])
        for many in (1, 200):  # parts of a row, and whole rows
            x = Rows(8 * many, n, dtype_of(t), data=rows.repeat(many, 1))
            for top in (1, 7, 128):
                check(x, None, call(x, t, None, top, skip=("logp",)), top)


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("m", [1, 700])
def test_masks(t, m):
    """Tokens of logit -infinity or the type's lowest value, rows of nothing else, single ones left."""
    import torch
    n = 5003
    lowest = torch.finfo(dtype_of(t)).min
    for mask in (-math.inf, lowest):
        x = logits(m, n, t, seed=3)
        x.t[torch.rand((m, n), generator=gen(1), device="cuda") < 0.9] = mask
        x.t[:, 17] = 1.0
        token = torch.full((m,), 17, dtype=torch.int32, device="cuda")
        check(x, token, call(x, t, token, 20), 20)
        x.t.fill_(mask)
        x.t[:, n - 1] = -2.5
        token.fill_(n - 1)
        got = call(x, t, token, 3)
        assert bool((got["logp"] == 0).all()) and bool((got["entropy"] == 0).all())
        assert got["index"].tolist() == [[n - 1, 0, 1]] * m
    x.t.fill_(lowest)
    got = call(x, t, token, 3)
    assert bool(((got["logp"] + math.log(n)).abs() <= (n + 40) * U).all())
    assert bool(((got["entropy"] - math.log(n)).abs() <= (n + 40) * U).all())
    x.t.fill_(-math.inf)
    got = call(x, t, token, 3)
    assert bool((got["lse"] == -math.inf).all()) and bool((got["logp"] == -math.inf).all())
    assert bool((got["entropy"] == 0).all()) and bool((got["value"] == -math.inf).all())
    assert got["index"].tolist() == [[0, 1, 2]] * m


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("m", [1, 600])
def test_rows_that_are_no_numbers(t, m):
    """A NaN or +infinity makes its row's numbers NaN, no other's, and the indexes still differ."""
    import torch
    n = 9000
    x = logits(m + 3, n, t, seed=5)
    token = torch.full((m + 3,), 100, dtype=torch.int32, device="cuda")
    clean = call(x, t, token, 16)
    x.t[0, 4321], x.t[1, 77] = float("nan"), math.inf
    x.t[2] = float("nan")
    got = call(x, t, token, 16)
    for k in ("logp", "entropy", "lse", "value"):
        assert bool(got[k][:3].isnan().all())
        assert torch.equal(got[k][3:], clean[k][3:])
    assert torch.equal(got["index"][3:], clean["index"][3:])
    for r in range(3):
        i = got["index"][r].tolist()
        assert len(set(i)) == 16 and all(0 <= v < n for v in i)


def test_what_is_asked_for():
    """Each output alone; tokens outside the row; entries beyond top stay."""
    import torch
    x = logits(5, 3001, "b", seed=1)
    token = torch.tensor([-1, 3001, 0, 3000, 1 << 30], dtype=torch.int32, device="cuda")
    whole = call(x, "b", token, 4, ldt=6)
    check(x, token, whole, 4)
    assert bool((whole["index"][:, 4:] == -7).all()) and bool((whole["value"][:, 4:] == 7).all())
    for keep in ("logp", "entropy", "lse"):
        got = call(x, "b", token if keep == "logp" else None, 0,
                   skip=[k for k in ("logp", "entropy", "lse", "index", "value") if k != keep])
        assert torch.equal(got[keep], whole[keep])
    got = call(x, "b", None, 4, ldt=6, skip=("logp", "entropy", "lse", "value"))
    assert torch.equal(got["index"], whole["index"])


@pytest.mark.parametrize("m", [1, 30])
def test_a_captured_call(m):
    """Without a workspace (rows whole) and with one (rows in parts): the same alternatives, numbers within
    the bound, replay after replay."""
    import torch
    import blas_symmetric_mat_amd as X
    x = logits(m, 70001, "h", seed=2)
    token = torch.zeros((m,), dtype=torch.int32, device="cuda")
    out = {"logp": torch.empty((m,), device="cuda"), "entropy": torch.empty((m,), device="cuda"),
           "lse": torch.empty((m,), device="cuda"), "index": torch.empty((m, 9), dtype=torch.int32, device="cuda"),
           "value": torch.empty((m, 9), device="cuda")}

    def run():
        X.xsymv_logp_h(m, x.n, x.t, x.ld, token, out["logp"], out["entropy"], out["lse"], 9, out["index"],
                       out["value"], 9)

    assert X.logp_workspace_bytes(m, x.n, 9) > 0
    for warm in (False, True):
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        if warm:
            with torch.cuda.stream(side):
                run()
            torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run()
        for seed in (3, 4, 5):
            x.t.copy_(torch.randn((m, x.n), generator=gen(seed), device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            check(x, token, out, 9)
        del graph


def test_many_rows_and_long_offsets():
    """Rows whose elements lie beyond 2^31."""
    import torch
    m, n, ld = 40, 1000, 1 << 26
    buf = torch.zeros((m * ld,), dtype=torch.bfloat16, device="cuda")
    x = Rows(1, 1, torch.bfloat16)
    x.m, x.n, x.ld = m, n, ld
    x.t = torch.as_strided(buf, (m, n), (ld, 1), 0)
    x.t.copy_(torch.randn((m, n), generator=gen(1), device="cuda"))
    token = torch.arange(m, device="cuda").to(torch.int32)
    check(x, token, call(x, "b", token, 10), 10)


def test_the_longest_row():
    """2^31 - 4096 logits: zeros but for two, the first and last of which are the largest.  l is exact up to
    the sums of the two (whole numbers of 8 a thread's step), so the bound is that of a few roundings."""
    import torch
    import blas_symmetric_mat_amd as X
    n = 2 ** 31 - 4096
    x = torch.zeros((1, n), dtype=torch.float16, device="cuda")
    x[0, 7] = x[0, n - 1] = 5.0
    token = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    f = [torch.empty((1,), device="cuda") for _ in range(3)]
    index, value = torch.empty((1, 3), dtype=torch.int32, device="cuda"), torch.empty((1, 3), device="cuda")
    X.xsymv_logp_h(1, n, x, n, token, *f, 3, index, value, 3)
    torch.cuda.synchronize()
    lse = math.log(n - 2 + 2 * math.exp(5.0))
    assert index.tolist() == [[7, n - 1, 0]]
    assert abs(f[2].item() - lse) < 64 * U * lse and abs(f[0].item() - (5 - lse)) < 64 * U * lse
    assert all(abs(a - b) < 64 * U * lse for a, b in zip(value[0].tolist(), (5 - lse, 5 - lse, -lse)))


def close(x, token, got):
    """As `check`, with what the sums are in fact.  A row is shared by `parts` workgroups of 256 threads, which take
    8 logits at a time: `loads` for a thread.  It adds the 8 by themselves, then to its sum; a workgroup's sums are
    added in eight steps, the row's in six: no logit passes more than loads + 30 additions.  The reference is the
    largest logit so far: a logit d below the row's is off by 3 u d + 2 u by its power and the reference's moves
    together, and by 3 u more for each of these, at most loads and 15 in joining."""
    import torch
    v, n = x.t.double(), x.n
    parts = max(1, min(1024 // x.m, -(-n // 2048), 64))  # (with lists of alternatives no fewer here)
    loads = -(-n // (2048 * parts)) + 1
    depth = loads + 30
    m = v.amax(1)
    d = m[:, None] - v
    e = (-d).exp()
    l = e.sum(1)
    log_l = l.log()
    some = e > 0
    d = torch.where(some, d, 0.0)
    rel = 3 * U * (d + loads + 15) + 2 * U
    err_l = (e * rel).sum(1) / l + depth * U
    # (logf within a step and a half)
    tol = err_l + 3 * U * log_l
    lse = m + log_l
    assert bool(((got["lse"].double() - lse).abs() <= tol + U * (lse.abs() + tol)).all())
    p = e / l[:, None]
    ent = log_l + (p * d).sum(1)
    err_s = (p * d * (rel + (depth + 4) * U)).sum(1) + (p * d).sum(1) * (err_l + 4 * U)
    assert bool(((got["entropy"].double() - ent).abs() <= tol + err_s + U * ent).all())
    want = v.gather(1, token.long()[:, None])[:, 0] - m - log_l
    off = (got["logp"].double() - want).abs()
    assert bool((off <= tol + 3 * U * want.abs()).all()), float((off - tol).max())


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("m,n", [(1, 1), (3, 9), (1, 2047), (5, 2049), (1, 32000), (37, 50021), (1500, 2500), (1, 262147),
                                 (9, 131072), (1100, 30001)])
def test_sizes_closely(t, m, n):
    import torch
    x = logits(m, n, t, seed=n + 1)
    token = torch.randint(0, n, (m,), generator=gen(m), device="cuda").to(torch.int32)
    for top in sorted({min(n, k) for k in (0, 5)}):
        close(x, token, call(x, t, token, top))


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("m,n", [(1, 262147), (1200, 8200)])
def test_rows_that_are_sure_of_a_token(t, m, n):
    """Two logits, 0 and d, the second in a later load of the first one's thread; nothing else.  The reference moves to
    the larger one, whose power is 1; the other's, below 0.78, is off by 2 u d + 5 u of itself, 5 u at most, its sum by
    1, the logarithm, below 0.58, by 2 more; so the likely token's log probability is within 10 u, however near 0 it
    is, the other's within 10 u and the rounding of a number as large as itself, and the entropy, which adds s / l
    with the errors of its power, product, quotient and constant, within 20 u."""
    import torch
    x = Rows(m, n, dtype_of(t))
    every = torch.linspace(0.25, 30.0, 240, device="cuda")
    token = torch.full((m,), 2048, dtype=torch.int32, device="cuda")
    for i in range(0, 240, 17 if m == 1 else 240):
        x.t.fill_(-math.inf)
        x.t[:, 0] = 0.0
        x.t[:, 2048] = every[i] if m == 1 else every.repeat(m // 240)
        d = x.t[:, 2048].double()
        rest = torch.log1p((-d).exp())
        for top in (0, 2):
            token.fill_(2048)
            got = call(x, t, token, top)
            assert bool(((got["logp"].double() + rest).abs() <= 10 * U).all()), (got["logp"].double() + rest).abs().max() / U
            assert bool(((got["lse"].double() - d - rest).abs() <= 10 * U + U * (d + 1)).all())
            ent = rest + d * (-d - rest).exp()
            assert bool(((got["entropy"].double() - ent).abs() <= 20 * U).all())
            token.fill_(0)
            got = call(x, t, token, top)
            assert bool(((got["logp"].double() + d + rest).abs() <= 10 * U + U * (d + 1)).all())
            if top:
                assert bool(((got["value"][:, 0].double() + rest).abs() <= 10 * U).all())


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("m,n", [(1, 40000), (2, 131073), (16, 70001), (300, 9001), (1500, 4099)])
def test_each_logit_counts_once(t, m, n):
    """Stretches of zeros, nothing else: l is the number of them exactly, lse and the entropy its logarithm (a step
    and a half, and a rounding).  They begin and end around loads', workgroups' and parts' ends."""
    import torch
    parts = max(1, min(1024 // m, -(-n // 2048), 64))
    each = -(-(-(-n // parts)) // 8) * 8
    ends = sorted({min(n, max(0, a + d)) for a in range(0, n + each, each) for d in (-9, -1, 0, 1, 8)}
                  | {min(n, 2048 * i + d) for i in range(0, 5) for d in (0, 7, 8)})
    pairs = list(zip(ends, ends[1:])) + [(a, n) for a in ends if a < n] + [(0, b) for b in ends if b]
    pairs += [pairs[-1]] * (-len(pairs) % m)
    x = Rows(m, n, dtype_of(t))
    token = torch.zeros((m,), dtype=torch.int32, device="cuda")
    at = torch.arange(n, device="cuda")
    for i in range(0, len(pairs), m):
        lo, hi = (torch.tensor(v, device="cuda")[:, None] for v in zip(*pairs[i:i + m]))
        x.t.copy_(torch.where((at >= lo) & (at < hi), 0.0, -math.inf))
        token.copy_(hi[:, 0] - 1)
        got = call(x, t, token, 0)
        want = (hi - lo)[:, 0].double().log()
        for k, sign in (("lse", 1), ("entropy", 1), ("logp", -1)):
            assert bool(((sign * got[k].double() - want).abs() <= 4 * U * want).all()), k


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("m", [1, 3000])
def test_rows_without_logits(t, m):
    """Nothing is likely: every output is written."""
    import torch
    x = Rows(m, 0, dtype_of(t))
    token = torch.zeros((m,), dtype=torch.int32, device="cuda")
    got = call(x, t, token, 0)
    assert bool((got["lse"] == -math.inf).all())
    assert bool((got["logp"] == 0).all()) and bool((got["entropy"] == 0).all())
