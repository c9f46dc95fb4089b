"""Attention over a cache of 8-bit rows in pages, against its definition in 64 bits.

The bound of an output, with u = 2^-24, w the exact weights and A = sum_t w_t |v_t|:

* a score is a sum of hd products and a few more roundings: off by (hd + 16) u times the sum of the
  products' sizes, and (letter s) by what 22 bits of a row of q leave out, 2^-22 max|q| times the sum of
  |k|; its power is off by that plus 4 u |s| (its argument in units of log 2) and 2 u;
* weights are rounded to 11 bits (h, b) or 22 (s) before the product with the values, and not below
  2^-39 of the largest scale of a token's values times the largest code;
* sums of n tokens in 32 bits add n u A; the weights' error counts twice, in the sum that divides too;
* the result is rounded to its type, by half a step.
"""
import itertools
import math
import random

import pytest

from tests.test_gpu_q8 import LETTERS, U, Rows, dtype_of, gen, half_step

pytestmark = pytest.mark.gpu

NAN = float("nan")


class Case:
    """Sequences on pages of a cache: `lens` tokens, `counts` rows each; `groups`: list of (sequences,
    shared tokens).  Rows of the cache that no sequence sees hold scales of NaN and infinity."""

    def __init__(self, t, heads, kvheads, hd, ps, lens, counts=None, groups=(), seed=0, pad=0, off=0,
                 spare=3, spread=2.5, lead=0, tail=0, room=0):
        import torch
        g = gen(seed)
        self.t, self.heads, self.kvheads, self.hd, self.ps = t, heads, kvheads, hd, ps
        self.lens, self.seqs = list(lens), len(lens)
        self.groups = list(groups)
        start = list(itertools.accumulate(counts if counts is not None else [1] * self.seqs, initial=lead))
        self.counts = [b - a for a, b in zip(start, start[1:])]
        self.rows = start[-1] + tail
        need = [max(0, -(-n // ps)) for n in lens]
        self.ldt = max(need, default=0) + room
        firsts = list(itertools.accumulate((c for c, _ in self.groups), initial=0))
        table, used = [[-1] * self.ldt for _ in lens], 0
        for (a, b), (_, shared) in zip(zip(firsts, firsts[1:]), self.groups):
            held = shared // ps
            for i in range(a, b):
                for j in range(min(held, need[i])):
                    table[i][j] = used + j
            used += held
        for i in range(self.seqs):
            for j in range(need[i]):
                if table[i][j] < 0:
                    table[i][j] = used
                    used += 1
        self.pages = used + spare
        order = list(range(self.pages))
        random.Random(seed).shuffle(order)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table = ints([[order[p] if p >= 0 else -1 for p in r] for r in table]).reshape(self.seqs, self.ldt)
        self.len = ints(self.lens)
        self.start = None if counts is None and not lead and not tail else ints(start)
        self.first = ints(firsts) if self.groups else None
        self.shared = ints([s for _, s in self.groups]) if self.groups else None
        cap = self.pages * kvheads * ps
        self.k, self.v = (Rows(cap, hd, torch.int8, pad, off,
                               data=torch.randint(-127, 128, (cap, hd), generator=g, device="cuda").to(torch.int8))
                          for _ in range(2))
        self.ks, self.vs = (0.005 + 0.02 * torch.rand((cap,), generator=g, device="cuda") for _ in range(2))
        self.q = Rows(self.rows, heads * hd, dtype_of(t), pad, off,
                      data=torch.randn((self.rows, heads * hd), generator=g, device="cuda") * spread)
        self.out = Rows(self.rows, heads * hd, dtype_of(t), pad, off, fill=7)
        self.lse = torch.full((self.rows, heads), 7.0, device="cuda")
        self.scale = 1 / math.sqrt(hd)

    def spoil(self):
        """Scales that no row sees are no numbers."""
        import torch
        seen = torch.zeros((self.pages * self.kvheads * self.ps,), dtype=torch.bool, device="cuda")
        for i in range(self.seqs):
            at, ok = self.places(i)
            seen[at[:, ok].flatten()] = True
        for s in (self.ks, self.vs):
            s[~seen] = NAN
            s[torch.arange(s.numel(), device="cuda") % 3 == 0] = torch.where(
                seen, s, math.inf)[torch.arange(s.numel(), device="cuda") % 3 == 0]
        return self

    def places(self, i):
        """Cache rows (head, token) of sequence i, and which tokens have a page."""
        import torch
        n = max(0, min(self.lens[i], self.ldt * self.ps))
        tok = torch.arange(n, device="cuda")
        page = self.table[i].long()[tok // self.ps] if n else tok
        ok = (page >= 0) & (page < self.pages)
        head = torch.arange(self.kvheads, device="cuda")[:, None]
        return (page.clamp(0, max(0, self.pages - 1)) * self.kvheads + head) * self.ps + tok % self.ps, ok

    def call(self, stream=None, lse=True):
        import blas_symmetric_mat_amd as X
        getattr(X, "xsymv_q8attn_" + self.t)(
            self.rows, self.heads, self.kvheads, self.hd, self.q.t, self.q.ld, self.seqs, self.start, self.len,
            self.table, self.ldt, len(self.groups), self.first, self.shared, self.k.t, self.k.ld, self.ks,
            self.v.t, self.v.ld, self.vs, self.pages, self.ps, self.scale, self.out.t, self.out.ld,
            self.lse if lse else None, stream=stream)

    def expected(self):
        """out, its bound, lse and its bound, NaN where nothing is written."""
        import torch
        f64 = torch.float64
        out = torch.full((self.rows, self.heads, self.hd), NAN, dtype=f64, device="cuda")
        err, lse, lerr = out.clone(), out[:, :, 0].clone(), out[:, :, 0].clone()
        share = self.heads // self.kvheads
        row = int(self.start[0]) if self.start is not None else 0
        for i, c in enumerate(self.counts):
            if c == 0:
                continue
            at, ok = self.places(i)
            n = at.shape[1]
            k, v = self.k.t[at].to(f64), self.v.t[at].to(f64)
            ks, vs = self.ks[at].to(f64), self.vs[at].to(f64)
            q = self.q.t[row:row + c].to(f64).reshape(c, self.kvheads, share, self.hd).permute(1, 0, 2, 3)
            q = q.reshape(self.kvheads, c * share, self.hd)
            limit = max(0, min(self.lens[i], self.ldt * self.ps)) - c + 1 + torch.arange(c, device="cuda")
            limit = limit.repeat_interleave(share)[:, None]
            see = ok & (torch.arange(n, device="cuda") < limit)
            kt = k.transpose(1, 2).contiguous()
            s = torch.where(see, q @ kt * (ks[:, None] * self.scale), -math.inf)
            big = torch.where(see, q.abs() @ kt.abs() * (ks[:, None] * abs(self.scale)), 0.0)
            es = (self.hd + 16) * U * big
            if self.t == "s":
                es = es + 2.0 ** -22 * q.abs().amax(2)[:, :, None] * torch.where(
                    see, kt.abs().sum(1)[:, None] * (ks[:, None] * abs(self.scale)), 0.0)
            es = es + torch.where(see, 4 * U * s.abs() + 2 * U, 0.0)
            empty = ~see.any(1)
            if n:
                m = s.amax(2, keepdim=True).nan_to_num(neginf=0.0)
                e = torch.where(see, (s - m).exp(), 0.0)
                l = e.sum(2, keepdim=True)
                w = e / l.clamp_min(1e-300)
                es = es.amax(2, keepdim=True) + 4 * U * m.abs()
                vv = torch.where(ok[None, :, None], v * vs[..., None], 0.0)
                o, a = w @ vv, w @ vv.abs()
                part = 2.0 ** -22 if self.t == "s" else 2.0 ** -11
                top = torch.where(see, torch.where(ok, vs, 0.0)[:, None], 0.0).amax(2, keepdim=True)
                e_out = a * (part + 2 * es + 2 * n * U) + n * 2.0 ** -39 * 127 * top + o.abs() * half_step(self.t) + 1e-30
                ls = m[..., 0] + l[..., 0].log()
                e_lse = es[..., 0] + n * U + 4 * U * ls.abs() + 4 * U
            else:
                o = e_out = torch.zeros_like(q)
                ls, e_lse = q[..., 0], q[..., 0]
            o = torch.where(empty[None, :, None], 0.0, o)
            e_out = torch.where(empty[None, :, None], 0.0, e_out)
            ls = torch.where(empty[None], -math.inf, ls)

            def back(x, tail):
                return x.reshape(self.kvheads, c, share, *tail).transpose(0, 1).reshape(c, self.heads, *tail)

            out[row:row + c], err[row:row + c] = back(o, (self.hd,)), back(e_out, (self.hd,))
            lse[row:row + c], lerr[row:row + c] = back(ls, ()), back(e_lse, ())
            row += c
        return out, err, lse, lerr

    def check(self):
        import torch
        want, err, lse, lerr = self.expected()
        torch.cuda.synchronize()
        got = self.out.t.double().reshape(self.rows, self.heads, self.hd)
        written = ~lse.isnan()
        assert bool((got[~written] == 7).all()) and bool((self.lse[~written] == 7).all())
        assert self.out.intact()
        assert bool(got[written].isfinite().all())
        over = ((got - want).abs() / err.clamp_min(1e-300))[written]
        assert over.numel() == 0 or float(over.max()) <= 1, float(over.max())
        none = lse == -math.inf
        assert bool((self.lse[none] == -math.inf).all())
        some = written & ~none
        off = ((self.lse.double() - lse).abs() / lerr)[some]
        assert off.numel() == 0 or float(off.max()) <= 1, float(off.max())


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("hd", [16, 17, 31, 33, 64, 80, 128, 129, 200, 256])
def test_widths(t, hd):
    """Single tokens, every kind of head width and page, rows of the cache at odd addresses."""
    for heads, kvheads, ps, pad, off in ((4, 4, 16, 0, 0), (6, 2, 7, 3, 1), (8, 1, 64, 16, 0)):
        c = Case(t, heads, kvheads, hd, ps, [1, 70, 301, 64, 129], pad=pad, off=off, seed=hd).spoil()
        c.call()
        c.check()


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("heads,kvheads", [(1, 1), (7, 7), (8, 1), (14, 2), (16, 1), (17, 1), (40, 2), (130, 1)])
def test_heads(t, heads, kvheads):
    for counts in (None, [3, 0, 1, 9]):
        c = Case(t, heads, kvheads, 64, 16, [200, 5, 33, 100], counts, seed=heads).spoil()
        c.call()
        c.check()


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("ps", [1, 2, 13, 16, 64, 100, 1000])
def test_pages(t, ps):
    """Lengths around a tile's and a page's ends."""
    lens = [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, ps, ps + 1, 2 * ps]
    c = Case(t, 4, 2, 128, ps, lens, seed=ps, room=2).spoil()
    c.call()
    c.check()


@pytest.mark.parametrize("t", LETTERS)
def test_prompts(t):
    """Rows that see up to their own token: whole prompts, chunks of them, single tokens among them."""
    for lens, counts in (([40, 300, 129, 64], [40, 300, 129, 64]), ([500, 333, 20], [100, 1, 20]),
                         ([1000], [37]), ([257, 1, 2], [130, 1, 2])):
        c = Case(t, 6, 2, 128, 16, lens, counts, seed=len(lens)).spoil()
        c.call()
        c.check()


@pytest.mark.parametrize("t", LETTERS)
def test_rows_that_see_nothing(t):
    """Fewer tokens than rows, no tokens, negative lengths, lengths beyond the table; rows outside start;
    tokens without a page, or whole sequences."""
    c = Case(t, 4, 2, 64, 16, [3, 0, 40, 17], [5, 2, 0, 17], lead=2, tail=3).spoil()
    c.call()
    c.check()
    c = Case(t, 4, 2, 64, 16, [100, 90, 80, 100], seed=3)
    c.table[0, 2] = -1
    c.table[0, 6] = c.pages
    c.table[1] = 1 << 30
    c.table[3, 0] = -(1 << 31)
    c.len[2] = c.lens[2] = -5
    c.len[3] = c.lens[3] = 2000000000
    c.spoil()
    c.call()
    c.check()
    c = Case(t, 2, 2, 64, 16, [0, 0], [0, 0], tail=2)
    c.call()
    c.check()


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("hd,heads,kvheads", [(128, 8, 2), (80, 15, 5), (64, 4, 4), (256, 8, 1)])
def test_shared_tokens(t, hd, heads, kvheads):
    """Groups of sequences with common tokens: one, several, of one sequence, of none, with nothing
    in common, with more in common than a sequence has."""
    for groups, extra, counts in (([(5, 320)], [1, 70, 16, 200, 33], None),
                                  ([(3, 64), (1, 160), (0, 0), (4, 0)], [3, 50, 17, 9, 100, 5, 1, 260], None),
                                  ([(2, 48), (20, 240)], list(range(1, 23)), None),
                                  ([(4, 160)], [40, 12, 70, 300], [30, 1, 0, 70]),
                                  ([(12, 512)], list(range(1, 13)), [1] * 12)):
        shared = [s for n, s in groups for _ in range(n)]
        lens = [a + b for a, b in zip(shared, extra)]
        c = Case(t, heads, kvheads, hd, 16, lens, counts, groups, seed=len(lens)).spoil()
        c.call()
        c.check()
    # the second and third sequence are shorter than what the group shares
    c = Case(t, heads, kvheads, hd, 16, [200, 30, 0, 170], None, [(4, 160)])
    c.call()
    c.check()
    c = Case(t, heads, kvheads, hd, 16, [300, 170, 165, 170], [60, 30, 5, 1], [(4, 160)])
    c.call()
    c.check()


def test_groups_that_are_not_in_order():
    """Whatever first and shared hold, nothing faults, and sequences whose tables agree are right."""
    import torch
    c = Case("b", 4, 2, 64, 16, [200] * 6, None, [(6, 160)]).spoil()
    c.groups = [0, 0, 0]
    for first, shared in (([0, 6, 6, 6], [160, -5, 1 << 30]), ([0, 2, 4, 6], [160, 0, 1]),
                          ([2, 3, 3, 5], [100, 100, 100]), ([-7, 3, 100, 1 << 30], [160, 96, -1])):
        c.first, c.shared = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (first, shared))
        c.call()
        if first[0] >= 0:
            c.check()
        torch.cuda.synchronize()


@pytest.mark.parametrize("t", LETTERS)
def test_many_tokens(t):
    """One sequence over all compute units; and lengths that differ a thousand times."""
    c = Case(t, 4, 1, 128, 64, [100003]).spoil()
    c.call()
    c.check()
    c = Case(t, 8, 2, 64, 32, [60000, 7, 900, 1, 20000] + [50] * 40, seed=2).spoil()
    c.call()
    c.check()
    c = Case(t, 8, 2, 128, 64, [30100 + 7 * i for i in range(40)], None, [(40, 29952)], seed=5)
    c.call()
    c.check()


@pytest.mark.parametrize("t", LETTERS)
def test_scales_that_differ(t):
    """Scores of hundreds, one token above all, values whose scales differ by 2^40, rows of zeros, and
    tokens whose weight vanishes."""
    import torch
    c = Case(t, 4, 2, 128, 16, [333, 64, 1], spread=30.0, seed=9)
    c.vs[::5] *= 2.0 ** -30
    c.vs[::7] *= 2.0 ** 10
    c.ks[::11] = 2.0 ** -100 / 127
    c.q.t[1] = 0
    c.call()
    c.check()
    c = Case(t, 4, 2, 128, 16, [333, 640], seed=10)
    c.ks[:] = 0.02
    c.vs[:] = torch.linspace(-60, 0, c.vs.numel(), device="cuda").exp2()
    c.call()
    c.check()


@pytest.mark.parametrize("t", LETTERS)
def test_rows_that_are_no_numbers(t):
    """An infinity or a NaN in a row of q makes that row's head NaN and nothing else."""
    import torch
    c = Case(t, 6, 2, 64, 16, [100, 50, 70, 1], [4, 1, 20, 1], seed=4)
    c.call()
    torch.cuda.synchronize()
    clean = c.out.t.clone()
    c.q.t[2, 3 * 64 + 5] = math.inf
    c.q.t[7, 64 + 1] = NAN
    c.call()
    torch.cuda.synchronize()
    bad = torch.zeros((c.rows, c.heads), dtype=torch.bool, device="cuda")
    bad[2, 3] = bad[7, 1] = True
    got = c.out.t.reshape(c.rows, c.heads, 64)
    assert bool(got[bad].isnan().all()) and bool(c.lse[bad].isnan().all())
    assert torch.equal(got[~bad], clean.reshape(c.rows, c.heads, 64)[~bad])


def test_offsets_beyond_32_bits():
    """A cache whose codes take more than 2^32 bytes; pages at both ends are used."""
    import torch
    c = Case("b", 4, 2, 128, 64, [500, 300], seed=1)
    ld, pages = 1024, 70000
    cap = pages * 2 * 64
    assert cap * ld > 1 << 33
    k, v = (torch.zeros((cap, ld), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((cap,), NAN, device="cuda") for _ in range(2))
    move = torch.arange(c.pages, device="cuda")
    move = torch.where(move % 2 == 0, move, pages - 1 - move)
    rows = (move[:, None] * 128 + torch.arange(128, device="cuda")).flatten()
    k[rows, :128], v[rows, :128], ks[rows], vs[rows] = c.k.t, c.v.t, c.ks, c.vs
    c.k.t, c.v.t, c.ks, c.vs, c.pages = k, v, ks, vs, pages
    c.k.ld = c.v.ld = ld
    c.table = torch.where(c.table >= 0, move[c.table.long().clamp_min(0)].to(torch.int32), -1).contiguous()
    c.call()
    c.k.t, c.v.t = k[:, :128], v[:, :128]
    c.check()


@pytest.mark.parametrize("t", LETTERS)
def test_the_same_bytes(t):
    """Every call gives the same bytes, on any stream, with and without lse."""
    import torch
    c = Case(t, 8, 2, 128, 16, [5000 + i for i in range(9)], None, [(9, 4000)], seed=6)
    c.call()
    torch.cuda.synchronize()
    want, lse = c.out.t.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    for stream in (None, side, None):
        c.out.t.zero_()
        torch.cuda.synchronize()
        c.call(stream=stream, lse=stream is None)
        torch.cuda.synchronize()
        assert torch.equal(c.out.t, want) and torch.equal(c.lse, lse)


def test_two_streams_at_once():
    import torch
    cases = [Case("b", 8, 2, 128, 16, [20000 + 1000 * i] * 3, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.call(stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_a_captured_call():
    """Replays see what the arrays hold then: sequences that grow, between other calls on the stream; one
    graph is captured where there is no workspace yet, and a later call outgrows another's."""
    import torch
    for warm in (False, True):
        c = Case("b", 8, 2, 128, 16, [900, 40, 300, 7], None, [(2, 32)], seed=8).spoil()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        if warm:
            c.call(stream=side)
            torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.call()
        other = Case("b", 8, 1, 128, 16, [50000] * 8, seed=3)
        for lens in ([900, 40, 300, 7], [450, 33, 1, 0], [899, 39, 299, 6]):
            c.lens = lens
            c.len.copy_(torch.tensor(lens, dtype=torch.int32))
            c.out.t.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            c.check()
            other.call(stream=side)
            torch.cuda.synchronize()
        other.check()
        del graph


def test_an_installed_workspace():
    import torch
    import blas_symmetric_mat_amd as X
    c = Case("b", 8, 2, 128, 16, [9000] * 3, seed=8)
    side = torch.cuda.Stream()
    want = X.q8attn_workspace_bytes(c.rows, 8, 2, 128, 3, 0)
    buf = torch.empty((max(want, 1),), dtype=torch.uint8, device="cuda")
    try:
        X.set_workspace(buf, want, stream=side)
        c.call(stream=side)
        torch.cuda.synchronize()
        c.check()
        if want > 64:
            X.set_workspace(buf, 64, stream=side)
            with pytest.raises(X.XsymvError) as e:
                c.call(stream=side)
            assert e.value.code == 2000
    finally:
        X.set_workspace(None, 0, stream=side)


@pytest.mark.parametrize("seed", range(12))
def test_any_sizes(seed):
    """Sizes as they fall."""
    rng = random.Random(seed)
    for i in range(6):
        kvheads = rng.randint(1, 6)
        ps = rng.choice([1, 3, 16, 64, rng.randint(1, 150)])
        seqs = rng.randint(1, 12)
        cut = sorted(rng.randint(0, seqs) for _ in range(rng.randint(0, 3)))
        groups = [(b - a, rng.choice([0, ps * rng.randint(0, max(1, 600 // ps))])) for a, b in zip([0] + cut, cut + [seqs])]
        if rng.random() < 0.3:
            groups = []
        shared = [s for n, s in groups for _ in range(n)] or [0] * seqs
        counts = None if rng.random() < 0.5 else [rng.choice([0, 1, 2, rng.randint(1, 90)]) for _ in range(seqs)]
        lens = [s + rng.choice([1, rng.randint(1, 50), rng.randint(1, 700)]) for s in shared]
        c = Case(rng.choice(LETTERS), kvheads * rng.randint(1, 9), kvheads, rng.choice([64, 128, rng.randint(16, 256)]),
                 ps, lens, counts, groups, seed=seed * 100 + i, pad=rng.choice([0, 16, rng.randint(1, 20)]),
                 off=rng.choice([0, 0, 1, 8])).spoil()
        c.call()
        c.check()


def test_many_more_rows_than_tokens():
    """Six million rows of a sequence of three tokens: all but the last three see nothing (how a block's
    tokens grow with its place would not fit an int here)."""
    import torch
    c = Case("h", 1, 1, 16, 16, [3], [6000000])
    c.call()
    torch.cuda.synchronize()
    assert not bool(c.out.t[:-3].any()) and bool((c.lse[:-3] == -math.inf).all())
    few = Case("h", 1, 1, 16, 16, [3], [3])
    for name in ("k", "v", "q"):
        getattr(few, name).t.copy_(getattr(c, name).t[-getattr(few, name).m:])
    for name in ("ks", "vs", "table"):
        getattr(few, name).copy_(getattr(c, name))
    few.call()
    torch.cuda.synchronize()
    assert torch.equal(c.out.t[-3:], few.out.t) and torch.equal(c.lse[-3:], few.lse)


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("lens", [[0, 0, 400, 500, 0, 390, 70, 450, 0, 401], [0] * 21 + [70, 384, 600] + [0] * 3,
                                  [0, 100, 33, 64, 383, 16, 0, 250]])
def test_groups_whose_first_sequences_have_ended(t, lens):
    """Sequences without tokens, whose rows of the table name no page, and shorter ones than the shared
    tokens stand before those that have all of them, or none has."""
    for counts in (None, [min(n, 5) for n in lens]):
        c = Case(t, 8, 2, 64, 16, lens, counts, groups=[(len(lens), 384)], seed=len(lens)).spoil()
        c.call()
        c.check()


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf, 1e37])
def test_scales_of_tokens_that_some_rows_do_not_see(t, hd, bad):
    """A values' scale that is no number: rows that see its token are not finite, the others, of the same
    jobs, keep their bytes (few rows and many, and rows of a group)."""
    import torch
    for lens, counts, groups in (([90, 40], [6, 3], ()), ([700, 300], [400, 150], ()),
                                 ([200, 215, 230], [12, 12, 12], [(3, 192)])):
        c = Case(t, 4, 2, hd, 16, lens, counts, groups, seed=hd)
        c.vs.clamp_(min=0.01)
        at = []
        for i in range(len(lens)):  # the last row's token but one or two, of each sequence
            places, _ = c.places(i)
            at += places[:, lens[i] - 2].tolist()
        c.vs[at] = 1e-4  # (not the largest, so that without it nothing else changes)
        c.call()
        torch.cuda.synchronize()
        clean = c.out.t.clone()
        c.vs[at] = bad
        c.call()
        torch.cuda.synchronize()
        ends = list(itertools.accumulate(counts))
        sees = torch.zeros((c.rows,), dtype=torch.bool, device="cuda")
        for e in ends:
            sees[e - 2:e] = True
        assert torch.equal(c.out.t[~sees], clean[~sees])
        # (a code of zero times infinity, or a weight that is nothing in 16 bits, aside)
        assert bool((~c.out.t[sees].isfinite()).any(1).all())


class Fine(Case):
    """A case whose half results may be small: below 2^-14 half's numbers lie 2^-24 apart, so that an output is
    rounded by up to 2^-25 there, whatever its size."""

    def expected(self):
        out, err, lse, lerr = super().expected()
        return out, err + (2.0 ** -25 if self.t == "h" else 0.0), lse, lerr


SCALES = [0.5, 0.75, 1.0, 2.0, 4.0, -1.0, -0.0625, 0.0]


def at_scale(c, scale, bad=True):
    """The case at another scale, its keys made smaller so that scores stay as large as they were."""
    c.scale = scale
    if bad:
        c.spoil()
    c.ks *= 0.125 / max(abs(scale), 0.125)
    c.call()
    c.check()


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("scale", SCALES)
def test_rows_that_see_nothing_at_any_scale(t, scale):
    """Rows without a token, of a sequence or of a piece of it: those of test_rows_that_see_nothing, and
    sequences whose first pages are not there, for one row each and for many."""
    at_scale(Fine(t, 4, 2, 64, 16, [3, 0, 40, 17], [5, 2, 0, 17], lead=2, tail=3), scale)
    c = Fine(t, 4, 2, 64, 16, [100, 90, 80, 100], seed=3)
    c.table[0, 2] = -1
    c.table[0, 6] = c.pages
    c.table[1] = 1 << 30
    c.table[3, 0] = -(1 << 31)
    c.len[2] = c.lens[2] = -5
    at_scale(c, scale)
    for counts in (None, [5, 3, 1], [250, 100, 60]):
        c = Fine(t, 4, 2, 64, 16, [300, 150, 100], counts, seed=4)
        c.table[0, :8] = -1
        c.table[1, 4:] = -1
        c.table[2] = c.pages
        at_scale(c, scale)


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_cut_prompts_at_any_scale(t, scale, hd):
    """Pieces that begin behind a row's last token: of many rows, of a few, of a group."""
    at_scale(Fine(t, 4, 2, hd, 16, [3000, 700], [300, 500], seed=5), scale)
    at_scale(Fine(t, 4, 2, hd, 16, [2000, 40], [5, 3], seed=6), scale)
    at_scale(Fine(t, 4, 2, hd, 16, [200, 30, 0, 170], None, [(4, 160)]), scale, bad=False)
    at_scale(Fine(t, 8, 2, hd, 16, [600, 370, 165, 370], [60, 30, 5, 1], [(4, 320)]), scale, bad=False)
    at_scale(Fine(t, 8, 2, hd, 16, [2100 + i for i in range(20)] + [7, 0, 33], None, [(23, 2048)]), scale, bad=False)


@pytest.mark.parametrize("t", ["s", "b"])
@pytest.mark.parametrize("up,scale", [(2.0 ** 16, 1.0), (2.0 ** 100, 0.125), (2.0 ** -60, 1.0), (2.0 ** -115, -0.125)])
def test_rows_of_large_and_small_numbers(t, up, scale):
    """q far from one, keys' scales by as much the other way."""
    for lens, counts in (([3, 0, 40, 17], [5, 2, 0, 17]), ([3000, 700], [300, 500]), ([2000, 40], None)):
        c = Fine(t, 4, 2, 64, 16, lens, counts, seed=7, spread=2.5 * up)
        c.ks /= up
        at_scale(c, scale)


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("up", [2.0 ** -121, 2.0 ** -118, 2.0 ** 100])
def test_scales_far_from_one(t, up):
    for lens, counts in (([300, 170], [30, 100]), ([2000, 40], None)):
        c = Fine(t, 4, 2, 64, 16, lens, counts, seed=8)
        c.scale *= up
        c.ks /= up
        c.call()
        c.check()


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("large", [1e6, 1e12, 1e30])
def test_large_scales_of_tokens_that_some_rows_do_not_see(t, hd, large):
    """A token's values as large as they like: rows of the same jobs that do not see it keep their bytes, and
    those that do are right (half, which does not hold them, aside)."""
    import torch
    for lens, counts, groups in (([90, 40], [6, 3], ()), ([700, 300], [400, 150], ()),
                                 ([200, 215, 230], [12, 12, 12], [(3, 192)]),
                                 ([200, 195, 230], [1, 1, 1], [(3, 224)])):
        c = Fine(t, 4, 2, hd, 16, lens, counts, groups, seed=hd)
        if groups and groups[0][1] > lens[0]:
            # (a token that only the last sequence of the group sees; the others end before it)
            places, _ = c.places(2)
            at, sees = places[:, 220].tolist(), [2]
        else:
            at = [p for i in range(len(lens)) for p in c.places(i)[0][:, lens[i] - 2].tolist()]
            sees = [r for e in itertools.accumulate(counts) for r in (e - 2, e - 1)]
        c.vs[at] = 1e-4
        c.call()
        torch.cuda.synchronize()
        clean = c.out.t.clone()
        c.check()
        c.vs[at] = large
        c.call()
        torch.cuda.synchronize()
        mask = torch.zeros((c.rows,), dtype=torch.bool, device="cuda")
        mask[sees] = True
        assert torch.equal(c.out.t[~mask], clean[~mask])
        if t != "h":
            c.check()


def test_many_more_heads_than_a_block():
    """One row of a hundred million heads that share their keys (what its blocks see, summed over them, fits no int
    if each counts for a token more): its first, middle and last heads are what they are among a few."""
    import torch
    heads, n = 100_000_000, 64
    c = Fine("h", 1, 1, 16, 16, [100], seed=11)
    few = Fine("h", 3 * n, 1, 16, 16, [100], seed=11)
    q = torch.randn((heads * 16,), generator=gen(1), device="cuda", dtype=torch.float16) * 2.5
    out, lse = torch.full_like(q, 7), torch.full((heads,), NAN, device="cuda")
    at = [0, heads // 2, heads - n]
    few.q.t.copy_(torch.cat([q[16 * a:16 * (a + n)] for a in at])[None])
    for name in ("k", "v"):
        getattr(few, name).t.copy_(getattr(c, name).t)
    for name in ("ks", "vs", "table"):
        getattr(few, name).copy_(getattr(c, name))
    few.call()
    few.check()
    import blas_symmetric_mat_amd as X
    X.xsymv_q8attn_h(1, heads, 1, 16, q, heads * 16, 1, None, c.len, c.table, c.ldt, 0, None, None, c.k.t, c.k.ld, c.ks,
                     c.v.t, c.v.ld, c.vs, c.pages, c.ps, c.scale, out, heads * 16, lse)
    torch.cuda.synchronize()
    few.out.t.copy_(torch.cat([out[16 * a:16 * (a + n)] for a in at])[None])
    few.lse.copy_(torch.cat([lse[a:a + n] for a in at])[None])
    few.check()
    left = int(lse.isnan().sum())
    assert left == 0


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("hd", [64, 128, 200, 256])
@pytest.mark.parametrize("how", ["any", "rising", "falling", "steps"])
def test_scales_that_differ_from_token_to_token(t, hd, how):
    """Values' scales from 2^-30 to 2^8 times the usual in any order, each larger than the one before (so that every
    token of a step in which rows end begins another stretch), smaller, in blocks, with zeros: every row is as close
    as the scales that it sees allow."""
    import torch
    for lens, counts, groups in (([300, 90], [300, 90], ()), ([700, 333], [400, 150], ()), ([100, 33], [6, 3], ()),
                                 ([200, 215, 30, 230], [12, 12, 5, 12], [(4, 192)]), ([900, 150], [100, 1], ())):
        c = Fine(t, 8, 2, hd, 16, lens, counts, groups, seed=hd + len(lens))
        for i, n in reversed(list(enumerate(lens))):
            at = torch.arange(n, device="cuda") / max(n - 1, 1)
            if how == "any":
                e = torch.rand((n,), generator=gen(i), device="cuda")
            else:
                e = {"rising": at, "falling": 1 - at, "steps": (at * 9.99).floor() / 9}[how]
            scale = 0.02 * (e * 38 - 30).exp2()
            if how == "any":
                scale[::13] = 0
            places, _ = c.places(i)
            c.vs[places] = scale.expand_as(places)
        c.call()
        c.check()


def each_token(c):
    """Keys of zeros, so that all tokens that a row sees have the same weight, whose sum is a whole number, and
    values that are zero but for one code of 127 in each column, another token's in each: a column is
    127 vs / (the tokens that the row sees), two roundings of it and the type's, or nothing.  Every token in turn."""
    import torch
    c.k.t.zero_()
    c.vs.fill_(2.0 ** -6)
    share, longest = c.heads // c.kvheads, max(c.lens)
    for base in range(0, longest, c.hd * c.kvheads):
        c.v.t.zero_()
        token = base + torch.arange(c.kvheads * c.hd, device="cuda").view(c.kvheads, c.hd)
        col = torch.arange(c.hd, device="cuda")
        for i in range(c.seqs):
            at, _ = c.places(i)
            for h in range(c.kvheads):
                some = token[h] < at.shape[1]
                c.v.t[at[h, token[h][some]], col[some]] = 127
        c.call()
        torch.cuda.synchronize()
        row = 0
        for i, n in enumerate(c.counts):
            limit = (c.lens[i] - n + 1 + torch.arange(n, device="cuda"))[:, None, None]
            want = torch.where(token.repeat_interleave(share, 0) < limit, 127 * 2.0 ** -6 / limit.double(), 0.0)
            got = c.out.t[row:row + n].reshape(n, c.heads, c.hd).double()
            assert bool(((got - want).abs() <= want * (3 * U + half_step(c.t) * (1 + 3 * U))).all()), (base, i)
            lse = limit[:, :, 0].double().log().expand(n, c.heads)
            # (log l within a step and a half, and its rounding)
            assert bool(((c.lse[row:row + n].double() - lse).abs() <= 4 * U * lse).all()), (base, i)
            row += n


@pytest.mark.parametrize("t", LETTERS)
@pytest.mark.parametrize("hd", [80, 256])
def test_each_token_counts_once(t, hd):
    """A sequence over all compute units, prompts, groups: no token of a piece's ends is lost or taken twice."""
    each_token(Case(t, 8, 8, hd, 64, [12345]))
    each_token(Case(t, 8, 8, hd, 16, [5000, 33, 700], [1, 1, 1], room=3))
    each_token(Case(t, 16, 8, hd, 16, [3100, 900], [600, 333]))
    each_token(Case(t, 32, 8, hd, 16, [2100 + 19 * i for i in range(9)], None, [(9, 2048)]))
    each_token(Case(t, 16, 8, hd, 16, [1100 + 19 * i for i in range(5)], [7, 1, 40, 19, 2], [(2, 1024), (3, 800)]))
