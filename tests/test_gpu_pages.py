"""The pages of a cache of 8-bit rows: every entry, count and byte against a plain model."""
import random

import pytest

from tests.pages_model import Model
from tests.test_gpu_q8 import Rows, gen

pytestmark = pytest.mark.gpu


def ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pages:
    """A model and the same on the device."""

    def __init__(self, seqs, ldt, pages, ps):
        self.m = Model(seqs, ldt, pages, ps)
        self.len, self.refs = ints(self.m.len), ints(self.m.refs)
        self.table = ints(self.m.table).reshape(seqs, ldt)

    @property
    def args(self):
        m = self.m
        return m.seqs, self.len, self.table, m.ldt, m.pages, m.ps

    def same(self):
        import torch
        torch.cuda.synchronize()
        assert self.len.tolist() == self.m.len
        assert self.refs.tolist() == self.m.refs
        for s, n in enumerate(self.m.len):  # entries behind a sequence's pages mean nothing
            held = -(-n // self.m.ps)
            assert self.table[s, :held].tolist() == self.m.table[s][:held]

    def grow(self, seq, add):
        import blas_symmetric_mat_amd as X
        got = ints([-9] * len(seq))
        X.xsymv_q8pages_grow(len(seq), ints(seq), ints(add), *self.args, self.refs, got)
        want = self.m.grow(seq, add)
        assert got.tolist() == want
        self.same()
        return want

    def fork(self, parent, child):
        import blas_symmetric_mat_amd as X
        src, dst = ints([-9] * len(parent)), ints([-9] * len(parent))
        X.xsymv_q8pages_fork(len(parent), ints(parent), ints(child), *self.args, self.refs, src, dst)
        want = self.m.fork(parent, child)
        assert (src.tolist(), dst.tolist()) == want
        self.same()
        return want

    def free(self, seq):
        import blas_symmetric_mat_amd as X
        X.xsymv_q8pages_free(len(seq), ints(seq), *self.args, self.refs)
        self.m.free(seq)
        self.same()

    def compact(self, place):
        """`place`: the results take the place of what they are made from."""
        import torch
        import blas_symmetric_mat_amd as X
        m = self.m
        out, ldo = (self.table, m.ldt) if place else (torch.full((m.seqs, m.ldt + 3), -9, dtype=torch.int32, device="cuda"), m.ldt + 3)
        rout = self.refs if place else ints([-9] * m.pages)
        src, dst, live = ints([-9] * (m.pages // 2)), ints([-9] * (m.pages // 2)), ints([-9])
        X.xsymv_q8pages_compact(m.seqs, self.table, m.ldt, out, ldo, m.pages, self.refs, rout, src, dst, live)
        torch.cuda.synchronize()
        table, refs, wsrc, wdst, wlive = m.compact()
        assert live.tolist() == [wlive] and src.tolist() == wsrc and dst.tolist() == wdst
        assert rout.tolist() == refs
        assert out[:, :m.ldt].tolist() == table
        if not place:
            assert bool((out[:, m.ldt:] == -9).all())
        m.table, m.refs = table, refs
        self.table, self.refs = out[:, :m.ldt].contiguous(), rout
        return wsrc, wdst, wlive


def test_a_life():
    """Sequences grown, forked, freed and moved together in any order, over small caches that run full."""
    for seed in range(25):
        rng = random.Random(seed)
        seqs, pages, ps = rng.randint(1, 12), rng.randint(1, 60), rng.choice([1, 4, 16])
        p = Pages(seqs, rng.randint(1, 12), pages, ps)
        for _ in range(14):
            n = rng.randint(1, 8)
            some = [rng.randint(-1, seqs) for _ in range(n)]
            what = rng.choice(["grow", "grow", "fork", "fork", "free", "compact"])
            if what == "grow":
                p.grow(some, [rng.choice([0, 1, 1, -3, ps, rng.randint(1, 3 * ps)]) for _ in some])
            elif what == "fork":
                p.fork(some, [rng.randint(-1, seqs) for _ in some])
            elif what == "free":
                p.free(some)
            else:
                p.compact(rng.random() < 0.5)


@pytest.mark.parametrize("n", [1, 16, 17, 1000, 1025, 8192])
def test_many_at_once(n):
    """Lists longer than a workgroup, more free pages asked for than there are, the last ones left out."""
    p = Pages(n + 2, 40, 3 * n + 7, 16)
    p.grow([n, n + 1], [16 * 5 + 3, 32])
    p.fork([n if i % 3 else n + 1 for i in range(n)], list(range(n)))
    p.grow(list(range(n)), [i % 40 for i in range(n)])
    p.free([i for i in range(n) if i % 2] + [1, 1])
    p.compact(False)
    p.grow(list(range(n)), [500] * n)
    p.free(list(range(n + 2)))
    assert not any(p.m.refs)


def test_long_tables():
    """Rows of the table of thousands of pages, shared by many; refs over several of the search's rounds."""
    p = Pages(40, 20000, 70001, 1)
    p.grow([0], [19990])
    p.fork([0] * 30, list(range(1, 31)))
    p.grow(list(range(40)), [9] * 40)
    p.grow([31, 32, 33], [19000, 19000, 19000])
    p.free([0, 31] + list(range(1, 20)))
    p.compact(False)
    p.compact(True)
    p.free(list(range(40)))
    p.compact(True)


def test_what_device_arrays_hold():
    """Lengths out of range, entries that are no pages: nothing faults, and what is said holds."""
    import torch
    p = Pages(6, 4, 20, 8)
    p.grow([0, 1, 2], [30, 8, 9])
    for t in (p.table[1], p.table[2]):
        t[0] = 1 << 30
    p.m.table[1][0] = p.m.table[2][0] = 1 << 30
    p.free([1, 2, 3])
    p.len[3] = p.m.len[3] = -7
    p.len[4] = p.m.len[4] = 2000000000
    p.m.free([3, 4])
    import blas_symmetric_mat_amd as X
    X.xsymv_q8pages_free(2, ints([3, 4]), *p.args, p.refs)
    p.same()
    p.grow([5, 5], [2000000000, 1])
    p.grow([0], [2147483647])
    torch.cuda.synchronize()


def test_slots():
    import torch
    import blas_symmetric_mat_amd as X
    for ps, kvheads in ((1, 3), (16, 8), (7, 1)):
        p = Pages(5, 9, 60, ps)
        p.grow([0, 1, 3, 4], [9 * ps, 1, 3, 2 * ps])
        p.table[4, 0] = p.m.table[4][0] = 60
        for start in (None, [0, 2, 3, 3, 9, 9 + ps]):
            rows = start[-1] + 2 if start else 5
            slot = ints([-9] * (rows * kvheads))
            X.xsymv_q8pages_slots(rows, kvheads, ints(start) if start else None, *p.args, slot)
            want = p.m.slots(start, kvheads)
            torch.cuda.synchronize()
            assert slot.tolist()[:len(want)] == want and set(slot.tolist()[len(want):]) <= {-9}


@pytest.mark.parametrize("hd,pad,rows,layers", [(128, 0, 128, 1), (80, 3, 35, 3), (1, 0, 5, 1), (15, 1, 7, 2),
                                                (17, 0, 3, 2), (256, 16, 512, 1), (64, 0, 4096, 2), (100, 0, 1, 1)])
def test_copy(hd, pad, rows, layers):
    """Pages copied in every layer, gaps and other pages left alone, numbers that are no pages passed over;
    keys and values, and one matrix alone."""
    import torch
    import blas_symmetric_mat_amd as X
    pages = 24
    stride = pages * rows + 5
    cap = stride * (layers - 1) + pages * rows
    g = gen(hd)
    src = [3, 5, -1, 7, 24, 2, 9, 9, 1, -2]
    dst = [10, 11, 12, 25, 13, -1, 14, 15, 1, -2]
    moves = [(3, 10), (5, 11), (9, 14), (9, 15)]
    for both in (True, False):
        k, v = (Rows(cap, hd, torch.int8, pad, 1, fill=5,
                     data=torch.randint(-127, 128, (cap, hd), generator=g, device="cuda").to(torch.int8)) for _ in range(2))
        ks, vs = (torch.rand((cap,), generator=g, device="cuda") for _ in range(2))
        want = [t.clone() for t in (k.t, ks, v.t, vs)]
        for w in want if both else want[:2]:
            for layer in range(layers):
                for a, b in moves:
                    at = layer * stride
                    w[at + b * rows:at + (b + 1) * rows] = w[at + a * rows:at + (a + 1) * rows].clone()
        X.xsymv_q8pages_copy(len(src), ints(src), ints(dst), pages, rows, hd, k.t, k.ld, ks, v.t if both else None,
                             v.ld, vs if both else None, layers, stride)
        torch.cuda.synchronize()
        for got, w in zip((k.t, ks, v.t, vs), want):
            assert torch.equal(got, w)
        assert k.intact() and v.intact()


def test_copy_beyond_32_bits():
    """Pages whose codes lie beyond 2^32 bytes."""
    import torch
    import blas_symmetric_mat_amd as X
    pages, rows, hd = 36000, 512, 256
    k = torch.zeros((pages * rows, hd), dtype=torch.int8, device="cuda")
    ks = torch.zeros((pages * rows,), device="cuda")
    k[-rows:] = 3
    ks[-rows:] = 0.5
    X.xsymv_q8pages_copy(1, ints([pages - 1]), ints([pages - 3]), pages, rows, hd, k, hd, ks, None, hd, None)
    torch.cuda.synchronize()
    at = (pages - 3) * rows
    assert bool((k[at:at + rows] == 3).all()) and bool((ks[at:at + rows] == 0.5).all())
    assert int(k[:at].count_nonzero()) == 0 and int(k[at + rows:-rows].count_nonzero()) == 0


def test_a_captured_step():
    """A search's step in a graph: answers end, the best are forked, take a token each; every replay does
    what the calls do eagerly."""
    import torch
    import blas_symmetric_mat_amd as X
    seqs, ldt, pages, ps = 9, 12, 80, 16
    p = Pages(seqs, ldt, pages, ps)
    p.grow([0], [100])
    parent, child, one = ints([0, 0, 0, 0]), ints([1, 2, 3, 4]), ints([1, 1, 1, 1])
    src, dst, got, slot = ints([0] * 4), ints([0] * 4), ints([0] * 4), ints([0] * 8)
    k = torch.randint(-127, 128, (pages * 2 * ps, 64), generator=gen(1), device="cuda").to(torch.int8)
    ks = torch.rand((pages * 2 * ps,), generator=gen(2), device="cuda")
    start = ints([0, 0, 1, 2, 3, 4, 4, 4, 4, 4])

    def step():
        X.xsymv_q8pages_free(4, child, *p.args, p.refs)
        X.xsymv_q8pages_fork(4, parent, child, *p.args, p.refs, src, dst)
        X.xsymv_q8pages_copy(4, src, dst, pages, 2 * ps, 64, k, 64, ks, None, 64, None)
        X.xsymv_q8pages_grow(4, child, one, *p.args, p.refs, got)
        X.xsymv_q8pages_slots(4, 2, start, *p.args, slot)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for grown in (0, 5, 7, 4):
        if grown:
            p.grow([0], [grown])
        graph.replay()
        torch.cuda.synchronize()
        p.m.free([1, 2, 3, 4])
        want = p.m.fork([0] * 4, [1, 2, 3, 4])
        assert (src.tolist(), dst.tolist()) == want
        p.m.grow([1, 2, 3, 4], [1] * 4)
        p.same()
        assert slot.tolist() == p.m.slots(start.tolist(), 2)
        for a, b in zip(*want):
            if a >= 0:
                assert torch.equal(k[a * 32:a * 32 + 32], k[b * 32:b * 32 + 32])
                assert torch.equal(ks[a * 32:a * 32 + 32], ks[b * 32:b * 32 + 32])


def test_the_most_pages():
    """As many pages as an int counts, of which the last three are free, and one used among free ones."""
    import torch
    import blas_symmetric_mat_amd as X
    pages = 2 ** 31 - 1
    length, table = ints([0, 0, 0]), torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    refs = torch.ones((pages,), dtype=torch.int32, device="cuda")
    refs[pages - 3:] = 0
    got = ints([0, 0])
    X.xsymv_q8pages_grow(2, ints([1, 0]), ints([2, 1]), 3, length, table, 4, pages, 1, refs, got)
    torch.cuda.synchronize()
    assert got.tolist() == [2, 1] and length.tolist() == [1, 2, 0]
    assert table[1, :2].tolist() == [pages - 3, pages - 2] and table[0, 0].item() == pages - 1
    assert refs[pages - 3:].tolist() == [1, 1, 1]
    refs.zero_()
    refs[pages - 2] = 5
    table.fill_(-1)
    table[2, 3] = pages - 2
    src, dst = (torch.zeros((pages // 2,), dtype=torch.int32, device="cuda") for _ in range(2))
    live = ints([7])
    X.xsymv_q8pages_compact(3, table, 4, table, 4, pages, refs, refs, src, dst, live)
    torch.cuda.synchronize()
    assert live.tolist() == [1] and src[:2].tolist() == [pages - 2, -1] and dst[:2].tolist() == [0, -1]
    assert refs[0].item() == 5 and not bool(refs[1:].any())
    assert table.flatten().tolist() == [-1] * 11 + [0]
    assert bool((src[1:] == -1).all()) and bool((dst[1:] == -1).all())


@pytest.mark.parametrize("mode", [1, 2])
def test_timing_records_each_call(mode):
    import blas_symmetric_mat_amd as X
    p = Pages(40, 30, 400, 4)
    p.grow([0, 1], [70, 41])
    X.timing_read()
    X.timing_enable(mode)
    try:
        p.fork([0, 1], [2, 3])           # one launch
        p.fork([0, 1] * 9, list(range(4, 22)))  # two
        p.grow([5], [3])
        p.free([0, 7])
        p.compact(True)
    finally:
        rec = X.timing_read()
        X.timing_enable(0)
    assert len(rec) == 5 and all(a > 0 and b >= 0 for a, b in rec)
    if mode == 1:
        assert [b > 0 for _, b in rec] == [False, True, False, False, True]


def test_refused_sequences_stay_as_they_are():
    """Lengths out of range of sequences that grow or fork refuses stay what they are, also where a sequence is
    listed twice; one that grows counts from none, or takes the place of an empty one."""
    import torch
    import blas_symmetric_mat_amd as X
    seqs, ldt, pages, ps = 8, 3, 7, 4
    table = torch.full((seqs, ldt), -1, dtype=torch.int32, device="cuda")
    refs = ints([0] * pages)
    big = 2000000000
    length = ints([-5, big, -(2 ** 31), -9, 13, -1, 2 ** 31 - 1, 0])
    got = ints([-9] * 9)
    # 2: more than its row has room for; 3: grows; 6: has no room; 5: not enough pages are left
    X.xsymv_q8pages_grow(9, ints([0, 1, 2, 2, 3, 4, 5, 6, 7]), ints([0, 1, 13, 1, 9, 1, 12, -1, 12]), seqs, length, table,
                         ldt, pages, ps, refs, got)
    torch.cuda.synchronize()
    assert got.tolist() == [0, 0, 0, 0, 9, 0, 12, 0, 0]
    assert length.tolist() == [-5, big, -(2 ** 31), 9, 13, 12, 2 ** 31 - 1, 0]
    assert table[3].tolist() == [0, 1, 2] and table[5].tolist() == [3, 4, 5] and refs.tolist() == [1] * 6 + [0]
    src, dst = ints([-9] * 7), ints([-9] * 7)
    # 0 takes the last page; 2 finds none; 9 does not exist; 5 and 1 are not empty
    X.xsymv_q8pages_fork(7, ints([3, 3, 3, 9, 3, 5, 5]), ints([0, 2, 2, 7, 5, 1, 9]), seqs, length, table, ldt, pages, ps,
                         refs, src, dst)
    torch.cuda.synchronize()
    assert src.tolist() == [2, -2, -2, -2, -2, -2, -2] and dst.tolist() == [6, -2, -2, -2, -2, -2, -2]
    assert length.tolist() == [9, big, -(2 ** 31), 9, 13, 12, 2 ** 31 - 1, 0]
    assert table[0].tolist() == [0, 1, 6] and refs.tolist() == [2, 2, 1, 1, 1, 1, 1]
    # many forks (tables in a launch of their own) of a sequence without a page left
    n = 40
    length, table = ints([6, -3] + [-i for i in range(n)]), torch.full((n + 2, 2), -1, dtype=torch.int32, device="cuda")
    table[0] = ints([0, 1])
    refs = ints([1, 1, 0])
    src, dst = ints([-9] * n), ints([-9] * n)
    X.xsymv_q8pages_fork(n, ints([0] * n), ints(list(range(2, n + 2))), n + 2, length, table, 2, 3, 4, refs, src, dst)
    torch.cuda.synchronize()
    assert src.tolist() == [1] + [-2] * (n - 1) and dst.tolist() == [2] + [-2] * (n - 1)
    assert length.tolist() == [6, -3, 6] + [-i for i in range(1, n)] and refs.tolist() == [2, 1, 1]
