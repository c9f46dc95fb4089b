"""Pages, attention and log probabilities as they are used together: several
answers to one prompt, against the layer of one sequence and against 64 bits."""
import pytest

from tests.test_gpu_q8 import gen, randn

pytestmark = pytest.mark.gpu

D, HEADS, F, PROMPT, LENGTH, ANSWERS = 512, 4, 1100, 37, 21, 5


def make(page=16, tokens=320):
    from blas_symmetric_mat_amd import q8_layer
    return q8_layer.Q8Answers(d=D, heads=HEADS, f=F, tokens=tokens, answers=ANSWERS, page=page, seed=3)


def tokens(seed):
    """x and r of the prompt, and of each answer's tokens (length x answers x d)."""
    g = gen(seed)
    return ([randn((PROMPT, D), g).bfloat16() for _ in range(2)],
            [randn((LENGTH, ANSWERS, D), g).bfloat16() for _ in range(2)])


def cached(layer, seq, count):
    """The codes and scales of a sequence's first tokens: (count x heads x hd, count x heads)."""
    t = layer.table.cpu()[seq]
    rows = [[(int(t[i // layer.page]) * HEADS + h) * layer.page + i % layer.page for h in range(HEADS)]
            for i in range(count)]
    return [(k[rows], s[rows]) for k, s in layer.kv]


@pytest.mark.parametrize("page", [1, 16, 64])
def test_answers_beside_single_sequences(page):
    """What an answer's tokens are in the cache depends on that token alone: the bytes are those of the layer
    of one sequence.  Outputs are what the layer is in 64 bits, as close as that layer's are: its attention is
    in 64 bits and rounded once, here the products' 16 bits add 2^-11 of the weights and values' sums to that
    rounding of 2^-8, which is one of the eight of the bound of 5 % there."""
    import torch
    from blas_symmetric_mat_amd import q8_layer
    many = make(page, 640)
    prompt, own = tokens(5)
    parts = [many.prompt(prompt[0][i:j], prompt[1][i:j]) for i, j in ((0, 20), (20, 21), (21, PROMPT))]
    many.fork()
    steps = [many.step(own[0][i], own[1][i]) for i in range(LENGTH)]
    torch.cuda.synchronize()
    for a in range(ANSWERS):
        x, r = (torch.cat([p, o[:, a]]) for p, o in zip(prompt, own))
        one = q8_layer.Q8Layer(d=D, heads=HEADS, f=F, tokens=PROMPT + LENGTH, seed=3)
        one(x, r)
        torch.cuda.synchronize()
        slots = one._slots(0, PROMPT + LENGTH).long()
        for (k, s), (k1, s1) in zip(cached(many, a + 1, PROMPT + LENGTH), one.kv):
            assert torch.equal(k.flatten(0, 1), k1[slots]) and torch.equal(s.flatten(), s1[slots])
        for part in (0, 1):
            got = torch.cat([p[part] for p in parts] + [s[part][a:a + 1] for s in steps]).double()
            want = q8_layer.plain(one, x, r)[part]
            assert ((got - want).norm() / want.norm()).item() < 0.05


def test_free_and_fork_again():
    """The pages of answers that have ended are there for others, whose outputs are those of the first."""
    import torch
    layer = make(16, 128)  # 8 pages: 3 of the prompt, one of each answer
    prompt, own = tokens(6)
    layer.prompt(*prompt)
    runs = []
    for _ in range(3):
        layer.fork()
        runs.append([layer.step(own[0][i], own[1][i]) for i in range(5)])
        with pytest.raises(ValueError):
            for i in range(LENGTH):
                layer.step(own[0][i], own[1][i])
        layer.free()
    torch.cuda.synchronize()
    for again in runs[1:]:
        for (y, h), (y2, h2) in zip(runs[0], again):
            assert torch.equal(y, y2) and torch.equal(h, h2)
    assert layer.refs.cpu().tolist() == [1] * 3 + [0] * 5
    assert layer.len.cpu().tolist() == [PROMPT] + [0] * ANSWERS


def test_a_captured_step():
    """A step with its logits and alternatives as a graph: replays with other rows, with eager work
    between, give the bytes of eager steps."""
    import torch
    from blas_symmetric_mat_amd import q8_layer
    eager, graphed = make(), make()
    prompt, own = tokens(7)
    head = q8_layer.Q8Weight(randn((1003, D), gen(8)))

    def step(layer, x, r):
        y, h = layer._step(x, r)
        return (y, h, *layer.likely(y, h, head, 9))

    for layer in (eager, graphed):
        layer.prompt(*prompt)
        layer.fork()
    x, r = own[0][0].clone(), own[1][0].clone()
    want = [step(eager, own[0][i], own[1][i]) for i in range(LENGTH)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [step(graphed, x, r)]  # the first step makes the workspaces of its stream
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(graphed, x, r)
    for i in range(1, LENGTH):
        x.copy_(own[0][i])
        r.copy_(own[1][i])
        graph.replay()
        got.append([t.clone() for t in out])
        if i % 5 == 0:
            assert int(torch.randn((1000, 100), device="cuda").isnan().sum()) == 0
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for t, u in zip(a, b):
            assert torch.equal(t, u)
    assert graphed.len.cpu().tolist() == [PROMPT] + [PROMPT + LENGTH] * ANSWERS


def test_moved_together():
    """Answers ended in the middle of the cache, the rest moved together: the others' next tokens stay as
    they would have been."""
    import torch
    import blas_symmetric_mat_amd as X
    a, b = make(4), make(4)
    prompt, own = tokens(9)
    for layer in (a, b):
        layer.prompt(*prompt)
        layer.fork()
        for i in range(LENGTH - 1):
            layer.step(own[0][i], own[1][i])
        X.xsymv_q8pages_free(2, layer.each[1:3].contiguous(), *layer._cache(), layer.refs)
    src, dst = (torch.empty((b.pages // 2,), dtype=torch.int32, device="cuda") for _ in range(2))
    live = torch.empty((1,), dtype=torch.int32, device="cuda")
    X.xsymv_q8pages_compact(b.seqs, b.table, b.pages, b.table, b.pages, b.pages, b.refs, b.refs, src, dst, live)
    rows = HEADS * b.page
    (k, ks), (v, vs) = b.kv
    X.xsymv_q8pages_copy(b.pages // 2, src, dst, b.pages, rows, b.hd, k, b.hd, ks, v, b.hd, vs, 1, b.pages * rows)
    torch.cuda.synchronize()
    count = int(live)
    assert bool((src[:1] >= count).all()) and bool((b.refs[:count] > 0).all()) and not bool(b.refs[count:].any())
    outs = [layer.step(own[0][LENGTH - 1], own[1][LENGTH - 1]) for layer in (a, b)]
    torch.cuda.synchronize()
    for t, u in zip(*outs):
        for row in (0, 3, 4):
            assert torch.equal(t[row], u[row])


@pytest.mark.parametrize("mode", [1, 2])
def test_timing_records_each_call(mode):
    """Calls with one kernel, with a join, with wide and narrow jobs: a record each, and the same bytes."""
    import torch
    import blas_symmetric_mat_amd as X
    many = make()
    prompt, own = tokens(11)
    y, h = many.prompt(*prompt)
    many.fork()
    head = q8_weight()
    many.likely(y, h, head, 5)
    many.likely(y[:1], h[:1], head, 5)
    torch.cuda.synchronize()
    X.timing_read()
    X.timing_enable(mode)
    try:
        index, value = many.likely(y, h, head, 5)
        single = many.likely(y[:1], h[:1], head, 5)
        many.step(own[0][0], own[1][0])
    finally:
        rec = X.timing_read()
        X.timing_enable(0)
    # a norm, a product and the log probabilities twice; the step's 13 calls, of which grow, slots and
    # three stores, a norm each, four products, the attention and the activation
    assert len(rec) >= 2 * 3 + 8 and all(a > 0 and b >= 0 for a, b in rec)
    assert torch.equal(index[:1], single[0]) and bool(((value[:1] - single[1]).abs() < 1e-5).all())


def q8_weight():
    from blas_symmetric_mat_amd import q8_layer
    return q8_layer.Q8Weight(randn((5003, D), gen(12)))
