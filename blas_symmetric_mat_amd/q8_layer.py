"""One layer of a decoder that serves from 8 bits, on the library's 8-bit row
operators: an example of their use together, and the path their tests run.
Q8Layer holds one sequence, Q8Answers several answers to one prompt.

    python -m blas_symmetric_mat_amd.q8_layer

The layer holds its weights as rows of codes with a scale each and keeps the
keys and values of a sequence in a cache of 8-bit rows, one row a token and
head.  A call takes a prompt's tokens or a single one:

    h  = x + r, normalised                         xsymv_q8norm_*
    q, k, v = h Wqkv^T                             xsymv_q8gemm_*
    k, v to their rows of the cache, read back     xsymv_q8store_*, xsymv_q8read_*
    attention over the sequence's tokens           (elementary torch operations)
    o  = attention Wo^T                            xsymv_q8store_* (rows in 8 bits), q8gemm
    h  = o + h, normalised                         xsymv_q8norm_*
    g, u = h Wgu^T;  g / (1 + exp(-g)) * u         xsymv_q8gemm_*, xsymv_q8glu_*
    x  = that Wd^T; the next layer adds h          xsymv_q8gemm_*

Q8Answers keeps the cache in pages that its answers share with the prompt:

    the prompt's tokens get pages, the answers get the prompt's
                                                   xsymv_q8pages_grow, _fork, _copy
    k, v to their rows of the cache                xsymv_q8pages_slots, xsymv_q8store_*
    attention, the prompt's tokens read once       xsymv_q8attn_*
    an answer's next token, from logits            xsymv_logp_*
    answers that have ended                        xsymv_q8pages_free
"""
from __future__ import annotations

import math

import blas_symmetric_mat_amd as X


class Q8Weight:
    """A matrix of n rows of k numbers as codes and scales."""

    def __init__(self, w):
        import torch
        self.n, self.k = w.shape
        w = w.float().contiguous()
        self.codes = torch.empty((self.n, self.k), dtype=torch.int8, device=w.device)
        self.scale = torch.empty((self.n,), dtype=torch.float32, device=w.device)
        X.xsymv_q8store_s(self.n, self.k, w, self.k, None, self.n, self.codes, self.k, self.scale)

    def values(self):
        return self.codes.double() * self.scale.double()[:, None]


class Q8Layer:
    """d: width, heads of size hd, f: width of the hidden layer, tokens: the
    cache's room; bfloat16 throughout, the residual stream included."""

    def __init__(self, d, heads, f, tokens, seed=0, eps=1e-5):
        import torch
        self.d, self.heads, self.hd, self.f, self.tokens, self.eps = d, heads, d // heads, f, tokens, eps
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.norm1 = (1 + 0.1 * normal(d)).bfloat16()
        self.norm2 = (1 + 0.1 * normal(d)).bfloat16()
        self.wqkv = Q8Weight(normal(3 * d, d) / math.sqrt(d))
        self.wo = Q8Weight(normal(d, d) / math.sqrt(d))
        self.wgu = Q8Weight(normal(2 * f, d) / math.sqrt(d))
        self.wd = Q8Weight(normal(d, f) / math.sqrt(f))
        rows = tokens * heads
        self.kv = [(torch.zeros((rows, self.hd), dtype=torch.int8, device="cuda"),
                    torch.zeros((rows,), dtype=torch.float32, device="cuda")) for _ in range(2)]
        # where a token's rows lie in the cache: its place is the sequence's choice
        self.place = torch.randperm(tokens, generator=g, device="cuda").to(torch.int32)
        self.used = 0

    def _slots(self, first, count):
        import torch
        head = torch.arange(self.heads, dtype=torch.int32, device=self.place.device)
        return (self.place[first:first + count, None] * self.heads + head).flatten().contiguous()

    def _rows(self, m, n):
        import torch
        dev = self.place.device
        return (torch.empty((m, n), dtype=torch.int8, device=dev),
                torch.empty((m,), dtype=torch.float32, device=dev))

    def _product(self, m, rows, w):
        import torch
        c = torch.empty((m, w.n), dtype=torch.bfloat16, device=self.place.device)
        X.xsymv_q8gemm_b(m, w.n, w.k, rows[0], w.k, rows[1], w.codes, w.k, w.scale, None, c, w.n)
        return c

    def _norm(self, m, x, r, weight):
        import torch
        d, rows = self.d, self._rows(m, self.d)
        h = torch.empty((m, d), dtype=torch.bfloat16, device=self.place.device)
        X.xsymv_q8norm_b(m, d, x, self._stride(x), "b", r, self._stride(r), "b", weight, self.eps,
                         h, d, rows[0], d, rows[1])
        return h, rows

    def _stride(self, t):
        return t.stride(0) if t.shape[0] > 1 else self.d

    def _check(self, name, t, m):
        import torch
        if t.dtype != torch.bfloat16 or t.device != self.place.device:
            raise ValueError(f"{name} is {t.dtype} on {t.device}, not bfloat16 on {self.place.device}")
        if tuple(t.shape) != (m, self.d):
            raise ValueError(f"{name} is {tuple(t.shape)}, not {(m, self.d)}")
        if (self.d > 1 and t.stride(1) != 1) or self._stride(t) < self.d:
            raise ValueError(f"{name}'s strides are {t.stride()}: rows lie one after the other")

    def __call__(self, x, r):
        """x, r: the next m tokens' rows and residuals (m x d, bfloat16, at any
        stride of rows); returns the layer's output and the new residual.
        ValueError, with nothing done, for other tensors and where the cache has
        no room for m tokens more."""
        m = x.shape[0]
        self._check("x", x, m)
        self._check("r", r, m)
        first, seen = self.used, self.used + m
        if seen > self.tokens:
            raise ValueError(f"the cache holds {self.tokens} tokens, {first} are there and {m} more "
                             "do not fit")
        out = self._layer(x, r, lambda qkv: self._attend(qkv, first, seen))
        self.used = seen
        return out

    def _layer(self, x, r, attend):
        """attend: of the rows' q, k, v."""
        m, d, f = x.shape[0], self.d, self.f
        h, rows = self._norm(m, x, r, self.norm1)
        att = attend(self._product(m, rows, self.wqkv))
        rows = self._rows(m, d)
        X.xsymv_q8store_b(m, d, att, d, None, m, rows[0], d, rows[1])
        o = self._product(m, rows, self.wo)
        h, rows = self._norm(m, o, h, self.norm2)
        gu = self._product(m, rows, self.wgu)
        rows = self._rows(m, f)
        X.xsymv_q8glu_b(m, f, gu, 2 * f, gu[:, f:], 2 * f, rows[0], f, rows[1])
        return self._product(m, rows, self.wd), h

    def _store(self, qkv, slots):
        d, heads, hd, m = self.d, self.heads, self.hd, qkv.shape[0]
        for part, (codes, scale) in enumerate(self.kv, start=1):
            new = qkv[:, part * d:(part + 1) * d].reshape(m * heads, hd)
            X.xsymv_q8store_b(m * heads, hd, new, hd, slots, self.tokens * heads, codes, hd, scale)

    def _attend(self, qkv, first, seen):
        import torch
        m, d, heads, hd = qkv.shape[0], self.d, self.heads, self.hd
        self._store(qkv, self._slots(first, m))
        past, read = self._slots(0, seen), []
        for codes, scale in self.kv:
            out = torch.empty((seen * heads, hd), dtype=torch.float32, device=codes.device)
            X.xsymv_q8read_s(seen * heads, hd, codes, hd, scale, past, self.tokens * heads, out, hd)
            read.append(out.view(seen, heads, hd).transpose(0, 1).double())
        q = qkv[:, :d].reshape(m, heads, hd).transpose(0, 1).double()
        score = q @ read[0].transpose(1, 2).contiguous() / math.sqrt(hd)
        token = torch.arange(seen, device=score.device)
        late = token[None, :] > token[first:, None]
        weight = torch.softmax(score.masked_fill(late, -math.inf), dim=-1)
        return (weight @ read[1].contiguous()).transpose(0, 1).reshape(m, d).bfloat16()


class Q8Answers(Q8Layer):
    """The layer for up to `answers` answers to one prompt, `page` tokens a page
    of the cache, which has room for `tokens` (a multiple of page).

        layer.prompt(x, r)   the prompt's next tokens, all of it before:
        layer.fork()         the answers begin, with the prompt's pages
        layer.step(x, r)     a token of each answer
        layer.free()         the answers end; fork may begin others

    Each returns or raises as Q8Layer does, and a call that fails takes no room."""

    def __init__(self, d, heads, f, tokens, answers, page=16, seed=0, eps=1e-5):
        super().__init__(d, heads, f, tokens, seed, eps)
        self._pages(answers, page)

    def _pages(self, answers, page):
        import torch
        if answers < 1 or page < 1 or self.tokens % page:
            raise ValueError(f"{answers} answers, {self.tokens} tokens in pages of {page}")
        self.answers, self.page, self.pages, self.seqs = answers, page, self.tokens // page, answers + 1

        def ints(v):
            return torch.tensor(v, dtype=torch.int32, device=self.place.device)

        # Sequence 0 is the prompt.  What calls take as device arrays is made once.
        self.len = ints([0] * self.seqs)
        self.table = ints([[-1] * self.pages] * self.seqs)
        self.refs = ints([0] * self.pages)
        self.each, self.zeros, self.ones = ints(list(range(1, self.seqs))), ints([0] * answers), ints([1] * answers)
        self.steps = ints([0] + list(range(self.seqs)))
        self.all, self.shared = ints([0, self.seqs]), ints([0])
        self.got, self.src, self.dst = (ints([0] * answers) for _ in range(3))
        self.used = self.more = 0     # tokens of the prompt, and of each answer behind it
        self.forked = False

    def _held(self, used, more, forked):
        """Pages that so many tokens are: a whole page of the prompt is held once."""
        whole = used // self.page
        own = -(-(used + more) // self.page) - whole
        return -(-used // self.page) + (self.answers * own if forked else 0)

    def _room(self, used, more, forked):
        if self._held(used, more, forked) > self.pages:
            raise ValueError(f"the cache holds {self.pages} pages of {self.page} tokens: {used} of a prompt"
                             + (f" and {more} of {self.answers} answers" if forked else "") + " do not fit")

    def _cache(self):
        return self.seqs, self.len, self.table, self.pages, self.pages, self.page

    def _answer(self, qkv, start, groups):
        import torch
        m, heads, hd = qkv.shape[0], self.heads, self.hd
        slots = torch.empty((m * heads,), dtype=torch.int32, device=self.place.device)
        X.xsymv_q8pages_slots(m, heads, start, self.seqs, self.len, self.table, self.pages, self.pages, self.page,
                              slots)
        self._store(qkv, slots)
        att = torch.empty((m, self.d), dtype=torch.bfloat16, device=self.place.device)
        (k, ks), (v, vs) = self.kv
        X.xsymv_q8attn_b(m, heads, heads, hd, qkv, 3 * self.d, self.seqs, start, self.len, self.table, self.pages,
                         groups, self.all, self.shared, k, hd, ks, v, hd, vs, self.pages, self.page,
                         1 / math.sqrt(hd), att, self.d, None)
        return att

    def prompt(self, x, r):
        import torch
        m = x.shape[0]
        self._check("x", x, m)
        self._check("r", r, m)
        if self.forked:
            raise ValueError("the prompt has answers")
        self._room(self.used + m, 0, False)
        add = torch.tensor([m], dtype=torch.int32, device=self.place.device)
        start = torch.tensor([0] + [m] * self.seqs, dtype=torch.int32, device=self.place.device)
        X.xsymv_q8pages_grow(1, self.zeros, add, *self._cache(), self.refs, self.got)
        try:
            out = self._layer(x, r, lambda qkv: self._answer(qkv, start, 0))
        except BaseException:
            self._shrink(0, 1)
            raise
        self.used += m
        return out

    def _shrink(self, first, count):
        """Sequences from `first` on give back the tokens that they were last grown by."""
        import torch
        n, table = self.len[first:first + count], self.table[first:first + count]
        old = n - self.got[:count]
        place = torch.arange(self.pages, device=n.device)
        last = table[(place >= (old[:, None] + self.page - 1) // self.page)
                     & (place < (n[:, None] + self.page - 1) // self.page)]
        self.refs[last.long()] = 0
        n.copy_(old)

    def fork(self):
        if self.forked:
            raise ValueError("the prompt has answers")
        self._room(self.used, 0, True)
        X.xsymv_q8pages_fork(self.answers, self.zeros, self.each, *self._cache(), self.refs, self.src, self.dst)
        rows = self.heads * self.page
        (k, ks), (v, vs) = self.kv
        try:
            X.xsymv_q8pages_copy(self.answers, self.src, self.dst, self.pages, rows, self.hd, k, self.hd, ks,
                                 v, self.hd, vs, 1, self.pages * rows)
            self.shared.fill_(self.used // self.page * self.page)
        except BaseException:
            X.xsymv_q8pages_free(self.answers, self.each, *self._cache(), self.refs)
            raise
        self.more, self.forked = 0, True

    def step(self, x, r):
        """x, r: row i is the next token of answer i."""
        self._check("x", x, self.answers)
        self._check("r", r, self.answers)
        if not self.forked:
            raise ValueError("the prompt has no answers")
        self._room(self.used, self.more + 1, True)
        self._grow()
        try:
            out = self._next(x, r)
        except BaseException:
            self._shrink(1, self.answers)
            raise
        self.more += 1
        return out

    def _grow(self):
        X.xsymv_q8pages_grow(self.answers, self.each, self.ones, *self._cache(), self.refs, self.got)

    def _next(self, x, r):
        return self._layer(x, r, lambda qkv: self._answer(qkv, self.steps, 1))

    def _step(self, x, r):
        """What a step does on the device (for a graph of it, whose replays are not counted here)."""
        self._grow()
        return self._next(x, r)

    def free(self):
        if not self.forked:
            raise ValueError("the prompt has no answers")
        X.xsymv_q8pages_free(self.answers, self.each, *self._cache(), self.refs)
        self.forked = False

    def likely(self, x, r, head, top):
        """The layer's output and residual as logits of `head` (a Q8Weight): the
        `top` most likely tokens of each row and their log probabilities."""
        import torch
        m = x.shape[0]
        rows = self._norm(m, x, r, self.norm1)[1]
        logits = self._product(m, rows, head)
        index = torch.empty((m, top), dtype=torch.int32, device=logits.device)
        value = torch.empty((m, top), dtype=torch.float32, device=logits.device)
        X.xsymv_logp_b(m, head.n, logits, head.n, None, None, None, None, top, index, value, top)
        return index, value


def plain(layer, x, r):
    """The same layer on the same weights in 64 bits, nothing rounded but the
    weights: what the 8-bit rows approximate (a whole prompt, an empty cache)."""
    import torch
    m, d, heads, hd = x.shape[0], layer.d, layer.heads, layer.hd

    def norm(v, w):
        return v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + layer.eps) * w.double()

    h = x.double() + r.double()
    qkv = norm(h, layer.norm1) @ layer.wqkv.values().t().contiguous()
    q, k, v = (t.reshape(m, heads, hd).transpose(0, 1) for t in qkv.split(d, dim=1))
    score = q @ k.transpose(1, 2).contiguous() / math.sqrt(hd)
    late = torch.ones((m, m), dtype=torch.bool, device="cuda").triu(1)
    att = (torch.softmax(score.masked_fill(late, -math.inf), dim=-1) @ v.contiguous())
    h = h + att.transpose(0, 1).reshape(m, d) @ layer.wo.values().t().contiguous()
    g, u = (norm(h, layer.norm2) @ layer.wgu.values().t().contiguous()).split(layer.f, dim=1)
    return (torch.nn.functional.silu(g) * u) @ layer.wd.values().t().contiguous(), h


def main():
    import time

    import torch
    layer = Q8Layer(d=4096, heads=32, f=11008, tokens=2048)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    prompt = 512
    x = torch.randn((prompt + 64, 4096), generator=g, device="cuda").bfloat16()
    r = torch.randn((prompt + 64, 4096), generator=g, device="cuda").bfloat16()
    y, h = layer(x[:prompt], r[:prompt])
    want, want_h = plain(layer, x[:prompt], r[:prompt])
    for name, a, b in (("output", y, want), ("residual", h, want_h)):
        print(f"prompt of {prompt} tokens: {name} off by {(a - b).norm() / b.norm():.3%} of its size "
              "against 64 bits")
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(prompt, prompt + 64):
        layer(x[i:i + 1], r[i:i + 1])
    torch.cuda.synchronize()
    print(f"64 single tokens: {(time.perf_counter() - t) / 64 * 1e6:.0f} us a token "
          "(attention in torch's elementary operations)")

    del layer, want, want_h
    answers, length, words = 16, 64, 32000
    layer = Q8Answers(d=4096, heads=32, f=11008, tokens=4096, answers=answers)
    head = Q8Weight(torch.randn((words, 4096), generator=g, device="cuda") / 64)

    def rows(tokens):
        return (head.codes[tokens].float() * head.scale[tokens, None] * 64).bfloat16()

    zero = torch.zeros((answers, 4096), dtype=torch.bfloat16, device="cuda")
    y, h = layer.prompt(x[:prompt], r[:prompt])
    index, value = layer.likely(y[-1:], h[-1:], head, answers)
    tokens, sums = index[0], value[0].clone()  # each answer begins with another token
    layer.fork()
    for i in range(length + 8):
        if i == 8:  # (the first steps make workspaces and load kernels)
            torch.cuda.synchronize()
            t = time.perf_counter()
        y, h = layer.step(rows(tokens), zero)
        index, value = layer.likely(y, h, head, 1)
        tokens = index[:, 0]
        sums += value[:, 0]
    torch.cuda.synchronize()
    print(f"{answers} answers of {length + 8} tokens: {(time.perf_counter() - t) / length * 1e6:.0f} us a token of each; "
          f"the likeliest has log probability {sums.max().item():.2f}")


if __name__ == "__main__":
    main()
