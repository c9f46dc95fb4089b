"""One layer of a decoder that serves from 8 bits, on the library's 8-bit row
operators: an example of their use together, and the path their tests run.

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
        import torch
        m, d, heads, hd = x.shape[0], self.d, self.heads, self.hd
        self._check("x", x, m)
        self._check("r", r, m)
        first, seen = self.used, self.used + m
        if seen > self.tokens:
            raise ValueError(f"the cache holds {self.tokens} tokens, {first} are there and {m} more "
                             "do not fit")
        h, rows = self._norm(m, x, r, self.norm1)
        qkv = self._product(m, rows, self.wqkv)
        slots, cap = self._slots(first, m), self.tokens * heads
        past, read = self._slots(0, seen), []
        for part, (codes, scale) in enumerate(self.kv, start=1):
            new = qkv[:, part * d:(part + 1) * d].reshape(m * heads, hd)
            X.xsymv_q8store_b(m * heads, hd, new, hd, slots, cap, codes, hd, scale)
            out = torch.empty((seen * heads, hd), dtype=torch.float32, device=codes.device)
            X.xsymv_q8read_s(seen * heads, hd, codes, hd, scale, past, cap, out, hd)
            read.append(out.view(seen, heads, hd).transpose(0, 1).double())
        q = qkv[:, :d].reshape(m, heads, hd).transpose(0, 1).double()
        score = q @ read[0].transpose(1, 2).contiguous() / math.sqrt(hd)
        token = torch.arange(seen, device=score.device)
        late = token[None, :] > token[first:, None]
        weight = torch.softmax(score.masked_fill(late, -math.inf), dim=-1)
        att = (weight @ read[1].contiguous()).transpose(0, 1).reshape(m, d).bfloat16()
        rows = self._rows(m, d)
        X.xsymv_q8store_b(m, d, att, d, None, m, rows[0], d, rows[1])
        o = self._product(m, rows, self.wo)
        h, rows = self._norm(m, o, h, self.norm2)
        gu, f = self._product(m, rows, self.wgu), self.f
        rows = self._rows(m, f)
        X.xsymv_q8glu_b(m, f, gu, 2 * f, gu[:, f:], 2 * f, rows[0], f, rows[1])
        y = self._product(m, rows, self.wd)
        self.used = seen
        return y, h


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


if __name__ == "__main__":
    main()
