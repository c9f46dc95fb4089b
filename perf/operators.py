"""What the 8-bit row operators are measured on: norm, gated activation, cache store and read, product.

The operators (``include/xsymv.h``, the xsymv_q8 entry points) keep a row of n numbers as n signed
8-bit codes and one 32-bit scale: with a = max(max_j |v_j|, 2^-100),

    code_j = round_half_even(v_j * (127 / a)),   scale = a / 127,   value_j = code_j * scale.

* norm:  h = x + r (rounded to r's type), v = h / sqrt(mean(h^2) + eps) * w, v as a row of codes.
* glu:   v = g / (1 + exp(-g)) * u, v as a row of codes.
* store: rows of keys or values written as codes into the rows ``slot`` of a cache; read: back.
* gemm:  C[i, j] = (sum_l A[i, l] * W[j, l]) * sa[i] * sw[j] + bias[j], the sum exact in integers.

``run`` gives the plain form where ``own`` is false, else the framework's calls.  Rows of codes are
returned as the values they stand for, which is what the read operator gives; in 16 bits, unless a
32-bit row was stored: a code holds 8 bits.
"""
import math

import torch

own = False

FLOOR = 2.0 ** -100
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LETTER = {"f32": "s", "f16": "h", "bf16": "b"}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # one token of one sequence between two layers: latency alone
        {"name": "norm-token", "op": "norm", "m": 1, "n": 4096, "type": "bf16", "res": "bf16", "pad": 0},
        # a prompt of 4096 tokens with the residual stream kept in 32 bits
        {"name": "norm-prompt", "op": "norm", "m": 4096, "n": 8192, "type": "bf16", "res": "f32", "pad": 0},
        # seven sequences' tokens, a width that no vector length divides, rows at an odd stride
        {"name": "glu-batch-odd", "op": "glu", "m": 7, "n": 11007, "type": "f16", "pad": 3},
        # a prompt's hidden layer, gate and up being the halves of one product's rows
        {"name": "glu-prompt", "op": "glu", "m": 4096, "n": 14336, "type": "bf16", "pad": 0},
        # 32 sequences add the keys of one token, 8 heads each, to their pages of a cache
        {"name": "store-batch", "op": "store", "m": 256, "n": 128, "cap": 1 << 17, "type": "bf16", "pad": 0},
        # a prompt of 16384 tokens, 8 heads, written to a cache and read back
        {"name": "store-prompt", "op": "store", "m": 131072, "n": 128, "cap": 1 << 18, "type": "f16", "pad": 0},
        # a sequence's scattered rows gathered out of a cache for a kernel that wants them in 32 bits
        {"name": "read-odd", "op": "read", "m": 20011, "n": 80, "cap": 1 << 16, "type": "f32", "pad": 0},
        # the attention's output projection for one token
        {"name": "gemm-token", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "type": "bf16", "bias": False, "pad": 0},
        # 16 sequences' tokens through the widest matrix of a layer: the weights' bytes bound it
        {"name": "gemm-batch", "op": "gemm", "m": 16, "n": 28672, "k": 8192, "type": "bf16", "bias": False, "pad": 0},
        # odd everything: tokens, outputs, inner length, row strides
        {"name": "gemm-odd", "op": "gemm", "m": 45, "n": 1003, "k": 2051, "type": "f32", "bias": True, "pad": 2},
        # a chunk of a prompt among single tokens: between bytes and arithmetic
        {"name": "gemm-chunk", "op": "gemm", "m": 256, "n": 8192, "k": 14336, "type": "f16", "bias": True, "pad": 0},
        # a prompt of 4096 tokens: arithmetic alone
        {"name": "gemm-prompt", "op": "gemm", "m": 4096, "n": 28672, "k": 8192, "type": "bf16", "bias": False, "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row length: half of them multiples of 128, the others as they fall."""
    n = _log(rng, lo, hi)
    return max(128, n // 128 * 128) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["norm", "glu", "store", "read", "gemm", "gemm"])
    t = rng.choice(["f32", "f16", "bf16", "bf16"])
    pad = rng.choice([0, 0, 16, rng.randint(1, 40)])
    if op == "norm":
        n = _width(rng, 128, 20000)
        return {"op": op, "m": _log(rng, 1, min(8192, (1 << 26) // n)), "n": n, "type": t,
                "res": rng.choice([t, "f32"]), "pad": pad}
    if op == "glu":
        n = _width(rng, 256, 40000)
        return {"op": op, "m": _log(rng, 1, min(8192, (1 << 26) // n)), "n": n, "type": t, "pad": pad}
    if op in ("store", "read"):
        n = rng.choice([64, 96, 128, 192, 256, rng.randint(33, 576)])
        m = _log(rng, 1, 131072)
        return {"op": op, "m": m, "n": n, "cap": m + _log(rng, 1, 131072), "type": t, "pad": pad}
    while True:
        m, n, k = _log(rng, 1, 8192), _width(rng, 128, 28672), _width(rng, 128, 28672)
        if m * n * k <= 1 << 39 and m * n <= 1 << 27:
            return {"op": op, "m": m, "n": n, "k": k, "type": t, "bias": rng.random() < 0.3, "pad": pad}


def _normal(shape, g, spread=1.0):
    return torch.randn(shape, generator=g, device="cuda") * spread


def _rows(m, n, pad, dtype):
    """An m x n tensor whose rows are n + pad elements apart."""
    return torch.zeros((m, n + pad), dtype=dtype, device="cuda")[:, :n]


def _codes(m, n, pad, g):
    q = _rows(m, n, pad, torch.int8)
    step = max(1, (1 << 27) // max(1, n))
    for i in range(0, m, step):
        part = q[i:i + step]
        part.copy_(_normal(part.shape, g, 30.0).round_().clamp_(-127, 127))
    return q


def prepare(case, seed):
    """Inputs, and the buffers that a serving loop keeps for the outputs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, m, n, pad = case["op"], case["m"], case["n"], case["pad"]
    dt = TYPES[case["type"]]
    s = {"op": op, "type": case["type"], "m": m, "n": n, "dtype": dt}
    # rows of codes are read back in 16 bits, but for a stored 32-bit row
    s["vtype"] = case["type"] if op in ("store", "read") or case["type"] != "f32" else "bf16"
    if op != "gemm":
        s["values"] = torch.empty((m, n), dtype=TYPES[s["vtype"]], device="cuda")
    if op in ("norm", "glu"):
        s["q"] = torch.empty((m, n), dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty((m,), dtype=torch.float32, device="cuda")
    if op == "norm":
        s["res"] = case["res"]
        s["x"] = _rows(m, n, pad, dt)
        s["x"].copy_(_normal((m, n), g))
        s["r"] = _rows(m, n, pad, TYPES[case["res"]])
        s["r"].copy_(_normal((m, n), g, 2.0))
        w = 1.0 + _normal((n,), g, 0.1)
        w[torch.randint(0, n, (max(1, n // 256),), generator=g, device="cuda")] *= 3.0  # channels that stand out
        s["w"] = w.to(dt)
        s["h"] = torch.empty((m, n), dtype=TYPES[case["res"]], device="cuda")
    elif op == "glu":
        gu = _rows(m, 2 * n, pad, dt)
        gu.copy_(_normal((m, 2 * n), g, 1.5))
        s["g"], s["u"] = gu[:, :n], gu[:, n:]
    elif op in ("store", "read"):
        cap = case["cap"]
        s["slot"] = torch.randperm(cap, generator=g, device="cuda")[:m].to(torch.int32)
        s["cap"] = cap
        if op == "store":
            s["x"] = _rows(m, n, pad, dt)
            s["x"].copy_(_normal((m, n), g))
            s["cache"] = torch.zeros((cap, n), dtype=torch.int8, device="cuda")
            s["cscale"] = torch.zeros((cap,), dtype=torch.float32, device="cuda")
        else:
            s["cache"] = _codes(cap, n, pad, g)
            s["cscale"] = 0.01 + 0.02 * torch.rand((cap,), generator=g, device="cuda")
    else:
        k = case["k"]
        s["k"] = k
        s["a"], s["wt"] = _codes(m, k, pad, g), _codes(n, k, pad, g)
        s["sa"] = 0.01 + 0.02 * torch.rand((m,), generator=g, device="cuda")
        s["sw"] = (0.5 + torch.rand((n,), generator=g, device="cuda")) / (30.0 * math.sqrt(k))
        s["bias"] = _normal((n,), g) if case["bias"] else None
        s["c"] = torch.empty((m, n), dtype=dt, device="cuda")
    return s


def _plain_codes(v):
    """Codes and scales of rows of 32-bit numbers."""
    a = v.abs().amax(dim=1, keepdim=True).clamp_min(FLOOR)
    return (v * (127.0 / a)).round(), a / 127.0


def _plain(s):
    op = s["op"]
    if op == "norm":
        h = (s["x"].float() + s["r"].float()).to(s["r"].dtype)
        f = h.float()
        v = f * (f.square().mean(dim=1, keepdim=True) + EPS).rsqrt() * s["w"].float()
        q, a = _plain_codes(v)
        return {"h": h, "values": (q * a).to(s["values"].dtype), "scale": a[:, 0]}
    if op == "glu":
        f = s["g"].float()
        v = f / (1.0 + (-f).exp()) * s["u"].float()
        q, a = _plain_codes(v)
        return {"values": (q * a).to(s["values"].dtype), "scale": a[:, 0]}
    if op in ("store", "read"):
        i = s["slot"].long()
        if op == "store":
            q, a = _plain_codes(s["x"].float())
            s["cache"][i] = q.to(torch.int8)
            s["cscale"][i] = a[:, 0]
        return {"values": (s["cache"][i].float() * s["cscale"][i][:, None]).to(s["values"].dtype)}
    c = s["a"].float() @ s["wt"].float().t()
    c = c * s["sa"][:, None] * s["sw"]
    if s["bias"] is not None:
        c = c + s["bias"]
    return {"c": c.to(s["c"].dtype)}


def _own(s):
    import blas_symmetric_mat_amd as X

    op, m, n = s["op"], s["m"], s["n"]
    t = LETTER[s["type"]]
    if op == "gemm":
        a, w, c = s["a"], s["wt"], s["c"]
        getattr(X, "xsymv_q8gemm_" + t)(m, n, s["k"], a, a.stride(0), s["sa"], w, w.stride(0), s["sw"], s["bias"], c, n)
        return {"c": c}
    v = s["values"]
    read = getattr(X, "xsymv_q8read_" + LETTER[s["vtype"]])
    if op in ("store", "read"):
        if op == "store":
            x = s["x"]
            getattr(X, "xsymv_q8store_" + t)(m, n, x, x.stride(0), s["slot"], s["cap"], s["cache"], n, s["cscale"])
        read(m, n, s["cache"], s["cache"].stride(0), s["cscale"], s["slot"], s["cap"], v, n)
        return {"values": v}
    q, scale = s["q"], s["scale"]
    if op == "norm":
        x, r, h = s["x"], s["r"], s["h"]
        getattr(X, "xsymv_q8norm_" + t)(m, n, x, x.stride(0), LETTER[s["res"]], r, r.stride(0), t, s["w"], EPS,
                                   h, n, q, n, scale)
        read(m, n, q, n, scale, None, m, v, n)
        return {"h": h, "values": v, "scale": scale}
    g, u = s["g"], s["u"]
    getattr(X, "xsymv_q8glu_" + t)(m, n, g, g.stride(0), u, u.stride(0), q, n, scale)
    read(m, n, q, n, scale, None, m, v, n)
    return {"values": v, "scale": scale}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """Bytes of the inputs and of the outputs, each once, and the operations on them."""
    op, m, n, b = case["op"], case["m"], case["n"], SIZE[case["type"]]
    if op == "gemm":
        k = case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + (4 * n if case["bias"] else 0) + b * m * n, "flops": 2 * m * n * k}
    if op == "read":
        return {"bytes": m * (n + 8 + b * n), "flops": m * n}
    if op == "store":
        return {"bytes": m * (b * n + 4 + n + 4 + b * n), "flops": 4 * m * n}
    v = 2
    if op == "norm":
        r = SIZE[case["res"]]
        return {"bytes": m * n * (b + 2 * r + v) + b * n + 4 * m, "flops": 8 * m * n}
    return {"bytes": m * n * (2 * b + v) + 4 * m, "flops": 9 * m * n}


def _exact_codes(v):
    a = v.abs().max(dim=1, keepdim=True).values
    step = torch.maximum(a, torch.full_like(a, FLOOR)) / 127
    return torch.round(v / step) * step, step[:, 0]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        # the products are whole numbers far below 2^53: the sums are exact
        c = torch.mm(s["a"].to(torch.float64), s["wt"].to(torch.float64).t().contiguous())
        c *= s["sa"].to(torch.float64)[:, None]
        c *= s["sw"].to(torch.float64)[None, :]
        if s["bias"] is not None:
            c += s["bias"].to(torch.float64)[None, :]
        return {"c": c}
    if op == "read":
        at = s["slot"].to(torch.int64)
        return {"values": torch.index_select(s["cache"], 0, at).to(torch.float64)
                * torch.index_select(s["cscale"], 0, at).to(torch.float64)[:, None]}
    if op == "store":
        return {"values": _exact_codes(s["x"].to(torch.float64))[0]}
    if op == "norm":
        # the row that is normalised is the one that is kept, in the residual's type
        whole = s["x"].to(torch.float64) + s["r"].to(torch.float64)
        kept = whole.to(s["r"].dtype).to(torch.float64)
        length = torch.linalg.vector_norm(kept, dim=1, keepdim=True)
        v = kept / torch.sqrt(length * length / case["n"] + EPS) * s["w"].to(torch.float64)
        values, step = _exact_codes(v)
        return {"h": whole, "values": values, "scale": step}
    gate = s["g"].to(torch.float64)
    values, step = _exact_codes(gate * torch.sigmoid(gate) * s["u"].to(torch.float64))
    return {"values": values, "scale": step}
