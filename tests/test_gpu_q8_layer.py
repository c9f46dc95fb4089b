"""The example layer on the GPU: rows at a stride, and a cache that is full."""
import pytest

pytestmark = pytest.mark.gpu


def layers(count):
    from blas_symmetric_mat_amd import q8_layer
    return [q8_layer.Q8Layer(d=256, heads=2, f=500, tokens=12, seed=3) for _ in range(count)]


def test_rows_at_a_stride():
    """x and r as column halves of wider matrices give the bytes of their
    contiguous copies."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    both = torch.randn((12, 512), generator=g, device="cuda").bfloat16()
    x, r = both[:, :256], both[:, 256:]
    a, b = layers(2)
    want = [a(x[i:j].contiguous(), r[i:j].contiguous()) for i, j in ((0, 7), (7, 8), (8, 12))]
    got = [b(x[i:j], r[i:j]) for i, j in ((0, 7), (7, 8), (8, 12))]
    torch.cuda.synchronize()
    for (y, h), (y2, h2) in zip(want, got):
        assert torch.equal(y, y2) and torch.equal(h, h2)


def test_a_full_cache_is_left_as_it_is():
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    x, r = (torch.randn((12, 256), generator=g, device="cuda").bfloat16() for _ in range(2))
    layer, = layers(1)
    layer(x, r)
    torch.cuda.synchronize()
    assert layer.used == 12
    before = [t.clone() for pair in layer.kv for t in pair]
    for m in (1, 12):
        with pytest.raises(ValueError):
            layer(x[:m], r[:m])
    torch.cuda.synchronize()
    assert layer.used == 12
    assert all(torch.equal(a, b) for a, b in zip(before, (t for pair in layer.kv for t in pair)))
