"""The example block: each stage against the definition in 64 bits, from the bits the stage before
left (the bounds of tests/_attention.py; the projections' from their roundings)."""
import pytest
import torch

from tests import _attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _projected(x, f, u, source=None):
    """x f (+ source) in 64 bits, and its bound: fp32 sums of exact products, rounded once."""
    x, f = x.double(), f.double()[0, 0]
    y, size = x @ f, x.abs() @ f.abs()
    if source is not None:
        y, size = y + source.double(), size + source.double().abs()
    return y, u * y.abs() + (1 + u) * (f.shape[0] + 2) * A.F32 * size + A.grain(u)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [(2, 9, 13, 320, 8, 77, 96), (1, 16, 16, 256, 4, 200, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_block(size, dtype):
    from examples.text_block import TextBlock
    n, h, w, c, heads, length, sc = size
    dt, u = A.TYPES[dtype], A.UNIT[dtype]
    gen = torch.Generator().manual_seed(3)
    block = TextBlock(n, h, w, c, heads, length, sc, dtype=dt, seed=4)
    block.q_weight.copy_(torch.randn(c // heads, generator=gen) + 1)
    block.k_weight.copy_(torch.randn(c // heads, generator=gen) + 1)
    x = torch.randn((n, h, w, c), generator=gen).to(dt).to(DEV)
    states = torch.randn((n, length, sc), generator=gen).to(dt).to(DEV)
    lengths = torch.randint(0, length + 1, (n,), generator=gen).to(torch.int32)
    block.set_states(states, lengths)
    out = block(x, torch.full_like(x, float("nan")))

    # The projections' own results are overwritten by the norm: they are made again.
    kv = block._project(states.view(n, 1, length, sc), "kv", torch.empty_like(block.kv))
    A.assert_within("kv", kv.view(n, length, 2 * c), *_projected(states, block.filters["kv"], u))
    q = block._project(x, "q", torch.empty_like(x))
    A.assert_within("q", q, *_projected(x, block.filters["q"], u))
    d = c // heads
    for name, raw, normed, weight in (
            ("q normed", block._rows(q), block._rows(block.q), block.q_weight),
            ("k normed", kv.view(n, length, 2, heads, d)[:, :, 0], block.k, block.k_weight)):
        ref = A.NormReference(raw, weight, block.cos, block.sin, None, 1e-6, False, u)
        A.assert_within(name, normed, ref.y, ref.y_tol)
    ref = A.Reference(block._rows(block.q), block.k, block.v, kv_lengths=lengths.to(DEV), u=u)
    A.assert_within("attended", block._rows(block.attended), ref.out, ref.out_tol)
    A.assert_within("out", out, *_projected(block.attended, block.filters["out"], u, source=x))
