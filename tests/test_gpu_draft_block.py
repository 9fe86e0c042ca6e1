"""The decoder operators run together as they would be used: each stage of the example block against
the definition in 64 bits, from the bits the stage before left; drafts as a tree against the same
tokens one by one; a captured step."""
import pytest
import torch

from tests import _attention as A
from tests import _decoder as D
from tests.test_gpu_text_block import _projected

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class _View(D.Cache):
    """The block's pages as the reference takes them."""

    def __init__(self, block):
        self.k, self.v, self.scales, self.block_table = block._pages()
        self.page = self.k.shape[1]


def _block(dtype, requests, drafts, tokens, channels, heads, kv_heads, page):
    from examples.draft_block import DraftBlock
    block = DraftBlock(requests, drafts, tokens, channels, heads, kv_heads, page=page, dtype=A.TYPES[dtype], seed=4)
    gen = torch.Generator().manual_seed(5)
    for w in (block.q_weight, block.k_weight, block.norm_weight):
        w.copy_(1 + 0.3 * torch.randn(w.shape, generator=gen))
    block.norm_bias.copy_(0.2 * torch.randn(channels, generator=gen))
    return block, gen


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [(3, 5, 90, 256, 4, 2, 16), (2, 24, 200, 640, 8, 2, 48)], ids=str)
def test_each_stage(size, dtype):
    requests, drafts, tokens, c, heads, kv_heads, page = size
    u, dt = A.UNIT[dtype], A.TYPES[dtype]
    block, gen = _block(dtype, *size)
    starts = torch.tensor([0] + [tokens - 2 * drafts - 3 * i for i in range(requests - 1)], dtype=torch.int32)
    # What lies in front: earlier tokens, written in one piece.
    d = c // heads
    import transposed_conv_implicit_gb300 as cg
    old = torch.randn((2, requests, tokens, kv_heads, d), generator=gen).to(dt).to(DEV)
    cg.kv_cache_write(old[0], old[1], *block._pages(), None, lengths=starts.to(DEV))
    x = (1.5 * torch.randn((requests, drafts, c), generator=gen) + 0.3).to(dt).to(DEV)
    up = (torch.rand((requests, drafts), generator=gen) * (torch.arange(drafts) + 1)).to(torch.int32) - 1
    depth = torch.zeros((requests, drafts), dtype=torch.int32)
    for b in range(requests):
        for i in range(drafts):
            depth[b, i] = 0 if up[b, i] < 0 else depth[b, up[b, i]] + 1
    positions = (starts[:, None] + depth).to(DEV)
    starts = starts.to(DEV)
    out = block(x, torch.full_like(x, float("nan")), starts, positions, parents=up.to(DEV))

    rows = requests * drafts
    ref = D.NormReference(x.view(rows, c), block.norm_weight, block.norm_bias, 1e-5, u)
    A.assert_within("normed", block.normed.view(rows, c), ref.y, ref.y_tol)
    # (The projection's own result is overwritten by the norm of heads: it is made again.)
    raw = block._project(block.normed, "qkv", torch.empty_like(block.qkv))
    A.assert_within("qkv", raw.view(rows, -1), *_projected(block.normed.view(rows, c), block.filters["qkv"], u))
    q, k, v = block.split(block.qkv)
    for name, was, now, weight in zip("qk", block.split(raw), (q, k), (block.q_weight, block.k_weight)):
        ref = A.NormReference(was, weight, block.cos, block.sin, positions, 1e-6, False, u)
        A.assert_within(name, now, ref.y, ref.y_tol)
    cache = _View(block)
    for b in range(requests):
        n = int(starts[b])
        got = cache.rows(b, n + drafts)
        for m, new in enumerate((k, v)):
            code, e = D.quantised(torch.cat((old[m, b, :n], new[b])))
            assert torch.equal(got[m], code * D.pow2(e)[..., None])
    ref = D.TreeReference(q, cache, (starts + drafts).tolist(), parents=up, u=u)
    A.assert_within("attended", block.attended.view(requests, drafts, heads, d), ref.out, ref.out_tol)
    A.assert_within("out", out.view(rows, c), *_projected(block.attended.view(rows, c), block.filters["out"], u,
                                                          source=x.view(rows, c)))


def test_a_chain_of_drafts_is_the_same_as_its_tokens_one_by_one():
    """The pages end up the same, bit for bit; the attention agrees within both calls' bounds."""
    size = (2, 6, 80, 256, 4, 2, 16)
    at_once, gen = _block("bf16", *size)
    one, _ = _block("bf16", 2, 1, *size[2:])
    x = torch.randn((2, 6, 256), generator=gen).bfloat16().to(DEV)
    starts = torch.zeros(2, dtype=torch.int32, device=DEV)
    place = torch.arange(6, dtype=torch.int32, device=DEV).expand(2, 6).contiguous()
    at_once(x, torch.empty_like(x), starts, place)
    ref = D.TreeReference(at_once.split(at_once.qkv)[0], _View(at_once), [6, 6], u=A.UNIT["bf16"])
    for i in range(6):
        token = x[:, i:i + 1].contiguous()
        one(token, torch.empty_like(token), starts + i, place[:, i:i + 1].contiguous())
        attended = one.attended.view(2, 4, 64)
        assert torch.equal(one.split(one.qkv)[0][:, 0], at_once.split(at_once.qkv)[0][:, i])
        A.assert_within("attended", attended, ref.out[:, i], ref.out_tol[:, i])
    for b in range(2):
        for got, want in zip(_View(one).rows(b, 6), _View(at_once).rows(b, 6)):
            assert torch.equal(got, want)


def test_an_accepted_branch_lies_in_the_text_s_order():
    size = (2, 7, 90, 256, 4, 2, 16)
    block, gen = _block("f16", *size)
    x = torch.randn((2, 7, 256), generator=gen).half().to(DEV)
    starts = torch.tensor([3, 40], dtype=torch.int32, device=DEV)
    parents = torch.tensor([-1, 0, 0, 1, 1, 2, 2], dtype=torch.int32, device=DEV)
    depth = torch.tensor([0, 1, 1, 2, 2, 2, 2], dtype=torch.int32, device=DEV)
    block(x, torch.empty_like(x), starts, starts[:, None] + depth, parents=parents)
    kept = torch.tensor([[0, 2, 6], [0, 1, 0]], dtype=torch.int32, device=DEV)
    before = _View(block).rows(1, 47)
    block.accept(starts, kept, torch.tensor([3, 2], dtype=torch.int32, device=DEV))
    _, k, v = block.split(block.qkv)
    for b, branch in ((0, [0, 2, 6]), (1, [0, 1])):
        got = _View(block).rows(b, int(starts[b]) + 7)
        for m, new in enumerate((k, v)):
            code, e = D.quantised(new[b, branch])
            first = int(starts[b])
            assert torch.equal(got[m][first:first + len(branch)], code * D.pow2(e)[..., None])
    assert torch.equal(_View(block).rows(1, 47)[0][42:], before[0][42:])


def test_a_captured_step():
    size = (2, 24, 200, 640, 8, 2, 48)
    block, gen = _block("bf16", *size)
    x = torch.randn((2, 24, 640), generator=gen).bfloat16().to(DEV)
    starts = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    place = starts[:, None] + torch.arange(24, dtype=torch.int32, device=DEV)
    out, again = torch.empty_like(x), torch.empty_like(x)
    block(x, out, starts, place)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, again, starts, place)
    for _ in range(2):
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, again)
