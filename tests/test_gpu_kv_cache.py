"""Writing the paged 8-bit cache and reading it back: codes and exponents have to be equal to the
definition's, whatever the sizes, strides, pages and values."""
import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _decoder as D
from tests._attention import TYPES

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, shape, dt):
    x = torch.randn(shape, generator=g, device=DEV)
    return (x * torch.exp(2 * torch.randn(shape[:-1] + (1,), generator=g, device=DEV))).to(dt)


def _same_codes(got, want):
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


CASES = [  # dtype, B, L, Hkv, D, page, starts, lengths, heads outside
    ("bf16", 1, 1, 1, 16, 16, [0], [1], True),
    ("f16", 3, 1, 8, 128, 64, [63, 0, 200], [1, 0, 1], True),
    ("bf16", 2, 37, 3, 80, 48, [11, 40], [37, 20], False),
    ("f16", 4, 130, 2, 112, 16, [0, 1, 15, 126], [130, 129, 0, 7], True),
    ("bf16", 2, 300, 4, 64, 256, [0, 100], None, True),
    ("f16", 2, 65, 5, 48, 32, None, [65, 3], False),
    ("bf16", 5, 20, 1, 32, 1024, [5, 0, 900, 1000, 1004], None, True),
    ("f16", 1, 3, 16, 96, 16, [-2], [3], True),           # two tokens in front of the table
    ("bf16", 2, 9, 2, 128, 16, [60, 64], None, False),    # some behind it
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_written_and_read_back(case):
    dtype, b, length, heads, d, page, starts, lengths, outside = case
    g, dt = _gen(b * 100 + length), TYPES[dtype]
    most = 64 if page == 16 and length == 9 else max(s for s in (starts or [0])) + length + 5
    cache = D.Cache(g, b, most, heads, d, page, outside=outside)
    fused = _rows(g, (b, length, 2, heads, d), dt)
    k, v = fused[:, :, 0], fused[:, :, 1]
    want = [cache.k.double(), cache.v.double()]
    scales = cache.scales.clone()
    s = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    back = [torch.full((b, length, heads, d), 3.0, dtype=dt, device=DEV) for _ in range(2)]
    expect = [x.clone() for x in back]
    end = cache.block_table.shape[1] * page
    for i in range(b):
        first = 0 if s is None else starts[i]
        for j in range(length if n is None else lengths[i]):
            at = first + j
            for m in range(2):
                expect[m][i, j] = 0
            if not 0 <= at < end:
                continue
            p, o = int(cache.block_table[i, at // page]), at % page
            for m, x in enumerate((k, v)):
                code, e = D.quantised(x[i, j])
                want[m][p, o] = code
                scales[p, :, o, m] = (e + 127).to(torch.uint8)
                expect[m][i, j] = (code * D.pow2(e)[:, None]).to(dt)
    got = cg.kv_cache_write(k, v, *cache.args(), s, lengths=n)
    assert got[0] is cache.k and got[2] is cache.scales
    _same_codes(cache.k, want[0])
    _same_codes(cache.v, want[1])
    assert torch.equal(cache.scales, scales)
    cg.kv_cache_read(*cache.args(), s, *back, lengths=n)
    assert torch.equal(back[0], expect[0]) and torch.equal(back[1], expect[1])


def test_values_at_the_types_ends():
    """Zeros, the largest and smallest numbers, infinities, NaN; rows whose largest element is on
    either side of 448 times a power of two; ties between codes."""
    for dt in (torch.bfloat16, torch.float16):
        big, least = torch.finfo(dt).max, torch.finfo(dt).smallest_normal / 2 ** (7 if dt is torch.bfloat16 else 10)
        rows = [[0.0] * 16, [big, -big, 1.0] + [0.0] * 13, [least, -least] + [0.0] * 14,
                [float("inf"), 2.0, -3.0] + [1.0] * 13, [float("-inf")] * 16,
                [float("nan"), 448.0] + [17.0] * 14, [float("nan")] * 16,
                [448.0, 17.0, 19.0, 18.0, -17.0] + [2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9] + [0.0] * 8,
                [449.0 if dt is torch.float16 else 450.0] + [17.0] * 15, [1.75, 1.0] + [0.3] * 14,
                [1.7578125] + [0.3] * 15, [-1.0] * 16, [2.0 ** -14, 2.0 ** -20] + [0.0] * 14]
        k = torch.tensor(rows, device=DEV).to(dt).view(1, len(rows), 1, 16)
        cache = D.Cache(_gen(1), 1, len(rows), 1, 16, 16)
        cg.kv_cache_write(k, k.flip(1), *cache.args(), None)
        at = int(cache.block_table[0, 0])
        for m, x in enumerate((k, k.flip(1))):
            code, e = D.quantised(x[0, :, 0])
            _same_codes((cache.k, cache.v)[m][at, :len(rows), 0], code)
            assert torch.equal(cache.scales[at, 0, :len(rows), m].long(), e.long() + 127)
            assert -64 <= int(e.min()) and int(e.max()) <= 120
        back, other = torch.empty_like(k), torch.empty_like(k)
        cg.kv_cache_read(*cache.args(), None, back, other)
        assert torch.equal(torch.nan_to_num(back), torch.nan_to_num(other.flip(1)))
        assert torch.equal(back.isnan(), k.isnan()) and not back.isinf().any()
        assert back[0, 1, 0, 0] >= 0.93 * big     # (a code above is limited to the largest number)
        # bfloat16's largest rows read as fp16: limited.
        half = torch.empty(k.shape, dtype=torch.float16, device=DEV)
        cg.kv_cache_read(*cache.args(), None, half, torch.empty_like(half))
        assert not half.isinf().any()


def test_pages_that_are_none():
    """Numbers outside [0, pages): nothing is written there, zeros are read."""
    g = _gen(2)
    cache = D.Cache(g, 2, 96, 2, 64, 32)
    cache.block_table[0, 1], cache.block_table[1, 0], cache.block_table[1, 2] = -1, 1 << 30, cache.k.shape[0]
    k, v = _rows(g, (2, 96, 2, 64), torch.bfloat16), _rows(g, (2, 96, 2, 64), torch.bfloat16)
    before = cache.scales.clone()
    cg.kv_cache_write(k, v, *cache.args(), None)
    back, other = torch.ones_like(k), torch.ones_like(v)
    cg.kv_cache_read(*cache.args(), None, back, other)
    for i, page in ((0, 1), (1, 0), (1, 2)):
        assert not back[i, page * 32:page * 32 + 32].any() and not other[i, page * 32:page * 32 + 32].any()
    assert int((cache.scales != before).any(3).any(2).any(1).sum()) == 3
    for i, page in ((0, 0), (0, 2), (1, 1)):
        x = k[i, page * 32:page * 32 + 32]
        code, e = D.quantised(x)
        assert torch.equal(back[i, page * 32:page * 32 + 32].double(), code * D.pow2(e)[..., None])


def test_rows_that_were_never_written_read_as_zeros():
    cache = D.Cache(_gen(3), 1, 40, 2, 32, 16)
    k, v = (torch.ones((1, 40, 2, 32), dtype=torch.float16, device=DEV) for _ in range(2))
    cg.kv_cache_read(*cache.args(), None, k, v)
    assert not k.any() and not v.any()


def test_token_by_token_is_the_same_as_at_once_and_replayed():
    g = _gen(4)
    k, v = _rows(g, (3, 50, 4, 128), torch.bfloat16), _rows(g, (3, 50, 4, 128), torch.bfloat16)
    once, steps = D.Cache(_gen(5), 3, 50, 4, 128, 16), D.Cache(_gen(5), 3, 50, 4, 128, 16)
    starts = torch.zeros(3, dtype=torch.int32, device=DEV)
    cg.kv_cache_write(k, v, *once.args(), None)
    one, two = torch.empty_like(k[:, :1]), torch.empty_like(v[:, :1])
    graph = torch.cuda.CUDAGraph()
    one.copy_(k[:, :1])
    two.copy_(v[:, :1])
    with torch.cuda.graph(graph):
        cg.kv_cache_write(one, two, *steps.args(), starts)
    for i in range(50):
        one.copy_(k[:, i:i + 1])
        two.copy_(v[:, i:i + 1])
        starts.fill_(i)
        graph.replay()
    assert torch.equal(once.k.view(torch.uint8), steps.k.view(torch.uint8))
    assert torch.equal(once.v.view(torch.uint8), steps.v.view(torch.uint8))
    assert torch.equal(once.scales, steps.scales)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    back, other = torch.empty_like(k), torch.empty_like(v)
    cg.kv_cache_read(*steps.args(), None, back, other, stream=side)
    side.synchronize()
    code, e = D.quantised(k)
    assert torch.equal(back.double(), code * D.pow2(e)[..., None])


def test_offsets_past_32_bits():
    """Pages of one cache more than 2^32 bytes apart."""
    pages, page, d = 40000, 1024, 128
    k_cache = torch.empty((pages, page, 1, d), dtype=torch.uint8, device=DEV).view(D.E4M3)
    scales = torch.zeros((pages, 1, page, 2), dtype=torch.uint8, device=DEV)
    table = torch.tensor([[39999, 2], [33555, 38000]], dtype=torch.int32, device=DEV)
    k = _rows(_gen(6), (2, 40, 1, d), torch.bfloat16)
    starts = torch.tensor([1000, 1010], dtype=torch.int32, device=DEV)
    cg.kv_cache_write(k, k, k_cache, k_cache, scales, table, starts)
    code, e = D.quantised(k)
    for i in range(2):
        for j in (0, 13, 14, 23, 24, 39):
            at = int(starts[i]) + j
            row = k_cache[int(table[i, at // page]), at % page, 0]
            _same_codes(row, code[i, j, 0])
    back, other = torch.empty_like(k), torch.empty_like(k)
    cg.kv_cache_read(k_cache, k_cache, scales, table, starts, back, other)
    assert torch.equal(back.double(), code * D.pow2(e)[..., None]) and torch.equal(back, other)


def test_refusals():
    i = cg.CONV_ERR_INVALID_VALUE
    k = torch.zeros((2, 5, 4, 64), dtype=torch.bfloat16, device=DEV)
    c = D.Cache(_gen(7), 2, 64, 4, 64, 16)
    good = dict(k=k, v=k, k_cache=c.k, v_cache=c.v, scales=c.scales, block_table=c.block_table, starts=None)

    def refused(status, lengths=None, **kw):
        a = dict(good, **kw)
        for read in (False, True):
            with pytest.raises(cg.ConvError) as e:
                if read:
                    cg.kv_cache_read(a["k_cache"], a["v_cache"], a["scales"], a["block_table"], a["starts"],
                                     a["k"].clone(), a["v"].clone(), lengths=lengths)
                else:
                    cg.kv_cache_write(*a.values(), lengths=lengths)
            assert e.value.status == status, str(e.value)

    refused(cg.CONV_ERR_NOT_SUPPORTED, k=k.float())
    refused(i, k=k.cpu())
    refused(i, k=k[0])
    refused(i, v=k.half())
    refused(i, v=k[:, :4])
    refused(i, k_cache=c.k.view(torch.uint8))
    refused(i, k_cache=c.k[:, :, :2])
    refused(i, v_cache=c.v[1:])
    refused(i, scales=c.scales[:-1])
    refused(i, scales=c.scales.int())
    refused(i, block_table=c.block_table.long())
    refused(i, block_table=c.block_table[:1])
    refused(i, block_table=c.block_table.t().contiguous().t())
    refused(i, block_table=c.block_table.cpu())
    refused(i, starts=torch.zeros(2, dtype=torch.int64, device=DEV))
    refused(i, starts=torch.zeros(3, dtype=torch.int32, device=DEV))
    refused(i, lengths=torch.zeros(2, dtype=torch.int32))
    odd = D.Cache(_gen(8), 2, 64, 4, 64, 24)
    refused(cg.CONV_ERR_NOT_SUPPORTED, k_cache=odd.k, v_cache=odd.v, scales=odd.scales, block_table=odd.block_table)
    thin = torch.zeros((2, 5, 4, 24), dtype=torch.bfloat16, device=DEV)
    t = D.Cache(_gen(9), 2, 64, 4, 24, 16)
    refused(cg.CONV_ERR_NOT_SUPPORTED, k=thin, v=thin, k_cache=t.k, v_cache=t.v, scales=t.scales,
            block_table=t.block_table)
    with pytest.raises(cg.ConvError) as e:       # one page's memory for all of them
        cg.kv_cache_write(k, k, c.k[:1].expand(c.k.shape), c.v, c.scales, c.block_table, None)
    assert e.value.status == i
    with pytest.raises(cg.ConvError) as e:
        cg.kv_cache_read(*c.args(), None, k[:1].expand(2, 5, 4, 64), k)
    assert e.value.status == i
    shifted = torch.zeros(k.numel() + 4, dtype=torch.bfloat16, device=DEV)[4:].view(k.shape)
    with pytest.raises(cg.ConvError) as e:
        cg.kv_cache_write(shifted, k, *c.args(), None)
    assert e.value.status == cg.CONV_ERR_MISALIGNED
    cg.kv_cache_write(k[:0], k[:0], c.k, c.v, c.scales, c.block_table[:0], None)
    cg.kv_cache_write(k[:, :0], k[:, :0], *c.args(), None)
