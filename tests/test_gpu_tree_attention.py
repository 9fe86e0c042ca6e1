"""Attention of drafted tokens to the paged 8-bit cache against its definition in 64 bits."""
import math

import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _decoder as D
from tests._attention import TYPES, UNIT, assert_within
from transposed_conv_implicit_gb300 import _lib, decoder

pytestmark = pytest.mark.gpu
DEV = "cuda"
MARK = 5.5


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _filled(g, dtype, keys, heads, d, page, *, outside=True, spread=0.5):
    """A cache whose requests hold keys[b] tokens; what lies behind is NaN."""
    dt, b, most = TYPES[dtype], len(keys), max(max(keys), 1)
    cache = D.Cache(g, b, most, heads, d, page, outside=outside)
    k, v = (torch.randn((b, most, heads, d), generator=g, device=DEV) for _ in range(2))
    k, v = ((x * torch.exp(spread * torch.randn((b, most, heads, 1), generator=g, device=DEV))).to(dt) for x in (k, v))
    cg.kv_cache_write(k, v, *cache.args(), None, lengths=torch.tensor(keys, dtype=torch.int32, device=DEV))
    # (Bytes of rows that were never written: any, where the length says that they are not there.)
    for i, n in enumerate(keys):
        at = torch.arange(n, cache.block_table.shape[1] * page, device=DEV)
        cache.scales[cache.block_table[i].long()[at // page], :, at % page] = 200
    return cache


def _tree(g, b, t, kind):
    if kind == "chain":
        return None
    up = (torch.rand((b, t), generator=g, device=DEV) * (torch.arange(t, device=DEV) + 1)).long() - 1
    if kind == "bushy":    # two levels
        up = torch.where(torch.arange(t, device=DEV) % 3 == 0, -1, (torch.arange(t, device=DEV) // 3 * 3)).expand(b, t)
    if kind == "line":     # the chain, said in parents
        up = (torch.arange(t, device=DEV) - 1).expand(b, t)
    if kind == "odd":      # numbers that are no earlier draft: the context
        up = torch.where(torch.arange(t, device=DEV) % 4 == 1, torch.arange(t, device=DEV) + 3, up)
        up = torch.where(torch.arange(t, device=DEV) % 4 == 2, -7, up)
        up = torch.where(torch.arange(t, device=DEV) % 8 == 3, torch.arange(t, device=DEV), up)
    up = up.to(torch.int32).contiguous()
    return up[0].contiguous() if kind == "shared" else up


def _run(dtype, q, cache, keys, t, parents, drafts, **kw):
    b, _, h, d = q.shape
    out = torch.full(q.shape, MARK, dtype=q.dtype, device=DEV)
    lse = torch.full((b, h, t), MARK, device=DEV)
    n = torch.tensor(keys, dtype=torch.int32, device=DEV)
    dl = None if drafts is None else torch.tensor(drafts, dtype=torch.int32, device=DEV)
    got = cg.tree_attention_fwd(q, *cache.args(), n, out, parents=parents, draft_lengths=dl, lse=lse, **kw)
    assert got is out
    ref = D.TreeReference(q, cache, keys, parents=parents, draft_lengths=drafts, scale=kw.get("scale"), u=UNIT[dtype])
    live = ref.written
    assert_within("out", out[live], ref.out[live], ref.out_tol[live])
    rows = live[:, None].expand(b, h, t)
    assert_within("lse", lse[rows], ref.lse[rows], ref.lse_tol[rows])
    assert (out[~live] == MARK).all() and (lse[~rows] == MARK).all()
    return out, lse


CASES = [  # dtype, T, H, Hkv, D, page, keys, drafts, tree, heads outside
    ("bf16", 1, 1, 1, 16, 16, [1], None, "chain", True),
    ("bf16", 1, 8, 8, 64, 16, [77], None, "chain", True),
    ("f16", 1, 12, 4, 80, 48, [531, 1, 128, 129, 127], None, "chain", True),
    ("bf16", 1, 32, 8, 128, 64, [700, 64, 0, 1000], None, "chain", False),
    ("bf16", 1, 20, 1, 128, 32, [300, 15, 16, 17], None, "chain", True),
    ("f16", 1, 40, 1, 96, 16, [260, 700], None, "chain", True),
    ("bf16", 7, 8, 4, 128, 64, [400, 7, 8, 133], [7, 7, 3, 5], "random", True),
    ("f16", 5, 6, 2, 112, 16, [5, 130, 260], None, "bushy", False),
    ("bf16", 8, 4, 2, 64, 256, [900, 8], None, "shared", True),
    ("f16", 3, 4, 4, 48, 16, [3, 1, 140], [3, 3, 0], "chain", True),       # more drafts than tokens
    ("bf16", 16, 2, 2, 128, 1024, [2000, 16], [16, 1], "odd", True),
    ("f16", 29, 12, 4, 80, 48, [531, 30, 333], [29, 20, 7], "random", True),
    ("bf16", 64, 8, 2, 128, 64, [700, 64, 129], [64, 60, 33], "random", True),
    ("f16", 100, 6, 2, 64, 32, [1000, 101], None, "line", False),
    ("bf16", 256, 4, 1, 128, 16, [300, 256], [256, 250], "random", True),
    ("f16", 256, 1, 1, 32, 16, [256, 1500], None, "chain", True),
    ("bf16", 33, 40, 8, 128, 48, [1000], None, "random", True),
    ("bf16", 13, 3, 1, 16, 16, [1, 13, 40, 0], [13, 13, 0, 5], "random", True),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_cases(case):
    dtype, t, h, hkv, d, page, keys, drafts, kind, outside = case
    g = _gen(t * 7 + h + d)
    b = len(keys)
    cache = _filled(g, dtype, keys, hkv, d, page, outside=outside)
    q = torch.randn((b, t, h, d), generator=g, device=DEV).to(TYPES[dtype])
    _run(dtype, q, cache, keys, t, _tree(g, b, t, kind), drafts)


@pytest.mark.parametrize("t,h,hkv", [(1, 4, 1), (9, 4, 2), (40, 8, 2)])
def test_long_contexts_cut_between_blocks(t, h, hkv):
    """Few requests and many keys: every row's keys are shared out."""
    g, keys = _gen(t), [30011, 9000]
    cache = _filled(g, "bf16", keys, hkv, 128, 64)
    q = torch.randn((2, t, h, 128), generator=g, device=DEV).bfloat16()
    _run("bf16", q, cache, keys, t, _tree(g, 2, t, "random"), None)


def test_strides_and_scale():
    """Queries and outputs as parts of fused projections; a scale of its own."""
    g, keys = _gen(11), [333, 90]
    cache = _filled(g, "f16", keys, 2, 64, 32, outside=False)
    fused = torch.randn((2, 6, 3, 4, 64), generator=g, device=DEV).half()
    q = fused[:, :, 1]
    wide = torch.full((2, 8, 6, 80), MARK, dtype=torch.float16, device=DEV)
    out = wide[:, 1:7, 1:5, 8:72]
    n = torch.tensor(keys, dtype=torch.int32, device=DEV)
    cg.tree_attention_fwd(q, *cache.args(), n, out, scale=0.05)
    ref = D.TreeReference(q, cache, keys, scale=0.05, u=UNIT["f16"])
    assert_within("out", out, ref.out, ref.out_tol)
    edge = wide.clone()
    edge[:, 1:7, 1:5, 8:72] = MARK
    assert (edge == MARK).all()
    heads = q.transpose(1, 2).contiguous().transpose(1, 2)
    other = torch.empty_like(heads)
    cg.tree_attention_fwd(heads, *cache.args(), n, other, scale=0.05)
    assert torch.equal(other, out)


def test_tables_and_trees_as_parts_of_larger_ones(monkeypatch):
    """Rows of the block table and of the parents further apart than they are long; the tensors' device
    not the current one, as far as one device can show."""
    g, keys, t = _gen(24), [333, 90], 30
    cache = _filled(g, "bf16", keys, 2, 64, 32)
    q = torch.randn((2, t, 6, 64), generator=g, device=DEV).bfloat16()
    up = _tree(g, 2, t, "random")
    n = torch.tensor(keys, dtype=torch.int32, device=DEV)
    want, got = torch.empty_like(q), torch.empty_like(q)
    cg.tree_attention_fwd(q, *cache.args(), n, want, parents=up)
    width = cache.block_table.shape[1]
    wide = torch.full((2, width + 3), 1 << 20, dtype=torch.int32, device=DEV)
    wide[:, :width] = cache.block_table
    more = torch.full((2, t + 5), 7, dtype=torch.int32, device=DEV)
    more[:, :t] = up
    monkeypatch.setattr(decoder, "_current_device", lambda: -1)
    cg.tree_attention_fwd(q, cache.k, cache.v, cache.scales, wide[:, :width], n, got, parents=more[:, :t])
    assert torch.equal(want, got)
    back = [torch.empty((2, 333, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    cg.kv_cache_read(*cache.args(), None, *back[:2], lengths=n)
    cg.kv_cache_read(cache.k, cache.v, cache.scales, wide[:, :width], None, *back[2:], lengths=n)
    for i, k in enumerate(keys):
        assert torch.equal(back[0][i, :k], back[2][i, :k]) and torch.equal(back[1][i, :k], back[3][i, :k])


def test_one_query_for_all():
    """Queries broadcast over heads and requests."""
    g, keys = _gen(12), [100, 300]
    cache = _filled(g, "bf16", keys, 2, 128, 16)
    q = torch.randn((1, 3, 1, 128), generator=g, device=DEV).bfloat16().expand(2, 3, 4, 128)
    _run("bf16", q, cache, keys, 3, None, None)


def test_tokens_that_are_none():
    """Pages that are none and tokens that were never written take no part, whatever lies there; a row
    that is left without any gives zeros and -inf."""
    g, keys = _gen(13), [200, 64, 90]
    cache = _filled(g, "bf16", keys, 2, 64, 32)
    cache.block_table[0, 2], cache.block_table[1, 0], cache.block_table[1, 1] = -1, 999, -5
    page = int(cache.block_table[2, 1])
    cache.scales[page, :, 3:17] = 0
    cache.k.view(torch.uint8)[page, 3:17] = 0x7F
    cache.v.view(torch.uint8)[page, 3:17] = 0xFF
    cache.scales[int(cache.block_table[2, 0]), 1] = 0         # of one head alone
    q = torch.randn((3, 4, 6, 64), generator=g, device=DEV).bfloat16()
    out, lse = _run("bf16", q, cache, keys, 4, None, None)
    assert not out[1].any() and (lse[1] == -math.inf).all()
    for t in (40,):        # more rows than go through the keys together
        q = torch.randn((3, t, 6, 64), generator=g, device=DEV).bfloat16()
        out, lse = _run("bf16", q, cache, keys, t, _tree(g, 3, t, "random"), None)
        assert not out[1].any() and (lse[1] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t", [2, 40])
def test_rows_of_very_different_size(dtype, t):
    """Exponents of keys and values far apart, large and small queries."""
    g, keys, dt = _gen(14), [700, 300], TYPES[dtype]
    cache = D.Cache(g, 2, 700, 2, 128, 64)
    top = 9 if dtype == "f16" else 30
    k, v = (torch.randn((2, 700, 2, 128), generator=g, device=DEV) for _ in range(2))
    k = k * torch.pow(2.0, torch.randint(-14, 2, (2, 700, 2, 1), generator=g, device=DEV).float())
    v = v * torch.pow(2.0, torch.randint(-top, top, (2, 700, 2, 1), generator=g, device=DEV).float())
    cg.kv_cache_write(k.to(dt), v.to(dt), *cache.args(), None)
    q = torch.randn((2, t, 4, 128), generator=g, device=DEV)
    q = (q * torch.pow(2.0, torch.randint(-12, 3, (2, t, 4, 128), generator=g, device=DEV).float())).to(dt)
    _run(dtype, q, cache, keys, t, _tree(g, 2, t, "random"), None)


def test_queries_of_any_size_in_bfloat16():
    """Rows near the type's ends: scores that are small, or that one key takes all of."""
    g, keys = _gen(15), [300]
    cache = _filled(g, "bf16", keys, 1, 64, 16)
    q = torch.randn((1, 12, 1, 64), generator=g, device=DEV)
    q *= torch.pow(2.0, torch.tensor([-130.0, -126, -100, -30, -14, -5, 0, 3, 5, 6, 7, 8], device=DEV))[:, None, None]
    _run("bf16", q.bfloat16(), cache, keys, 12, None, None)


def test_a_query_that_is_not_finite_stays_alone():
    g, keys = _gen(16), [200]
    cache = _filled(g, "bf16", keys, 2, 64, 16)
    for t in (5, 40):
        q = torch.randn((1, t, 4, 64), generator=g, device=DEV).bfloat16()
        clean, out = torch.empty_like(q), torch.empty_like(q)
        n = torch.tensor(keys, dtype=torch.int32, device=DEV)
        cg.tree_attention_fwd(q, *cache.args(), n, clean)
        q[0, 1, 2, 7] = float("nan")
        q[0, 3, 0, 0] = float("inf")
        cg.tree_attention_fwd(q, *cache.args(), n, out)
        keep = torch.ones((1, t, 4), dtype=torch.bool, device=DEV)
        keep[0, 1, 2] = keep[0, 3, 0] = False
        assert torch.equal(out[keep], clean[keep])
        assert out[0, 1, 2].isnan().all()


def test_requests_do_not_depend_on_one_another():
    """A request alone gives the same numbers, up to where its keys are cut."""
    g, keys, t = _gen(17), [500, 40, 900], 6
    cache = _filled(g, "bf16", keys, 2, 128, 32)
    q = torch.randn((3, t, 8, 128), generator=g, device=DEV).bfloat16()
    up = _tree(g, 3, t, "random")
    out, _ = _run("bf16", q, cache, keys, t, up, None)
    for i in range(3):
        alone = torch.empty_like(q[i:i + 1])
        cg.tree_attention_fwd(q[i:i + 1], cache.k, cache.v, cache.scales, cache.block_table[i:i + 1],
                              torch.tensor(keys[i:i + 1], dtype=torch.int32, device=DEV), alone, parents=up[i:i + 1])
        ref = D.TreeReference(q, cache, keys, parents=up, u=UNIT["bf16"])
        assert_within("out", alone[0], ref.out[i], ref.out_tol[i])


def test_equal_calls_give_equal_bits_and_share_workspaces():
    """Two captured graphs over one workspace, replayed in turn, its contents foreign."""
    g = _gen(18)
    sets = []
    for keys, t in (([3000, 700], 3), ([1500, 64], 40)):
        cache = _filled(g, "bf16", keys, 2, 128, 64)
        q = torch.randn((2, t, 8, 128), generator=g, device=DEV).bfloat16()
        sets.append((q, cache, torch.tensor(keys, dtype=torch.int32, device=DEV), _tree(g, 2, t, "random")))
    size = max(cg.tree_attention_workspace_size(2, 8, 2, q.shape[1], c.block_table.shape[1] * 64, 128)
               for q, c, _, _ in sets)
    ws = cg.new_workspace(size, DEV)
    first, graphs, outs = [], [], []
    for q, c, n, up in sets:
        o = torch.empty_like(q)
        cg.tree_attention_fwd(q, *c.args(), n, o, parents=up)
        first.append(o)
        outs.append(torch.empty_like(q))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cg.tree_attention_fwd(q, *c.args(), n, outs[-1], parents=up, workspace=ws)
        graphs.append(graph)
    ws[cg.CONV_STATUS_BYTES:] = 0xFF
    for _ in range(3):
        for graph, o, want in zip(graphs, outs, first):
            o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want)
    assert cg.conv_check_device_status(ws) == (0, 0)


def test_another_stream_with_its_own_workspace():
    g, keys = _gen(19), [2000, 900]
    cache = _filled(g, "f16", keys, 2, 64, 64)
    q = torch.randn((2, 4, 4, 64), generator=g, device=DEV).half()
    n = torch.tensor(keys, dtype=torch.int32, device=DEV)
    want, got = torch.empty_like(q), torch.empty_like(q)
    cg.tree_attention_fwd(q, *cache.args(), n, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cg.tree_attention_fwd(q, *cache.args(), n, got, stream=side)
    side.synchronize()
    assert torch.equal(want, got)


@pytest.mark.parametrize("t,h,hkv,d", [(1, 4, 1, 128), (6, 8, 2, 64), (50, 4, 1, 128)])
def test_guard_bytes_behind_an_exact_workspace(t, h, hkv, d):
    g, keys = _gen(20), [5000, 129]
    cache = _filled(g, "bf16", keys, hkv, d, 64)
    q = torch.randn((2, t, h, d), generator=g, device=DEV).bfloat16()
    size = cg.tree_attention_workspace_size(2, h, hkv, t, cache.block_table.shape[1] * 64, d)
    ws = torch.zeros(size + 8192, dtype=torch.uint8, device=DEV)
    ws[size:] = 0x5A
    cg.tree_attention_fwd(q, *cache.args(), torch.tensor(keys, dtype=torch.int32, device=DEV), torch.empty_like(q),
                          workspace=ws[:size])
    assert (ws[size:] == 0x5A).all() and not ws[:cg.CONV_STATUS_BYTES].any()


@pytest.mark.parametrize("t", [20, 64, 100])
def test_a_wait_that_runs_out_is_reported(t):
    """Many rows: the widened keys are not announced, every wait for them ends, and the next call is
    right again."""
    g, keys = _gen(23), [700, 300]
    cache = _filled(g, "bf16", keys, 2, 128, 64)
    q = torch.randn((2, t, 8, 128), generator=g, device=DEV).bfloat16()
    out, n = torch.empty_like(q), torch.tensor(keys, dtype=torch.int32, device=DEV)
    ws = cg.new_workspace(cg.tree_attention_workspace_size(2, 8, 2, t, cache.block_table.shape[1] * 64, 128), DEV)
    lib = _lib.lib()
    try:
        lib.conv_testing_set_wait_fault(1, 5_000_000)
        cg.tree_attention_fwd(q, *cache.args(), n, out, workspace=ws)
        status, bits = cg.conv_check_device_status(ws)
    finally:
        lib.conv_testing_set_wait_fault(0, 0)
    assert status == cg.CONV_ERR_DEVICE_TIMEOUT and bits != 0 and bits & ~7 == 0, (status, bits)
    cg.tree_attention_fwd(q, *cache.args(), n, out, workspace=ws)
    assert cg.conv_check_device_status(ws) == (0, 0)
    ref = D.TreeReference(q, cache, keys, u=UNIT["bf16"])
    assert_within("out", out, ref.out, ref.out_tol)


def test_offsets_past_32_bits():
    pages, page, d = 40000, 1024, 128
    g = _gen(21)
    cache = D.Cache(g, 1, 2048, 1, d, page)
    store = torch.zeros((pages, page, 1, d), dtype=torch.uint8, device=DEV).view(D.E4M3)
    cache.k = cache.v = store
    cache.scales = torch.zeros((pages, 1, page, 2), dtype=torch.uint8, device=DEV)
    cache.block_table = torch.tensor([[39999, 33555]], dtype=torch.int32, device=DEV)
    k = torch.randn((1, 1500, 1, d), generator=g, device=DEV).bfloat16()
    cg.kv_cache_write(k, k, *cache.args(), None)
    for t in (2, 40):
        q = torch.randn((1, t, 2, d), generator=g, device=DEV).bfloat16()
        _run("bf16", q, cache, [1500], t, None, None)


def test_refusals():
    i, ns = cg.CONV_ERR_INVALID_VALUE, cg.CONV_ERR_NOT_SUPPORTED
    c = D.Cache(_gen(22), 2, 64, 2, 64, 16)
    q = torch.zeros((2, 5, 4, 64), dtype=torch.bfloat16, device=DEV)
    n = torch.zeros(2, dtype=torch.int32, device=DEV)
    good = dict(q=q, k_cache=c.k, v_cache=c.v, scales=c.scales, block_table=c.block_table, kv_lengths=n,
                output=torch.empty_like(q))

    def refused(status, kw=None, **change):
        with pytest.raises(cg.ConvError) as e:
            cg.tree_attention_fwd(*dict(good, **change).values(), **(kw or {}))
        assert e.value.status == status, str(e.value)

    refused(ns, q=q.float())
    refused(i, q=q.cpu())
    refused(i, q=q[0])
    refused(i, q=q[..., :32])
    refused(i, q=q[:, :, :3], output=q[:, :, :3].clone())      # heads no multiple
    refused(i, output=q[:, :4])
    refused(i, output=q.half())
    refused(i, output=q[:1].expand(2, 5, 4, 64))
    refused(i, k_cache=c.k.view(torch.uint8))
    refused(i, v_cache=c.v[1:])
    refused(i, scales=c.scales[..., :1])
    refused(i, block_table=c.block_table.long())
    refused(i, kv_lengths=None)
    refused(i, kv_lengths=n.long())
    refused(i, kv_lengths=n[:1])
    refused(i, dict(draft_lengths=n.float()))
    refused(i, dict(parents=torch.zeros((2, 4), dtype=torch.int32, device=DEV)))
    refused(i, dict(parents=torch.zeros((2, 5), dtype=torch.int64, device=DEV)))
    refused(i, dict(parents=torch.zeros((5, 2), dtype=torch.int32, device=DEV).t()))
    refused(i, dict(lse=torch.zeros((2, 5, 4), device=DEV)))
    for scale in (0.0, -1.0, math.inf, math.nan):
        refused(i, dict(scale=scale))
    refused(i, dict(workspace=torch.zeros(1 << 22, dtype=torch.uint8)))
    size = cg.tree_attention_workspace_size(2, 4, 2, 5, 64, 64)
    refused(cg.CONV_ERR_WORKSPACE_TOO_SMALL, dict(workspace=cg.new_workspace(size, DEV)[:size - 1]))
    refused(cg.CONV_ERR_MISALIGNED, dict(workspace=cg.new_workspace(size + 16, DEV)[8:]))
    many = torch.zeros((2, 257, 4, 64), dtype=torch.bfloat16, device=DEV)
    refused(ns, q=many, output=many.clone())
    for bad in ((2, 4, 3, 5, 64, 64), (2, 4, 2, 257, 64, 64), (2, 4, 2, 5, 64, 72), (-1, 4, 2, 5, 64, 64)):
        with pytest.raises(cg.ConvError):
            cg.tree_attention_workspace_size(*bad)
    cg.tree_attention_fwd(*good.values(), workspace=cg.new_workspace(size, DEV))
    cg.tree_attention_fwd(q[:0], c.k, c.v, c.scales, c.block_table[:0], n[:0], q[:0].clone())
    none = q[:, :0]
    cg.tree_attention_fwd(none, *c.args(), n, none.clone())
