"""The decoder operators at drawn sizes and layouts, against 64 bits (bounds: tests/_decoder.py)."""
import random

import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _decoder as D
from tests._attention import TYPES, UNIT, assert_within
from tests.test_gpu_layer_norm import _check, _rows
from tests.test_gpu_tree_attention import DEV, _filled, _gen, _run, _tree

pytestmark = pytest.mark.gpu


def _spread(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(60))
def test_trees(seed):
    rng = random.Random(seed)
    while True:
        b, hkv, group = rng.choice([1, 2, 3, 5]), rng.choice([1, 1, 2, 3, 8]), rng.choice([1, 1, 2, 3, 4, 7])
        t, most = rng.choice([1, 1, 2, _spread(rng, 1, 256)]), _spread(rng, 1, 3000)
        if b * hkv * group * t * most <= 6e6:
            break
    dtype, d, page = rng.choice(["bf16", "f16"]), 16 * rng.randint(1, 8), 16 * rng.choice([1, 1, 2, 3, 5, 16])
    keys = [rng.choice([most, rng.randint(0, most)]) for _ in range(b)]
    drafts = rng.choice([None, [rng.randint(0, t) for _ in range(b)]])
    g = _gen(seed)
    cache = _filled(g, dtype, keys, hkv, d, page, outside=rng.random() < 0.6, spread=rng.choice([0.1, 0.5, 2.0]))
    if rng.random() < 0.3:      # a token that was never written
        page_of = int(cache.block_table[0, 0])
        cache.scales[page_of, :, 0] = 0
        cache.k.view(torch.uint8)[page_of, 0] = cache.v.view(torch.uint8)[page_of, 0] = 0x7F
    q = (rng.choice([0.1, 1.0, 3.0]) * torch.randn((b, t, hkv * group, d), generator=g, device=DEV)).to(TYPES[dtype])
    kind = rng.choice(["chain", "random", "bushy", "shared", "line", "odd"])
    _run(dtype, q, cache, keys, t, _tree(g, b, t, kind), drafts)


@pytest.mark.parametrize("seed", range(40))
def test_norms(seed):
    rng = random.Random(seed)
    c, rows = _spread(rng, 1, 9000), _spread(rng, 1, 4000)
    if rng.random() < 0.6:
        c = max(8, c // 8 * 8)
    rows = max(1, min(rows, 2000000 // c))
    dtype = rng.choice(["bf16", "f16"])
    g, dt = _gen(seed), TYPES[dtype]
    wide = c + rng.choice([0, 0, 3, 8])      # rows further apart than they are long
    x, dy = _rows(g, rows, wide, dt)[:, :c], torch.randn((rows, wide), generator=g, device=DEV).to(dt)[:, :c]
    wt = rng.choice([dt, torch.float32])
    w = None if rng.random() < 0.2 else (1 + 0.2 * torch.randn(c, generator=g, device=DEV)).to(wt)
    b = None if rng.random() < 0.2 else (0.1 * torch.randn(c, generator=g, device=DEV)).to(wt)
    y, dx = torch.empty((rows, c), dtype=dt, device=DEV), torch.empty((rows, c), dtype=dt, device=DEV)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dw, db = torch.empty(c, device=DEV), torch.empty(c, device=DEV)
    eps = rng.choice([1e-5, 1e-3])
    cg.layer_norm_fwd(x, w, b, y, mean=mean, rstd=rstd, eps=eps)
    cg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)
    _check(x, w, b, y, mean, rstd, dy, dx, dw, db, eps, UNIT[dtype])


@pytest.mark.parametrize("seed", range(30))
def test_caches(seed):
    """Written in pieces of drawn lengths, read back whole: the rows' own values."""
    rng = random.Random(seed)
    b, heads, d = rng.choice([1, 2, 4]), rng.choice([1, 2, 3, 8]), 16 * rng.randint(1, 8)
    page, length = 16 * rng.choice([1, 2, 3, 8]), _spread(rng, 1, 400)
    dtype = rng.choice(["bf16", "f16"])
    g, dt = _gen(seed), TYPES[dtype]
    cache = D.Cache(g, b, length, heads, d, page, outside=rng.random() < 0.5)
    x = torch.randn((2, b, length, heads, d), generator=g, device=DEV)
    x = (x * torch.exp(3 * torch.randn((2, b, length, heads, 1), generator=g, device=DEV))).to(dt)
    at = 0
    while at < length:
        n = rng.randint(1, length - at)
        starts = torch.full((b,), at, dtype=torch.int32, device=DEV)
        cg.kv_cache_write(x[0, :, at:at + n], x[1, :, at:at + n], *cache.args(), starts)
        at += n
    k, v = torch.empty_like(x[0]), torch.empty_like(x[1])
    cg.kv_cache_read(*cache.args(), None, k, v)
    for got, was in zip((k, v), x):
        code, e = D.quantised(was)
        want = (code * D.pow2(e)[..., None]).clamp(-torch.finfo(dt).max, torch.finfo(dt).max)
        assert_within("rows", got, want, torch.zeros_like(want) if dt is torch.bfloat16 else 2.0 ** -25 + 0 * want)
