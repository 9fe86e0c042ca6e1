"""Tree attention with many more items than thread blocks, where a block writes items that it has whole
and leaves shares of others, against the definition in 64 bits."""
import math
import random

import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _decoder as D
from tests._attention import TYPES, UNIT, assert_within
from tests.test_gpu_tree_attention import DEV, _filled, _gen, _run, _tree
from transposed_conv_implicit_gb300 import _lib

pytestmark = pytest.mark.gpu


def _ragged(seed, n, lo, hi):
    rng = random.Random(seed)
    return [rng.randint(lo, hi) for _ in range(n)]


CASES = [  # dtype, T, H, Hkv, D, page, keys, drafts, tree
    ("bf16", 24, 32, 8, 128, 64, [928] * 25, None, "random"),
    ("bf16", 24, 32, 8, 128, 64, [4096] * 64, None, "shared"),
    ("f16", 30, 24, 8, 80, 48, _ragged(1, 40, 30, 400), _ragged(2, 40, 0, 30), "random"),     # some of one key tile
    ("bf16", 94, 8, 2, 64, 32, _ragged(3, 60, 94, 700), None, "random"),                      # 256 rows and 120
    ("f16", 75, 16, 4, 128, 16, [900] * 40, None, "chain"),                                   # 256 rows and 44
    ("bf16", 100, 1, 1, 16, 128, [100, 128, 101], None, "random"),                            # no share anywhere
    ("f16", 70, 2, 2, 48, 16, _ragged(4, 100, 70, 300), None, "line"),
    ("bf16", 13, 40, 8, 112, 64, _ragged(5, 64, 0, 900), _ragged(6, 64, 0, 13), "odd"),
    ("bf16", 33, 4, 2, 32, 16, _ragged(7, 90, 33, 129), None, "bushy"),
    ("f16", 128, 2, 1, 96, 256, _ragged(8, 64, 128, 1100), _ragged(9, 64, 1, 128), "random"), # one and two groups' items
    ("bf16", 7, 32, 8, 128, 64, _ragged(10, 64, 7, 600), None, "random"),                     # few rows
    ("f16", 1, 16, 8, 64, 16, _ragged(11, 100, 0, 900), None, "chain"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-%dx%d-%d-%d-%s" % (c[0], len(c[6]), c[1], c[2], c[4], c[8]))
def test_cases(case):
    dtype, t, h, hkv, d, page, keys, drafts, kind = case
    g, b = _gen(t * 11 + h + d), len(keys)
    cache = _filled(g, dtype, keys, hkv, d, page)
    q = torch.randn((b, t, h, d), generator=g, device=DEV).to(TYPES[dtype])
    up = _tree(g, b, t, kind)
    out, lse = _run(dtype, q, cache, keys, t, up, drafts)
    again, _ = _run(dtype, q, cache, keys, t, up, drafts)
    assert torch.equal(out, again)


@pytest.mark.parametrize("seed", range(20))
def test_drawn(seed):
    rng = random.Random(1000 + seed)
    while True:
        b, hkv, group = rng.randint(16, 64), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        t, most = rng.choice([9, 17, 24, 33, 64, 100, 140, 256]), int(2 ** rng.uniform(6, 11))
        if t * group > 64 and t <= most and b * hkv * group * t * most <= 1e8:
            break
    dtype, d, page = rng.choice(["bf16", "f16"]), 16 * rng.randint(1, 8), 16 * rng.choice([1, 2, 4, 8])
    keys = [rng.choice([most, rng.randint(0, most)]) for _ in range(b)]
    drafts = rng.choice([None, [rng.randint(0, t) for _ in range(b)]])
    g = _gen(seed)
    cache = _filled(g, dtype, keys, hkv, d, page, outside=rng.random() < 0.5)
    q = torch.randn((b, t, hkv * group, d), generator=g, device=DEV).to(TYPES[dtype])
    _run(dtype, q, cache, keys, t, _tree(g, b, t, rng.choice(["chain", "random", "line"])), drafts)


def test_rows_without_keys_and_rows_that_are_not_finite():
    """In items that a block has whole: pages that are none for a tile, or for all; queries with NaN."""
    g, t, b = _gen(3), 40, 40
    keys = [300 + 5 * i for i in range(b)]
    cache = _filled(g, "bf16", keys, 4, 64, 64)
    cache.block_table[::4] = -1                       # no keys
    cache.block_table[1::4, :2] = 1 << 20             # the first tile is none
    cache.block_table[2::4, 2:4] = -3                 # the second
    q = torch.randn((b, t, 8, 64), generator=g, device=DEV).bfloat16()
    out, lse = _run("bf16", q, cache, keys, t, _tree(g, b, t, "random"), None)
    assert not out[::4].any() and (lse[::4] == -math.inf).all()
    q[5, 7, 3, 1], q[6, 0, 0, 0] = float("nan"), float("inf")
    other = torch.empty_like(out)
    cg.tree_attention_fwd(q, *cache.args(), torch.tensor(keys, dtype=torch.int32, device=DEV), other,
                          parents=_tree(_gen(3), b, t, "line"))
    assert other[5, 7, 3].isnan().all() and not other[5, 7, 2].isnan().any() and not other[4].isnan().any()


def test_a_wait_that_runs_out_is_reported():
    g, keys, t = _gen(4), [200] * 40, 20
    cache = _filled(g, "bf16", keys, 8, 64, 64)
    q = torch.randn((40, t, 32, 64), generator=g, device=DEV).bfloat16()
    out, n = torch.empty_like(q), torch.tensor(keys, dtype=torch.int32, device=DEV)
    ws = cg.new_workspace(cg.tree_attention_workspace_size(40, 32, 8, t, cache.block_table.shape[1] * 64, 64), DEV)
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
