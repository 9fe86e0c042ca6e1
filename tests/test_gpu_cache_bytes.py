"""A key's byte of 0 says that nothing was written, whatever the value's byte is."""
import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests.test_gpu_tree_attention import DEV, _filled, _gen, _run, _tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("byte", [1, 126, 254, 255])
@pytest.mark.parametrize("t", [1, 5, 40])      # a few rows of a key head, two groups of rows, more
def test_a_value_without_a_key(t, byte):
    g, keys = _gen(t + byte), [300, 64, 129]
    cache = _filled(g, "bf16", keys, 2, 64, 32)
    for b, first in ((0, 0), (1, 1), (2, 2)):
        page = int(cache.block_table[b, first])
        cache.scales[page, :, 3:17, 0] = 0
        cache.scales[page, :, 3:17, 1] = byte
        cache.k.view(torch.uint8)[page, 3:17] = 0x7F
        cache.v.view(torch.uint8)[page, 3:17] = 0xFF
    q = torch.randn((3, t, 8, 64), generator=g, device=DEV).bfloat16()
    _run("bf16", q, cache, keys, t, _tree(g, 3, t, "random"), None)
    k, v = (torch.ones((3, 32, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cg.kv_cache_read(*cache.args(), None, k, v)
    assert not k[0, 3:17].any() and not v[0, 3:17].any()
