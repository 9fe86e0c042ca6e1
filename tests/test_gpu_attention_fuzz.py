"""Cross attention at drawn sizes, masks and layouts, against 64 bits (bounds: tests/_attention.py)."""
import random

import pytest
import torch

from tests import _attention as A
from tests.test_gpu_attention import DEV, _compare, _gen, _make_mask, _normal, _run

pytestmark = pytest.mark.gpu


def _spread(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _draw(seed):
    rng = random.Random(seed)
    while True:
        b, hkv, group = rng.choice([1, 2, 3, 7]), _spread(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5])
        lq, lk, d = _spread(rng, 1, 900), _spread(rng, 1, 1800), 8 * rng.randint(1, 16)
        if b * hkv * group * lq * lk <= 3e7:
            break
    kind = rng.choice(["none", "none", "lengths", "keys", "rows", "heads", "tail"])
    return (rng.choice(["bf16", "f16"]), b, lq, lk, hkv * group, hkv, d, kind, rng.random() < 0.3,
            rng.random() < 0.6)


@pytest.mark.parametrize("seed", range(64))
def test_drawn(seed):
    dtype, b, lq, lk, h, hkv, d, kind, heads_first, train = _draw(seed)
    g, dt = _gen(seed), A.TYPES[dtype]

    def tensor(length, heads):
        if heads_first:      # [B, heads, length, D], seen as [B, length, heads, D]
            return _normal(g, (b, heads, length, d), dt).transpose(1, 2)
        return _normal(g, (b, length, heads, d), dt)

    q, k, v = tensor(lq, h), tensor(lk, hkv), tensor(lk, hkv)
    dout = tensor(lq, h) if train else None
    n, m = _make_mask(kind, g, b, h, lq, lk)
    got = _run(q, k, v, dout, kv_lengths=n, mask=m)
    _compare(got, A.Reference(q, k, v, kv_lengths=n, mask=m, dout=dout, u=A.UNIT[dtype]))
