"""The norm with the rotation at sizes where every warp walks many rows: tokens whose heads it walks
with their angles held, and rows back to back; with several steps of the backward pass's ring."""
import math

import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _attention as A
from tests.test_gpu_attention import DEV, _gen, _normal, _tables

pytestmark = pytest.mark.gpu

WALKS = [  # b, lq, lk, h, hkv, d, rot
    (2, 5001, 2503, 3, 7, 128, 128),     # tokens' heads: odd heads, two tokens a warp or more
    (3, 9001, 77, 4, 8, 40, 32),         # lanes that are no power of two (halves: 2 + 1; adjacent: 3)
    (2, 3001, 3001, 15, 1, 64, 64),      # k: one head each, rows back to back
    (4, 5003, 0, 4, 4, 72, 24),          # words of 4 elements (halves)
    (1, 20011, 10007, 2, 2, 24, 24),
    (1, 5000, 2600, 3, 4, 256, 64),
    (5, 2600, 1300, 1, 3, 120, 0),       # no rotation
    (2, 6007, 5, 4, 1, 96, 96),
    (1, 700, 3, 37, 8, 80, 80),          # few tokens with many heads: rows back to back
    (7, 301, 299, 9, 5, 104, 104),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("size", WALKS, ids=lambda s: "x".join(map(str, s)))
def test_walks(size, adjacent, dtype):
    b, lq, lk, h, hkv, d, rot = size
    g, dt, u = _gen(sum(size)), A.TYPES[dtype], A.UNIT[dtype]
    rows = max(lq, lk) + 100
    cos, sin = _tables(rows, rot) if rot else (None, None)
    sizes = {"q": (lq, h), "k": (lk, hkv)}
    x, w, pos, dy, y, dx, dw = {}, {}, {}, {}, {}, {}, {}
    for n, (length, heads) in sizes.items():
        if not length:
            for part in (x, w, pos, dy, y, dx, dw):
                part[n] = None
            continue
        x[n] = _normal(g, (b, length, heads, d), dt, 1.5)
        w[n] = _normal(g, (d,), torch.float32 if n == "q" else dt) + 1
        first = torch.randint(0, 100, (b, 1), generator=g, device=DEV)
        pos[n] = (first + torch.arange(length, device=DEV)).to(torch.int32)   # each request's own
        dy[n] = _normal(g, x[n].shape, dt)
        y[n] = torch.full_like(x[n], math.nan)
        dx[n] = torch.full_like(x[n], math.nan)
        dw[n] = torch.full((d,), math.nan, device=DEV)
    kw = dict(cos=cos, sin=sin, q_positions=pos["q"], k_positions=pos["k"], eps=1e-5,
              adjacent_pairs=adjacent)
    cg.qk_norm_rope_fwd(x["q"], x["k"], w["q"], w["k"], y["q"], y["k"], **kw)
    cg.qk_norm_rope_bwd(dy["q"], dy["k"], x["q"], x["k"], w["q"], w["k"], dx["q"], dx["k"], dw["q"],
                        dw["k"], **kw)
    for n in x:
        if x[n] is None:
            continue
        ref = A.NormReference(x[n], w[n], cos, sin, pos[n], 1e-5, adjacent, u, dy[n])
        A.assert_within(n, y[n], ref.y, ref.y_tol)
        A.assert_within("d" + n, dx[n], ref.dx, ref.dx_tol)
        A.assert_within("d%s_weight" % n, dw[n], ref.dw, ref.dw_tol)
