"""Workspaces of exactly the size that is asked for: nothing behind them is written."""
import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _attention as A
from tests.test_gpu_attention import DEV, _gen, _normal, _tables

pytestmark = pytest.mark.gpu
GUARD = 0xA5


def guarded(size, room=1 << 16):
    """(a workspace of `size` bytes, the bytes behind it)."""
    buf = torch.full((size + room,), GUARD, dtype=torch.uint8, device=DEV)
    buf[:cg.CONV_STATUS_BYTES] = 0
    return buf[:size], buf[size:]


NORMS = [  # b, lq, lk, h, hkv, d: as many rows as fill the GPU
    (1, 607, 609, 16, 16, 128),
    (1, 1215, 1, 16, 16, 128),
    (2, 1139, 77, 8, 8, 128),
    (1, 3, 1213, 16, 16, 128),
    (1, 1500, 700, 16, 16, 128),
]


@pytest.mark.parametrize("size", NORMS, ids=lambda s: "x".join(map(str, s)))
def test_norm_backward_keeps_to_its_workspace(size):
    b, lq, lk, h, hkv, d = size
    g, dt, u = _gen(sum(size)), torch.bfloat16, A.UNIT["bf16"]
    cos, sin = _tables(max(lq, lk), d)
    x = {"q": _normal(g, (b, lq, h, d), dt), "k": _normal(g, (b, lk, hkv, d), dt)}
    dy = {n: _normal(g, x[n].shape, dt) for n in x}
    w = {n: _normal(g, (d,), dt) + 1 for n in x}
    dx = {n: torch.empty_like(x[n]) for n in x}
    dw = {n: torch.empty((d,), device=DEV) for n in x}
    ws, behind = guarded(cg.qk_norm_rope_workspace_size(d))
    cg.qk_norm_rope_bwd(dy["q"], dy["k"], x["q"], x["k"], w["q"], w["k"], dx["q"], dx["k"], dw["q"],
                        dw["k"], cos=cos, sin=sin, workspace=ws)
    assert (behind == GUARD).all()
    for n in x:
        ref = A.NormReference(x[n], w[n], cos, sin, None, 1e-6, False, u, dy[n])
        A.assert_within("d" + n, dx[n], ref.dx, ref.dx_tol)
        A.assert_within("d%s_weight" % n, dw[n], ref.dw, ref.dw_tol)
