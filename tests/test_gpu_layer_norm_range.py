"""Layer norm of rows whose squares, or sums, pass fp32's range, and of rows without variance."""
import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _decoder as D
from tests._attention import UNIT, assert_within
from tests.test_gpu_layer_norm import DEV, _gen, _rows

pytestmark = pytest.mark.gpu

# Part of a warp, a warp, a block; rows that begin inside words; element by element.
CHANNELS = [1, 8, 24, 64, 320, 333, 1280, 1281, 2056, 4096, 4099, 8192, 9001, 16384]


def _norm(x, w, b, dy, eps):
    rows, c = x.shape
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dw, db = torch.empty(c, device=DEV), torch.empty(c, device=DEV)
    cg.layer_norm_fwd(x, w, b, y, mean=mean, rstd=rstd, eps=eps)
    cg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("c", CHANNELS)
def test_far_rows(c):
    """Deviations up to 1e37, means up to 1e37 that sum to more than fp32 holds, beside rows of
    ordinary size, whose bits stay."""
    g = _gen(c)
    x, dy = _rows(g, 24, c, torch.float32), torch.randn((24, c), generator=g, device=DEV).bfloat16()
    plain = x.bfloat16()
    for row, size in ((1, 1e17), (4, 1e18), (5, 1e19), (6, 1e20), (9, 1e25), (14, 1e30), (15, 1e37)):
        x[row] *= size
    for row, size in ((2, 1e20), (7, 1e30), (20, 1e37)):
        x[row] = size * (1 + 0.25 * x[row])
    x = x.bfloat16()
    w = (1 + 0.2 * torch.randn(c, generator=g, device=DEV)).bfloat16()
    b = (0.1 * torch.randn(c, generator=g, device=DEV)).bfloat16()
    got, was = _norm(x, w, b, dy, 1e-5), _norm(plain, w, b, dy, 1e-5)
    ref = D.NormReference(x, w, b, 1e-5, UNIT["bf16"], dy)
    # dx of the largest rows lies among bfloat16's subnormal numbers, multiples of 2^-133: rounding to
    # those is off by up to 2^-134 (the reference's grain is fp16's or less), and up to eight roundings to
    # fp32's, multiples of 2^-149, by 2^-150 each.
    ref.dx_tol = ref.dx_tol + 2.0 ** -134 + 8 * 2.0 ** -150
    for name, t in zip(("y", "mean", "rstd", "dx", "dweight", "dbias"), got):
        assert_within(name, t, getattr(ref, name), getattr(ref, name + "_tol"))
    same = (x == plain).all(1)
    assert int(same.sum()) >= 14
    for t, u in list(zip(got, was))[:4]:
        assert torch.equal(t[same], u[same])


def test_a_far_row_beside_one_that_is_not_finite():
    g = _gen(1)
    x = _rows(g, 9, 64, torch.bfloat16)
    x[3] *= 1e25
    x[4, 5], x[5, 0] = float("nan"), float("inf")
    y, mean, rstd, dx, _, _ = _norm(x, None, None, torch.ones_like(x), 1e-5)
    assert y[4].isnan().all() and y[5].isnan().all()
    keep = torch.tensor([i not in (4, 5) for i in range(9)], device=DEV)
    ref = D.NormReference(x[keep], None, None, 1e-5, UNIT["bf16"])
    assert_within("y", y[keep], ref.y, ref.y_tol)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_no_variance_and_no_eps(dt):
    x = _rows(_gen(2), 5, 320, dt)
    x[1], x[3] = 0.0, 2.0
    y, _, rstd, _, _, _ = _norm(x, None, None, torch.ones_like(x), 0.0)
    assert (rstd[1::2] == float("inf")).all() and rstd[::2].isfinite().all()
    assert y[::2].isfinite().all()


@pytest.mark.parametrize("c", [1, 7, 64, 333, 4099, 9001])
def test_far_rows_of_one_value_leave_the_others_gradients(c):
    """(0 - mean) * rstd, of what lies behind a row or of a row that is not there, is infinite."""
    g = _gen(c)
    x = torch.full((700, c), 3e37, dtype=torch.bfloat16, device=DEV)
    dy = torch.randn((700, c), generator=g, device=DEV).bfloat16()
    y, mean, rstd, dx, dw, db = _norm(x, None, None, dy, 1e-5)
    assert not y.any() and not dw.any() and torch.equal(mean, x[:, 0].float())
    assert dx.isfinite().all() and db.isfinite().all()
