"""Layer norm of rows of one value, or nearly of one: deviations are the rows' own, not the rounding of
a sum."""
import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests._attention import F32, TYPES, UNIT, assert_within
from tests.test_gpu_layer_norm import DEV, _gen

pytestmark = pytest.mark.gpu

CHANNELS = [1, 3, 8, 40, 321, 1000, 1281, 2056, 4099, 4104, 9000, 9001, 16384]
EPS = 1e-5


def _norm(x, w, b, dy):
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(x.shape[0], device=DEV) for _ in range(2))
    dw, db = (torch.empty(x.shape[1], device=DEV) for _ in range(2))
    cg.layer_norm_fwd(x, w, b, y, mean=mean, rstd=rstd, eps=EPS)
    cg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("c", CHANNELS)
def test_rows_of_one_value(c, dtype):
    """The first sum is off by less than 2^-14 of it (fewer than 600 additions follow one another), so its
    mean rounds to the value itself: deviations of 0, y the bias, no gradient of the weights."""
    g, dt = _gen(c), TYPES[dtype]
    values = [3.1, -0.1, 1000.0, 60000.0, -777.7, 1e-3] + ([1e8, -1e18] if dtype == "bf16" else [])
    x = torch.tensor(values, device=DEV).to(dt)[:, None].expand(-1, c).contiguous()
    dy = torch.randn(x.shape, generator=g, device=DEV).to(dt)
    w = (1 + 0.2 * torch.randn(c, generator=g, device=DEV)).to(dt)
    b = torch.randn(c, generator=g, device=DEV).to(dt)
    y, mean, rstd, dx, dw, db = _norm(x, w, b, dy)
    assert torch.equal(y, b.expand_as(y)) and torch.equal(mean, x[:, 0].float())
    want = torch.full_like(rstd, EPS).double() ** -0.5
    assert_within("rstd", rstd, want, 4 * F32 * want)
    assert not dw.any()
    gw = dy.double() * w.double()
    ref = want[:, None] * (gw - gw.mean(1, keepdim=True))
    size = gw.abs() + (c + 8) * gw.abs().mean(1, keepdim=True)
    assert_within("dx", dx, ref, UNIT[dtype] * ref.abs() + want[:, None] * 16 * F32 * size + 1e-7)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("c", [c for c in CHANNELS if c > 1])
def test_rows_whose_elements_differ_by_a_step(c, dtype):
    """Few or half of a row's elements one step of the type above the others: the deviations' sums, of
    numbers that are exact, are all that is rounded."""
    g, dt = _gen(c + 1), TYPES[dtype]
    base = torch.tensor([200.0, 1000.0, 33.0, 5000.0], device=DEV).to(dt)
    step = torch.nextafter(base, base + base) - base
    share = torch.tensor([0.5, 0.1, 0.9, 1.5 / c], device=DEV)[:, None]
    up = torch.rand((4, c), generator=g, device=DEV) < share
    up[:, 0], up[:, 1] = True, False
    x = torch.where(up, (base + step)[:, None], base[:, None]).contiguous()
    dy = torch.randn(x.shape, generator=g, device=DEV).to(dt)
    y, mean, rstd, dx, _, _ = _norm(x, None, None, dy)
    xd, u = x.double(), UNIT[dtype]
    m = xd.mean(1, keepdim=True)
    dev = xd - m
    r = ((dev * dev).mean(1, keepdim=True) + EPS) ** -0.5
    # Sums of C numbers of up to a step; the variance loses one bit at most against their squares.
    steps = step.double()[:, None]
    dev_err = (c + 8) * F32 * steps + 2 * F32 * dev.abs()
    rel = (2 * (c + 8) + 8) * F32
    h, h_err = dev * r, r * dev_err + (dev * r).abs() * rel
    assert_within("y", y, h, u * h.abs() + 2 * h_err + 1e-7)
    assert_within("mean", mean[:, None], m, F32 * m.abs() + (c + 8) * F32 * steps)
    assert_within("rstd", rstd[:, None], r, (rel + 4 * F32) * r)
    gd = dy.double()
    mg, mgh = gd.mean(1, keepdim=True), (gd * h).mean(1, keepdim=True)
    ref = r * (gd - mg - h * mgh)
    # (Backward the mean is one in 32 bits.)
    back = h_err + r * (F32 * m.abs() + dev_err)
    tol = u * ref.abs() + r * ((c + 16) * F32 * (gd.abs() + gd.abs().mean(1, keepdim=True) * (1 + h.abs()) + h.abs())
                               + back * mgh.abs() + h.abs() * (gd.abs() * back).mean(1, keepdim=True)) \
        + (rel + 4 * F32) * ref.abs() + 1e-7
    assert_within("dx", dx, ref, tol)
