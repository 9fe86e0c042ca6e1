"""float16 gradients where rows of dout differ by large factors.  Scaling a row of dout by a power of
two scales its dq by the same (nothing is lost as long as both stay within the type's normal numbers),
and one request's or key head's gradients do not depend on another's size."""
import pytest
import torch

from tests import _attention as A
from tests.test_gpu_attention import DEV, _compare, _gen, _make_mask, _normal, _run

pytestmark = pytest.mark.gpu
DT = torch.float16
STEP = 2.0 ** -24        # of float16's subnormal numbers

CASES = [  # b, lq, lk, h, hkv, d, mask
    (1, 200, 2048, 4, 2, 128, "none"),
    (2, 300, 700, 2, 2, 64, "lengths"),
    (1, 333, 900, 6, 2, 80, "rows"),
    (2, 130, 100, 3, 3, 96, "none"),       # one tile of keys
    (2, 150, 128, 4, 2, 40, "heads"),
    (2, 400, 77, 4, 4, 40, "none"),        # one tile of keys, narrow heads, no mask
    (3, 300, 128, 8, 2, 64, "lengths"),
]


def _tensors(case, seed):
    b, lq, lk, h, hkv, d, kind = case
    g = _gen(seed)
    # Keys four times as large and queries a quarter: larger dq for the same scores.
    q, k = _normal(g, (b, lq, h, d), DT, 0.25), _normal(g, (b, lk, hkv, d), DT, 4.0)
    v = _normal(g, (b, lk, hkv, d), DT)
    # Multiples of 2^-6, so that small powers of two scale them exactly.
    dout = (torch.randint(-128, 129, (b, lq, h, d), generator=g, device=DEV) / 64).to(DT)
    n, m = _make_mask(kind, g, b, h, lq, lk)
    return g, q, k, v, dout, dict(kv_lengths=n, mask=m)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_a_row_of_dout_scales_its_dq(case):
    g, q, k, v, dout, kw = _tensors(case, 31)
    b, lq, _, h, _, _, _ = case
    power = torch.randint(-8, -5, (b, lq, h, 1), generator=g, device=DEV)
    power[:, 7::50] = 8
    power[:, 5::60, ::2] = 3
    scale = torch.exp2(power.float())
    scaled = (dout.float() * scale).to(DT)
    assert torch.equal(scaled.float(), dout.float() * scale)
    base = _run(q, k, v, dout, **kw)[2].float()
    got = _run(q, k, v, scaled, **kw)[2].float()
    off = (got - base * scale).abs()
    # Subnormal results are rounded by steps of 2^-24, twice.
    assert (off <= torch.where((base * scale).abs() < 2.0 ** -14, STEP, 0.0)).all(), float(
        (off / (base * scale).abs().clamp(min=STEP)).max())


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** -6])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_gradients_do_not_depend_on_other_requests_and_key_heads(case, size):
    b, lq, lk, h, hkv, d, kind = case
    g, q, k, v, dout, kw = _tensors(case, 32)
    group = h // hkv
    factor = torch.ones((b, 1, hkv, 1), device=DEV)
    factor[:, :, 1::2] = size
    factor[1:] = size
    factor = factor * torch.ones((b, 1, hkv, 1), device=DEV)
    scaled = (dout.float() * factor.repeat_interleave(group, dim=2)).to(DT)
    base, got = _run(q, k, v, dout, **kw), _run(q, k, v, scaled, **kw)
    same_k = (factor == 1).expand(b, lk, hkv, d)
    same_q = (factor == 1).repeat_interleave(group, dim=2).expand(b, lq, h, d)
    assert torch.equal(base[2][same_q], got[2][same_q])
    assert torch.equal(base[3][same_k], got[3][same_k])
    assert torch.equal(base[4][same_k], got[4][same_k])
    # Values' sizes do not matter to other key heads either.
    big = torch.where(factor == 1, v.float(), v.float() * 2.0 ** 8).to(DT)
    base, got = _run(q, k, v, dout, **kw), _run(q, k, big, dout, **kw)
    assert torch.equal(base[2][same_q], got[2][same_q])
    assert torch.equal(base[3][same_k], got[3][same_k])


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_rows_of_very_different_size_within_bounds(case):
    g, q, k, v, dout, kw = _tensors(case, 33)
    b, lq, lk, h, hkv, d, kind = case
    power = torch.randint(-9, -5, (b, lq, h, 1), generator=g, device=DEV)
    power[:, 3::40] = 7
    dout = (dout.float() * torch.exp2(power.float())).to(DT)
    got = _run(q, k, v, dout, **kw)
    _compare(got, A.Reference(q, k, v, dout=dout, u=A.UNIT["f16"], **kw))


@pytest.mark.parametrize("case", [
    (2, 200, 700, 4, 2, 64, "keys"), (1, 300, 1500, 2, 2, 128, "tail"), (2, 150, 400, 4, 2, 80, "rows"),
    (2, 200, 100, 4, 1, 40, "keys"), (1, 260, 600, 6, 2, 24, "heads"), (3, 100, 500, 3, 3, 8, "tail"),
    (2, 300, 640, 2, 1, 48, "lengths")], ids=lambda c: "x".join(map(str, c)))
def test_large_values_that_no_query_attends_change_nothing(case):
    """Masked padding that holds large finite numbers: the same bits as with zeros there."""
    b, lq, lk, h, hkv, d, kind = case
    g, q, k, v, dout, kw = _tensors(case, 34)
    if kind in ("rows", "heads"):
        kw["mask"][..., lk // 3:lk // 2] = 0
    keep = A.pairs(b, h, lq, lk, **kw)
    live = keep.any(2).reshape(b, hkv, h // hkv, lk).any(2).transpose(1, 2)
    dout = (dout.float() / 256).to(DT)
    runs = []
    for fill in (0.0, 6e4):
        k2, v2 = k.clone(), v.clone()
        k2[~live] = fill
        v2[~live] = fill
        runs.append(_run(q, k2, v2, dout, **kw))
    assert not live.all()
    for x, y in zip(*runs):
        assert torch.equal(x, y)
    _compare(runs[1], A.Reference(q, k, v, dout=dout, u=A.UNIT["f16"], **kw))


SMALL = [  # b, lq, lk, h, hkv, d: one tile of keys, shares of the keys, pairs
    (2, 300, 120, 4, 4, 40), (3, 1, 3000, 8, 2, 128), (1, 5, 4000, 2, 2, 64), (2, 1500, 2000, 16, 16, 64),
    (2, 200, 100, 2, 2, 128),
]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("size", SMALL, ids=lambda s: "x".join(map(str, s)))
def test_many_small_probabilities_beside_a_large_one(size, masked):
    """One key takes nearly all of every row and holds zeros; the output is what the others add, whose
    probabilities lie between 2^-20 and 2^-28 of its own.  Their roundings are half a step of float16's
    subnormals at most, of P times 2^7: 2^-32 each."""
    b, lq, lk, h, hkv, d = size
    g = _gen(sum(size))
    q = torch.full((b, lq, h, d), 1.0, dtype=DT, device=DEV)
    k = _normal(g, (b, lk, hkv, d), DT, 0.01)
    # scale * q.k = ln 2 * (0 for the first key, -20 .. -28 for the others)
    drop = 20 + 8 * torch.rand((b, lk, hkv, 1), generator=g, device=DEV)
    drop[:, 0] = 0
    k[..., :1] -= (drop * 0.6931 / 0.25 / 8).to(DT)
    for i in range(1, 8):
        k[..., i:i + 1] -= (drop * 0.6931 / 0.25 / 8).to(DT)
    v = (torch.rand((b, lk, hkv, d), generator=g, device=DEV) * 200 + 100).to(DT)
    v[:, 0] = 0
    mask = None
    if masked:
        mask = torch.rand((b, 1, lq, lk), generator=g, device=DEV) < 0.7
        mask[..., 0] = True
    out, lse = _run(q, k, v, mask=mask, scale=0.25)
    ref = A.Reference(q, k, v, mask=mask, scale=0.25, u=A.UNIT["f16"])
    keep = A.pairs(b, h, lq, lk, None, mask).double()
    total = (keep @ v.double().transpose(1, 2).repeat_interleave(h // hkv, dim=1)).transpose(1, 2)
    bound = ref.out_tol - (2.0 ** -24 - 2.0 ** -31) * total     # (the general bound allows 2^-24 each)
    assert (ref.out > 4 * bound).all()
    A.assert_within("out", out, ref.out, bound)
    A.assert_within("lse", lse, ref.lse, ref.lse_tol)
