"""Cross attention and the norm with the rotation against their definitions in 64 bits, at the
sizes, layouts and masks where they can go wrong.  Bounds: tests/_attention.py."""
import math

import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dt, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device=DEV)).to(dt)


def _make_mask(kind, g, b, h, lq, lk):
    """(kv_lengths, mask) of a kind."""
    if kind == "none":
        return None, None
    if kind == "lengths":
        n = torch.randint(0, lk + 1, (b,), generator=g, device=DEV).to(torch.int32)
        n[0] = lk
        if b > 1:
            n[1] = 0            # a request without any key
        if b > 2:
            n[2] = lk + 5       # taken as lk
        return n, None
    if kind == "keys":          # padding by a mask shared by heads and queries
        return None, torch.rand((b, 1, 1, lk), generator=g, device=DEV) < 0.6
    if kind == "rows":          # shared by heads; some rows empty
        m = torch.rand((b, 1, lq, lk), generator=g, device=DEV) < 0.3
        m[:, :, ::3] = False
        return None, m
    if kind == "heads":         # everything of its own, bytes, with lengths too
        m = (torch.rand((b, h, lq, lk), generator=g, device=DEV) < 0.5).to(torch.uint8) * 7
        n = torch.randint(0, lk + 1, (b,), generator=g, device=DEV).to(torch.int32)
        return n, m
    if kind == "tail":          # a strided mask: only the last keys
        m = torch.zeros((b, 1, lk, lq), dtype=torch.bool, device=DEV)
        m[:, :, lk - max(1, lk // 5):] = True
        return None, m.transpose(2, 3)
    raise ValueError(kind)


def _run(q, k, v, dout=None, *, kv_lengths=None, mask=None, scale=None, guard=float("nan")):
    """Forward (and backward) into outputs full of `guard`."""
    b, lq, h, d = q.shape
    out = torch.full_like(q, guard, memory_format=torch.contiguous_format)
    lse = torch.full((b, h, lq), guard, dtype=torch.float32, device=DEV)
    kw = dict(kv_lengths=kv_lengths, mask=mask, scale=scale)
    ws = cg.new_workspace(cg.cross_attention_workspace_size(
        b, h, k.shape[2], lq, k.shape[1], d, masked=mask is not None, mask_heads=h, backward=True), DEV)
    cg.cross_attention_fwd(q, k, v, out, lse=lse, workspace=ws, **kw)
    if dout is None:
        assert cg.conv_check_device_status(ws) == (0, 0)
        return out, lse
    dq = torch.full_like(out, guard)
    dk = torch.full(k.shape, guard, dtype=k.dtype, device=DEV)
    dv = torch.full(k.shape, guard, dtype=k.dtype, device=DEV)
    cg.cross_attention_bwd(dout, q, k, v, out, lse, dq, dk, dv, workspace=ws, **kw)
    assert cg.conv_check_device_status(ws) == (0, 0)
    return out, lse, dq, dk, dv


def _compare(got, ref):
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), got):
        A.assert_within(name, x, getattr(ref, name), getattr(ref, name + "_tol"))


def _check(dtype, b, lq, lk, h, hkv, d, kind, *, train=True, seed=0, scale=None, spread=1.0):
    g, dt = _gen(seed), A.TYPES[dtype]
    q = _normal(g, (b, lq, h, d), dt, spread)
    kv = _normal(g, (b, lk, 2, hkv, d), dt)
    k, v = kv[:, :, 0], kv[:, :, 1]
    dout = _normal(g, (b, lq, h, d), dt) if train else None
    n, m = _make_mask(kind, g, b, h, lq, lk)
    got = _run(q, k, v, dout, kv_lengths=n, mask=m, scale=scale)
    _compare(got, A.Reference(q, k, v, scale=scale, kv_lengths=n, mask=m, dout=dout, u=A.UNIT[dtype]))


SIZES = [  # b, lq, lk, h, hkv, d
    (1, 1, 1, 1, 1, 8),
    (2, 1, 77, 4, 4, 64),
    (3, 5, 16, 2, 1, 16),
    (2, 128, 128, 2, 2, 128),
    (1, 129, 127, 2, 1, 128),
    (3, 257, 129, 4, 2, 40),
    (2, 300, 77, 3, 3, 40),
    (1, 64, 513, 5, 1, 80),
    (2, 200, 640, 2, 2, 72),
    (1, 600, 300, 6, 2, 96),
    (4, 31, 33, 8, 8, 24),
    (1, 513, 260, 1, 1, 120),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["none", "lengths", "keys", "rows", "heads", "tail"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_gradients(size, kind, dtype):
    _check(dtype, *size, kind, seed=sum(size))


LONG = [  # many tiles for each thread block, cut in the middle of rows
    (2, 1021, 523, 12, 4, 80, "none", "bf16"),
    (2, 1021, 523, 12, 4, 80, "rows", "f16"),
    (2, 1021, 523, 12, 12, 80, "keys", "bf16"),
    (5, 700, 900, 8, 4, 128, "lengths", "bf16"),
    (2, 1024, 512, 12, 12, 128, "heads", "f16"),
    (1, 2048, 2000, 16, 16, 128, "none", "bf16"),
    (2, 3000, 1100, 8, 2, 40, "rows", "f16"),
    (16, 1024, 77, 8, 8, 40, "lengths", "bf16"),
    (1, 100, 9000, 4, 4, 64, "lengths", "bf16"),
    (8, 2500, 77, 8, 4, 48, "lengths", "bf16"),      # one tile of keys
    (3, 3001, 128, 8, 2, 64, "lengths", "bf16"),
    (5, 2000, 90, 6, 6, 64, "none", "f16"),
    (40, 700, 30, 4, 1, 32, "lengths", "f16"),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "x".join(map(str, c)))
def test_long(case):
    _check(case[7], *case[:7], seed=3)


ALONE = [  # row tiles without a partner in a pair, more of them than SMs: b, lq, lk, h, hkv, d
    (3, 100, 300, 60, 60, 128),
    (2, 300, 300, 40, 40, 128),
    (1, 260, 290, 90, 90, 72),
    (4, 70, 270, 50, 50, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["none", "lengths", "rows"])
@pytest.mark.parametrize("size", ALONE, ids=lambda s: "x".join(map(str, s)))
def test_rows_without_a_partner(size, kind, dtype):
    _check(dtype, *size, kind)


TOKENS = [  # b, lq, lk, h, hkv, d: few queries over many keys
    (1, 1, 5000, 8, 8, 64),
    (3, 1, 4097, 32, 8, 128),
    (2, 2, 2049, 10, 2, 80),
    (5, 3, 1000, 4, 4, 128),
    (1, 1, 20000, 16, 1, 128),
    (40, 1, 300, 8, 2, 64),
    (1, 17, 3000, 128, 1, 32),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["none", "lengths", "rows"])
@pytest.mark.parametrize("size", TOKENS, ids=lambda s: "x".join(map(str, s)))
def test_single_tokens(size, kind, dtype):
    _check(dtype, *size, kind, train=False, seed=sum(size))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_peaked_scores_rise_along_the_keys(dtype):
    """Scores far apart, the largest last: the running maximum moves at almost every tile."""
    g, dt = _gen(5), A.TYPES[dtype]
    b, lq, lk, h, d = 1, 130, 900, 2, 64
    q = _normal(g, (b, lq, h, d), dt)
    k = _normal(g, (b, lk, h, d), dt) + (
        torch.arange(lk, device=DEV)[None, :, None, None] / 60.0).to(dt) * q[:, :1].sign()
    k = k.to(dt)
    v, dout = _normal(g, (b, lk, h, d), dt), _normal(g, (b, lq, h, d), dt)
    _compare(_run(q, k, v, dout), A.Reference(q, k, v, dout=dout, u=A.UNIT[dtype]))


def test_scale_is_taken():
    _check("bf16", 1, 140, 150, 2, 2, 64, "none", scale=0.31)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_rows_left_out_may_hold_anything(bad, dtype):
    """Keys past the lengths, keys masked for every query, and (backward) queries without keys
    hold NaN or infinities: nothing of it arrives anywhere."""
    g, dt = _gen(9), A.TYPES[dtype]
    for kind, lq, lk in (("lengths", 200, 333), ("keys", 133, 290), ("rows", 150, 140),
                         ("lengths", 1, 700), ("keys", 2, 500)):
        b, h, hkv, d = 3, 4, 2, 64
        q, dout = _normal(g, (b, lq, h, d), dt), _normal(g, (b, lq, h, d), dt)
        k, v = _normal(g, (b, lk, hkv, d), dt), _normal(g, (b, lk, hkv, d), dt)
        n, m = _make_mask(kind, g, b, h, lq, lk)
        if kind == "rows":
            m[..., 20:40] = False
        keep = A.pairs(b, h, lq, lk, n, m)
        live_k = keep.any(2).any(1)
        k[~live_k] = bad
        v[~live_k] = bad
        live_q = keep.any(3).transpose(1, 2)
        q[~live_q] = bad
        dout[~live_q] = bad
        got = _run(q, k, v, dout, kv_lengths=n, mask=m)
        ref = A.Reference(q, k, v, kv_lengths=n, mask=m, dout=dout, u=A.UNIT[dtype])
        _compare(got, ref)
        assert (got[1] == -math.inf).equal(~keep.any(3))
        assert not got[0][~live_q].any() and not got[2][~live_q].any()
        assert not got[3][~live_k].any() and not got[4][~live_k].any()


def test_a_value_that_is_not_finite_arrives():
    """A NaN in a row that takes part is not hidden."""
    g = _gen(10)
    q, k, v = (_normal(g, (1, 130, 1, 64), torch.bfloat16) for _ in range(3))
    v[0, 7, 0, 3] = math.nan
    out, lse = _run(q, k, v)
    assert torch.isnan(out[..., 3]).all() and torch.isfinite(out[..., :3]).all()
    k[0, 7, 0, 3] = math.nan
    out, lse = _run(q, k, v)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("sizes", [(0, 5, 5), (2, 0, 5), (2, 5, 0), (2, 0, 0)])
def test_lengths_of_zero(sizes):
    b, lq, lk = sizes
    g = _gen(1)
    q, dout = (_normal(g, (b, lq, 2, 64), torch.bfloat16) for _ in range(2))
    k, v = (_normal(g, (b, lk, 2, 64), torch.bfloat16) for _ in range(2))
    out, lse, dq, dk, dv = _run(q, k, v, dout)
    assert not out.any() and not dq.any() and not dk.any() and not dv.any()
    assert (lse == -math.inf).all()


@pytest.mark.parametrize("lq,lk", [(150, 290), (1, 400)])
def test_layouts(lq, lk):
    """Heads outside tokens, padded rows, broadcast batch and heads, views into larger tensors."""
    g, dt = _gen(3), torch.bfloat16
    b, h, d = 2, 4, 40
    q = _normal(g, (b, h, lq, d), dt).transpose(1, 2)
    k = _normal(g, (b, lk, 2, 64), dt)[..., 8:48]
    v = _normal(g, (1, lk, 1, d), dt).expand(b, lk, 2, d)
    dout = _normal(g, (lq, b, h, d), dt).transpose(0, 1)
    out_all = torch.zeros((b, lq, 3, h, d), dtype=dt, device=DEV)
    dq_all = torch.zeros((b, h, lq + 2, d + 16), dtype=dt, device=DEV)
    dkv_all = torch.zeros((b, lk, 3, 2, d), dtype=dt, device=DEV)
    out, dq = out_all[:, :, 1], dq_all[:, :, 1:-1, 8:8 + d].transpose(1, 2)
    lse = torch.empty((b, h, lq), dtype=torch.float32, device=DEV)
    cg.cross_attention_fwd(q, k, v, out, lse=lse)
    cg.cross_attention_bwd(dout, q, k, v, out, lse, dq, dkv_all[:, :, 0], dkv_all[:, :, 2])
    _compare((out, lse, dq, dkv_all[:, :, 0], dkv_all[:, :, 2]),
             A.Reference(q, k, v, dout=dout, u=A.UNIT["bf16"]))
    # Nothing beside the outputs was written.
    assert not out_all[:, :, 0].any() and not out_all[:, :, 2].any() and not dkv_all[:, :, 1].any()
    assert not dq_all[:, :, 0].any() and not dq_all[:, :, -1].any()
    assert not dq_all[..., :8].any() and not dq_all[..., 8 + d:].any()


def test_equal_calls_give_equal_bits_and_streams_are_honoured():
    g = _gen(4)
    q, dout = (_normal(g, (2, 700, 4, 64), torch.bfloat16) for _ in range(2))
    k, v = (_normal(g, (2, 500, 2, 64), torch.bfloat16) for _ in range(2))
    first = _run(q, k, v, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _run(q, k, v, dout)
    side.synchronize()
    for x, y in zip(first, again):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_small_and_large_output_gradients(dtype):
    """dout far from 1, as loss scaling leaves it."""
    g, dt = _gen(6), A.TYPES[dtype]
    for size in (2.0 ** -9, 2.0 ** 7):
        q, k, v = (_normal(g, (1, 300, 2, 64), dt) for _ in range(3))
        dout = _normal(g, (1, 300, 2, 64), dt, size)
        ref = A.Reference(q, k, v, dout=dout, u=A.UNIT[dtype])
        _compare(_run(q, k, v, dout), ref)


def test_gradient_against_differences():
    """Directional derivatives of the 64-bit definition by central differences."""
    g, dt = _gen(8), torch.float16
    b, lq, lk, h, hkv, d = 1, 70, 150, 4, 2, 32
    q, k, v = _normal(g, (b, lq, h, d), dt), _normal(g, (b, lk, hkv, d), dt), _normal(g, (b, lk, hkv, d), dt)
    dout = _normal(g, (b, lq, h, d), dt)
    n = torch.tensor([101], dtype=torch.int32, device=DEV)
    _, _, dq, dk, dv = _run(q, k, v, dout, kv_lengths=n)
    ref = A.Reference(q, k, v, kv_lengths=n, dout=dout, u=A.UNIT["f16"])

    def loss(q, k, v):
        return float((A.Reference(q, k, v, kv_lengths=n, u=1e-3).out * dout.double()).sum())

    eps = 1e-4
    for i, (name, grad) in enumerate((("dq", dq), ("dk", dk), ("dv", dv))):
        x = [t.double() for t in (q, k, v)]
        step = torch.randn(x[i].shape, generator=g, device=DEV, dtype=torch.float64)
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + eps * step, x[i] - eps * step
        slope = (loss(*up) - loss(*down)) / (2 * eps)
        bound = float((getattr(ref, name + "_tol") * step.abs()).sum()) + 1e-6 * abs(slope)
        assert abs(float((grad.double() * step).sum()) - slope) <= bound, name


# ------------------------------------------------------------------ norm and rotation
def _tables(rows, rot):
    angle = torch.arange(rows, device=DEV, dtype=torch.float32)[:, None] * (
        10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float32) / max(1, rot // 2)))
    return angle.cos().contiguous(), angle.sin().contiguous()


NORMS = [  # b, lq, lk, h, hkv, d, rot
    (1, 1, 0, 1, 1, 8, 8),
    (2, 1, 3, 32, 8, 128, 128),
    (3, 17, 5, 8, 8, 40, 32),
    (2, 65, 77, 8, 2, 40, 40),       # halves of 20: words of 4
    (1, 100, 9, 3, 1, 24, 8),
    (2, 33, 40, 1, 1, 256, 64),
    (1, 700, 300, 16, 4, 80, 0),
    (4, 5, 1, 5, 5, 120, 120),
    (2, 300, 11, 2, 1, 64, 48),
    (1, 3, 2000, 40, 2, 96, 96),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("size", NORMS, ids=lambda s: "x".join(map(str, s)))
def test_norm_rope(size, adjacent, dtype):
    b, lq, lk, h, hkv, d, rot = size
    g, dt, u = _gen(sum(size)), A.TYPES[dtype], A.UNIT[dtype]
    cos, sin = _tables(400, rot) if rot else (None, None)
    x = {"q": _normal(g, (b, lq, h, d), dt, 1.5), "k": _normal(g, (b, lk, 2, hkv, d), dt, 0.4)[:, :, 1]}
    if d % 16 == 0:
        x["q"][:, :1, :1] = 0        # a row of zeros: only eps keeps it
    w = {"q": _normal(g, (d,), dt) + 1, "k": _normal(g, (d,), torch.float32)}
    pos = {"q": torch.randint(0, 400, (b, lq), generator=g, device=DEV).to(torch.int32), "k": None}
    dy = {n: _normal(g, x[n].shape, dt) for n in x}
    y = {n: torch.full(x[n].shape, math.nan, dtype=dt, device=DEV) for n in x}
    dx = {n: torch.full(x[n].shape, math.nan, dtype=dt, device=DEV) for n in x}
    dw = {n: torch.full((d,), math.nan, device=DEV) for n in x}
    kw = dict(cos=cos, sin=sin, q_positions=pos["q"], eps=1e-5, adjacent_pairs=adjacent)
    cg.qk_norm_rope_fwd(x["q"], x["k"], w["q"], w["k"], y["q"], y["k"], **kw)
    cg.qk_norm_rope_bwd(dy["q"], dy["k"], x["q"], x["k"], w["q"], w["k"], dx["q"], dx["k"], dw["q"],
                        dw["k"], **kw)
    again = {n: torch.empty_like(dw[n]) for n in x}
    cg.qk_norm_rope_bwd(dy["q"], dy["k"], x["q"], x["k"], w["q"], w["k"], dx["q"], dx["k"], again["q"],
                        again["k"], **kw)
    for n in x:
        ref = A.NormReference(x[n], w[n], cos, sin, pos[n], 1e-5, adjacent, u, dy[n])
        A.assert_within(n, y[n], ref.y, ref.y_tol)
        A.assert_within("d" + n, dx[n], ref.dx, ref.dx_tol)
        A.assert_within("d%s_weight" % n, dw[n], ref.dw, ref.dw_tol)
        assert torch.equal(dw[n], again[n])


def test_norm_rope_in_place_alone_and_strided():
    g, dt = _gen(2), torch.bfloat16
    cos, sin = _tables(64, 64)
    qkv = _normal(g, (2, 50, 3, 4, 64), dt)
    w = _normal(g, (64,), dt)
    ref_q = A.NormReference(qkv[:, :, 0], w, cos, sin, None, 1e-6, False, A.UNIT["bf16"])
    ref_k = A.NormReference(qkv[:, :, 1].transpose(1, 2)[:, :50], w, cos, sin, None, 1e-6, False,
                            A.UNIT["bf16"])
    rest = qkv[:, :, 2].clone()
    kt = torch.empty((2, 4, 50, 64), dtype=dt, device=DEV)
    cg.qk_norm_rope_fwd(None, qkv[:, :, 1].transpose(1, 2)[:, :50], None, w, None, kt, cos=cos, sin=sin)
    cg.qk_norm_rope_fwd(qkv[:, :, 0], None, w, None, qkv[:, :, 0], None, cos=cos, sin=sin)
    A.assert_within("q", qkv[:, :, 0], ref_q.y, ref_q.y_tol)
    A.assert_within("k", kt, ref_k.y, ref_k.y_tol)
    assert torch.equal(rest, qkv[:, :, 2])


def test_norm_rope_positions_are_clamped_and_shared():
    g, dt = _gen(12), torch.float16
    cos, sin = _tables(16, 32)
    x, w = _normal(g, (3, 20, 2, 32), dt), _normal(g, (32,), dt)
    pos = torch.arange(-2, 18, device=DEV, dtype=torch.int32)
    y = torch.empty_like(x)
    cg.qk_norm_rope_fwd(x, None, w, None, y, None, cos=cos, sin=sin, q_positions=pos)
    ref = A.NormReference(x, w, cos, sin, pos, 1e-6, False, A.UNIT["f16"])
    A.assert_within("y", y, ref.y, ref.y_tol)


def test_norm_gradient_against_differences():
    g = _gen(13)
    cos, sin = _tables(64, 24)
    x, dy, w = (_normal(g, s, torch.float16) for s in ((1, 30, 3, 40), (1, 30, 3, 40), (40,)))
    dx, dw = torch.empty_like(x), torch.empty((40,), device=DEV)
    cg.qk_norm_rope_bwd(dy, None, x, None, w, None, dx, None, dw, None, cos=cos, sin=sin)
    ref = A.NormReference(x, w, cos, sin, None, 1e-6, False, A.UNIT["f16"], dy)

    def loss(x, w):
        return float((A.NormReference(x, w, cos, sin, None, 1e-6, False, 1e-3).y * dy.double()).sum())

    eps = 1e-5
    step = torch.randn(x.shape, generator=g, device=DEV, dtype=torch.float64)
    slope = (loss(x.double() + eps * step, w) - loss(x.double() - eps * step, w)) / (2 * eps)
    assert abs(float((dx.double() * step).sum()) - slope) <= float(
        (ref.dx_tol * step.abs()).sum()) + 1e-6 * abs(slope)
    step = torch.randn(w.shape, generator=g, device=DEV, dtype=torch.float64)
    slope = (loss(x, w.double() + eps * step) - loss(x, w.double() - eps * step)) / (2 * eps)
    assert abs(float((dw.double() * step).sum()) - slope) <= float(
        (ref.dw_tol * step.abs()).sum()) + 1e-6 * abs(slope)
