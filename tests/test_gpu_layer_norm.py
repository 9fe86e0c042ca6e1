"""Layer norm against its definition in 64 bits: types, sizes on both sides of every layout, strides,
broadcasts, aliases, gradients against differences."""
import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _decoder as D
from tests._attention import TYPES, UNIT, assert_within

pytestmark = pytest.mark.gpu
DEV = "cuda"
MARK = 7.25


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, rows, c, dt):
    return (1.7 * torch.randn((rows, c), generator=g, device=DEV)
            + 0.5 * torch.randn(c, generator=g, device=DEV)).to(dt)


def _check(x, w, b, y, mean, rstd, dy, dx, dw, db, eps, u):
    ref = D.NormReference(x, w, b, eps, u, dy)
    for name, got in (("y", y), ("mean", mean), ("rstd", rstd), ("dx", dx), ("dweight", dw), ("dbias", db)):
        if got is not None:
            assert_within(name, got, getattr(ref, name), getattr(ref, name + "_tol"))


# Channels on both sides of the layouts: part of a warp, a warp, a block; words of 8 and single elements.
SIZES = [(1, 1), (3, 2), (1, 8), (300, 8), (5, 24), (77, 40), (1000, 64), (9, 72), (2049, 320), (13, 333),
         (65, 640), (7, 1000), (33, 1280), (3, 1281), (31, 1288), (5, 2048), (11, 2056), (17, 4096),
         (3, 4099), (2, 8192), (3, 10240), (2, 16383), (2, 16384), (0, 64), (20011, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,c", SIZES)
def test_sizes(rows, c, dtype):
    g, dt = _gen(rows * 31 + c), TYPES[dtype]
    x, dy = _rows(g, rows, c, dt), torch.randn((rows, c), generator=g, device=DEV).to(dt)
    kind = (rows + c) % 4     # of the weights
    wt = torch.float32 if kind == 1 else dt
    w = None if kind == 2 else (1 + 0.2 * torch.randn(c, generator=g, device=DEV)).to(wt)
    b = None if kind == 3 else (0.1 * torch.randn(c, generator=g, device=DEV)).to(wt)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dw, db = torch.full((c,), MARK, device=DEV), torch.full((c,), MARK, device=DEV)
    assert cg.layer_norm_fwd(x, w, b, y, mean=mean, rstd=rstd) is y
    cg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)
    if rows == 0:
        assert not dw.any() and not db.any()
        return
    _check(x, w, b, y, mean, rstd, dy, dx, dw, db, 1e-5, UNIT[dtype])
    # Without the statistics, and without the weights' gradients: the same bits.
    again, dx2 = torch.empty_like(x), torch.empty_like(x)
    cg.layer_norm_fwd(x, w, b, again)
    cg.layer_norm_bwd(dy, x, w, mean, rstd, dx2, None, None)
    assert torch.equal(again, y) and torch.equal(dx2, dx)
    one = torch.full((c,), MARK, device=DEV)
    cg.layer_norm_bwd(dy, x, w, mean, rstd, dx2, None, one)
    assert torch.equal(one, db)


@pytest.mark.parametrize("c", [64, 333, 2048])
def test_strides(c):
    """A feature map's pixels, a slice of a fused projection, rows apart from the outputs' in stride,
    a gradient that repeats one row."""
    g, dt, eps = _gen(c), torch.bfloat16, 1e-3
    wide = torch.randn((3, 10, 3, c), generator=g, device=DEV).to(dt)
    x = wide[:, :, 1]                                        # two strides
    out = torch.full((3, 12, c), MARK, dtype=dt, device=DEV)
    y = out[:, 1:11]
    w = torch.randn(c, generator=g, device=DEV).to(dt)
    mean, rstd = torch.empty((3, 10), device=DEV), torch.empty((3, 10), device=DEV)
    cg.layer_norm_fwd(x, w, None, y, mean=mean, rstd=rstd, eps=eps)
    assert (out[:, 0] == MARK).all() and (out[:, 11] == MARK).all()
    dy = torch.randn((1, 1, c), generator=g, device=DEV).to(dt).expand(3, 10, c)
    dx = torch.empty((3, 10, c), dtype=dt, device=DEV)
    dw, db = torch.empty(c, device=DEV), torch.empty(c, device=DEV)
    cg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)
    flat = [t.reshape(30, c) for t in (x, dy)]
    _check(flat[0], w, None, y.reshape(30, c), mean.view(30), rstd.view(30), flat[1], dx.view(30, c), dw, db,
           eps, UNIT["bf16"])
    # In place, and over the gradient that came in: the same bits.
    x2, dy2 = x.clone(), dy.contiguous()
    cg.layer_norm_fwd(x2, w, None, x2, eps=eps)
    assert torch.equal(x2, y)
    cg.layer_norm_bwd(dy2, x, w, mean, rstd, dy2, None, None)
    assert torch.equal(dy2, dx)


@pytest.mark.parametrize("c", [1, 5, 7, 9, 15, 63, 64, 65, 130, 321, 333, 643, 1281, 1288, 2047, 4099, 8185, 8186])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_that_begin_inside_a_word(c, dtype):
    """Every place of a 16-byte word, another one in each tensor: what lies around a row stays, and a
    row's bits do not depend on where it lies."""
    g, dt, rows = _gen(c), TYPES[dtype], 21 if c < 2000 else 6
    x, dy = _rows(g, rows, c, dt), torch.randn((rows, c), generator=g, device=DEV).to(dt)
    w = (1 + 0.2 * torch.randn(c, generator=g, device=DEV)).to(torch.float32 if c % 4 == 1 else dt)
    b = torch.randn(c, generator=g, device=DEV).to(w.dtype)
    first = None
    for turn in range(4):
        views, flats = [], []
        for n in range(4):                                  # x, dy, y, dx
            at, apart = (2 * turn + 3 * n) % 8 if turn else 0, c + (turn + n) * (turn > 1)
            flat = torch.full((at + rows * apart + 8,), MARK, dtype=dt, device=DEV)
            views.append(flat[at:].as_strided((rows, c), (apart, 1), flat.storage_offset() + at))
            flats.append(flat)
        views[0].copy_(x)
        views[1].copy_(dy)
        mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        dw, db = torch.empty(c, device=DEV), torch.empty(c, device=DEV)
        cg.layer_norm_fwd(views[0], w, b, views[2], mean=mean, rstd=rstd)
        cg.layer_norm_bwd(views[1], views[0], w, mean, rstd, views[3], dw, db)
        got = [views[2].clone(), views[3].clone(), mean, rstd, dw, db]
        _check(x, w, b, got[0], mean, rstd, dy, got[1], dw, db, 1e-5, UNIT[dtype])
        for flat, view in list(zip(flats, views))[2:]:
            view.fill_(MARK)
            assert (flat == MARK).all()
        if c % 8 and c < 8186:
            first = first or got
            assert all(torch.equal(p, q) for p, q in zip(got, first))


def test_a_map_and_an_unaligned_view():
    g, dt = _gen(3), torch.float16
    x = _rows(g, 2 * 5 * 7, 48, dt).view(2, 5, 7, 48)
    y = torch.empty_like(x)
    cg.layer_norm_fwd(x, None, None, y)
    ref = D.NormReference(x.view(-1, 48), None, None, 1e-5, UNIT["f16"])
    assert_within("y", y.view(-1, 48), ref.y, ref.y_tol)
    flat = torch.zeros(70 * 48 + 3, dtype=dt, device=DEV)
    moved = flat[3:].view(2, 5, 7, 48)
    moved.copy_(x)
    cg.layer_norm_fwd(moved, None, None, moved)
    assert_within("y", moved.reshape(-1, 48), ref.y, ref.y_tol)
    assert not flat[:3].any()


def test_rows_of_a_far_mean_and_of_one_value():
    """Deviations are taken from the row's own mean; a constant row gives the bias."""
    g = _gen(4)
    x = (200.0 + torch.randn((40, 512), generator=g, device=DEV)).half()
    x[7] = 3.0
    b = torch.randn(512, generator=g, device=DEV).half()
    y = torch.empty_like(x)
    cg.layer_norm_fwd(x, None, b, y)
    ref = D.NormReference(x, None, b, 1e-5, UNIT["f16"])
    assert_within("y", y, ref.y, ref.y_tol)
    assert torch.equal(y[7], b)


def test_a_row_that_is_not_finite_stays_alone():
    g, dt = _gen(5), torch.bfloat16
    x, dy = _rows(g, 50, 320, dt), _rows(g, 50, 320, dt)
    y, clean = torch.empty_like(x), torch.empty_like(x)
    cg.layer_norm_fwd(x, None, None, clean)
    x[9, 3], x[20, 0] = float("nan"), float("inf")
    cg.layer_norm_fwd(x, None, None, y)
    keep = torch.ones(50, dtype=torch.bool, device=DEV)
    keep[9] = keep[20] = False
    assert torch.equal(y[keep], clean[keep])
    assert y[9].isnan().all()


def test_gradients_against_differences():
    """Central differences of the definition in 64 bits along random directions."""
    g, c, rows = _gen(6), 40, 6
    x, dy = _rows(g, rows, c, torch.float16), torch.randn((rows, c), generator=g, device=DEV).half()
    w = (1 + 0.2 * torch.randn(c, generator=g, device=DEV)).half()
    b = torch.zeros(c, dtype=torch.float16, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dw, db = torch.empty(c, device=DEV), torch.empty(c, device=DEV)
    cg.layer_norm_fwd(x, w, b, y, mean=mean, rstd=rstd)
    cg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)

    def loss(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return ((d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * w + b) * dy.double()).sum()

    at = [t.double() for t in (x, w, b)]
    for i, grad in enumerate((dx, dw, db)):
        for _ in range(4):
            way = torch.randn(at[i].shape, generator=g, device=DEV).double()
            h = 1e-6
            near = [[t + s * h * way if j == i else t for j, t in enumerate(at)] for s in (1, -1)]
            want = (loss(*near[0]) - loss(*near[1])) / (2 * h)
            got = (grad.double() * way).sum()
            # dx is rounded to fp16 (2^-11 of each); the differences are good to some 1e-8 of the sums.
            slack = 2.0 ** -11 if i == 0 else 1e-6
            assert abs(got - want) <= (slack + 1e-7) * (grad.double() * way).abs().sum() + 1e-7


def test_captured_and_replayed_with_a_shared_workspace():
    g, c = _gen(8), 320
    x, dy = _rows(g, 700, c, torch.bfloat16), _rows(g, 700, c, torch.bfloat16)
    w = torch.ones(c, dtype=torch.bfloat16, device=DEV)
    ws = cg.new_workspace(cg.layer_norm_workspace_size(c), DEV)
    outs = [dict(y=torch.empty_like(x), mean=torch.empty(700, device=DEV), rstd=torch.empty(700, device=DEV),
                 dx=torch.empty_like(x), dw=torch.empty(c, device=DEV), db=torch.empty(c, device=DEV))
            for _ in range(3)]

    def step(o):
        cg.layer_norm_fwd(x, w, None, o["y"], mean=o["mean"], rstd=o["rstd"])
        cg.layer_norm_bwd(dy, x, w, o["mean"], o["rstd"], o["dx"], o["dw"], o["db"], workspace=ws)

    step(outs[0])
    graphs = []
    for o in outs[1:]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(o)
        graphs.append(graph)
    ws[cg.CONV_STATUS_BYTES:] = 0xA5
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        for n in o:
            assert torch.equal(o[n], outs[0][n]), n


def test_another_stream():
    g = _gen(9)
    x = _rows(g, 3000, 640, torch.bfloat16)
    y, z = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(3000, device=DEV), torch.empty(3000, device=DEV)
    cg.layer_norm_fwd(x, None, None, y, mean=mean, rstd=rstd)
    dx, dw = torch.empty_like(x), torch.empty(640, device=DEV)
    cg.layer_norm_bwd(x, x, None, mean, rstd, dx, dw, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dx2, dw2 = torch.empty_like(x), torch.empty(640, device=DEV)
    cg.layer_norm_fwd(x, None, None, z, stream=side)
    cg.layer_norm_bwd(x, x, None, mean, rstd, dx2, dw2, None, stream=side)
    side.synchronize()
    assert torch.equal(y, z) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_guard_bytes_behind_an_exact_workspace():
    for c in (8, 320, 333, 4096, 16384):
        size = cg.layer_norm_workspace_size(c)
        ws = torch.zeros(size + 4096, dtype=torch.uint8, device=DEV)
        ws[size:] = 0x5A
        x = _rows(_gen(c), 700, c, torch.bfloat16)
        mean, rstd = torch.zeros(700, device=DEV), torch.ones(700, device=DEV)
        cg.layer_norm_bwd(x, x, None, mean, rstd, torch.empty_like(x), torch.empty(c, device=DEV),
                          torch.empty(c, device=DEV), workspace=ws[:size])
        assert (ws[size:] == 0x5A).all() and not ws[:cg.CONV_STATUS_BYTES].any()


def test_refusals():
    x = torch.zeros((4, 10, 64), dtype=torch.bfloat16, device=DEV)
    w, f = torch.ones(64, dtype=torch.bfloat16, device=DEV), torch.ones(64, device=DEV)
    stat = torch.zeros((4, 10), device=DEV)
    i = cg.CONV_ERR_INVALID_VALUE

    def refused(status, x=x, w=w, b=w, y=None, **kw):
        with pytest.raises(cg.ConvError) as e:
            cg.layer_norm_fwd(x, w, b, torch.empty_like(x) if y is None else y, **kw)
        assert e.value.status == status, str(e.value)

    refused(cg.CONV_ERR_NOT_SUPPORTED, x=x.float())
    refused(i, x=x.cpu())
    refused(i, x=torch.zeros((), dtype=torch.bfloat16, device=DEV))
    refused(i, y=x[:, :9])
    refused(i, y=x.half())
    refused(i, y=x[:1].expand(4, 10, 64))
    refused(i, y=torch.empty((4, 64, 10), dtype=torch.bfloat16, device=DEV).transpose(1, 2))
    refused(i, w=w[:32])
    refused(i, w=w.half())
    refused(i, b=f)
    refused(i, w=torch.ones(128, dtype=torch.bfloat16, device=DEV)[::2])
    refused(i, mean=stat.double())
    refused(i, rstd=stat[:2])
    for eps in (-1e-5, float("nan"), float("inf")):
        refused(i, eps=eps)
    refused(cg.CONV_ERR_NOT_SUPPORTED, x=torch.zeros((2, 16385), dtype=torch.bfloat16, device=DEV), w=None, b=None)
    three = torch.zeros((8, 12, 6, 64), dtype=torch.bfloat16, device=DEV)[::2, ::2, ::2]
    refused(i, x=three, y=torch.empty((4, 6, 3, 64), dtype=torch.bfloat16, device=DEV))

    def refused_back(status, dy=x, m=stat, r=stat, dx=None, dw=f, db=f, **kw):
        with pytest.raises(cg.ConvError) as e:
            cg.layer_norm_bwd(dy, x, w, m, r, torch.empty_like(x) if dx is None else dx, dw, db, **kw)
        assert e.value.status == status, str(e.value)

    refused_back(i, dy=x[:2])
    refused_back(i, dy=x.half())
    refused_back(i, m=None)
    refused_back(i, r=stat[0])
    refused_back(i, dx=x[:1].expand(4, 10, 64))
    refused_back(i, dw=w)
    refused_back(i, db=f[:3])
    refused_back(i, workspace=torch.zeros(1 << 22, dtype=torch.uint8))
    size = cg.layer_norm_workspace_size(64)
    refused_back(cg.CONV_ERR_WORKSPACE_TOO_SMALL, workspace=cg.new_workspace(size, DEV)[:size - 1])
    refused_back(cg.CONV_ERR_MISALIGNED, workspace=cg.new_workspace(size + 16, DEV)[8:])
    for c in (0, -1, 16385):
        with pytest.raises(cg.ConvError):
            cg.layer_norm_workspace_size(c)
