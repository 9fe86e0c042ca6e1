"""Workspaces of exactly the size that is asked for: nothing behind them is written."""
import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _attention as A
from tests.test_gpu_attention import DEV, _gen, _make_mask, _normal, _tables

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


# A stream-K convolution keeps flags and partial tiles in its workspace; what other calls leave
# there must not be taken for them.
DEEP = dict(n=2, hw=8, c=1024, f=256)


def _deep_conv(ws):
    """A convolution that the planner runs in stream-K, as (call, output, exact result)."""
    n, hw, c, f = DEEP["n"], DEEP["hw"], DEEP["c"], DEEP["f"]
    g = _gen(21)
    # Small whole numbers: every sum is exact.
    x = torch.randint(-2, 3, (n, hw, hw, c), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randint(-1, 2, (3, 3, c, f), generator=g, device=DEV).to(torch.bfloat16)
    out = torch.empty((n, hw // 2, hw // 2, f), dtype=torch.bfloat16, device=DEV)
    packed = cg.conv2d_pack_filter(w, filter_is_fcrs=False)
    want = torch.nn.functional.conv2d(x.double().permute(0, 3, 1, 2), w.double().permute(3, 2, 0, 1),
                                      stride=2, padding=1).permute(0, 2, 3, 1).to(torch.bfloat16)

    def call():
        out.fill_(float("nan"))
        cg.conv2d_fwd_packed(x, packed, out, r=3, s=3, stride=(2, 2), symmetric_padding=(1, 1),
                             workspace=ws)
    return call, out, want


def _streamk_workspace():
    return cg.new_workspace(cg.CONV_STATUS_BYTES + cg.conv_streamk_workspace_size(), DEV)


@pytest.mark.parametrize("left", [0, 1, 7, 0x7F800000, -1])
def test_streamk_does_not_take_what_lies_in_its_workspace_for_flags(left):
    ws = _streamk_workspace()
    call, out, want = _deep_conv(ws)
    words = ws.view(torch.int32)
    for i in range(4):
        words[cg.CONV_STATUS_BYTES // 4:] = left if i else torch.arange(
            1, words.numel() - cg.CONV_STATUS_BYTES // 4 + 1, dtype=torch.int32, device=DEV)
        call()
        assert cg.conv_check_device_status(ws) == (0, 0)
        assert torch.equal(out, want)


def test_streamk_beside_masked_attention_and_the_norm_in_one_workspace():
    ws = _streamk_workspace()
    call, out, want = _deep_conv(ws)
    g = _gen(22)
    q, dout = (_normal(g, (1, 100, 2, 64), torch.bfloat16) for _ in range(2))
    k, v = (_normal(g, (1, 100, 2, 64), torch.bfloat16) for _ in range(2))
    mask = torch.ones((1, 1, 100, 100), dtype=torch.bool, device=DEV).tril()
    attended, dq, dk, dv = (torch.empty_like(q) for _ in range(4))
    lse = torch.empty((1, 2, 100), device=DEV)
    w, dw = torch.ones(64, dtype=torch.bfloat16, device=DEV), torch.empty(64, device=DEV)
    ref = A.Reference(q, k, v, mask=mask, dout=dout, u=A.UNIT["bf16"])
    for _ in range(40):
        cg.cross_attention_fwd(q, k, v, attended, lse=lse, mask=mask, workspace=ws)
        call()
        assert torch.equal(out, want)
        cg.cross_attention_bwd(dout, q, k, v, attended, lse, dq, dk, dv, mask=mask, workspace=ws)
        call()
        assert torch.equal(out, want)
        cg.qk_norm_rope_bwd(dq, None, q, None, w, None, torch.empty_like(q), None, dw, None, workspace=ws)
        call()
        assert torch.equal(out, want)
    assert cg.conv_check_device_status(ws) == (0, 0)
    A.assert_within("dq", dq, ref.dq, ref.dq_tol)


def test_streamk_in_a_graph_that_is_replayed():
    ws = _streamk_workspace()
    call, out, want = _deep_conv(ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(5):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert cg.conv_check_device_status(ws) == (0, 0)


@pytest.mark.parametrize("by_number", [False, True])
def test_default_workspaces_belong_to_the_stream_of_the_call(by_number):
    """A call on another stream without a workspace of its own: memory freed by the call is not handed
    to the current stream while the call still waits there."""
    g, dt = _gen(41), torch.bfloat16
    q, dout = _normal(g, (1, 300, 4, 64), dt), _normal(g, (1, 300, 4, 64), dt)
    k, v = _normal(g, (1, 700, 2, 64), dt), _normal(g, (1, 700, 2, 64), dt)
    mask = torch.rand((1, 1, 300, 700), generator=g, device=DEV) < 0.5
    out, dq, dk, dv = (torch.empty_like(t) for t in (q, q, k, v))
    lse = torch.empty((1, 4, 300), device=DEV)
    w, normed, dw = torch.ones(64, dtype=dt, device=DEV), torch.empty_like(q), torch.empty(64, device=DEV)
    busy = _normal(g, (4096, 4096), dt)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if by_number else side
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(50):
            busy = busy @ busy * 1e-2
    cg.cross_attention_fwd(q, k, v, out, lse=lse, mask=mask, stream=stream)
    cg.cross_attention_bwd(dout, q, k, v, out, lse, dq, dk, dv, mask=mask, stream=stream)
    cg.qk_norm_rope_bwd(dout, None, q, None, w, None, normed, None, dw, None, stream=stream)
    held = [torch.full((1 << n,), 0xFF, dtype=torch.uint8, device=DEV) for n in range(9, 25) for _ in range(4)]
    torch.cuda.synchronize()
    assert all((h == 0xFF).all() for h in held)
    ref = A.Reference(q, k, v, mask=mask, dout=dout, u=A.UNIT["bf16"])
    for name, x in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        A.assert_within(name, x, getattr(ref, name), getattr(ref, name + "_tol"))
    norm = A.NormReference(q, w, None, None, None, 1e-6, False, A.UNIT["bf16"], dout)
    A.assert_within("dw", dw, norm.dw, norm.dw_tol)


def test_a_new_workspace_is_cleared_on_its_stream():
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0, torch.cuda.default_stream().cuda_stream):
        ws = cg.new_workspace(1000, DEV, stream)
        torch.cuda.synchronize()
        assert ws.numel() == 1000 and not ws.any()
        assert torch.cuda.current_stream() == torch.cuda.default_stream()


ATTENTION = [  # b, lq, lk, h, hkv, d, mask: exact workspaces of each schedule
    (2, 300, 77, 4, 4, 40, "lengths"), (1, 260, 290, 90, 90, 72, "none"), (4, 1, 3000, 8, 2, 128, "lengths"),
    (2, 333, 700, 6, 2, 80, "rows"), (1, 500, 100, 4, 2, 96, "heads"), (3, 130, 260, 4, 1, 8, "keys"),
    (2, 1021, 523, 12, 4, 80, "rows"), (1, 129, 2000, 2, 2, 24, "tail"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "x".join(map(str, c)))
def test_attention_keeps_to_its_workspace(case, dtype):
    b, lq, lk, h, hkv, d, kind = case
    g, dt = _gen(sum(case[:6])), A.TYPES[dtype]
    q, dout = _normal(g, (b, lq, h, d), dt), _normal(g, (b, lq, h, d), dt)
    k, v = _normal(g, (b, lk, hkv, d), dt), _normal(g, (b, lk, hkv, d), dt)
    n, m = _make_mask(kind, g, b, h, lq, lk)
    out, dq, dk, dv = (torch.empty_like(t) for t in (q, q, k, v))
    lse = torch.empty((b, h, lq), device=DEV)
    kw = dict(kv_lengths=n, mask=m)
    masked = dict(masked=m is not None, mask_heads=1 if m is None else m.shape[1])
    for backward in (False, True):
        ws, behind = guarded(cg.cross_attention_workspace_size(b, h, hkv, lq, lk, d, backward=backward, **masked))
        cg.cross_attention_fwd(q, k, v, out, lse=lse, workspace=ws, **kw)
        if backward:
            cg.cross_attention_bwd(dout, q, k, v, out, lse, dq, dk, dv, workspace=ws, **kw)
        assert cg.conv_check_device_status(ws) == (0, 0)
        assert (behind == GUARD).all()
    ref = A.Reference(q, k, v, dout=dout, u=A.UNIT[dtype], **kw)
    for name, x in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        A.assert_within(name, x, getattr(ref, name), getattr(ref, name + "_tol"))
