"""What the binding of the attention refuses, and the bounded waits of its kernels: a wait that can
only run out is reported in the workspace's status, and the next call is right again."""
import math

import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests import _attention as A
from tests.test_gpu_attention import DEV, _gen, _make_mask, _normal
from transposed_conv_implicit_gb300 import _lib

pytestmark = pytest.mark.gpu


def _tensors(b=2, lq=10, lk=20, h=4, hkv=2, d=64, dt=torch.bfloat16):
    def t(*shape):
        return torch.zeros(shape, dtype=dt, device=DEV)
    return dict(q=t(b, lq, h, d), k=t(b, lk, hkv, d), v=t(b, lk, hkv, d), output=t(b, lq, h, d),
                lse=torch.zeros((b, h, lq), device=DEV), dout=t(b, lq, h, d), dq=t(b, lq, h, d),
                dk=t(b, lk, hkv, d), dv=t(b, lk, hkv, d))


def _refused(status, call, *args, **kw):
    with pytest.raises(cg.ConvError) as e:
        call(*args, **kw)
    assert e.value.status == status, str(e.value)


FWD = ("q", "k", "v", "output")
BWD = ("dout", "q", "k", "v", "output", "lse", "dq", "dk", "dv")


def _wrong(t):
    """(tensor, a wrong one, status)."""
    i = cg.CONV_ERR_INVALID_VALUE
    yield "q", t["q"].float(), cg.CONV_ERR_NOT_SUPPORTED
    yield "q", t["q"].cpu(), i
    yield "q", t["q"][0], i
    yield "q", t["q"].transpose(1, 3), i
    yield "k", t["k"][..., :32], i
    yield "k", t["k"][:1], i
    yield "k", t["k"].half(), i
    yield "k", torch.zeros((2, 20, 3, 64), dtype=torch.bfloat16, device=DEV), i
    yield "v", t["v"][:, :19], i
    yield "v", t["v"].half(), i
    yield "output", t["output"][:, :9], i
    yield "output", t["output"][:1].expand(2, 10, 4, 64), i


@pytest.mark.parametrize("backward", [False, True])
def test_tensors_that_do_not_fit(backward):
    t = _tensors()
    names, call = (BWD, cg.cross_attention_bwd) if backward else (FWD, cg.cross_attention_fwd)
    for name, wrong, status in _wrong(t):
        if backward and name == "output" and wrong.shape == t["output"].shape:
            continue        # only read there: a broadcast is fine
        args = dict(t, **{name: wrong})
        _refused(status, call, *(args[n] for n in names))
    if backward:
        for name in ("dout", "dq", "dk", "dv"):
            args = dict(t, **{name: t[name][:, :-1]})
            _refused(cg.CONV_ERR_INVALID_VALUE, call, *(args[n] for n in names))
        for lse in (None, t["lse"].double(), t["lse"].transpose(1, 2), t["lse"][:1]):
            args = dict(t, lse=lse)
            _refused(cg.CONV_ERR_INVALID_VALUE, call, *(args[n] for n in names))


def test_options_that_do_not_fit():
    t = _tensors()
    i, args = cg.CONV_ERR_INVALID_VALUE, [t[n] for n in FWD]

    def refused(status, **kw):
        _refused(status, cg.cross_attention_fwd, *args, **kw)

    refused(i, kv_lengths=torch.zeros(2, dtype=torch.int64, device=DEV))
    refused(i, kv_lengths=torch.zeros(3, dtype=torch.int32, device=DEV))
    refused(i, kv_lengths=torch.zeros(2, dtype=torch.int32))
    refused(i, mask=torch.ones((2, 4, 10, 20), device=DEV))
    refused(i, mask=torch.ones((10, 20), dtype=torch.bool, device=DEV))
    refused(i, mask=torch.ones((2, 4, 10, 19), dtype=torch.bool, device=DEV))
    refused(i, mask=torch.ones((2, 2, 10, 20), dtype=torch.bool, device=DEV))
    refused(i, mask=torch.ones((2, 4, 10, 20), dtype=torch.bool))
    refused(i, lse=torch.zeros((2, 10, 4), device=DEV))
    for scale in (0.0, -1.0, math.inf, math.nan):
        refused(i, scale=scale)
    refused(i, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    size = cg.cross_attention_workspace_size(2, 4, 2, 10, 20, 64)
    small = cg.new_workspace(size, DEV)[:size - 1]
    refused(cg.CONV_ERR_WORKSPACE_TOO_SMALL, workspace=small)
    refused(cg.CONV_ERR_MISALIGNED, workspace=cg.new_workspace(size + 16, DEV)[8:])
    x = torch.zeros(2 * 10 * 4 * 64 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(2, 10, 4, 64)
    _refused(cg.CONV_ERR_MISALIGNED, cg.cross_attention_fwd, x, *args[1:])
    wide = torch.zeros((2, 10, 4, 144), dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros((2, 20, 2, 144), dtype=torch.bfloat16, device=DEV)
    _refused(cg.CONV_ERR_NOT_SUPPORTED, cg.cross_attention_fwd, wide, kv, kv, wide)
    with pytest.raises(cg.ConvError):
        cg.cross_attention_workspace_size(2, 4, 3, 10, 20, 64)
    cg.cross_attention_fwd(*args, workspace=cg.new_workspace(size, DEV))


def test_norm_refuses():
    t = _tensors(d=64)
    q, k, i = t["q"], t["k"], cg.CONV_ERR_INVALID_VALUE
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    cos = torch.ones((32, 16), device=DEV)

    def refused(status, q=q, k=k, qw=w, kw=w, qo=t["dq"], ko=t["dk"], **rest):
        rest = dict(dict(cos=cos, sin=cos), **rest)
        _refused(status, cg.qk_norm_rope_fwd, q, k, qw, kw, qo, ko, **rest)

    refused(i, q=None, k=None)
    refused(cg.CONV_ERR_NOT_SUPPORTED, q=q.float())
    refused(i, q=q.cpu())
    refused(i, q=q[0])
    refused(i, k=k[0])
    refused(i, k=k[:1])
    refused(i, k=k.half())
    refused(i, qw=None)
    refused(i, kw=w[:32])
    refused(i, kw=w.half())
    refused(i, qo=None)
    refused(i, qo=t["dq"][:, :9])
    refused(i, ko=t["dk"][:1].expand(2, 20, 2, 64))
    refused(i, sin=None)
    refused(i, cos=cos[:, :8])
    refused(i, cos=cos[0])
    refused(i, cos=cos.double(), sin=cos.double())
    refused(cg.CONV_ERR_NOT_SUPPORTED, cos=cos[:, :6].contiguous(), sin=cos[:, :6].contiguous())
    refused(i, cos=torch.ones((32, 36), device=DEV), sin=torch.ones((32, 36), device=DEV))
    refused(i, eps=-1.0)
    refused(i, q_positions=torch.zeros(9, dtype=torch.int32, device=DEV))
    refused(i, q_positions=torch.zeros(10, dtype=torch.int64, device=DEV))
    refused(i, k_positions=torch.zeros((20, 2), dtype=torch.int32, device=DEV).t())
    dw = torch.zeros(64, device=DEV)

    def refused_back(status, dqo=t["dout"], dko=t["dv"], dqw=dw, dkw=dw, **rest):
        _refused(status, cg.qk_norm_rope_bwd, dqo, dko, q, k, w, w, t["dq"], t["dk"], dqw, dkw, **rest)

    refused_back(i, dqo=None)
    refused_back(i, dqo=t["dout"][:, :9])
    refused_back(i, dqw=None)
    refused_back(i, dkw=dw.bfloat16())
    refused_back(i, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    size = cg.qk_norm_rope_workspace_size(64)
    refused_back(cg.CONV_ERR_WORKSPACE_TOO_SMALL, workspace=cg.new_workspace(size, DEV)[:size - 1])
    cg.qk_norm_rope_bwd(t["dout"], t["dv"], q, k, w, w, t["dq"], t["dk"], dw, dw,
                        workspace=cg.new_workspace(size, DEV))


# ------------------------------------------------------------------ bounded waits
WAITS = [  # b, lq, lk, h, hkv, d, mask: one for each kernel and schedule
    (2, 300, 77, 4, 4, 40, "none"),        # one key tile
    (8, 2500, 300, 8, 8, 64, "none"),      # pairs of row tiles
    (8, 2500, 300, 8, 8, 128, "rows"),
    (4, 1, 3000, 8, 2, 128, "lengths"),    # split along the keys
    (1, 200, 900, 2, 2, 72, "heads"),
]


@pytest.mark.parametrize("case", WAITS, ids=lambda c: "x".join(map(str, c)))
def test_a_wait_that_runs_out_is_reported(case):
    b, lq, lk, h, hkv, d, kind = case
    g, dt = _gen(7), torch.bfloat16
    q, dout = _normal(g, (b, lq, h, d), dt), _normal(g, (b, lq, h, d), dt)
    k, v = _normal(g, (b, lk, hkv, d), dt), _normal(g, (b, lk, hkv, d), dt)
    n, m = _make_mask(kind, g, b, h, lq, lk)
    out, dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    lse = torch.empty((b, h, lq), device=DEV)
    ws = cg.new_workspace(cg.cross_attention_workspace_size(
        b, h, hkv, lq, lk, d, masked=m is not None, mask_heads=h, backward=True), DEV)
    kw = dict(kv_lengths=n, mask=m, workspace=ws)
    calls = [lambda: cg.cross_attention_fwd(q, k, v, out, lse=lse, **kw),
             lambda: cg.cross_attention_bwd(dout, q, k, v, out, lse, dq, dk, dv, **kw)]
    lib = _lib.lib()
    for call in calls:
        try:
            lib.conv_testing_set_wait_fault(1, 5_000_000)
            call()
            status, bits = cg.conv_check_device_status(ws)
        finally:
            lib.conv_testing_set_wait_fault(0, 0)
        assert status == cg.CONV_ERR_DEVICE_TIMEOUT and bits != 0 and bits & ~7 == 0, (status, bits)
        call()
        assert cg.conv_check_device_status(ws) == (0, 0)
    ref = A.Reference(q, k, v, kv_lengths=n, mask=m, dout=dout, u=A.UNIT["bf16"])
    for name, x in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        A.assert_within(name, x, getattr(ref, name), getattr(ref, name + "_tol"))
