"""The refusals of the attention entry points that need no GPU: validation returns its status
before any CUDA call (the pointers here are never dereferenced), and the sizes a call may have."""
import ctypes

import pytest

from transposed_conv_implicit_gb300 import _lib, attention, build

OK, INVALID, NOTSUP, MISALIGNED = 0, 1, 2, 3
P = {name: 0x10000 * (i + 1) for i, name in enumerate(
    ("q", "k", "v", "out", "lse", "kv_lengths", "mask", "dout", "dq", "dk", "dv"))}
WS = ctypes.c_void_p(0x1000000)
FIELDS = ("dtype", "batch", "heads", "kv_heads", "q_len", "kv_len", "head_dim", "scale")
TENSORS = ("q", "k", "v", "out", "dout", "dq", "dk", "dv")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def _attn(**change):
    """A call's arguments, dense, with changes: a size, a pointer, or NAME_stride = (b, token, head)."""
    a = dict(dtype=0, batch=2, heads=4, kv_heads=2, q_len=10, kv_len=20, head_dim=64, scale=0.125)
    a.update({f: change.pop(f) for f in FIELDS if f in change})
    strides = {}
    for t in TENSORS:
        heads, length = (a["kv_heads"], a["kv_len"]) if t in ("k", "v", "dk", "dv") else (
            a["heads"], a["q_len"])
        row = heads * a["head_dim"]
        strides[t] = change.pop(t + "_stride", (length * row, row, a["head_dim"]))
    ptrs = [change.pop(n, p) for n, p in P.items()]
    mask = change.pop("mask_stride", (0, 0, a["kv_len"], 1))
    assert not change, change
    return attention._ATTN.pack(*(a[f] for f in FIELDS), *ptrs,
                                *(s for t in TENSORS for s in strides[t]), *mask)


BOTH = [
    (dict(dtype=2), NOTSUP), (dict(dtype=7), NOTSUP),
    (dict(head_dim=0), INVALID), (dict(head_dim=-8), INVALID), (dict(head_dim=36), NOTSUP),
    (dict(head_dim=136), NOTSUP),
    (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(heads=3), INVALID),
    (dict(batch=-1), INVALID), (dict(q_len=-1), INVALID), (dict(kv_len=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID),
    # rows that 31 bits do not count
    (dict(batch=1 << 20, q_len=1 << 10), NOTSUP), (dict(batch=1 << 20, kv_len=1 << 11), NOTSUP),
    (dict(q_len=0x7FFFFFFF), NOTSUP),
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(out=0), INVALID),
    (dict(q=P["q"] + 8), MISALIGNED), (dict(k=P["k"] + 2), MISALIGNED), (dict(v=P["v"] + 4), MISALIGNED),
    (dict(out=P["out"] + 8), MISALIGNED), (dict(lse=P["lse"] + 2), MISALIGNED),
    (dict(kv_lengths=P["kv_lengths"] + 1), MISALIGNED),
    (dict(q_stride=(4096, 260, 64)), MISALIGNED), (dict(k_stride=(4096, 128, 68)), MISALIGNED),
    (dict(q_stride=(2560, 0, 64)), INVALID), (dict(v_stride=(2560, 0, 64)), INVALID),
    (dict(k_stride=(2560, -128, 64)), INVALID),
]
FORWARD = [(dict(out_stride=(0, 256, 64)), INVALID), (dict(out_stride=(2560, 256, 0)), INVALID),
           (dict(out_stride=(2560, 252, 64)), MISALIGNED)]
BACKWARD = [(dict([(n, 0)]), INVALID) for n in ("lse", "dout", "dq", "dk", "dv")]
BACKWARD += [(dict([(n, P[n] + 8)]), MISALIGNED) for n in ("dout", "dq", "dk", "dv")]
BACKWARD += [(dict([(n + "_stride", (0, 256, 64))]), INVALID) for n in ("dq", "dk", "dv")]
BACKWARD += [(dict(dout_stride=(2560, 256, 60)), MISALIGNED)]


@pytest.mark.parametrize("change,status", BOTH + FORWARD, ids=str)
def test_forward_refuses(lib, change, status):
    assert lib.cross_attention_fwd(_attn(**change), WS, 1 << 40, None) == status


@pytest.mark.parametrize("change,status", BOTH + BACKWARD, ids=str)
def test_backward_refuses(lib, change, status):
    assert lib.cross_attention_bwd(_attn(**change), WS, 1 << 40, None) == status


def test_attention_refuses_its_workspace(lib):
    for call in (lib.cross_attention_fwd, lib.cross_attention_bwd):
        assert call(None, WS, 1 << 40, None) == INVALID
        assert call(_attn(), None, 1 << 40, None) == INVALID
        assert call(_attn(), ctypes.c_void_p(WS.value + 8), 1 << 40, None) == MISALIGNED


@pytest.mark.parametrize("change", [c for c, _ in BOTH[:11]], ids=str)
def test_no_workspace_size_for_sizes_that_are_refused(lib, change):
    assert lib.cross_attention_workspace_size(_attn(**change), 0) == 0
    assert lib.cross_attention_workspace_size(_attn(**change), 1) == 0


# ------------------------------------------------------------------ norm and rotation
def _norm(backward, **change):
    """Arguments of the norm of q and k, with changes; q_NAME and k_NAME change one tensor."""
    a = dict(dtype=0, batch=2, head_dim=64, rot_dim=32, table_rows=50, adjacent_pairs=0, eps=1e-6,
             cos=0x100000, sin=0x200000)
    a.update({f: change.pop(f) for f in list(a) if f in change})
    out = attention._NORM_HEAD.pack(*a.values())
    for i, (name, length, heads) in enumerate((("q", 10, 4), ("k", 20, 2))):
        base = 0x1000000 * (i + 1)
        row = heads * a["head_dim"]
        dense = (length * row, row, a["head_dim"])
        t = dict(x=base, weight=base + 0x10000, positions=base + 0x20000,
                 y=0 if backward else base + 0x30000, dy=base + 0x40000 if backward else 0,
                 dx=base + 0x50000 if backward else 0, dweight=base + 0x60000 if backward else 0,
                 length=length, heads=heads, weight_f32=0, position_stride=length,
                 x_stride=dense, y_stride=dense, dy_stride=dense, dx_stride=dense)
        t.update({f: change.pop("%s_%s" % (name, f)) for f in list(t) if "%s_%s" % (name, f) in change})
        out += attention._NORM_TENSOR.pack(*list(t.values())[:11], *t["x_stride"], *t["y_stride"],
                                           *t["dy_stride"], *t["dx_stride"])
    assert not change, change
    return out


NORM_BOTH = [
    (dict(dtype=2), NOTSUP), (dict(batch=-1), INVALID), (dict(head_dim=0), INVALID),
    (dict(head_dim=44), NOTSUP), (dict(head_dim=264), NOTSUP), (dict(rot_dim=-8), INVALID),
    (dict(rot_dim=72), INVALID), (dict(rot_dim=12), NOTSUP),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(cos=0), INVALID), (dict(sin=0), INVALID), (dict(table_rows=0), INVALID),
    (dict(cos=0x100004), MISALIGNED), (dict(sin=0x200008), MISALIGNED),
    (dict(q_length=-1), INVALID), (dict(k_heads=0), INVALID), (dict(q_weight=0), INVALID),
    (dict(k_x=0x2000008), MISALIGNED), (dict(q_weight=0x1010004), MISALIGNED),
    (dict(k_positions=0x2020002), MISALIGNED),
    (dict(q_x_stride=(2560, 252, 64)), MISALIGNED), (dict(k_x_stride=(2560, -128, 64)), INVALID),
    (dict(q_x_stride=(1 << 36, 256, 64)), NOTSUP), (dict(q_length=0x7FFFFFFF), NOTSUP),
]


@pytest.mark.parametrize("change,status", NORM_BOTH + [
    (dict(q_y=0), INVALID), (dict(k_y=0x2030008), MISALIGNED), (dict(q_y_stride=(2560, 256, 0)), INVALID),
    (dict(k_y_stride=(2560, 124, 64)), MISALIGNED)], ids=str)
def test_norm_forward_refuses(lib, change, status):
    assert lib.qk_norm_rope_fwd(_norm(False, **change), None) == status


@pytest.mark.parametrize("change,status", NORM_BOTH + [
    (dict(q_dy=0), INVALID), (dict(q_dx=0), INVALID), (dict(k_dweight=0), INVALID),
    (dict(k_dy=0x2040008), MISALIGNED), (dict(q_dx=0x1050002), MISALIGNED),
    (dict(q_dweight=0x1060002), MISALIGNED), (dict(k_dx_stride=(0, 128, 64)), INVALID),
    (dict(q_dy_stride=(2560, 256, 60)), MISALIGNED)], ids=str)
def test_norm_backward_refuses(lib, change, status):
    assert lib.qk_norm_rope_bwd(_norm(True, **change), WS, 1 << 40, None) == status


def test_norm_refuses_its_workspace(lib):
    assert lib.qk_norm_rope_fwd(None, None) == INVALID
    assert lib.qk_norm_rope_bwd(None, WS, 1 << 40, None) == INVALID
    assert lib.qk_norm_rope_bwd(_norm(True), None, 1 << 40, None) == INVALID
    assert lib.qk_norm_rope_bwd(_norm(True), ctypes.c_void_p(WS.value + 4), 1 << 40, None) == MISALIGNED
