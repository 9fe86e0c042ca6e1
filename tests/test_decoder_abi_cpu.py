"""The refusals of the decoder's entry points that need no GPU: validation returns its status before
any CUDA call (the pointers here are never dereferenced)."""
import ctypes

import pytest

from transposed_conv_implicit_gb300 import _lib, build, decoder

OK, INVALID, NOTSUP, MISALIGNED = 0, 1, 2, 3
WS = ctypes.c_void_p(0x1000000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def _packed(layout, a, change):
    for name, value in change.items():
        assert name in a, name
        a[name] = value
    flat = []
    for v in a.values():
        flat += v if isinstance(v, tuple) else (v,)
    return layout.pack(*flat)


def _norm(**change):
    row, names = (640, 64), ("x", "weight", "bias", "y", "mean", "rstd", "dy", "dx", "dweight", "dbias")
    a = dict(dtype=0, batch=4, length=10, channels=64, weight_f32=0, eps=1e-5)
    a.update({n: 0x10000 * (i + 1) for i, n in enumerate(names)})
    a.update(x_stride=row, y_stride=row, dy_stride=row, dx_stride=row)
    return _packed(decoder._NORM, a, change)


def _cache_fields():
    return dict(k_cache_stride=(8192, 64, 1024), v_cache_stride=(8192, 64, 1024))


def _cache(**change):
    a = dict(dtype=0, batch=2, length=5, kv_heads=8, head_dim=64, pages=20, page_size=16, table_width=4)
    names = ("k", "v", "k_cache", "v_cache", "scales", "block_table", "starts", "lengths")
    a.update({n: 0x10000 * (i + 1) for i, n in enumerate(names)})
    a.update(table_stride=4, k_stride=(2560, 512, 64), v_stride=(2560, 512, 64), **_cache_fields())
    return _packed(decoder._CACHE, a, change)


def _tree(**change):
    a = dict(dtype=0, batch=2, heads=16, kv_heads=8, q_len=5, head_dim=64, pages=20, page_size=16, table_width=4,
             scale=0.125)
    names = ("q", "k_cache", "v_cache", "scales", "block_table", "kv_lengths", "draft_lengths", "parents", "out",
             "lse")
    a.update({n: 0x10000 * (i + 1) for i, n in enumerate(names)})
    a.update(table_stride=4, parent_stride=5, q_stride=(5120, 1024, 64), out_stride=(5120, 1024, 64),
             **_cache_fields())
    return _packed(decoder._TREE, a, change)


NORM = [
    (dict(dtype=2), NOTSUP), (dict(batch=-1), INVALID), (dict(length=-1), INVALID), (dict(channels=0), INVALID),
    (dict(channels=16385), NOTSUP), (dict(batch=1 << 16, length=1 << 15), NOTSUP), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(x=0), INVALID), (dict(x=0x10001), MISALIGNED),
    (dict(weight=0x20001), MISALIGNED), (dict(weight_f32=1, weight=0x20002), MISALIGNED),
    (dict(mean=0x50002), MISALIGNED), (dict(x_stride=(640, -64)), INVALID), (dict(x_stride=(1 << 40, 64)), NOTSUP),
]


@pytest.mark.parametrize("change,status", NORM + [
    (dict(y=0), INVALID), (dict(y=0x40001), MISALIGNED), (dict(bias=0x30001), MISALIGNED),
    (dict(y_stride=(640, 0)), INVALID)], ids=str)
def test_norm_forward_refuses(lib, change, status):
    assert lib.layer_norm_fwd(_norm(**change), None) == status


@pytest.mark.parametrize("change,status", NORM + [
    (dict(dy=0), INVALID), (dict(dx=0), INVALID), (dict(mean=0), INVALID), (dict(rstd=0), INVALID),
    (dict(dweight=0x90002), MISALIGNED), (dict(dbias=0xA0001), MISALIGNED), (dict(dx=0x80001), MISALIGNED),
    (dict(dx_stride=(0, 64)), INVALID), (dict(dy_stride=(-1, 64)), INVALID)], ids=str)
def test_norm_backward_refuses(lib, change, status):
    assert lib.layer_norm_bwd(_norm(**change), WS, 1 << 40, None) == status


def test_norm_refuses_its_workspace(lib):
    assert lib.layer_norm_fwd(None, None) == INVALID
    assert lib.layer_norm_bwd(None, WS, 1 << 40, None) == INVALID
    assert lib.layer_norm_bwd(_norm(), None, 1 << 40, None) == INVALID
    assert lib.layer_norm_bwd(_norm(), ctypes.c_void_p(WS.value + 8), 1 << 40, None) == MISALIGNED
    assert lib.layer_norm_workspace_size(0) == 0 and lib.layer_norm_workspace_size(16385) == 0


PAGES = [
    (dict(dtype=2), NOTSUP), (dict(batch=-1), INVALID), (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(head_dim=72), NOTSUP), (dict(head_dim=144), NOTSUP), (dict(page_size=0), INVALID),
    (dict(page_size=24), NOTSUP), (dict(pages=-1), INVALID), (dict(pages=0), INVALID), (dict(table_width=-1), INVALID),
    (dict(table_width=1 << 27), NOTSUP), (dict(k_cache=0), INVALID), (dict(v_cache=0), INVALID),
    (dict(scales=0), INVALID), (dict(block_table=0), INVALID), (dict(k_cache=0x30008), MISALIGNED),
    (dict(scales=0x50002), MISALIGNED), (dict(block_table=0x60002), MISALIGNED), (dict(table_stride=-4), INVALID),
    (dict(k_cache_stride=(8192, 72, 1024)), MISALIGNED), (dict(v_cache_stride=(8192, 64, -1024)), INVALID),
    (dict(v_cache_stride=(1 << 40, 64, 1024)), NOTSUP),
]


@pytest.mark.parametrize("change,status", PAGES + [
    (dict(length=-1), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(k=0x10008), MISALIGNED),
    (dict(starts=0x70001), MISALIGNED), (dict(lengths=0x80002), MISALIGNED), (dict(k_stride=(2560, 516, 64)), MISALIGNED),
    (dict(v_stride=(2560, -512, 64)), INVALID), (dict(batch=1 << 16, length=1 << 13), NOTSUP)], ids=str)
def test_cache_refuses(lib, change, status):
    assert lib.kv_cache_write(_cache(**change), None) == status
    assert lib.kv_cache_read(_cache(**change), None) == status


def test_what_is_written_may_not_repeat(lib):
    assert lib.kv_cache_write(_cache(k_cache_stride=(0, 64, 1024)), None) == INVALID
    assert lib.kv_cache_write(_cache(v_cache_stride=(8192, 0, 1024)), None) == INVALID
    assert lib.kv_cache_read(_cache(k_stride=(0, 512, 64)), None) == INVALID
    assert lib.kv_cache_read(_cache(v_stride=(2560, 512, 0)), None) == INVALID
    assert lib.kv_cache_write(None, None) == INVALID and lib.kv_cache_read(None, None) == INVALID


@pytest.mark.parametrize("change,status", PAGES + [
    (dict(heads=0), INVALID), (dict(heads=12), INVALID), (dict(q_len=-1), INVALID), (dict(q_len=257), NOTSUP),
    (dict(batch=1 << 24, q_len=16), NOTSUP), (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(kv_lengths=0), INVALID), (dict(q=0x10008), MISALIGNED),
    (dict(out=0x90008), MISALIGNED), (dict(lse=0xA0002), MISALIGNED), (dict(parents=0x80001), MISALIGNED),
    (dict(parent_stride=-1), INVALID), (dict(q_stride=(5120, 1020, 64)), MISALIGNED),
    (dict(out_stride=(5120, 0, 64)), INVALID), (dict(out_stride=(5120, 1024, 60)), MISALIGNED)], ids=str)
def test_tree_attention_refuses(lib, change, status):
    if "k_cache" in change and change["k_cache"] == 0x30008:
        change = dict(k_cache=0x20008)
    assert lib.tree_attention_fwd(_tree(**change), WS, 1 << 40, None) == status


def test_tree_attention_refuses_its_workspace(lib):
    assert lib.tree_attention_fwd(None, WS, 1 << 40, None) == INVALID
    assert lib.tree_attention_fwd(_tree(), None, 1 << 40, None) == INVALID
    assert lib.tree_attention_fwd(_tree(), ctypes.c_void_p(WS.value + 8), 1 << 40, None) == MISALIGNED
    for change in (dict(dtype=2), dict(head_dim=24), dict(heads=12), dict(q_len=300), dict(batch=-1)):
        assert lib.tree_attention_workspace_size(_tree(**change)) == 0
