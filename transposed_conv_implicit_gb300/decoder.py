"""The layer norm, the paged 8-bit cache of keys and values, and the attention of drafted tokens to
it: the binding of include/conv_gb300_decoder.h.

As elsewhere the functions only check and marshal arguments; every step of the computation runs in
the library's sm_103a kernels.

The cache of a layer: k_cache and v_cache float8_e4m3fn [pages, page_size, kv_heads, D] with any
strides whose innermost is 1 (a transposed view keeps a head's tokens side by side), scales uint8
[pages, kv_heads, page_size, 2], the exponents plus 127 of each row of k and of v (0: nothing was
written there, so a new cache's scales start as zeros), block_table int32 [batch, pages of a
request].  Token p of request b is token p % page_size of page block_table[b][p // page_size].
"""
from __future__ import annotations

import math
import struct

from . import _lib
from . import attention as _a
from ._lib import CONV_ERR_NOT_SUPPORTED, CONV_OK, CONV_STATUS_BYTES
from .attention import _common, _dense, _error, _invalid, _pack, _stream, _strides, _workspace

__all__ = ["layer_norm_fwd", "layer_norm_bwd", "layer_norm_workspace_size", "kv_cache_write",
           "kv_cache_read", "tree_attention_fwd", "tree_attention_workspace_size"]

_NORM = struct.Struct("@5if10Q8q")     # layer_norm_args_t
_CACHE = struct.Struct("@8i8Q13q")     # kv_cache_args_t
_TREE = struct.Struct("@9if10Q14q")    # tree_attention_args_t


_current_device = None    # filled on first use


def _call(fn, name, device, *args):
    """Calls with the tensors' device current: the library launches on the current one."""
    global _current_device
    if _current_device is None:
        torch = _a._torch
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if _current_device() == device:
        status = fn(*args)
    else:
        with _a._torch.cuda.device(device):
            status = fn(*args)
    if status != CONV_OK:
        raise _error(status, name)


def _sized(fn, device, *args):
    """A workspace size for calls on this device."""
    with _a._torch.cuda.device(device):
        return fn(*args)


# ------------------------------------------------------------------ layer norm
def _like(t, name, x):
    if t.shape != x.shape:
        raise _invalid("%s has shape %s, not %s" % (name, tuple(t.shape), tuple(x.shape)))
    if t.dtype is not x.dtype or t.get_device() != x.get_device():
        raise _invalid("%s must be %s on cuda:%d" % (name, x.dtype, x.get_device()))


def _rows(t, name, x):
    """(extent, stride) of [..., C]'s leading dimensions, those that run into one another joined (a
    feature map's pixels, a slice of a fused projection)."""
    _like(t, name, x)
    shape = x.shape
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise _invalid("%s: the innermost dimension must be contiguous" % name)
    dims = []
    for n, s in zip(shape[:-1], t.stride()[:-1]):
        if n == 1:
            continue
        if dims and dims[-1][1] == n * s:
            dims[-1] = (dims[-1][0] * n, s)
        else:
            dims.append((n, s))
    return dims


def _two(all_dims, names):
    """The tensors' rows as [batch][length] of one shape, and their strides."""
    cut = None    # a size of the inner dimension that every tensor can be cut at
    for dims in all_dims:
        if len(dims) > 2:
            raise _invalid("%s: the rows have more than two strides" % " or ".join(names))
        if len(dims) == 2:
            if cut is not None and cut != dims[1][0]:
                raise _invalid("%s: the rows are strided differently" % " and ".join(names))
            cut = dims[1][0]
    rows = 1
    for n, _ in all_dims[0]:
        rows *= n
    if cut is None:
        cut = rows
    strides = []
    for dims in all_dims:
        if len(dims) == 2:
            strides.append((dims[0][1], dims[1][1]))
        else:
            s = dims[0][1] if dims else 0
            strides.append((s * cut, s))
    return rows // cut if cut else 0, cut, strides


def _norm_common(x, name):
    codes = _a._codes or _a._fill_codes()
    code = codes.get(x.dtype)
    if code is None:
        raise _error(CONV_ERR_NOT_SUPPORTED, "dtype %s" % x.dtype)
    if not x.is_cuda:
        raise _invalid("%s must be a CUDA tensor" % name)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise _invalid("%s must be [..., channels]" % name)
    return code, x.get_device()


def _norm_weight(w, name, c, dtype, device):
    torch = _a._torch
    if w is None:
        return 0, None
    if w.shape != (c,) or w.get_device() != device or not w.is_contiguous() or (
            w.dtype is not dtype and w.dtype is not torch.float32):
        raise _invalid("%s must be a contiguous [%d] tensor of %s or float32" % (name, c, dtype))
    return w.data_ptr(), w.dtype


def _norm_size(x, others, names):
    """(batch, length, strides of x and of the others), which are (tensor, name)."""
    rows = x.numel() // x.shape[-1]
    if x.is_contiguous():     # (without the walk over the dimensions: a call of few tokens is its launch)
        for t, name in others:
            if not t.is_contiguous():
                break
            _like(t, name, x)
        else:
            return 1, rows, [(0, x.shape[-1])] * (1 + len(others))
    dims = [_rows(x, names[0], x)] + [_rows(t, name, x) for t, name in others]
    if rows == 0:
        return 0, 0, [(0, 0)] * len(dims)
    return _two(dims, names)


def layer_norm_fwd(x, weight, bias, y, *, mean=None, rstd=None, eps=1e-5, stream=None):
    """y = (x - mean) / sqrt(var + eps) * weight + bias over the last dimension; returns `y`.

    x [..., C]; weight and bias [C], of x's type or float32 (both of one), or None.  mean and rstd
    (float32 [...], optional) receive each row's mean and 1 / sqrt(var + eps), which layer_norm_bwd
    needs.  y may be x."""
    code, device = _norm_common(x, "x")
    torch, dtype, shape = _a._torch, x.dtype, x.shape
    c = shape[-1]
    w, wt = _norm_weight(weight, "weight", c, dtype, device)
    b, bt = _norm_weight(bias, "bias", c, dtype, device)
    if wt is not None and bt is not None and wt is not bt:
        raise _invalid("weight and bias must be of one type")
    m = 0 if mean is None else _dense(mean, "mean", shape[:-1], torch.float32, device)
    r = 0 if rstd is None else _dense(rstd, "rstd", shape[:-1], torch.float32, device)
    batch, length, (xs, ys) = _norm_size(x, ((y, "y"),), ("x", "y"))
    args = _pack(_NORM, code, batch, length, c, torch.float32 in (wt, bt), eps, x.data_ptr(), w, b,
                 y.data_ptr(), m, r, 0, 0, 0, 0, *xs, *ys, 0, 0, 0, 0)
    _call(_lib.lib().layer_norm_fwd, "layer_norm_fwd", device, args, _stream(stream, device))
    return y


def layer_norm_workspace_size(channels) -> int:
    """Workspace bytes of layer_norm_bwd (CONV_STATUS_BYTES do where neither dweight nor dbias is wanted)."""
    size = _lib.lib().layer_norm_workspace_size(int(channels))
    if size == 0:
        raise _error(CONV_ERR_NOT_SUPPORTED, "layer_norm_workspace_size")
    return size


def layer_norm_bwd(dy, x, weight, mean, rstd, dx, dweight, dbias, *, workspace=None, stream=None):
    """Gradients of layer_norm_fwd: dx like x, dweight and dbias float32 [C] (either may be None),
    summed in a fixed order; returns the three.  mean and rstd are the forward pass's.  dx may be
    dy or x."""
    code, device = _norm_common(x, "x")
    torch, dtype, shape = _a._torch, x.dtype, x.shape
    c = shape[-1]
    w, wt = _norm_weight(weight, "weight", c, dtype, device)
    if mean is None or rstd is None:
        raise _invalid("the backward pass needs mean and rstd")
    m = _dense(mean, "mean", shape[:-1], torch.float32, device)
    r = _dense(rstd, "rstd", shape[:-1], torch.float32, device)
    dw = 0 if dweight is None else _dense(dweight, "dweight", (c,), torch.float32, device)
    db = 0 if dbias is None else _dense(dbias, "dbias", (c,), torch.float32, device)
    batch, length, (xs, ds, dxs) = _norm_size(x, ((dy, "dy"), (dx, "dx")), ("x", "dy", "dx"))
    args = _pack(_NORM, code, batch, length, c, wt is torch.float32, 0.0, x.data_ptr(), w, 0, 0, m, r,
                 dy.data_ptr(), dx.data_ptr(), dw, db, *xs, 0, 0, *ds, *dxs)
    lib = _lib.lib()
    if workspace is None:
        from . import new_workspace
        size = _sized(lib.layer_norm_workspace_size, device, c) if dw or db else CONV_STATUS_BYTES
        workspace = new_workspace(size, x.device, stream, status_only=True)
    _call(lib.layer_norm_bwd, "layer_norm_bwd", device, args, *_workspace(workspace, device),
          _stream(stream, device))
    return dx, dweight, dbias


# ------------------------------------------------------------------ the cache
# (The calls below run before every launch, single tokens' among them: a tensor's shape and strides
# are asked for once, which takes longer than anything that is done with them.)
def _cache(k_cache, v_cache, scales, block_table, batch, kv_heads, d, device):
    """(pages, page_size, table_width), the pointers, the table's stride and the cache's strides.
    kv_heads None: as k_cache has them."""
    torch = _a._torch
    shape = k_cache.shape
    if len(shape) != 4 or shape[3] != d or (shape[2] != kv_heads if kv_heads else shape[2] < 1):
        raise _invalid("k_cache must be [pages, page_size, %s, %d]" % (kv_heads or "kv_heads", d))
    pages, page_size, kv_heads, _ = shape
    ks = _strides(k_cache, "k_cache", shape, torch.float8_e4m3fn, device)
    vs = _strides(v_cache, "v_cache", shape, torch.float8_e4m3fn, device)
    s = _dense(scales, "scales", (pages, kv_heads, page_size, 2), torch.uint8, device)
    table, stride = block_table.shape, block_table.stride()
    if (len(table) != 2 or table[0] != batch or block_table.dtype is not torch.int32
            or block_table.get_device() != device or (stride[1] != 1 and table[1] > 1)):
        raise _invalid("block_table must be int32 [%d, pages of a request] on cuda:%d, contiguous "
                       "along the pages" % (batch, device))
    return ((pages, page_size, table[1]), kv_heads,
            (k_cache.data_ptr(), v_cache.data_ptr(), s, block_table.data_ptr()), stride[0], ks + vs)


def _per_request(t, name, batch, device):
    return 0 if t is None else _dense(t, name, (batch,), _a._torch.int32, device)


def _leading(x, name):
    """The dtype's code, the device's number, the dtype and the shape of [batch, length, heads, D]."""
    code, device = _common(x, name)
    return code, device, x.dtype, x.shape


def _move(name, k, v, k_cache, v_cache, scales, block_table, starts, lengths, stream):
    code, device, dtype, shape = _leading(k, "k")
    b, length, heads, d = shape
    strides = _strides(k, "k", shape, dtype, device) + _strides(v, "v", shape, dtype, device)
    if heads < 1:
        raise _invalid("k must have heads")
    sizes, _, ptrs, table_stride, cache_strides = _cache(k_cache, v_cache, scales, block_table, b, heads, d,
                                                         device)
    args = _pack(_CACHE, code, b, length, heads, d, *sizes, k.data_ptr(), v.data_ptr(), *ptrs,
                 _per_request(starts, "starts", b, device), _per_request(lengths, "lengths", b, device),
                 table_stride, *strides, *cache_strides)
    _call(getattr(_lib.lib(), name), name, device, args, _stream(stream, device))


def kv_cache_write(k, v, k_cache, v_cache, scales, block_table, starts, *, lengths=None, stream=None):
    """Quantises k and v [B, L, kv_heads, D] into the cache as tokens starts[b] .. of request b, and
    their exponents into scales; returns (k_cache, v_cache, scales).

    starts and lengths: int32 [B]; starts may be None (0), lengths[b] tokens of request b are taken
    (default: all).  A row's scale is the smallest power of two, 2^-64 at least, that brings its
    largest finite element to 448 or below (1 for rows of zeros); codes are rounded to nearest;
    infinities become the largest code, NaN stays.  Tokens outside the table, or on pages that it gives no number of, are left out.  No two
    tokens of a call may go to the same place."""
    _move("kv_cache_write", k, v, k_cache, v_cache, scales, block_table, starts, lengths, stream)
    return k_cache, v_cache, scales


def kv_cache_read(k_cache, v_cache, scales, block_table, starts, k, v, *, lengths=None, stream=None):
    """Tokens starts[b] .. of the cache as k and v [B, L, kv_heads, D] in 16 bits; returns (k, v).

    Arguments as kv_cache_write's; rows from lengths[b] on keep what they hold; tokens outside the
    table, and those that were never written, read as zeros."""
    _move("kv_cache_read", k, v, k_cache, v_cache, scales, block_table, starts, lengths, stream)
    return k, v


# ------------------------------------------------------------------ tree attention
def tree_attention_workspace_size(batch, heads, kv_heads, q_len, max_keys, head_dim, *,
                                  dtype="bf16") -> int:
    """Workspace bytes of tree_attention_fwd with these sizes; max_keys is what the block table
    covers: its pages of a request times page_size."""
    width = -(-int(max_keys) // 16)
    args = _pack(_TREE, _lib.DTYPE_CODES[dtype], batch, heads, kv_heads, q_len, head_dim, 0, 16, width, 1.0,
                 *([0] * 24))
    size = _lib.lib().tree_attention_workspace_size(args)
    if size == 0:
        raise _error(CONV_ERR_NOT_SUPPORTED, "tree_attention_workspace_size")
    return size


def tree_attention_fwd(q, k_cache, v_cache, scales, block_table, kv_lengths, output, *, parents=None,
                       draft_lengths=None, lse=None, scale=None, workspace=None, stream=None):
    """Attention of each request's drafted tokens to its cache; returns `output`.

    q [B, T, H, D] holds the drafts' queries (T up to 256; T = 1: one token).  Request b has
    kv_lengths[b] tokens in the cache, the last draft_lengths[b] (default T) of them the drafts,
    written there before.  Draft i attends the tokens in front of the drafts, itself, and its
    ancestors: parents (int32 [B, T], or [T] for all requests) gives the draft in front of each, a
    smaller number, anything else (such as -1) where the context is; without parents draft i attends
    all drafts up to i.  Rows of output (and lse, float32 [B, H, T], optional) from draft_lengths[b]
    on keep what they hold.  scale defaults to 1 / sqrt(D).  Calls that may overlap on the GPU need
    workspaces of their own."""
    code, device, dtype, shape = _leading(q, "q")
    torch = _a._torch
    b, t, h, d = shape
    strides = _strides(q, "q", shape, dtype, device) + _strides(output, "output", shape, dtype, device)
    sizes, hkv, ptrs, table_stride, cache_strides = _cache(k_cache, v_cache, scales, block_table, b, None, d,
                                                           device)
    up, up_stride = 0, 0
    if parents is not None:
        tree, steps = parents.shape, parents.stride()
        if (parents.dtype is not torch.int32 or parents.get_device() != device
                or (tree != (b, t) and tree != (t,)) or (steps[-1] != 1 and t > 1)):
            raise _invalid("parents must be int32 [%d, %d] or [%d] on cuda:%d, contiguous along the drafts"
                           % (b, t, t, device))
        up, up_stride = parents.data_ptr(), steps[0] if len(tree) == 2 else 0
    if kv_lengths is None:
        raise _invalid("kv_lengths is missing")
    if lse is not None:
        lse = _dense(lse, "lse", (b, h, t), torch.float32, device)
    if scale is None:
        scale = 1.0 / math.sqrt(d) if d else 1.0
    args = _pack(_TREE, code, b, h, hkv, t, d, *sizes, scale, q.data_ptr(), *ptrs,
                 _per_request(kv_lengths, "kv_lengths", b, device),
                 _per_request(draft_lengths, "draft_lengths", b, device), up, output.data_ptr(), lse or 0,
                 table_stride, up_stride, *strides, *cache_strides)
    lib = _lib.lib()
    if workspace is None:
        from . import new_workspace
        workspace = new_workspace(_sized(lib.tree_attention_workspace_size, device, args), q.device, stream,
                                  status_only=True)
    _call(lib.tree_attention_fwd, "tree_attention_fwd", device, args, *_workspace(workspace, device),
          _stream(stream, device))
    return output
