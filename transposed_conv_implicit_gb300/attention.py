"""Cross attention to an encoder's states, and the per-head norm of queries and
keys with the position rotation: the binding of include/conv_gb300_attention.h.

As for the convolutions, the functions only check and marshal arguments; every
step of the computation runs in the library's sm_103a kernels.

Layouts: q [B, Lq, H, D]; k, v [B, Lk, Hkv, D] with H a multiple of Hkv, any
strides whose innermost is 1 (a feature map [N, h, w, H*D] viewed as
[N, h*w, H, D]; the two halves of a fused key/value projection).  Dtypes:
bfloat16 and float16; lse and the weight gradients are float32.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import _lib
from ._lib import CONV_ERR_INVALID_VALUE, CONV_ERR_NOT_SUPPORTED, CONV_OK

__all__ = [
    "cross_attention_fwd", "cross_attention_bwd", "cross_attention_workspace_size",
    "qk_norm_rope_fwd", "qk_norm_rope_bwd", "qk_norm_rope_workspace_size",
]

# cross_attention_args_t: 7 ints, the scale, 11 pointers, 8 strides of 3, 1 of 4.
_ATTN = struct.Struct("@7if11Q28q")
# qk_norm_rope_tensor_t and the head of qk_norm_rope_args_t.
_NORM_TENSOR = struct.Struct("@7Q3i4x13q")
_NORM_HEAD = struct.Struct("@6if4x2Q")
_NO_TENSOR = bytes(_NORM_TENSOR.size)
_NO_STRIDES = (0, 0, 0)

_torch = None         # with the next two, filled on first use
_codes = None         # torch dtype -> conv_dtype_t
_raw_stream = None


def _fill_codes():
    global _torch, _codes, _raw_stream
    import torch
    _torch = torch
    # The current stream as a plain number, without building a Stream object.
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _codes = {torch.bfloat16: 0, torch.float16: 1}
    return _codes


def _error(status, where):
    from . import ConvError
    return ConvError(status, where)


def _invalid(what):
    return _error(CONV_ERR_INVALID_VALUE, what)


def _check(status, where):
    if status != CONV_OK:
        raise _error(status, where)


def _pack(layout, *values):
    """The values as a C struct; numbers that its fields cannot hold are refused."""
    try:
        return layout.pack(*values)
    except (struct.error, OverflowError) as e:
        raise _invalid("a size, a stride or a factor is out of range (%s)" % e) from None


# The calls below run before every launch, single tokens' among them: devices are
# compared as numbers and shapes as they come (a torch.device or a tuple for each
# tensor made a call of one token half as long again).
def _stream(stream, device):
    if stream is None:
        return _raw_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _workspace(workspace, device):
    """Address and bytes of the caller's workspace."""
    if workspace.get_device() != device:
        raise _invalid("workspace must be on cuda:%d" % device)
    return workspace.data_ptr(), workspace.nbytes


def _common(x, name):
    """The dtype code and the device's number of the leading tensor."""
    codes = _codes or _fill_codes()
    if x.dim() != 4:
        raise _invalid("%s must be [batch, length, heads, head_dim]" % name)
    code = codes.get(x.dtype)
    if code is None:
        raise _error(CONV_ERR_NOT_SUPPORTED, "dtype %s" % x.dtype)
    if not x.is_cuda:
        raise _invalid("%s must be a CUDA tensor" % name)
    return code, x.get_device()


def _strides(t, name, shape, dtype, device):
    """{batch, token, head} strides of a tensor of this shape, type and device."""
    if t.shape != shape:
        raise _invalid("%s has shape %s, not %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype is not dtype or t.get_device() != device:
        raise _invalid("%s must be %s on cuda:%d" % (name, dtype, device))
    b, l, h, d = t.stride()
    if d != 1 and shape[3] > 1:
        raise _invalid("%s: the innermost dimension must be contiguous" % name)
    return b, l, h


def _dense(t, name, shape, dtype, device):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise _invalid("%s must be a contiguous %s tensor of shape %s on cuda:%d"
                       % (name, dtype, tuple(shape), device))
    return t.data_ptr()


def _attention(backward, q, k, v, output, lse, kv_lengths, mask, scale, grads, workspace, stream):
    code, device = _common(q, "q")
    torch, dtype, shape = _torch, q.dtype, q.shape
    b, lq, h, d = shape
    if k.dim() != 4 or k.shape[0] != b or k.shape[3] != d:
        raise _invalid("k must be [batch, kv_len, kv_heads, head_dim] of q's batch and head_dim")
    kshape = k.shape
    lk, hkv = kshape[1], kshape[2]
    strides = (_strides(q, "q", shape, dtype, device) + _strides(k, "k", kshape, dtype, device)
               + _strides(v, "v", kshape, dtype, device)
               + _strides(output, "output", shape, dtype, device))
    if lse is not None:
        lse = _dense(lse, "lse", (b, h, lq), torch.float32, device)
    elif backward:
        raise _invalid("the backward pass needs lse")
    if kv_lengths is not None:
        kv_lengths = _dense(kv_lengths, "kv_lengths", (b,), torch.int32, device)
    mask_ptr, mask_strides = 0, (0, 0, 0, 0)
    if mask is not None:
        if (mask.dim() != 4 or mask.dtype not in (torch.bool, torch.uint8)
                or mask.get_device() != device):
            raise _invalid("mask must be a bool or uint8 tensor of 4 dimensions on cuda:%d" % device)
        for have, want in zip(mask.shape, (b, h, lq, lk)):
            if have != want and have != 1:
                raise _invalid("mask has shape %s, not broadcast to %s"
                               % (tuple(mask.shape), (b, h, lq, lk)))
        mask_ptr = mask.data_ptr()
        mask_strides = tuple(st if n > 1 else 0 for n, st in zip(mask.shape, mask.stride()))
    if grads is None:
        ptrs, gstrides = (0, 0, 0, 0), _NO_STRIDES * 4
    else:
        dout, dq, dk, dv = grads
        gstrides = (_strides(dout, "dout", shape, dtype, device)
                    + _strides(dq, "dq", shape, dtype, device)
                    + _strides(dk, "dk", kshape, dtype, device)
                    + _strides(dv, "dv", kshape, dtype, device))
        ptrs = (dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr())
    if scale is None:
        scale = 1.0 / math.sqrt(d) if d else 1.0
    args = _pack(_ATTN, code, b, h, hkv, lq, lk, d, scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                 output.data_ptr(), lse or 0, kv_lengths or 0, mask_ptr, *ptrs, *strides, *gstrides,
                 *mask_strides)
    lib = _lib.lib()
    if workspace is None:
        from . import new_workspace
        workspace = new_workspace(lib.cross_attention_workspace_size(args, int(backward)), q.device,
                                  stream)
    call = lib.cross_attention_bwd if backward else lib.cross_attention_fwd
    status = call(args, *_workspace(workspace, device), _stream(stream, device))
    if status != CONV_OK:
        raise _error(status, "cross_attention_bwd" if backward else "cross_attention_fwd")


def cross_attention_workspace_size(batch, heads, kv_heads, q_len, kv_len, head_dim, *, masked=False,
                                   mask_heads=1, backward=False, dtype="bf16") -> int:
    """Workspace bytes for calls of these sizes.  `masked`: a mask with its own rows for every
    batch and query (for `mask_heads` heads) is given; narrower masks need no more."""
    args = _pack(_ATTN, _lib.DTYPE_CODES[dtype], batch, heads, kv_heads, q_len, kv_len, head_dim, 1.0,
                 0, 0, 0, 0, 0, 0, int(masked), 0, 0, 0, 0, *(_NO_STRIDES * 8), 1, int(mask_heads > 1), 1, 1)
    size = _lib.lib().cross_attention_workspace_size(args, int(backward))
    if size == 0:
        raise _error(CONV_ERR_NOT_SUPPORTED, "cross_attention_workspace_size")
    return size


def cross_attention_fwd(q, k, v, output, *, lse=None, kv_lengths=None, mask=None, scale=None,
                        workspace=None, stream=None):
    """output = softmax(scale * q k^T) v over each query head's key head; returns `output`.

    lse (float32 [B, H, Lq], optional) receives the log of each query's softmax sum, which
    cross_attention_bwd needs.  kv_lengths (int32 [B]): keys from there on take no part.  mask
    (bool or uint8, broadcast to [B, H, Lq, Lk]): pairs where it is 0 take no part.  A query
    without keys gives zeros and lse = -inf.  scale defaults to 1/sqrt(D).  Calls that may
    overlap on the GPU need workspaces of their own."""
    _attention(False, q, k, v, output, lse, kv_lengths, mask, scale, None, workspace, stream)
    return output


def cross_attention_bwd(dout, q, k, v, output, lse, dq, dk, dv, *, kv_lengths=None, mask=None,
                        scale=None, workspace=None, stream=None):
    """Gradients of cross_attention_fwd into dq, dk and dv (returned); `output` and `lse` are
    the forward pass's.  Key heads shared by several query heads get their sum.  The sums run in
    a fixed order: equal calls give equal bits."""
    _attention(True, q, k, v, output, lse, kv_lengths, mask, scale, (dout, dq, dk, dv), workspace,
               stream)
    return dq, dk, dv


def _norm_tensor(name, x, weight, positions, y, dy, dx, dweight, batch, d, dtype, device):
    if x is None:
        return _NO_TENSOR
    torch, shape = _torch, x.shape
    if shape[0] != batch or shape[3] != d:
        raise _invalid("%s differs from the other tensor in batch or head_dim" % name)
    if weight is None:
        raise _invalid("%s needs its weight" % name)
    if weight.shape != (d,) or weight.get_device() != device or not weight.is_contiguous() or (
            weight.dtype is not dtype and weight.dtype is not torch.float32):
        raise _invalid("%s_weight must be a contiguous [%d] tensor of %s or float32" % (name, d, dtype))
    pos, pos_stride = 0, 0
    if positions is not None:
        if positions.dim() == 1 and positions.shape[0] == shape[1]:
            stride = (0, positions.stride(0))
        elif positions.shape == (batch, shape[1]):
            stride = positions.stride()
        else:
            raise _invalid("%s_positions must be [length] or [batch, length]" % name)
        if positions.dtype is not torch.int32 or positions.get_device() != device or (
                stride[1] != 1 and shape[1] > 1):
            raise _invalid("%s_positions must be int32 on cuda:%d, contiguous along the length"
                           % (name, device))
        pos, pos_stride = positions.data_ptr(), stride[0]
    xs = _strides(x, name, shape, dtype, device)
    if dy is None:
        if y is None:
            raise _invalid("%s needs its output" % name)
        out, rest = y.data_ptr(), (0, 0, 0)
        strides = (*xs, *_strides(y, name + "_out", shape, dtype, device), 0, 0, 0, 0, 0, 0)
    else:
        if dx is None or dweight is None:
            raise _invalid("%s needs d%s and d%s_weight" % (name, name, name))
        out, rest = 0, (dy.data_ptr(), dx.data_ptr(),
                        _dense(dweight, "d%s_weight" % name, (d,), torch.float32, device))
        strides = (*xs, 0, 0, 0, *_strides(dy, "d%s_out" % name, shape, dtype, device),
                   *_strides(dx, "d" + name, shape, dtype, device))
    return _pack(_NORM_TENSOR, x.data_ptr(), weight.data_ptr(), pos, out, *rest, shape[1], shape[2],
                 weight.dtype is not dtype, pos_stride, *strides)


def _norm_head(q, k, cos, sin, eps, adjacent_pairs):
    lead = q if q is not None else k
    if lead is None:
        raise _invalid("q and k are both missing")
    code, device = _common(lead, "q" if q is not None else "k")
    if k is not None and k.dim() != 4:
        raise _invalid("k must be [batch, length, heads, head_dim]")
    if cos is None or sin is None:
        if cos is not None or sin is not None:
            raise _invalid("cos and sin come together")
        rows, half, cp, sp = 0, 0, 0, 0
    else:
        if cos.dim() != 2:
            raise _invalid("cos must be [rows, rot_dim / 2]")
        shape = cos.shape
        rows, half = shape
        cp = _dense(cos, "cos", shape, _torch.float32, device)
        sp = _dense(sin, "sin", shape, _torch.float32, device)
    head = _pack(_NORM_HEAD, code, lead.shape[0], lead.shape[3], 2 * half, rows,
                 1 if adjacent_pairs else 0, eps, cp, sp)
    return head, lead, device


def qk_norm_rope_fwd(q, k, q_weight, k_weight, q_out, k_out, *, cos=None, sin=None, q_positions=None,
                     k_positions=None, eps=1e-6, adjacent_pairs=False, stream=None):
    """q_out and k_out: each head's row of q and k over its root mean square, times the weight,
    its first 2 * cos.shape[1] elements turned by the row's position; returns (q_out, k_out).

    q and k may differ in length and heads, either may be None (with its weight and output).
    cos and sin are float32 tables [rows, rot_dim / 2]; positions int32 [B, L] or [L] (default
    0 .. L-1) select their rows.  Pairs are (i, i + rot_dim/2), or (2i, 2i+1) with
    adjacent_pairs.  q_out may be q itself, and k_out k."""
    head, lead, device = _norm_head(q, k, cos, sin, eps, adjacent_pairs)
    b, d = lead.shape[0], lead.shape[3]
    args = (head
            + _norm_tensor("q", q, q_weight, q_positions, q_out, None, None, None, b, d, lead.dtype, device)
            + _norm_tensor("k", k, k_weight, k_positions, k_out, None, None, None, b, d, lead.dtype, device))
    _check(_lib.lib().qk_norm_rope_fwd(args, _stream(stream, device)), "qk_norm_rope_fwd")
    return q_out, k_out


def qk_norm_rope_workspace_size(head_dim) -> int:
    """Workspace bytes of qk_norm_rope_bwd."""
    return _lib.lib().qk_norm_rope_workspace_size(int(head_dim))


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, dq, dk, dq_weight, dk_weight, *,
                     cos=None, sin=None, q_positions=None, k_positions=None, eps=1e-6,
                     adjacent_pairs=False, workspace=None, stream=None):
    """Gradients of qk_norm_rope_fwd: dq and dk like q and k, dq_weight and dk_weight float32 [D]
    (summed in a fixed order); returns the four.  q and k are the forward pass's inputs."""
    if (q is None) != (dq_out is None) or (k is None) != (dk_out is None):
        raise _invalid("q comes with dq_out, and k with dk_out")
    head, lead, device = _norm_head(q, k, cos, sin, eps, adjacent_pairs)
    b, d = lead.shape[0], lead.shape[3]
    args = (head
            + _norm_tensor("q", q, q_weight, q_positions, None, dq_out, dq, dq_weight, b, d, lead.dtype,
                           device)
            + _norm_tensor("k", k, k_weight, k_positions, None, dk_out, dk, dk_weight, b, d, lead.dtype,
                           device))
    if workspace is None:
        from . import new_workspace
        workspace = new_workspace(qk_norm_rope_workspace_size(d), lead.device, stream)
    _check(_lib.lib().qk_norm_rope_bwd(args, *_workspace(workspace, device), _stream(stream, device)),
           "qk_norm_rope_bwd")
    return dq, dk, dq_weight, dk_weight
