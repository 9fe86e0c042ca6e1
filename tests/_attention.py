"""The attention operators' definitions in 64 bits, and error bounds that follow
from where the library rounds: probabilities and score gradients once to the
tensors' type (unit roundoff u), results once, everything else fp32."""
import math

import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
F32 = 2.0 ** -24


def grain(u):
    """Half the step of fp16's subnormal numbers, below which a relative roundoff does not hold
    (bfloat16's are out of reach)."""
    return 2.0 ** -25 if u < 2.0 ** -9 else 0.0


def pairs(b, h, lq, lk, kv_lengths=None, mask=None, device="cuda"):
    keep = torch.ones((b, h, lq, lk), dtype=torch.bool, device=device)
    if kv_lengths is not None:
        keep &= torch.arange(lk, device=device) < kv_lengths[:, None, None, None]
    if mask is not None:
        keep &= mask.bool()
    return keep


class Reference:
    """cross attention in 64 bits with elementwise error bounds (out, lse, dq, dk, dv).  Pairs
    that are left out take no part, whatever their rows hold."""

    def __init__(self, q, k, v, *, scale=None, kv_lengths=None, mask=None, dout=None, u):
        b, lq, h, d = q.shape
        lk, hkv = k.shape[1], k.shape[2]
        g = h // hkv
        scale = 1.0 / math.sqrt(d) if scale is None else scale
        keep = pairs(b, h, lq, lk, kv_lengths, mask, q.device)
        live_k = keep.reshape(b, hkv, g, lq, lk).any(3).any(2)            # [B, Hkv, Lk]
        live_q = keep.any(3)                                              # [B, H, Lq]

        def clean(x, live):
            x = x.double().transpose(1, 2)
            return torch.where(live[..., None], x, torch.zeros_like(x))

        q64 = clean(q, live_q)
        k64 = clean(k, live_k).repeat_interleave(g, dim=1)
        v64 = clean(v, live_k).repeat_interleave(g, dim=1)
        s = (q64 @ k64.transpose(2, 3) * scale).masked_fill(~keep, -math.inf)
        lse = torch.logsumexp(s, dim=3)
        base = torch.where(live_q, lse, torch.zeros_like(lse))[..., None]
        p = torch.exp(s - base)
        o = p @ v64
        # A score's fp32 sum is off by at most (D + 2) roundings of its absolute sum, and the
        # exponent's argument in base 2 by two more of its own size: p is off by that share.
        s_abs = (q64.abs() @ k64.abs().transpose(2, 3)) * scale
        ds_err = F32 * ((d + 2) * s_abs + 4 * (s_abs + base.abs() + 1))
        ds_err = torch.where(keep, ds_err, torch.zeros_like(ds_err)).amax(3, keepdim=True)
        share = u + 2 * ds_err + lk * F32        # of each p: rounding, its score, its row's sum
        mag = p @ v64.abs()
        tiny = 2.0 ** -24 * (keep.double() @ v64.abs()) if u < 2.0 ** -9 else 0.0  # fp16's smallest step
        self.out = o.transpose(1, 2)
        self.out_tol = (u * o.abs() + share * (1 + u) * mag + tiny + grain(u)).transpose(1, 2)
        self.lse = lse
        self.lse_tol = (ds_err + lk * F32).squeeze(3) + 4 * F32 * base.abs().squeeze(3)
        if dout is None:
            return
        do = clean(dout, live_q)
        dp = do @ v64.transpose(2, 3)
        delta = (do * o).sum(3, keepdim=True)
        ds = p * (dp - delta)
        dp_abs = do.abs() @ v64.abs().transpose(2, 3)
        o_tol = self.out_tol.transpose(1, 2)
        # delta comes from the rounded out or from the rounded products: off by at most
        # |dout| times out's bound.
        delta_err = (do.abs() * o_tol).sum(3, keepdim=True) + d * F32 * dp_abs.amax(3, keepdim=True)
        ds_tol = u * ds.abs() + p * (delta_err + d * F32 * dp_abs) + (2 * ds_err + lk * F32) * p * (
            (dp - delta).abs())

        def shared(x):
            return x.reshape(b, hkv, g, lk, d).sum(2).transpose(1, 2)

        def bound(value, err):
            return u * value.abs() + (1 + u) * err + grain(u)

        rows = lq * g * F32
        dq, dq_err = ds @ k64 * scale, (ds_tol + rows * ds.abs()) @ k64.abs() * scale
        dk = shared(ds.transpose(2, 3) @ q64) * scale
        dk_err = shared((ds_tol + rows * ds.abs()).transpose(2, 3) @ q64.abs()) * scale
        dv = shared(p.transpose(2, 3) @ do)
        dv_err = shared(((share + rows) * p).transpose(2, 3) @ do.abs())
        self.dq, self.dq_tol = dq.transpose(1, 2), bound(dq, dq_err).transpose(1, 2)
        self.dk, self.dk_tol = dk, bound(dk, dk_err)
        self.dv, self.dv_tol = dv, bound(dv, dv_err)


def assert_within(name, got, want, tol):
    """Elementwise; infinities have to be equal."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine]), "%s: not-finite places differ" % name
    err = torch.where(fine, (got - torch.where(fine, want, torch.zeros_like(want))).abs(),
                      torch.zeros_like(got))
    bad = ~(err <= torch.where(fine, tol, torch.ones_like(err)))
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError("%s: %d of %d outside the bound, first at %s: got %g, want %g, bound %g" % (
            name, int(bad.sum()), bad.numel(), at, got[tuple(at)], want[tuple(at)], tol[tuple(at)]))


class NormReference:
    """The norm with the rotation in 64 bits; rounding u on the results only."""

    def __init__(self, x, weight, cos, sin, positions, eps, adjacent, u, dy=None):
        b, length, heads, d = x.shape
        x64, w = x.double(), weight.double()
        r = 1 / torch.sqrt(x64.square().mean(3, keepdim=True) + eps)
        rot = 0 if cos is None else 2 * cos.shape[1]
        if positions is None:
            positions = torch.arange(length, device=x.device)
        positions = positions.long().expand(b, length)
        i = torch.arange(rot // 2, device=x.device)
        first, second = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
        if rot:
            at = positions.clamp(0, cos.shape[0] - 1)
            c, s = cos.double()[at][:, :, None], sin.double()[at][:, :, None]

        def turned(z, sign):
            z = z.clone()
            if rot:
                a, e = z[..., first].clone(), z[..., second].clone()
                z[..., first], z[..., second] = a * c - sign * e * s, e * c + sign * a * s
            return z

        def reach(z):   # the size of what a turned element sums
            z = z.abs()
            if rot:
                both = z[..., first] + z[..., second]
                z = z.clone()
                z[..., first], z[..., second] = both, both
            return z

        y = x64 * r * w
        self.y = turned(y, 1)
        self.y_tol = u * self.y.abs() + (d + 8) * F32 * reach(y) + grain(u)
        if dy is None:
            return
        dy64 = dy.double()
        g = turned(dy64, -1)
        xhat = x64 * r
        gw = g * w
        self.dx = r * (gw - xhat * (gw * xhat).mean(3, keepdim=True))
        size = r * (reach(dy64) * w.abs() + xhat.abs() * (reach(dy64) * (w * xhat).abs()).mean(3, keepdim=True))
        self.dx_tol = u * self.dx.abs() + 2 * (d + 8) * F32 * size + grain(u)
        self.dw = (g * xhat).sum((0, 1, 2))
        rows = b * length * heads
        self.dw_tol = (d + 8 + min(rows, 4096)) * F32 * (reach(dy64) * xhat.abs()).sum((0, 1, 2)) + 1e-30
