"""The decoder operators' definitions in 64 bits, and error bounds that follow from where the library
rounds: results once to the tensors' type (unit roundoff u), probabilities once to fp16, everything
else fp32."""
import math

import torch

from tests._attention import F32, grain

E4M3 = torch.float8_e4m3fn


class NormReference:
    """Layer norm of rows x [R, C] in 64 bits with elementwise bounds."""

    def __init__(self, x, weight, bias, eps, u, dy=None):
        rows, c = x.shape
        x = x.double()
        w = torch.ones(c, dtype=torch.float64, device=x.device) if weight is None else weight.double()
        b = torch.zeros(c, dtype=torch.float64, device=x.device) if bias is None else bias.double()
        mean = x.mean(1, keepdim=True)
        dev = x - mean
        var = (dev * dev).mean(1, keepdim=True)
        rstd = 1 / torch.sqrt(var + eps)
        h = dev * rstd
        # A deviation is off by the mean's error and a rounding, the variance by its own sum's
        # roundings and by what the deviations' errors make of it.
        mean_err = (c + 8) * F32 * x.abs().mean(1, keepdim=True)
        dev_err = mean_err + 2 * F32 * (x.abs() + mean.abs())
        rel = (c + 8) * F32 + (2 * dev.abs() * dev_err + dev_err ** 2).mean(1, keepdim=True) / (var + eps)
        h_err = rstd * dev_err + h.abs() * (rel + 4 * F32)
        self.mean, self.mean_tol = mean[:, 0], mean_err[:, 0] + F32 * mean[:, 0].abs()
        self.rstd, self.rstd_tol = rstd[:, 0], rstd[:, 0] * (rel[:, 0] + 4 * F32)
        self.y = h * w + b
        self.y_tol = u * self.y.abs() + w.abs() * h_err + 4 * F32 * ((h * w).abs() + b.abs()) + grain(u)
        if dy is None:
            return
        dy = dy.double()
        g = dy * w
        mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
        self.dx = rstd * (g - mg - h * mgh)
        mg_err = (c + 8) * F32 * g.abs().mean(1, keepdim=True)
        mgh_err = (c + 8) * F32 * (g * h).abs().mean(1, keepdim=True) + (g.abs() * h_err).mean(1, keepdim=True)
        size = g.abs() + mg.abs() + (h * mgh).abs()
        self.dx_tol = u * self.dx.abs() + grain(u) + rstd * (
            8 * F32 * size + mg_err + h.abs() * mgh_err + h_err * mgh.abs()) + (rel + 4 * F32) * self.dx.abs()
        self.dweight = (dy * h).sum(0)
        self.dweight_tol = (dy.abs() * h_err).sum(0) + (rows + 16) * F32 * (dy * h).abs().sum(0) + 1e-37
        self.dbias = dy.sum(0)
        self.dbias_tol = (rows + 16) * F32 * dy.abs().sum(0)


def pow2(e):
    """2^e in 64 bits, exact (the GPU's power function is not)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantised(x):
    """(values of the codes, exponents) of rows, in 64 bits."""
    x = x.double()
    size = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x))
    top = size.amax(-1, keepdim=True)
    m, e = torch.frexp(top / 448.0)                     # (0.5 only where top is 448 times a power of two)
    e = (e - (m == 0.5).to(e.dtype)).clamp(min=-64)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    z = x * pow2(-e)
    step = pow2(torch.frexp(z.abs().clamp(2.0 ** -6, 448.0))[1] - 4)
    code = (torch.round(z / step) * step).clamp(-448.0, 448.0)
    return torch.where(x.isnan(), x, code), e[..., 0]


class Cache:
    """A paged cache, its pages in a random order.  `outside`: heads outside the tokens, or inside."""

    def __init__(self, gen, batch, max_keys, heads, d, page, *, spare=3, outside=True, fill=0xFF, device="cuda"):
        per = -(-max_keys // page)
        pages = batch * per + spare
        order = torch.randperm(pages, generator=gen, device=device)[:batch * per]
        self.block_table = order.view(batch, per).to(torch.int32)
        shape = (pages, heads, page, d) if outside else (pages, page, heads, d)

        def store():   # what was never written: NaN codes
            t = torch.full(shape, fill, dtype=torch.uint8, device=device).view(E4M3)
            return t.transpose(1, 2) if outside else t

        self.k, self.v = store(), store()
        self.scales = torch.zeros((pages, heads, page, 2), dtype=torch.uint8, device=device)
        self.page = page

    def args(self):
        return self.k, self.v, self.scales, self.block_table

    def rows(self, b, keys):
        """Values of the first `keys` tokens in 64 bits: k, v [keys, heads, D], exponents [keys, heads, 2],
        and which were written (with a page that exists)."""
        at = torch.arange(keys, device=self.k.device)
        page, off = self.block_table[b].long()[at // self.page], at % self.page
        real = (page >= 0) & (page < self.k.shape[0])
        page = torch.where(real, page, torch.zeros_like(page))
        e = self.scales[page, :, off].long() - 127
        live = (e[..., 0] > -127) & real[:, None]
        out = []
        for i, t in enumerate((self.k, self.v)):
            x = t.view(torch.uint8)[page, off].view(E4M3).double() * pow2(e[..., i])[..., None]
            out.append(torch.where(live[..., None], x, torch.zeros_like(x)))
        return out[0], out[1], e, live


def ancestors(parents, t):
    """sees [T, T] of one request."""
    sees = torch.zeros((t, t), dtype=torch.bool)
    for i in range(t):
        at = i
        while True:
            sees[i, at] = True
            up = at - 1 if parents is None else int(parents[at])
            if up < 0 or up >= at:
                break
            at = up
    return sees


class TreeReference:
    """Tree attention in 64 bits: out, lse of the rows that are written, with bounds; `written` says
    which [B, T]."""

    def __init__(self, q, cache, kv_lengths, *, parents=None, draft_lengths=None, scale=None, u):
        b, t, h, d = q.shape
        hkv = cache.k.shape[2]
        group = h // hkv
        scale = 1.0 / math.sqrt(d) if scale is None else scale
        like = dict(dtype=torch.float64, device=q.device)
        self.out, self.out_tol = torch.zeros((b, t, h, d), **like), torch.zeros((b, t, h, d), **like)
        self.lse, self.lse_tol = torch.zeros((b, h, t), **like), torch.zeros((b, h, t), **like)
        self.written = torch.zeros((b, t), dtype=torch.bool, device=q.device)
        most = cache.block_table.shape[1] * cache.page
        for i in range(b):
            n = max(0, min(int(kv_lengths[i]), most))
            drafts = min(t if draft_lengths is None else max(0, min(int(draft_lengths[i]), t)), n)
            if drafts == 0:
                continue
            self.written[i, :drafts] = True
            up = None if parents is None else (parents if parents.dim() == 1 else parents[i]).tolist()
            sees = torch.ones((drafts, n), dtype=torch.bool)
            sees[:, n - drafts:] = ancestors(up, drafts)
            k, v, e, live = cache.rows(i, n)
            for g in range(hkv):
                keep = sees.to(q.device) & live[None, :, g]
                qg = q[i, :drafts, g * group:(g + 1) * group].double().transpose(0, 1)   # [G, drafts, D]
                kg, vg, ev = k[:, g], v[:, g], e[:, g, 1].double()
                s = (qg @ kg.T * scale).masked_fill(~keep, -math.inf)
                lse = torch.logsumexp(s, dim=2)
                has = lse > -math.inf
                base = torch.where(has, lse, torch.zeros_like(lse))[..., None]
                p = torch.exp(s - base)
                o = p @ vg
                # A score: D + 2 roundings of its absolute sum, the small elements of a query that is
                # held as fp16, and the exponent's argument, which has the value's exponent added.
                s_abs = qg.abs() @ kg.abs().T * scale
                # (In the type's half steps: at most 2^-25 of an element held at 2^14 and more.)
                low = 2.0 ** -39 * qg.abs().amax(2, keepdim=True) * kg.abs().sum(1) * scale
                off = F32 * ((d + 2) * s_abs + 4 * (s_abs + base.abs() + 4) + 2 * (ev.abs() + 16)) + low
                off = torch.where(keep, off, torch.zeros_like(off)).amax(2, keepdim=True)
                share = 2.0 ** -11 + 2 * off + 2.0 ** -21 + n * F32
                # A probability is held as w = p 2^f, with f its value's exponent, or (more than 64 rows) the
                # largest of the 16 tokens it lies among.  The largest w of a row is held at 2^4 at least,
                # and those below fp16's normal numbers are off by 2^-25: by 2^-29 of the largest.  The
                # value that w meets is v 2^-f.
                f = ev
                if t * group > 64:
                    fill = torch.where(live[:, g], ev, torch.full_like(ev, -1000.0))
                    fill = torch.nn.functional.pad(fill, (0, -n % 16), value=-1000.0)
                    f = fill.view(-1, 16).amax(1).repeat_interleave(16)[:n].clamp(min=-64)
                weight = torch.where(keep, p * pow2(f), torch.zeros_like(p))
                tiny = 2.0 ** -29 * weight.amax(2, keepdim=True) * (
                    keep.double() @ (vg * pow2(-f)[:, None]).abs())
                tol = u * o.abs() + (1 + u) * share * (p @ vg.abs()) + tiny + grain(u)
                rows = slice(g * group, (g + 1) * group)
                self.out[i, :drafts, rows], self.out_tol[i, :drafts, rows] = o.transpose(0, 1), tol.transpose(0, 1)
                self.lse[i, rows, :drafts] = lse
                self.lse_tol[i, rows, :drafts] = (off + 2.0 ** -21 + n * F32)[..., 0] + 4 * F32 * base[..., 0].abs()
