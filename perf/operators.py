"""The attention operators' measured cases: cross attention to an encoder's states
(forward, forward + backward, single tokens) and the per-head norm of queries and
keys with the position rotation (forward, backward).

Each case can run in its plain form (elementary torch operations in 32 bits) or
through the library (`own`), on the same inputs; `exact` gives the definition in
64 bits.  Layouts: q [B, Lq, H, D], k and v [B, Lk, Hkv, D] as views of the fused
key/value projection [B, Lk, 2, Hkv, D]; lse and all weight gradients are fp32.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # A denoiser's 64 x 64 map (16 images, 320 channels = 8 heads of 40) reads captions
        # of up to 77 tokens: the ordinary inference call, bound by memory.
        dict(name="fwd_map64_text", op="attn", dir="fwd", dtype="bf16", B=16, Lq=4096, Lk=77, H=8,
             Hkv=8, D=40, mask="lengths"),
        # A 128 x 128 map against 4096 encoder states: the largest call, bound by the products.
        dict(name="fwd_map128_long", op="attn", dir="fwd", dtype="bf16", B=2, Lq=16384, Lk=4096, H=16,
             Hkv=16, D=128, mask="none"),
        # Text reading interleaved images: each query sees its own image's states only, the
        # queries before the first image none; shared key heads, odd lengths.
        dict(name="fwd_interleaved_odd", op="attn", dir="fwd", dtype="f16", B=3, Lq=1021, Lk=1531, H=12,
             Hkv=4, D=80, mask="rows"),
        # One token of one request against a short caption: latency alone.
        dict(name="token_one", op="attn", dir="fwd", dtype="bf16", B=1, Lq=1, Lk=77, H=8, Hkv=8, D=64,
             mask="none"),
        # One token for each of 64 requests against up to 4096 cached states, 4 query heads to
        # a key head: serving, bound by reading the cache.
        dict(name="token_serve", op="attn", dir="fwd", dtype="bf16", B=64, Lq=1, Lk=4096, H=32, Hkv=8,
             D=128, mask="lengths"),
        # The training step of the first case.
        dict(name="train_map64_text", op="attn", dir="train", dtype="bf16", B=16, Lq=4096, Lk=77, H=8,
             Hkv=8, D=40, mask="lengths"),
        # Training on long states: bound by the products.
        dict(name="train_long", op="attn", dir="train", dtype="bf16", B=2, Lq=8192, Lk=2048, H=16,
             Hkv=16, D=128, mask="none"),
        # Training with the interleaved mask, shared key heads and odd lengths.
        dict(name="train_interleaved_odd", op="attn", dir="train", dtype="f16", B=2, Lq=1021, Lk=523,
             H=12, Hkv=4, D=80, mask="rows"),
        # The queries of one new token for 8 requests (the keys are in the cache): latency alone.
        dict(name="norm_token", op="norm", dir="fwd", dtype="bf16", B=8, Lq=1, Lk=0, H=32, Hkv=8, D=128,
             rot=128, pairs="half"),
        # Queries and keys of a long sequence, as in prompt processing: bound by memory.
        dict(name="norm_long", op="norm", dir="fwd", dtype="bf16", B=8, Lq=8192, Lk=4096, H=16, Hkv=16,
             D=128, rot=128, pairs="half"),
        # The 64 x 64 map's queries (8 heads of 40, 32 of them rotated, neighbouring pairs) and the
        # caption's keys, backward.
        dict(name="norm_bwd_map64", op="norm", dir="bwd", dtype="f16", B=16, Lq=4096, Lk=77, H=8, Hkv=8,
             D=40, rot=32, pairs="adjacent"),
        # The long case, backward.
        dict(name="norm_bwd_long", op="norm", dir="bwd", dtype="bf16", B=8, Lq=4096, Lk=2048, H=16,
             Hkv=4, D=128, rot=128, pairs="half"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm; 3072 is left to its neighbour."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v + 1 if v == 3072 else v


def draw(rng):
    kind = rng.choice(["fwd", "token", "train", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "f16"])
    d = rng.choice([16, 24, 32, 40, 56, 64, 72, 80, 96, 104, 120, 128])
    while True:
        hkv = rng.choice([1, 2, 3, 4, 8, 16])
        h = hkv * rng.choice([1, 1, 2, 4, 5])
        b = _spread(rng, 1, 64)
        if kind == "token":
            lq, lk = rng.choice([1, 1, 1, 2, 5]), _spread(rng, 1, 16384)
            cost = b * lk * hkv * d / (64 * 4096 * 8 * 128)
        elif kind in ("fwd", "train"):
            lq, lk = _spread(rng, 1, 16384), _spread(rng, 1, 8192)
            most = 2 * 16 * (16384 * 4096 if kind == "fwd" else 8192 * 2048)
            cost = max(b * h * lq * lk / most, b * h * lq * d / (2 * 16384 * 16 * 128))
        else:
            lq, lk = _spread(rng, 1, 16384), rng.choice([0, _spread(rng, 1, 8192)])
            cost = b * (lq * h + lk * hkv) * d / (8 * (8192 * 16 + 4096 * 16) * 128)
        if cost <= 0.5 and 3072 not in (h * d, hkv * d):
            break
    if kind.startswith("norm"):
        rot = rng.choice([d, d, max(8, d // 16 * 8)])
        return dict(op="norm", dir=kind[5:], dtype=dtype, B=b, Lq=lq, Lk=lk, H=h, Hkv=hkv, D=d, rot=rot,
                    pairs=rng.choice(["half", "adjacent"]))
    mask = rng.choice(["none", "lengths"] if kind == "token" else ["none", "lengths", "lengths", "rows"])
    return dict(op="attn", dir="train" if kind == "train" else "fwd", dtype=dtype, B=b, Lq=lq, Lk=lk, H=h,
                Hkv=hkv, D=d, mask=mask)


# ------------------------------------------------------------------ the cases' masks
def _lengths(case):
    """Valid keys of each request: spread evenly over the upper half of [0, Lk], the full
    length first (a fixed set; the seed deals it out)."""
    b, lk = case["B"], case["Lk"]
    return [lk - (lk * i) // (2 * b) for i in range(b)]


SEGMENTS = 4


def _segments(length, extra):
    """Positions' segments: `extra` leading shares without one (-1), then SEGMENTS equal shares."""
    shares = SEGMENTS + extra
    return [i * shares // length - extra for i in range(length)]


def _pairs(case):
    """(query, key) pairs of one head that the mask leaves, over the batch."""
    if case["mask"] == "none":
        return case["B"] * case["Lq"] * case["Lk"]
    if case["mask"] == "lengths":
        return case["Lq"] * sum(_lengths(case))
    qs, ks = _segments(case["Lq"], 1), _segments(case["Lk"], 0)
    return case["B"] * sum(qs.count(s) * ks.count(s) for s in range(SEGMENTS))


# ------------------------------------------------------------------ inputs
def _prepare_attn(case, gen):
    dev, dt = "cuda", TYPES[case["dtype"]]
    b, lq, lk, h, hkv, d = (case[n] for n in ("B", "Lq", "Lk", "H", "Hkv", "D"))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev).to(dt)

    kv = normal(b, lk, 2, hkv, d)
    s = dict(case=case, q=normal(b, lq, h, d), k=kv[:, :, 0], v=kv[:, :, 1], kv_lengths=None, mask=None,
             scale=1.0 / math.sqrt(d), out=torch.empty((b, lq, h, d), dtype=dt, device=dev))
    if case["mask"] == "lengths":
        order = torch.randperm(b, generator=gen, device=dev)
        s["kv_lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)[order].contiguous()
    elif case["mask"] == "rows":
        qs = torch.tensor(_segments(lq, 1), device=dev)
        ks = torch.tensor(_segments(lk, 0), device=dev)
        s["mask"] = (qs[:, None] == ks[None, :]).expand(b, 1, lq, lk).contiguous()
    if case["dir"] == "train":
        s["dout"] = normal(b, lq, h, d)
        s["lse"] = torch.empty((b, h, lq), dtype=torch.float32, device=dev)
        s["dq"] = torch.empty_like(s["q"])
        s["dkv"] = torch.empty_like(kv)
    return s


def _prepare_norm(case, gen):
    dev, dt = "cuda", TYPES[case["dtype"]]
    b, lq, lk, h, hkv, d, rot = (case[n] for n in ("B", "Lq", "Lk", "H", "Hkv", "D", "rot"))
    most = max(lq, lk, 64) + 64
    angle = (torch.arange(most, device=dev, dtype=torch.float32)[:, None]
             * (10000.0 ** (-torch.arange(rot // 2, device=dev, dtype=torch.float32) / (rot // 2))))
    s = dict(case=case, cos=angle.cos(), sin=angle.sin(), adjacent=case["pairs"] == "adjacent")
    for name, length, heads in (("q", lq, h), ("k", lk, hkv)):
        if not length:
            s.update({name: None, name + "_weight": None, name + "_positions": None, name + "_out": None})
            continue
        s[name] = (1.7 * torch.randn((b, length, heads, d), generator=gen, device=dev)).to(dt)
        s[name + "_weight"] = (1.0 + 0.2 * torch.randn((d,), generator=gen, device=dev)).to(dt)
        first = torch.randint(0, 64, (b, 1), generator=gen, device=dev)
        s[name + "_positions"] = (first + torch.arange(length, device=dev)).to(torch.int32)
        if case["dir"] == "fwd":
            s[name + "_out"] = torch.empty_like(s[name])
        else:
            s["d" + name + "_out"] = torch.randn((b, length, heads, d), generator=gen, device=dev).to(dt)
            s["d" + name] = torch.empty_like(s[name])
            s["d" + name + "_weight"] = torch.empty((d,), dtype=torch.float32, device=dev)
    if case["dir"] == "bwd" and not lk:
        s.update(dk_out=None, dk=None, dk_weight=None)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (_prepare_attn if case["op"] == "attn" else _prepare_norm)(case, gen)


# ------------------------------------------------------------------ plain forms
def _plain_attn(s):
    case = s["case"]
    group = case["H"] // case["Hkv"]
    q = s["q"].float().transpose(1, 2)                                    # [B, H, Lq, D]
    k = s["k"].float().transpose(1, 2).repeat_interleave(group, dim=1)    # [B, H, Lk, D]
    v = s["v"].float().transpose(1, 2).repeat_interleave(group, dim=1)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    if s["kv_lengths"] is not None:
        keys = torch.arange(case["Lk"], device=x.device)
        keep = keys < s["kv_lengths"][:, None, None, None]
    else:
        keep = s["mask"]
    if keep is not None:
        x = x.masked_fill(~keep, -math.inf)
    top = x.amax(dim=3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    del x
    total = p.sum(dim=3, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.matmul(p, v)
    outs = {"out": out.transpose(1, 2).to(s["q"].dtype)}
    if case["dir"] == "fwd":
        return outs
    dout = s["dout"].float().transpose(1, 2)
    dp = torch.matmul(dout, v.transpose(2, 3))
    ds = p * (dp - (dout * out).sum(dim=3, keepdim=True)) * s["scale"]
    del dp
    dq = torch.matmul(ds, k)

    def shared(g):  # the gradient of a key head sums over the query heads that share it
        return g.reshape(case["B"], case["Hkv"], group, case["Lk"], case["D"]).sum(dim=2)

    dk, dv = shared(torch.matmul(ds.transpose(2, 3), q)), shared(torch.matmul(p.transpose(2, 3), dout))
    outs["lse"] = (torch.log(total) + top).squeeze(3)
    outs["dq"] = dq.transpose(1, 2).to(s["q"].dtype)
    outs["dkv"] = torch.stack((dk, dv), dim=1).permute(0, 3, 1, 2, 4).to(s["q"].dtype)
    return outs


def _halves(x, rot, adjacent):
    """The two members of each rotated pair and the rest."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if adjacent else (r[..., : rot // 2], r[..., rot // 2:])
    return a, b, x[..., rot:]


def _joined(a, b, rest, adjacent):
    r = torch.stack((a, b), dim=-1).flatten(-2) if adjacent else torch.cat((a, b), dim=-1)
    return torch.cat((r, rest), dim=-1)


def _plain_norm(s):
    case, outs = s["case"], {}
    rot, adj = case["rot"], s["adjacent"]
    for n in ("q", "k"):
        if s[n] is None:
            continue
        x, w = s[n].float(), s[n + "_weight"].float()
        at = s[n + "_positions"].long()
        cos, sin = s["cos"][at][:, :, None, :], s["sin"][at][:, :, None, :]
        r = torch.rsqrt((x * x).mean(dim=3, keepdim=True) + EPS)
        if case["dir"] == "fwd":
            a, b, rest = _halves(x * r * w, rot, adj)
            outs[n + "_out"] = _joined(a * cos - b * sin, b * cos + a * sin, rest, adj).to(s[n].dtype)
            continue
        a, b, rest = _halves(s["d" + n + "_out"].float(), rot, adj)
        g = _joined(a * cos + b * sin, b * cos - a * sin, rest, adj)
        xhat = x * r
        outs["d" + n + "_weight"] = (g * xhat).sum(dim=(0, 1, 2))
        g = g * w
        outs["d" + n] = (r * (g - xhat * (g * xhat).mean(dim=3, keepdim=True))).to(s[n].dtype)
    return outs


# ------------------------------------------------------------------ the library's calls
def _own_attn(s):
    import transposed_conv_implicit_gb300 as cg
    if "workspace" not in s:
        c = s["case"]
        s["workspace"] = cg.new_workspace(cg.cross_attention_workspace_size(
            c["B"], c["H"], c["Hkv"], c["Lq"], c["Lk"], c["D"], masked=s["mask"] is not None,
            backward=c["dir"] == "train"), s["q"].device)
    kw = dict(kv_lengths=s["kv_lengths"], mask=s["mask"], scale=s["scale"], workspace=s["workspace"])
    if s["case"]["dir"] == "fwd":
        cg.cross_attention_fwd(s["q"], s["k"], s["v"], s["out"], **kw)
        return {"out": s["out"]}
    dkv = s["dkv"]
    cg.cross_attention_fwd(s["q"], s["k"], s["v"], s["out"], lse=s["lse"], **kw)
    cg.cross_attention_bwd(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["dq"], dkv[:, :, 0],
                           dkv[:, :, 1], **kw)
    return {"out": s["out"], "lse": s["lse"], "dq": s["dq"], "dkv": dkv}


def _own_norm(s):
    import transposed_conv_implicit_gb300 as cg
    kw = dict(cos=s["cos"], sin=s["sin"], q_positions=s["q_positions"], k_positions=s["k_positions"],
              eps=EPS, adjacent_pairs=s["adjacent"])
    if s["case"]["dir"] == "fwd":
        cg.qk_norm_rope_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["q_out"], s["k_out"], **kw)
        return {n: s[n] for n in ("q_out", "k_out") if s[n] is not None}
    if "workspace" not in s:
        s["workspace"] = cg.new_workspace(cg.qk_norm_rope_workspace_size(s["case"]["D"]), s["q"].device)
    cg.qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["dq"],
                        s["dk"], s["dq_weight"], s["dk_weight"], workspace=s["workspace"], **kw)
    return {n: s[n] for n in ("dq", "dk", "dq_weight", "dk_weight") if s[n] is not None}


def run(state):
    if state["case"]["op"] == "attn":
        return _own_attn(state) if own else _plain_attn(state)
    return _own_norm(state) if own else _plain_norm(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    b, lq, lk, h, hkv, d = (case[n] for n in ("B", "Lq", "Lk", "H", "Hkv", "D"))
    if case["op"] == "norm":
        rows = b * (lq * h + lk * hkv)
        passes = 2 if case["dir"] == "fwd" else 3            # x in, y out; or x and dy in, dx out
        tables = 4 * case["rot"] * (max(lq, lk) + 64) + 4 * b * (lq + lk)
        return {"bytes": passes * rows * d * 2 + tables, "flops": rows * d * (8 if passes == 2 else 16)}
    keys = sum(_lengths(case)) if case["mask"] == "lengths" else b * lk
    q_bytes, kv_bytes = b * lq * h * d * 2, 2 * keys * hkv * d * 2
    mask = b * lq * lk if case["mask"] == "rows" else 4 * b
    flops = 4 * d * h * _pairs(case)
    if case["dir"] == "fwd":
        return {"bytes": 2 * q_bytes + kv_bytes + mask, "flops": flops}
    # A training step reads q, dout, k and v and writes out, lse, dq, dk and dv; 2 products
    # forward and 5 backward.
    return {"bytes": 4 * q_bytes + 2 * kv_bytes + 4 * b * h * lq + mask, "flops": flops * 7 // 2}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_attn(case, s):
    b, h, hkv, d = case["B"], case["H"], case["Hkv"], case["D"]
    lq, lk = case["Lq"], case["Lk"]
    train = case["dir"] == "train"
    like = dict(dtype=torch.float64, device="cuda")
    out = torch.zeros((b, lq, h, d), **like)
    lse = torch.full((b, h, lq), -math.inf, **like)
    dq = torch.zeros((b, lq, h, d), **like)
    dkv = torch.zeros((b, lk, 2, hkv, d), **like)
    step = max(1, (1 << 27) // max(1, lk))
    for i in range(b):
        n = lk if s["kv_lengths"] is None else int(s["kv_lengths"][i])
        if n == 0:
            continue
        for j in range(h):
            kj = j * hkv // h
            keys, values = s["k"][i, :n, kj].double(), s["v"][i, :n, kj].double()
            for at in range(0, lq, step):
                rows = slice(at, min(lq, at + step))
                q = s["q"][i, rows, j].double()
                score = (q @ keys.T) / math.sqrt(d)
                if s["mask"] is not None:
                    score[~s["mask"][i, 0, rows, :n]] = -math.inf
                norm = torch.logsumexp(score, dim=1)
                live = norm > -math.inf
                prob = torch.exp(score - torch.where(live, norm, torch.zeros_like(norm))[:, None])
                del score
                o = prob @ values
                out[i, rows, j] = o
                if not train:
                    continue
                lse[i, j, rows] = norm
                do = s["dout"][i, rows, j].double()
                grad = do @ values.T
                grad -= (do * o).sum(1)[:, None]
                grad *= prob
                dkv[i, :n, 1, kj] += prob.T @ do
                dq[i, rows, j] = grad @ keys / math.sqrt(d)
                dkv[i, :n, 0, kj] += grad.T @ q / math.sqrt(d)
    return {"out": out, "lse": lse, "dq": dq, "dkv": dkv} if train else {"out": out}


def _exact_norm(case, s):
    """Each pair (a, b) as the complex number a + ib, times e^{i angle}; the gradient from the
    Jacobian of x -> x / rms(x)."""
    outs, rot = {}, case["rot"]
    turn = torch.complex(s["cos"].double(), s["sin"].double())
    first = torch.arange(0, rot, 2, device="cuda") if s["adjacent"] else torch.arange(rot // 2, device="cuda")
    second = first + (1 if s["adjacent"] else rot // 2)
    for n in ("q", "k"):
        if s[n] is None:
            continue
        dx, dw = [], torch.zeros(case["D"], dtype=torch.float64, device="cuda")
        w = s[n + "_weight"].double()
        for i in range(case["B"]):
            x = s[n][i].double()
            phase = turn[s[n + "_positions"][i].long()][:, None]
            rms = torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
            y = x / rms * w if case["dir"] == "fwd" else s["d" + n + "_out"][i].double()
            z = torch.complex(y[..., first], y[..., second])
            z = z * phase if case["dir"] == "fwd" else z * phase.conj()
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            if case["dir"] == "bwd":
                dw += (y * x / rms).sum((0, 1))
                u = y * w
                y = u / rms - x * (u * x).sum(-1, keepdim=True) / (case["D"] * rms ** 3)
            dx.append(y)
        if case["dir"] == "fwd":
            outs[n + "_out"] = torch.stack(dx)
        else:
            outs["d" + n], outs["d" + n + "_weight"] = torch.stack(dx), dw
    return outs


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attn(case, s) if case["op"] == "attn" else _exact_norm(case, s)
