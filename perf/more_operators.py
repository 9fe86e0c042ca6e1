"""The decoder operators' measured cases: the layer norm (forward, training), the paged 8-bit cache
of keys and values (writing, reading back) and the attention of drafted tokens' trees to it.

Each case can run in its plain form (elementary torch operations in 32 bits) or through the
library (`own`), on the same inputs; `exact` gives the definition in 64 bits.

The cache: k_cache and v_cache e4m3 [pages, page_size, Hkv, D] (stored with the heads outside the
tokens), scales uint8 [pages, Hkv, page_size, 2], the exponents plus 127 of a row of k and of v;
block_table int32 [B, pages of a request].
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


def listed():
    return [
        # One decoding step's tokens of 8 requests: latency alone.
        dict(name="norm_token", op="norm", dir="fwd", dtype="bf16", rows=8, C=1280),
        # The pixels of 16 64 x 64 maps of 320 channels, in front of an attention's projections.
        dict(name="norm_map64", op="norm", dir="fwd", dtype="bf16", rows=65536, C=320),
        # The same maps in training: forward and backward with the weights' gradients.
        dict(name="norm_train_map64", op="norm", dir="train", dtype="f16", rows=65536, C=320),
        # A long batch of wide rows in training; an odd number of them.
        dict(name="norm_train_wide", op="norm", dir="train", dtype="bf16", rows=16381, C=4096),
        # One new token for each of 64 requests goes into the cache: latency alone.
        dict(name="write_token", op="write", dtype="bf16", B=64, L=1, Hkv=8, D=128, keys=4096, page=64,
             ragged=True),
        # Prompts of up to 4096 tokens go into the cache: bound by memory.
        dict(name="write_prompt", op="write", dtype="bf16", B=16, L=4096, Hkv=8, D=128, keys=4096, page=64,
             ragged=True),
        # Cached states come back in 16 bits (for a model that wants them dense); odd lengths.
        dict(name="read_odd", op="read", dtype="f16", B=12, L=3001, Hkv=4, D=80, keys=4096, page=48,
             ragged=True),
        # One token of one request, a short context: latency alone.
        dict(name="tree_one", op="tree", dtype="bf16", B=1, T=1, H=8, Hkv=8, D=64, keys=77, page=16,
             ragged=False),
        # One token for each of 64 requests against up to 4096 keys, 4 query heads to a key head:
        # serving without drafts, bound by reading the cache.
        dict(name="tree_token_serve", op="tree", dtype="bf16", B=64, T=1, H=32, Hkv=8, D=128, keys=4096,
             page=64, ragged=True),
        # Small trees of up to 7 drafts, long contexts: still bound by the cache.
        dict(name="tree_draft", op="tree", dtype="bf16", B=32, T=7, H=32, Hkv=8, D=128, keys=8192, page=64,
             ragged=True),
        # Wide trees of 64 drafts: 256 rows to a key head, bound by the products.
        dict(name="tree_wide", op="tree", dtype="bf16", B=16, T=64, H=32, Hkv=8, D=128, keys=8192, page=64,
             ragged=False),
        # Odd sizes throughout.
        dict(name="tree_odd", op="tree", dtype="f16", B=5, T=29, H=12, Hkv=4, D=80, keys=2531, page=48,
             ragged=True),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["norm", "norm", "write", "read", "tree", "tree", "tree"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "norm":
        while True:
            c = _spread(rng, 3, 8192)
            if rng.random() < 0.7:
                c = max(8, c // 8 * 8)
            rows = _spread(rng, 1, 131072)
            if rows * c <= 16381 * 4096:
                return dict(op=op, dir=rng.choice(["fwd", "train"]), dtype=dtype, rows=rows, C=c)
    page = rng.choice([16, 32, 48, 64, 128, 256, 1024])
    d = rng.choice([16, 32, 48, 64, 80, 96, 112, 128])
    hkv, ragged = rng.choice([1, 2, 3, 4, 8, 16]), rng.random() < 0.7
    while True:
        b, keys = _spread(rng, 1, 64), _spread(rng, 1, 32768)
        if op == "tree":
            t = min(keys, rng.choice([1, 1, 2, 3, 5, 8, 13, 24, 47, 64, 100, 256]))
            h = hkv * rng.choice([1, 2, 3, 4, 5, 8])
            cost = max(b * keys * hkv * d / (64 * 4096 * 8 * 128), b * keys * t * h * d / (16 * 8192 * 64 * 32 * 128))
            if cost <= 0.5:
                return dict(op=op, dtype=dtype, B=b, T=t, H=h, Hkv=hkv, D=d, keys=keys, page=page, ragged=ragged)
        elif b * keys * hkv * d <= 16 * 4096 * 8 * 128:
            length = min(keys, rng.choice([1, _spread(rng, 1, 32768)]))
            return dict(op=op, dtype=dtype, B=b, L=length, Hkv=hkv, D=d, keys=keys, page=page, ragged=ragged)


# ------------------------------------------------------------------ a case's lengths
def _lengths(case):
    """(keys, tokens) of each request: all of them, or (ragged) spread over the upper half of the
    range, the full ones first.  A fixed set; the seed deals it out."""
    b, most = case["B"], case["T"] if case["op"] == "tree" else case["L"]
    if not case["ragged"]:
        return [(case["keys"], most)] * b
    tokens = [most - (most * i) // (2 * b) for i in range(b)]
    return [(max(t, case["keys"] - (case["keys"] * i) // (2 * b)), t) for i, t in enumerate(tokens)]


# ------------------------------------------------------------------ inputs
def _quantise(x):
    """e4m3 codes and exponents of rows (the last dimension), in 32 bits: the scale is the smallest
    power of two that brings the largest finite element to 448 or below (1 for rows of zeros)."""
    x = x.float()
    top = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(dim=-1)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, e - 9 + (m > 0.875).to(e.dtype), torch.zeros_like(e)).clamp(min=-126)
    code = torch.ldexp(x, -e[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return code, (e + 127).to(torch.uint8)


def _empty_cache(case, gen):
    """Pages for all requests in a random order, and some more, and the table."""
    per = -(-case["keys"] // case["page"])
    used = case["B"] * per
    order = torch.randperm(used + 5, generator=gen, device="cuda")[:used]
    shape = (used + 5, case["Hkv"], case["page"], case["D"])
    cache = [torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).transpose(1, 2)
             for _ in range(2)]
    scales = torch.full((used + 5, case["Hkv"], case["page"], 2), 127, dtype=torch.uint8, device="cuda")
    return dict(k_cache=cache[0], v_cache=cache[1], scales=scales,
                block_table=order.view(case["B"], per).to(torch.int32))


def _fill(s, gen):
    """Values of a model in every page: rows of differing size, some channels larger."""
    pages, page, hkv, d = s["k_cache"].shape
    at = 0
    step = max(1, (1 << 26) // (page * hkv * d))
    loud = 1.0 + 3.0 * (torch.rand((2, hkv, 1, d), generator=gen, device="cuda") > 0.97)
    while at < pages:
        n = min(step, pages - at)
        for i, name in enumerate(("k_cache", "v_cache")):
            x = torch.randn((n, hkv, page, d), generator=gen, device="cuda") * loud[i]
            x *= torch.exp(0.5 * torch.randn((n, hkv, page, 1), generator=gen, device="cuda"))
            code, e = _quantise(x)
            s[name].transpose(1, 2)[at : at + n].view(torch.uint8).copy_(code.view(torch.uint8))
            s["scales"][at : at + n, :, :, i] = e
        at += n


def _trees(case, gen):
    """A random parent for each draft (an earlier draft, or -1: the context), and who sees whom."""
    b, t = case["B"], case["T"]
    index = torch.arange(t, device="cuda")
    parents = (torch.rand((b, t), generator=gen, device="cuda") * (index + 1)).long() - 1
    sees = torch.zeros((b, t, t), dtype=torch.bool, device="cuda")
    at = index.expand(b, t).clone()
    while bool((at >= 0).any()):
        sees |= (index == at[..., None]) & (at >= 0)[..., None]
        at = torch.where(at >= 0, parents.gather(1, at.clamp(min=0)), at)
    return parents.to(torch.int32), sees


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] == "norm":
        rows, c = case["rows"], case["C"]
        s = dict(case=case, x=(1.7 * normal(rows, c) + 0.5 * normal(c)).to(dt),
                 y=torch.empty((rows, c), dtype=dt, device="cuda"), weight=(1.0 + 0.2 * normal(c)).to(dt),
                 bias=(0.1 * normal(c)).to(dt))
        if case["dir"] == "train":
            s["dy"], s["dx"] = normal(rows, c).to(dt), torch.empty((rows, c), dtype=dt, device="cuda")
            s.update({n: torch.empty(rows, dtype=torch.float32, device="cuda") for n in ("mean", "rstd")})
            s.update({n: torch.empty(c, dtype=torch.float32, device="cuda") for n in ("dweight", "dbias")})
        return s
    s = dict(case=case, **_empty_cache(case, gen))
    deal = torch.randperm(case["B"], generator=gen, device="cuda")
    sizes = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")[deal]
    s["kv_lengths"], s["lengths"] = sizes[:, 0].contiguous(), sizes[:, 1].contiguous()
    s["starts"] = s["kv_lengths"] - s["lengths"]
    if case["op"] == "write":
        kv = normal(case["B"], case["L"], 2, case["Hkv"], case["D"])
        kv *= torch.exp(0.5 * normal(case["B"], case["L"], 2, case["Hkv"], 1))
        kv = kv.to(dt)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        return s
    _fill(s, gen)
    if case["op"] == "read":
        shape = (case["B"], case["L"], case["Hkv"], case["D"])
        s["k"], s["v"] = (torch.zeros(shape, dtype=dt, device="cuda") for _ in range(2))
        return s
    shape = (case["B"], case["T"], case["H"], case["D"])
    s["q"], s["out"] = normal(*shape).to(dt), torch.zeros(shape, dtype=dt, device="cuda")
    s["parents"], s["sees"] = _trees(case, gen)
    s["scale"] = 1.0 / math.sqrt(case["D"])
    return s


# ------------------------------------------------------------------ plain forms
def _plain_norm(s):
    x, w = s["x"].float(), s["weight"].float()
    mean = x.mean(dim=1, keepdim=True)
    centred = x - mean
    rstd = torch.rsqrt((centred * centred).mean(dim=1, keepdim=True) + EPS)
    xhat = centred * rstd
    outs = {"y": (xhat * w + s["bias"].float()).to(s["x"].dtype)}
    if s["case"]["dir"] == "fwd":
        return outs
    dy = s["dy"].float()
    g = dy * w
    dx = rstd * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
    return dict(outs, mean=mean[:, 0], rstd=rstd[:, 0], dx=dx.to(s["x"].dtype), dweight=(dy * xhat).sum(dim=0),
                dbias=dy.sum(dim=0))


def _places(s, length):
    """(page, offset) [B, length] of the requests' tokens from `starts` on, and which there are."""
    i = torch.arange(length, device="cuda")
    there = i < s["lengths"][:, None]
    at = torch.where(there, s["starts"][:, None] + i, 0).long()
    page = s["case"]["page"]
    return s["block_table"].gather(1, at // page).long(), at % page, there


def _plain_write(s):
    pages, offsets, there = _places(s, s["case"]["L"])
    pages, offsets = pages[there], offsets[there]
    for i, (x, name) in enumerate(((s["k"], "k_cache"), (s["v"], "v_cache"))):
        code, e = _quantise(x[there])
        s[name].view(torch.uint8)[pages, offsets] = code.view(torch.uint8)
        s["scales"][..., i].transpose(1, 2)[pages, offsets] = e
    return {n: s[n] for n in ("k_cache", "v_cache", "scales")}


def _rows(s, name, i, pages, offsets):
    """Rows of the cache as 32-bit numbers."""
    code = s[name].view(torch.uint8)[pages, offsets].view(torch.float8_e4m3fn).float()
    e = s["scales"][..., i].transpose(1, 2)[pages, offsets].int() - 127
    return torch.ldexp(code, e[..., None])


def _plain_read(s):
    pages, offsets, there = _places(s, s["case"]["L"])
    for i, n in enumerate(("k", "v")):
        x = _rows(s, n + "_cache", i, pages, offsets)
        s[n].copy_(torch.where(there[..., None, None], x, 0.0))
    return {"k": s["k"], "v": s["v"]}


def _plain_tree(s):
    case = s["case"]
    b, t, hkv, d, most = case["B"], case["T"], case["Hkv"], case["D"], case["keys"]
    group = case["H"] // hkv
    key = torch.arange(most, device="cuda")
    pages, offsets = s["block_table"].long()[:, key // case["page"]], (key % case["page"]).expand(b, most)
    q = s["q"].float().view(b, t, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * group, d)
    x = torch.matmul(q, _rows(s, "k_cache", 0, pages, offsets).permute(0, 2, 3, 1)) * s["scale"]
    # A draft sees the context, and of the drafts those that `sees` says.
    draft = key - s["starts"][:, None]
    there = (draft >= 0) & (key < s["kv_lengths"][:, None])
    seen = s["sees"].gather(2, draft.clamp(0, t - 1)[:, None].expand(b, t, most)) & there[:, None]
    seen = (seen | (draft < 0)[:, None]) & (torch.arange(t, device="cuda") < s["lengths"][:, None])[..., None]
    seen = seen[:, None, :, None].expand(b, 1, t, group, most).reshape(b, 1, t * group, most)
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(dim=3, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    del x
    total = p.sum(dim=3, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.matmul(p, _rows(s, "v_cache", 1, pages, offsets).permute(0, 2, 1, 3))
    out = out.view(b, hkv, t, group, d).permute(0, 2, 1, 3, 4).reshape(b, t, hkv * group, d)
    return {"out": out.to(s["q"].dtype)}


# ------------------------------------------------------------------ the library's calls
def _own_norm(s):
    import transposed_conv_implicit_gb300 as cg
    if s["case"]["dir"] == "fwd":
        return {"y": cg.layer_norm_fwd(s["x"], s["weight"], s["bias"], s["y"], eps=EPS)}
    if "workspace" not in s:
        s["workspace"] = cg.new_workspace(cg.layer_norm_workspace_size(s["case"]["C"]), s["x"].device)
    cg.layer_norm_fwd(s["x"], s["weight"], s["bias"], s["y"], mean=s["mean"], rstd=s["rstd"], eps=EPS)
    cg.layer_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                      workspace=s["workspace"])
    return {n: s[n] for n in ("y", "mean", "rstd", "dx", "dweight", "dbias")}


def _own_write(s):
    import transposed_conv_implicit_gb300 as cg
    cg.kv_cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["scales"], s["block_table"], s["starts"],
                      lengths=s["lengths"])
    return {n: s[n] for n in ("k_cache", "v_cache", "scales")}


def _own_read(s):
    import transposed_conv_implicit_gb300 as cg
    cg.kv_cache_read(s["k_cache"], s["v_cache"], s["scales"], s["block_table"], s["starts"], s["k"], s["v"],
                     lengths=s["lengths"])
    return {"k": s["k"], "v": s["v"]}


def _own_tree(s):
    import transposed_conv_implicit_gb300 as cg
    if "workspace" not in s:
        c = s["case"]
        s["workspace"] = cg.new_workspace(cg.tree_attention_workspace_size(
            c["B"], c["H"], c["Hkv"], c["T"], s["block_table"].shape[1] * c["page"], c["D"]), s["q"].device)
    cg.tree_attention_fwd(s["q"], s["k_cache"], s["v_cache"], s["scales"], s["block_table"], s["kv_lengths"],
                          s["out"], parents=s["parents"], draft_lengths=s["lengths"], scale=s["scale"],
                          workspace=s["workspace"])
    return {"out": s["out"]}


_PLAIN = {"norm": _plain_norm, "write": _plain_write, "read": _plain_read, "tree": _plain_tree}
_OWN = {"norm": _own_norm, "write": _own_write, "read": _own_read, "tree": _own_tree}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        rows, c = case["rows"], case["C"]
        if case["dir"] == "fwd":
            return {"bytes": 4 * rows * c + 4 * c, "flops": 8 * rows * c}
        # x and dy in, y and dx out, the statistics and the weights' gradients.
        return {"bytes": 8 * rows * c + 8 * rows + 12 * c, "flops": 22 * rows * c}
    b, hkv, d = case["B"], case["Hkv"], case["D"]
    sizes = _lengths(case)
    tables = 4 * b * -(-case["keys"] // case["page"]) + 8 * b
    if case["op"] != "tree":  # a row in 16 bits, and in 8 with its exponent; k and v
        rows = 2 * hkv * sum(t for _, t in sizes)
        return {"bytes": rows * (3 * d + 1) + tables, "flops": 3 * rows * d}
    t, h = case["T"], case["H"]
    # (A draft sees about as many others as the logarithm of their number: none are counted.)
    pairs = h * sum(n_t * (n - n_t) for n, n_t in sizes)
    return {"bytes": hkv * sum(n for n, _ in sizes) * (2 * d + 2) + 4 * h * d * sum(n_t for _, n_t in sizes)
            + tables + 4 * b * t, "flops": 4 * d * pairs + 4 * d * h * sum(n_t for _, n_t in sizes)}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_norm(case, s):
    x, w = s["x"].double(), s["weight"].double()
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    std = torch.sqrt(var + EPS)
    y = (x - mean) / std * w + s["bias"].double()
    if case["dir"] == "fwd":
        return {"y": y}
    # The gradient through the Jacobian of x -> (x - mean) / std.
    dy, c = s["dy"].double(), case["C"]
    u = dy * w
    along = (u * (x - mean)).sum(1, keepdim=True)
    dx = (u - u.sum(1, keepdim=True) / c) / std - (x - mean) * along / (c * std ** 3)
    return {"y": y, "mean": mean[:, 0], "rstd": 1 / std[:, 0], "dx": dx,
            "dweight": torch.einsum("rc,rc->c", dy, (x - mean) / std), "dbias": dy.sum(0)}


def _exact_cache(case, s):
    """Token by token of a request: the place, the exponent by logarithms, the rounding by steps."""
    write, page = case["op"] == "write", case["page"]
    outs = {}
    scales = s["scales"].clone()
    for i, n in enumerate(("k", "v")):
        cache = s[n + "_cache"].double()
        dense = torch.zeros((case["B"], case["L"], case["Hkv"], case["D"]), dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            first, count = int(s["starts"][b]), int(s["lengths"][b])
            at = torch.arange(first, first + count, device="cuda")
            pages, offsets = s["block_table"][b].long()[torch.div(at, page, rounding_mode="floor")], at.remainder(page)
            if write:
                x = s[n][b, :count].double()
                top = x.abs().amax(-1, keepdim=True)
                # (16-bit numbers are 448 times a power of two, or 2^-12 of it away: the logarithm's own
                # error, which may lift a whole number, is taken off.)
                e = torch.where(top > 0, torch.ceil(torch.log2(top / 448.0) - 1e-9), torch.zeros_like(top))
                z = x / torch.exp2(e)
                step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
                cache[pages, offsets] = torch.round(z / step) * step
                scales[pages, :, offsets, i] = (e[..., 0] + 127).to(torch.uint8)
            else:
                dense[b, :count] = cache[pages, offsets] * torch.exp2(
                    scales[pages, :, offsets, i].double() - 127)[..., None]
        outs[n + "_cache" if write else n] = cache if write else dense
    return dict(outs, scales=None) if write else outs


def _exact_tree(case, s):
    """One draft after the other along its way to the root, one key head at a time."""
    b, t, h, hkv, d = (case[n] for n in ("B", "T", "H", "Hkv", "D"))
    group = h // hkv
    out = torch.zeros((b, t, h, d), dtype=torch.float64, device="cuda")
    for i in range(b):
        n, count = int(s["kv_lengths"][i]), int(s["lengths"][i])
        parents = s["parents"][i].tolist()
        at = torch.arange(n, device="cuda")
        pages, offsets = s["block_table"][i].long()[at // case["page"]], at % case["page"]
        hide = torch.zeros((count, n), dtype=torch.bool, device="cuda")
        way = []
        for j in range(count):
            way.append(([] if parents[j] < 0 else way[parents[j]]) + [j])
        left_out = [(j, n - count + k) for j in range(count) for k in set(range(count)) - set(way[j])]
        if left_out:
            rows, keys = torch.tensor(left_out, device="cuda").T
            hide[rows, keys] = True
        for g in range(hkv):
            k, v = (s[name][pages, offsets, g].double()
                    * torch.exp2(s["scales"][pages, g, offsets, m].double() - 127)[:, None]
                    for m, name in enumerate(("k_cache", "v_cache")))
            heads = slice(g * group, (g + 1) * group)
            score = torch.einsum("thd,nd->htn", s["q"][i, :count, heads].double(), k) / math.sqrt(d)
            score.masked_fill_(hide, -math.inf)
            out[i, :count, heads] = torch.einsum("htn,nd->thd", torch.softmax(score, dim=2), v)
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    return _exact_tree(case, s) if case["op"] == "tree" else _exact_cache(case, s)
