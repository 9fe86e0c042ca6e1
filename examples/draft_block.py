"""A block of a text decoder that checks trees of drafted tokens, from the library's operators end to end:

    h        = layer norm of x
    q, k, v  = conv1x1(h)                      the new tokens' queries, keys and values, fused
    q, k     = norm and rotation of each head, at each token's place
    k, v     quantised into the request's pages, behind what lies there
    y        = x + conv1x1(attention of q to the pages, each draft to its ancestors)

Tokens are a map of one row, [requests, 1, tokens, channels], so the projections are the library's
convolutions.  `accept` writes the branch that a model keeps over the drafts' place in the pages.

    python examples/draft_block.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import transposed_conv_implicit_gb300 as cg  # noqa: E402
from examples.text_block import angle_tables  # noqa: E402


class DraftBlock:
    """Buffers, pages, workspace and packed weights for `requests` of up to `max_tokens` tokens and
    `drafts` new ones a call; random weights."""

    def __init__(self, requests, drafts, max_tokens, channels, heads, kv_heads, *, page=64,
                 dtype=torch.bfloat16, device="cuda:0", seed=0):
        gen = torch.Generator().manual_seed(seed)
        d = channels // heads
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, d
        self.drafts = drafts

        def filt(c_in, c_out):
            f = torch.randn((1, 1, c_in, c_out), generator=gen) * c_in ** -0.5
            return f.to(dtype).to(device)

        def empty(*shape):
            return torch.empty(shape, dtype=dtype, device=device)

        self.filters = {"qkv": filt(channels, (heads + 2 * kv_heads) * d), "out": filt(channels, channels)}
        self.packed = {n: cg.conv2d_pack_filter(f, filter_is_fcrs=False) for n, f in self.filters.items()}
        self.norm_weight = torch.ones(channels, dtype=dtype, device=device)
        self.norm_bias = torch.zeros(channels, dtype=dtype, device=device)
        self.q_weight, self.k_weight = (torch.ones(d, dtype=dtype, device=device) for _ in range(2))
        self.cos, self.sin = angle_tables(max_tokens, d // 8 * 8, device)
        self.normed, self.attended = empty(requests, 1, drafts, channels), empty(requests, 1, drafts, channels)
        self.qkv = empty(requests, 1, drafts, (heads + 2 * kv_heads) * d)
        # The pages, a head's tokens side by side; the scales' zeros say that they are empty.
        per = -(-max_tokens // page)
        shape = (requests * per, kv_heads, page, d)
        self.k_cache, self.v_cache = (
            torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn).transpose(1, 2)
            for _ in range(2))
        self.scales = torch.zeros((requests * per, kv_heads, page, 2), dtype=torch.uint8, device=device)
        self.block_table = torch.randperm(requests * per, generator=gen).view(requests, per).to(
            torch.int32).to(device)
        # One workspace: the block's calls run one after another on one stream.
        self.workspace = cg.new_workspace(cg.tree_attention_workspace_size(
            requests, heads, kv_heads, drafts, per * page, d), device)

    def _project(self, x, name, out, source=None):
        return cg.conv2d_fwd_packed(x, self.packed[name], out, r=1, s=1, has_residual=source is not None,
                                    source=source, beta=1.0 if source is not None else 0.0,
                                    workspace=self.workspace)

    def split(self, qkv):
        """q, k and v of the fused projection, as views."""
        n, _, t, _ = qkv.shape
        rows = qkv.view(n, t, self.heads + 2 * self.kv_heads, self.head_dim)
        h, hkv = self.heads, self.kv_heads
        return rows[:, :, :h], rows[:, :, h:h + hkv], rows[:, :, h + hkv:]

    def _pages(self):
        return self.k_cache, self.v_cache, self.scales, self.block_table

    def __call__(self, x, out, starts, positions, *, parents=None):
        """out = the block of x (both [requests, drafts, channels]); starts int32 [requests]: tokens
        that lie in the pages already; positions int32 [requests, drafts]: each draft's place in the
        text (siblings share one); parents as cg.tree_attention_fwd's.  Returns out."""
        n, t, c = x.shape
        cg.layer_norm_fwd(x, self.norm_weight, self.norm_bias, self.normed.view(n, t, c))
        q, k, v = self.split(self._project(self.normed, "qkv", self.qkv))
        cg.qk_norm_rope_fwd(q, k, self.q_weight, self.k_weight, q, k, cos=self.cos, sin=self.sin,
                            q_positions=positions, k_positions=positions)
        cg.kv_cache_write(k, v, *self._pages(), starts)
        cg.tree_attention_fwd(q, *self._pages(), starts + t, self.attended.view(n, t, self.heads, self.head_dim),
                              parents=parents, workspace=self.workspace)
        return self._project(self.attended, "out", out.view(n, 1, t, c), source=x.view(n, 1, t, c)).view(n, t, c)

    def accept(self, starts, kept, lengths):
        """Writes the drafts kept[b][:lengths[b]] (of the last call, in the text's order) as the tokens
        from starts[b] on."""
        _, k, v = self.split(self.qkv)
        index = kept.long()[:, :, None, None].expand(-1, -1, self.kv_heads, self.head_dim)
        cg.kv_cache_write(k.gather(1, index), v.gather(1, index), *self._pages(), starts, lengths=lengths)


def main():
    requests, drafts, tokens, channels, heads, kv_heads = 32, 7, 8192, 4096, 32, 8
    block = DraftBlock(requests, drafts, tokens, channels, heads, kv_heads)
    gen = torch.Generator().manual_seed(1)
    x = torch.randn((requests, drafts, channels), generator=gen).bfloat16().cuda()
    starts = torch.full((requests,), tokens - drafts, dtype=torch.int32).cuda()
    parents = torch.tensor([-1, 0, 0, 1, 1, 2, 2], dtype=torch.int32).cuda()
    depth = torch.tensor([0, 1, 1, 2, 2, 2, 2], dtype=torch.int32).cuda()
    block.scales.fill_(127)       # (contexts of zeros)
    out = torch.empty_like(x)

    def step():
        block(x, out, starts, starts[:, None] + depth, parents=parents)

    for _ in range(5):
        step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    steps = 100
    begin.record()
    for _ in range(steps):
        step()
    end.record()
    status, _ = cg.conv_check_device_status(block.workspace)
    print("%d requests of %d tokens, trees of %d drafts, %d channels, %d/%d heads: %.1f us a step (%s)"
          % (requests, tokens, drafts, channels, heads, kv_heads, begin.elapsed_time(end) * 1e3 / steps,
             cg.conv_status_string(status)))


if __name__ == "__main__":
    main()
