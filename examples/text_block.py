"""A text-conditioned block of an image model, from the library's operators end to end:

    q        = conv1x1(x)                      the map's pixels as queries
    k, v     = conv1x1(states)                 a caption's states, once per caption
    q, k     = norm and rotation of each head
    y        = x + conv1x1(cross attention of q to k, v)

The map stays NHWC throughout: [n, h, w, heads * d] is the query tensor [n, h * w, heads, d] as it
stands, so nothing is copied between the convolutions and the attention.  A denoising loop sets the
caption once (`set_states`) and calls the block for every step.

    python examples/text_block.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import transposed_conv_implicit_gb300 as cg  # noqa: E402


def angle_tables(positions, rot, device, base=10000.0):
    """cos and sin of position * base^(-2i / rot), i < rot / 2."""
    rate = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * rate
    return angle.cos().float().to(device), angle.sin().float().to(device)


class TextBlock:
    """Buffers, workspaces and packed weights for maps [n, h, w, channels] and captions of up to
    `states_len` states of `state_channels`; random weights."""

    def __init__(self, n, h, w, channels, heads, states_len, state_channels, *, dtype=torch.bfloat16,
                 device="cuda:0", seed=0):
        gen = torch.Generator().manual_seed(seed)

        def filt(c_in, c_out):
            f = torch.randn((1, 1, c_in, c_out), generator=gen) * c_in ** -0.5
            return f.to(dtype).to(device)

        def empty(*shape):
            return torch.empty(shape, dtype=dtype, device=device)

        d = channels // heads
        self.heads, self.head_dim = heads, d
        self.filters = {"q": filt(channels, channels), "kv": filt(state_channels, 2 * channels),
                        "out": filt(channels, channels)}
        self.packed = {name: cg.conv2d_pack_filter(f, filter_is_fcrs=False)
                       for name, f in self.filters.items()}
        self.q_weight = torch.ones(d, dtype=dtype, device=device)
        self.k_weight = torch.ones(d, dtype=dtype, device=device)
        self.cos, self.sin = angle_tables(max(h * w, states_len), d // 8 * 8, device)
        self.q = empty(n, h, w, channels)
        self.kv = empty(n, 1, states_len, 2 * channels)
        self.attended = empty(n, h, w, channels)
        self.lengths = torch.full((n,), states_len, dtype=torch.int32, device=device)
        # One workspace: the block's calls run one after another on one stream.
        self.workspace = cg.new_workspace(
            cg.cross_attention_workspace_size(n, heads, heads, h * w, states_len, d), device)

    def _project(self, x, name, out, source=None):
        return cg.conv2d_fwd_packed(x, self.packed[name], out, r=1, s=1, has_residual=source is not None,
                                    source=source, beta=1.0 if source is not None else 0.0,
                                    workspace=self.workspace)

    def _rows(self, x):
        n, h, w, c = x.shape
        return x.view(n, h * w, self.heads, self.head_dim)

    def set_states(self, states, lengths):
        """states [n, states_len, state_channels]; lengths int32 [n]: the states that count."""
        n, length, c = states.shape
        self._project(states.view(n, 1, length, c), "kv", self.kv)
        kv = self.kv.view(n, length, 2, self.heads, self.head_dim)
        self.k, self.v = kv[:, :, 0], kv[:, :, 1]
        cg.qk_norm_rope_fwd(None, self.k, None, self.k_weight, None, self.k, cos=self.cos, sin=self.sin)
        self.lengths.copy_(lengths)

    def __call__(self, x, out):
        """out = the block of x (both [n, h, w, channels]); returns out."""
        q = self._rows(self._project(x, "q", self.q))
        cg.qk_norm_rope_fwd(q, None, self.q_weight, None, q, None, cos=self.cos, sin=self.sin)
        cg.cross_attention_fwd(q, self.k, self.v, self._rows(self.attended), kv_lengths=self.lengths,
                               workspace=self.workspace)
        return self._project(self.attended, "out", out, source=x)


def main():
    n, h, w, channels, heads, length = 16, 64, 64, 320, 8, 77
    block = TextBlock(n, h, w, channels, heads, length, 768)
    gen = torch.Generator().manual_seed(1)
    x = torch.randn((n, h, w, channels), generator=gen).bfloat16().cuda()
    states = torch.randn((n, length, 768), generator=gen).bfloat16().cuda()
    lengths = torch.randint(2, length + 1, (n,), generator=gen).to(torch.int32)
    block.set_states(states, lengths)
    out = torch.empty_like(x)
    for _ in range(5):
        block(x, out)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    steps = 100
    begin.record()
    for _ in range(steps):
        block(x, out)
    end.record()
    status, _ = cg.conv_check_device_status(block.workspace)
    print("%d x %dx%d map, %d channels, %d heads, captions of up to %d states: %.1f us a step (%s)"
          % (n, h, w, channels, heads, length, begin.elapsed_time(end) * 1e3 / steps,
             cg.conv_status_string(status)))


if __name__ == "__main__":
    main()
