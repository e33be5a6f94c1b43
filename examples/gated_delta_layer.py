"""One gated delta-rule layer as a server runs it: packed prompts into slots of a state pool,
then one token a row.

    residual -> norm -> in-projection (4-bit) -> z | q k v | beta | dt
    q k v -> causal convolution -> gated delta rule -> norm, gated by z
    out-projection (4-bit) -> added to the residual, and the norm for the next block

Prompts of different lengths are packed on one axis and go through ``causal_conv1d`` and
``gated_delta_scan``, which leave both states in the pools; every further token goes through
``causal_conv1d_update`` and ``gated_delta_update``.  Weights and inputs are random.

    python examples/gated_delta_layer.py            # a small layer, checked against itself
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import depthwise_causal_conv1d_amd as dc  # noqa: E402
from examples.state_space_layer import quantize  # noqa: E402


class GatedDeltaLayer:
    def __init__(self, width, heads, value_size, groups, key_size, slots, group_size=64, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, generator=gen, device=device) * scale
        self.H, self.P, self.G, self.K, self.gs = heads, value_size, groups, key_size, group_size
        self.inner, self.keys = heads * value_size, groups * key_size
        self.channels = 2 * self.keys + self.inner                  # of the convolution: q | k | v
        # the row's end is padded so that rows start on 16 bytes
        self.row = -(-(self.inner + self.channels + 2 * heads) // 8) * 8
        self.w_in = quantize(normal(self.row, width, scale=width ** -0.5), group_size)
        self.w_out = quantize(normal(width, self.inner, scale=self.inner ** -0.5), group_size)
        self.conv_w = normal(self.channels, 4, scale=0.5).to(torch.bfloat16)
        self.conv_b = normal(self.channels, scale=0.1).to(torch.bfloat16)
        self.norm_w = (1 + normal(self.P, scale=0.1)).to(torch.bfloat16)
        self.block_w = (1 + normal(width, scale=0.1)).to(torch.bfloat16)
        self.A = -16 * torch.rand(heads, generator=gen, device=device)
        self.dt_bias = -5 + 2 * torch.rand(heads, generator=gen, device=device)
        self.conv_state = torch.zeros(slots, 3, self.channels, dtype=torch.bfloat16, device=device).permute(0, 2, 1)
        self.state = torch.zeros(slots, heads, value_size, key_size, device=device)
        self.rule = dict(dt_bias=self.dt_bias, dt_softplus=True, beta_sigmoid=True, qk_l2norm=True)

    def project(self, weights, x):
        q, scales, zeros = weights
        return dc.w4_matvec(x, q, scales, zeros, group_size=self.gs)

    def split(self, row):
        z, qkv, beta, dt, _ = row.split([self.inner, self.channels, self.H, self.H,
                                         row.shape[-1] - self.inner - self.channels - 2 * self.H], -1)
        return z.unflatten(-1, (self.H, self.P)), qkv, beta, dt

    def heads(self, qkv):
        q, k, v = qkv.split([self.keys, self.keys, self.inner], -1)
        return (q.unflatten(-1, (self.G, self.K)), k.unflatten(-1, (self.G, self.K)), v.unflatten(-1, (self.H, self.P)))

    def finish(self, y, z, residual):
        """The rule's output [..., H, P] into the residual stream; its norm for the next block."""
        y = dc.gated_rms_norm(y, z, self.norm_w)
        return dc.add_rms_norm(self.project(self.w_out, y.flatten(-2).flatten(0, -2)), residual, self.block_w)

    def prompts(self, x, residual, starts, slots):
        """x [tokens, width]: normed prompts packed one behind the other, sequence i from starts[i] to
        starts[i + 1] into slot slots[i] (int32 tensors on the device); residual likewise, advanced."""
        z, qkv, beta, dt = self.split(self.project(self.w_in, x)[None])
        qkv = dc.causal_conv1d(qkv.transpose(1, 2), self.conv_w, self.conv_b, "silu", conv_state=self.conv_state,
                               conv_state_indices=slots, seq_starts=starts).transpose(1, 2)
        y = dc.gated_delta_scan(*self.heads(qkv), dt, self.A, beta, state=self.state, state_indices=slots,
                                seq_starts=starts, **self.rule)
        return self.finish(y, z, residual)

    def token(self, x, residual, slots):
        """x [rows, width]: the next token of the sequences in slots (-1: no sequence)."""
        z, qkv, beta, dt = self.split(self.project(self.w_in, x))
        qkv = dc.causal_conv1d_update(qkv, self.conv_state, self.conv_w, self.conv_b, "silu", conv_state_indices=slots)
        y = dc.gated_delta_update(*self.heads(qkv), dt, self.A, beta, self.state, state_indices=slots, **self.rule)
        return self.finish(y, z, residual)


def run(width=512, heads=8, value_size=64, groups=4, key_size=64, lengths=(5, 130, 64, 1), more=6, seed=1):
    """Prompts, then `more` tokens of each; the same tokens as longer prompts must give the same
    outputs.  Returns the largest difference over the outputs' root mean square."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = len(lengths)
    residual = [torch.randn(length + more, width, generator=gen, device="cuda") for length in lengths]
    slots = torch.arange(n, device="cuda", dtype=torch.int32).flip(0).contiguous()

    def starts(extra):
        return torch.tensor([0] + [length + extra for length in lengths]).cumsum(0).to(torch.int32).cuda()

    def inputs(parts):
        """The block's normed input and its residual stream."""
        r = torch.cat(parts) if len(parts[0].shape) > 1 else torch.stack(parts)
        return dc.add_rms_norm(torch.zeros_like(r, dtype=torch.bfloat16), r, layer.block_w), r

    args = (width, heads, value_size, groups, key_size, n)
    layer, whole = GatedDeltaLayer(*args), GatedDeltaLayer(*args)
    want = whole.prompts(*inputs(residual), starts(more), slots).split([length + more for length in lengths])
    layer.prompts(*inputs([r[:length] for r, length in zip(residual, lengths)]), starts(0), slots)
    worst = 0.0
    for i in range(more):
        got = layer.token(*inputs([r[length + i] for r, length in zip(residual, lengths)]), slots)
        ref = torch.stack([w[length + i] for w, length in zip(want, lengths)])
        worst = max(worst, float((got.float() - ref.float()).abs().max() / ref.float().square().mean().sqrt()))
    return worst


if __name__ == "__main__":
    print(f"largest difference between stepping and prompting: {run():.4f} of the outputs' root mean square")
