"""One state-space layer as a server runs it: packed prompts into slots of a state
pool, then one token a row.

    in-projection (4-bit) -> z | x B C | dt
    x B C -> causal convolution -> recurrence, gated by z
    out-projection (4-bit)

Prompts of different lengths are packed on one axis and go through ``w4_matvec``,
``causal_conv1d`` and ``selective_scan``, which leave both states in the pools; every
further token is ``w4_matvec``, ``causal_conv1d_selective_update`` and ``w4_matvec``: three
launches.  Weights and inputs are random.

    python examples/state_space_layer.py            # a small layer, checked against itself
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import depthwise_causal_conv1d_amd as dc  # noqa: E402


def quantize(w, group_size):
    """Rows of w [N, K] to 4-bit codes with a scale and zero point a group of inputs."""
    N, K = w.shape
    groups = -(-K // group_size)  # the last may be shorter
    v = torch.nn.functional.pad(w, (0, groups * group_size - K)).view(N, groups, group_size)
    lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)   # a zero point is a code: zero is in the range
    scale = ((hi - lo) / 15).to(torch.bfloat16)
    step = torch.where(scale > 0, scale.float(), 1.0)            # (a group of zeros has none)
    zero = (-lo / step).round().clamp(0, 15)
    codes = (v / step[..., None] + zero[..., None]).round().clamp(0, 15)
    return (dc.w4_pack(codes.to(torch.uint8).view(N, -1)[:, :K].contiguous()), scale.t().contiguous(),
            zero.to(torch.uint8).t().contiguous())


class StateSpaceLayer:
    def __init__(self, width, heads, head_size, groups, state_size, slots, group_size=64, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, generator=gen, device=device) * scale
        self.H, self.P, self.G, self.K, self.gs = heads, head_size, groups, state_size, group_size
        self.inner, self.bc = heads * head_size, groups * state_size
        self.channels = self.inner + 2 * self.bc                    # of the convolution: x | B | C
        # dt's columns are padded so that a row of the projection starts on 16 bytes
        self.row = -(-(self.inner + self.channels + heads) // 8) * 8
        self.w_in = quantize(normal(self.row, width, scale=width ** -0.5), group_size)
        self.w_out = quantize(normal(width, self.inner, scale=self.inner ** -0.5), group_size)
        self.conv_w = normal(self.channels, 4, scale=0.5).to(torch.bfloat16)
        self.conv_b = normal(self.channels, scale=0.1).to(torch.bfloat16)
        self.A = -1 - 15 * torch.rand(heads, generator=gen, device=device)
        self.D = normal(heads)
        self.dt_bias = -5 + 2 * torch.rand(heads, generator=gen, device=device)
        self.conv_state = torch.zeros(slots, 3, self.channels, dtype=torch.bfloat16, device=device).permute(0, 2, 1)
        self.ssm_state = torch.zeros(slots, heads, head_size, state_size, device=device)
        self.workspace = dc.selective_update_workspace(slots, groups, device)

    def project(self, weights, x):
        q, scales, zeros = weights
        return dc.w4_matvec(x, q, scales, zeros, group_size=self.gs)

    def split(self, row):
        z, xbc, dt = row.split([self.inner, self.channels, row.shape[-1] - self.inner - self.channels], -1)
        return z.unflatten(-1, (self.H, self.P)), xbc, dt[..., :self.H]

    def prompts(self, x, starts, slots):
        """x [tokens, width]: prompts packed one behind the other, sequence i from
        starts[i] to starts[i + 1] into slot slots[i] (int32 tensors on the device)."""
        z, xbc, dt = self.split(self.project(self.w_in, x)[None])
        y = dc.causal_conv1d(xbc.transpose(1, 2), self.conv_w, self.conv_b, "silu", conv_state=self.conv_state,
                             conv_state_indices=slots, seq_starts=starts).transpose(1, 2)
        u, B, C = y.split([self.inner, self.bc, self.bc], -1)
        out = dc.selective_scan(u.unflatten(-1, (self.H, self.P)), dt, self.A, B.unflatten(-1, (self.G, self.K)),
                                C.unflatten(-1, (self.G, self.K)), D=self.D, z=z, dt_bias=self.dt_bias,
                                dt_softplus=True, ssm_state=self.ssm_state, state_indices=slots, seq_starts=starts)
        return self.project(self.w_out, out[0].flatten(1))

    def token(self, x, slots):
        """x [rows, width]: the next token of the sequences in slots (-1: no sequence)."""
        z, xbc, dt = self.split(self.project(self.w_in, x))
        out = dc.causal_conv1d_selective_update(xbc, self.conv_state, self.conv_w, self.conv_b, "silu", dt, self.A,
                                                self.ssm_state, groups=self.G, D=self.D, z=z, dt_bias=self.dt_bias,
                                                dt_softplus=True, state_indices=slots, workspace=self.workspace)
        return self.project(self.w_out, out.flatten(1))


def run(width=512, heads=8, head_size=64, groups=2, state_size=128, lengths=(5, 130, 64, 1), more=6, seed=1):
    """Prompts, then `more` tokens of each; the same tokens as longer prompts must give the
    same outputs.  Returns the largest difference over the outputs' root mean square."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = len(lengths)
    tokens = [torch.randn(length + more, width, generator=gen, device="cuda").to(torch.bfloat16) for length in lengths]
    slots = torch.arange(n, device="cuda", dtype=torch.int32).flip(0).contiguous()

    def starts(extra):
        return torch.tensor([0] + [length + extra for length in lengths]).cumsum(0).to(torch.int32).cuda()

    args = (width, heads, head_size, groups, state_size, n)
    layer, whole = StateSpaceLayer(*args), StateSpaceLayer(*args)
    want = whole.prompts(torch.cat(tokens), starts(more), slots).split([length + more for length in lengths])
    layer.prompts(torch.cat([t[:length] for t, length in zip(tokens, lengths)]), starts(0), slots)
    worst = 0.0
    for i in range(more):
        got = layer.token(torch.stack([t[length + i] for t, length in zip(tokens, lengths)]), slots)
        ref = torch.stack([w[length + i] for w, length in zip(want, lengths)])
        worst = max(worst, float((got.float() - ref.float()).abs().max() / ref.float().square().mean().sqrt()))
    return worst


if __name__ == "__main__":
    print(f"largest difference between stepping and prompting: {run():.4f} of the outputs' root mean square")
