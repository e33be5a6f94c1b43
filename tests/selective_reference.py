"""Plain 64-bit forms of the state-space operators, and the bounds their kernels meet
(not a test module).

``recurrence`` steps through the tokens one by one in float64.  Beside each result it
returns the same sum with every term's magnitude (``*_abs``): rounding one factor of
every term by a relative e moves the result by at most e times that.

Bounds, per element, with u = 2^-8 the largest relative error of one rounding to BF16
(eight significant bits, to nearest):

* one token: products and sums in FP32 over at most 256 terms, a step through log1p
  and two exponentials of arguments below 32: under 2^-18 of the magnitudes, and u of
  the result where it is stored as BF16.
* whole sequences: the same, and the copy of the state that C reads, or the products
  of C and B, rounded to BF16 once: u of the magnitudes of y.  A chunk's prefix sums
  of dt A stay below 2^8 here, which moves an exponential by under 2^-13 of itself
  where that is not yet negligible: 2^-13 of the magnitudes of y.  A state of 32 bits
  is built from operands that carry all 24 bits and from suffix sums: 2^-17 of its
  magnitudes.  One of 16 bits is built from the scaled x rounded once: u of its
  magnitudes, and u for its own rounding.
"""
from __future__ import annotations

import torch

U = 2.0 ** -8
TINY = 1e-30


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def silu(v):
    return v * torch.sigmoid(v)


def recurrence(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False, h0=None):
    """One sequence: x, z [T, H, P], dt [T, H], B, C [T, G, K], h0 [H, P, K], float64.
    Returns (out, out_abs, state, state_abs)."""
    T, H, P = x.shape
    G, K = B.shape[1:]
    group = torch.arange(H) // (H // G)
    d = dt + (0 if dt_bias is None else dt_bias)
    if dt_softplus:
        d = softplus(d)
    h = torch.zeros(H, P, K, dtype=torch.float64) if h0 is None else h0.clone()
    ha = h.abs()
    out, out_abs = torch.empty_like(x), torch.empty_like(x)
    for t in range(T):
        decay = torch.exp(d[t] * A)[:, None, None]
        add = (d[t][:, None] * x[t])[:, :, None] * B[t, group][:, None, :]
        h, ha = h * decay + add, ha * decay + add.abs()
        y = (h * C[t, group][:, None, :]).sum(-1)
        ya = (ha * C[t, group].abs()[:, None, :]).sum(-1)
        if D is not None:
            y, ya = y + D[:, None] * x[t], ya + (D[:, None] * x[t]).abs()
        if z is not None:
            y, ya = y * silu(z[t]), ya * silu(z[t]).abs()
        out[t], out_abs[t] = y, ya
    return out, out_abs, h, ha


def convolve(history, x, weight, bias, act):
    """One token of the width-4 convolution: history [Dc, 3] oldest first, x [Dc]."""
    v = (torch.cat([history, x[:, None]], 1) * weight).sum(1)
    if bias is not None:
        v = v + bias
    return silu(v) if act in ("silu", "swish") else v


def close(got, want, bound, what):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= bound + TINY)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / (bound + TINY)).nan_to_num(1e9).max()):.3g} times its bound")
