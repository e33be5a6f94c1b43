"""Plain 64-bit forms of the gated delta rule and of the norms, and the bounds their kernels
meet (not a test module).

``recurrence`` steps through the tokens one by one in float64.  ``bounds`` says how far a
kernel may be from it, with u = 2^-8 the largest relative error of one rounding to BF16
(eight significant bits, to nearest) and keys no longer than one, weights b in [0, 2].

* one token (``step_bounds``): products and sums in FP32 over at most 256 terms, and a step
  through log1p, exponentials and reciprocal square roots of moderate arguments: under 2^-18
  of the magnitudes (the same sums with every term's absolute value), and u of the result
  where it is stored as BF16.

* whole sequences.  The kernel takes chunks of C tokens as matrix products,

      R = v - e^c S k,  U = T R,  out = e^c S q + P U,  S' = e^{c_C} S + (w U)^T k

  with T the inverse of a unit lower triangular matrix times b, P the decayed products of q
  and k.  A relative error eS, eT, eR, eU, eP of an operand moves a sum by at most that times
  the sum of magnitudes, so within a chunk

      dR <= eS e^c |S| |k| + eR |R|,   dU <= |T| dR + eT |T| |R|
      dout <= u e^c |S| |q| + |P| dU + (u + eU2) |P| |U|
      dS' <= (w (dU + eU |U|))^T |k|          (the local error, and its norm over a row)

  An error that the state ahead of the chunk already has passes through the recurrence
  itself: a token multiplies it by e^g (I - b k k^T), whose norm is at most e^g, so a row's
  2-norm of the error shrinks with the decay, the local norms add up, and the output sees
  at most e^c times it times |q|.
  With an F32 state the operands carry two BF16 parts or more: e = u^2 = 2^-16.  With a BF16
  state (or none to hand out) eS, eR and eU are u, eT is 2^-16.  All of them gain 2^-18 for FP32 sums,
  exponentials (differences of prefix sums that carry 48 bits) and the factors of q and k.
"""
from __future__ import annotations

import torch

U = 2.0 ** -8
F32 = 2.0 ** -18
TINY = 1e-30


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def silu(v):
    return v * torch.sigmoid(v)


def factors(dt, A, beta, dt_bias=None, dt_softplus=False, beta_sigmoid=False):
    """(log-decay, weight) [T, H] of float64 operands."""
    d = dt if dt_bias is None else dt + dt_bias
    d = softplus(d) if dt_softplus else d
    return d * A, torch.sigmoid(beta) if beta_sigmoid else beta


def unit(v, l2norm, eps=1e-6):
    return v / (v.square().sum(-1, keepdim=True) + eps).sqrt() if l2norm else v


def recurrence(q, k, v, g, b, scale, s0=None):
    """One sequence: q, k [T, H, K], v [T, H, P], g, b [T, H], s0 [H, P, K], float64.
    Returns (out [T, H, P], state)."""
    T, H, P = v.shape
    s = torch.zeros(H, P, k.shape[-1], dtype=torch.float64) if s0 is None else s0.clone()
    out = torch.empty_like(v)
    for t in range(T):
        s = s * torch.exp(g[t])[:, None, None]
        u = b[t][:, None] * (v[t] - (s * k[t][:, None, :]).sum(-1))
        s = s + u[:, :, None] * k[t][:, None, :]
        out[t] = scale * (s * q[t][:, None, :]).sum(-1)
    return out, s


def step_bounds(q, k, v, g, b, scale, s0):
    """For one token of n rows (v [n, H, P], s0 [n, H, P, K]): (out, state, bound of out before
    its rounding, bound of the state before its rounding)."""
    decay = torch.exp(g)[..., None, None]
    s = s0 * decay
    u = b[..., None] * (v - (s * k[..., None, :]).sum(-1))
    ua = b.abs()[..., None] * (v.abs() + (s * k[..., None, :]).abs().sum(-1))
    new = s + u[..., None] * k[..., None, :]
    newa = s.abs() + ua[..., None] * k.abs()[..., None, :]
    out = scale * (new * q[..., None, :]).sum(-1)
    outa = abs(scale) * (newa * q.abs()[..., None, :]).sum(-1)
    return out, new, F32 * outa, F32 * newa


def bounds(q, k, v, g, b, scale, s0, chunk, exact):
    """How far a kernel's (output before its rounding, state before its rounding) may be from
    one sequence's recurrence.  exact: an F32 state is handed out."""
    T, H, P = v.shape
    K = k.shape[-1]
    eS = eR = eU = (2.0 ** -16 if exact else U) + F32
    eT = 2.0 ** -16 + F32
    s = torch.zeros(H, P, K, dtype=torch.float64) if s0 is None else s0.clone()
    row = ahead = torch.zeros(H, P, dtype=torch.float64)
    local = F32 * s.abs()
    dout = torch.empty_like(v)
    for t0 in range(0, T, chunk):
        sl = slice(t0, min(T, t0 + chunk))
        qc, kc, vc = (x[sl].transpose(0, 1) for x in (q, k, v))               # [H, C, .]
        c, w = g[sl].t().cumsum(-1), b[sl].t()
        n = c.shape[-1]
        low = torch.ones(n, n, dtype=torch.bool).tril()
        decay = torch.exp((c[:, :, None] - c[:, None, :]).masked_fill(~low, -torch.inf))
        gram = (kc @ kc.transpose(1, 2)) * decay
        T_ = torch.linalg.inv(torch.eye(n, dtype=torch.float64) + (w[:, :, None] * gram).tril(-1)) * w[:, None, :]
        Pm = (qc @ kc.transpose(1, 2)) * decay * scale
        ec = torch.exp(c)[..., None]
        R = vc - ec * (kc @ s.transpose(1, 2))
        Um = T_ @ R
        dR = eS * ec * (kc.abs() @ s.abs().transpose(1, 2)) + eR * (R.abs() + F32 * vc.abs())
        dU = T_.abs() @ dR + eT * (T_.abs() @ R.abs())
        do = (U + F32) * abs(scale) * ec * (qc.abs() @ s.abs().transpose(1, 2)) \
            + Pm.abs() @ dU + (U + 2.0 ** -16 + F32) * (Pm.abs() @ Um.abs())
        do = do + abs(scale) * ec * qc.norm(dim=-1)[..., None] * row[:, None, :]
        dout[sl] = do.transpose(0, 1)
        tail = torch.exp(c[:, -1:] - c)[..., None]
        local = (tail * (dU + eU * Um.abs())).transpose(1, 2) @ kc.abs()       # [H, P, K]
        s = s * torch.exp(c[:, -1])[:, None, None] + (tail * Um).transpose(1, 2) @ kc
        local = local + F32 * s.abs()
        ahead = row * torch.exp(c[:, -1])[:, None]
        row = ahead + local.norm(dim=-1)
    return dout, ahead[..., None] + local


def close(got, want, bound, what):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= bound + TINY)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / (bound + TINY)).nan_to_num(1e9).max()):.3g} times its bound")
