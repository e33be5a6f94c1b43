"""The 64-bit forms that the GPU tests compare with, against the formulas written out:
every output as a double sum over tokens and states instead of a recurrence."""
import numpy as np
import torch

from selective_reference import convolve, recurrence, silu, softplus


def draw(seed, T=7, H=4, P=3, G=2, K=5):
    gen = torch.Generator().manual_seed(seed)
    x, z = torch.randn(T, H, P, generator=gen).double(), torch.randn(T, H, P, generator=gen).double()
    B, C = torch.randn(T, G, K, generator=gen).double(), torch.randn(T, G, K, generator=gen).double()
    dt, A = torch.rand(T, H, generator=gen).double(), -torch.rand(H, generator=gen).double()
    D, h0 = torch.randn(H, generator=gen).double(), torch.randn(H, P, K, generator=gen).double()
    return x, z, dt, A, B, C, D, h0


def test_recurrence_is_the_double_sum():
    x, z, dt, A, B, C, D, h0 = draw(1)
    T, H, P = x.shape
    out, out_abs, state, state_abs = recurrence(x, dt, A, B, C, D, z, h0=h0)
    for h in range(H):
        g = h // 2
        for t in range(T):
            decay = lambda u: np.exp(float(A[h]) * float(dt[u + 1:t + 1, h].sum()))  # noqa: E731
            for p in range(P):
                y = float(D[h] * x[t, h, p]) + decay(-1) * float(h0[h, p] @ C[t, g])
                y += sum(decay(u) * float(dt[u, h] * x[u, h, p]) * float(B[u, g] @ C[t, g]) for u in range(t + 1))
                y *= float(z[t, h, p]) / (1 + np.exp(-float(z[t, h, p])))
                assert abs(y - float(out[t, h, p])) < 1e-12
    assert bool((out_abs >= out.abs() - 1e-12).all() and (state_abs >= state.abs() - 1e-12).all())


def test_no_decay_sums_up():
    x, _, dt, A, B, C, _, _ = draw(2)
    _, _, state, _ = recurrence(x, dt, 0 * A, B, C)
    group = torch.arange(4) // 2
    want = sum((dt[t, :, None] * x[t])[:, :, None] * B[t, group][:, None, :] for t in range(x.shape[0]))
    assert torch.allclose(state, want, atol=1e-13)


def test_steps_are_biased_and_softplused():
    x, _, dt, A, B, C, _, _ = draw(3)
    bias = torch.tensor([0.5, -3.0, 0.0, 20.0]).double()
    a = recurrence(x, dt, A, B, C, dt_bias=bias, dt_softplus=True)
    b = recurrence(x, torch.log1p(torch.exp(dt + bias)), A, B, C)
    assert torch.allclose(a[0], b[0], atol=1e-11)


def test_parts():
    v = torch.tensor([-800.0, -1.0, 0.0, 2.0, 800.0]).double()
    assert torch.allclose(softplus(v), torch.tensor([0.0, 0.31326168751822286, 0.6931471805599453, 2.1269280110429727,
                                                     800.0]).double(), atol=1e-14)
    assert torch.allclose(silu(v)[1:4], v[1:4] / (1 + torch.exp(-v[1:4])))
    history = torch.tensor([[1.0, 2.0, 3.0]]).double()
    got = convolve(history, torch.tensor([4.0]).double(), torch.tensor([[0.5, -1.0, 2.0, 3.0]]).double(),
                   torch.tensor([0.25]).double(), None)
    assert float(got) == 0.5 - 2.0 + 6.0 + 12.0 + 0.25
