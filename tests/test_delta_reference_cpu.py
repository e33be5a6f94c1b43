"""The 64-bit forms that the GPU tests compare with, against the formulas written out: the rule as
products of transition matrices, and its chunk form, whose error bounds the tests use."""
import torch

from delta_reference import U, bounds, factors, recurrence, step_bounds, unit


def draw(seed, T=9, H=2, P=3, K=5):
    gen = torch.Generator().manual_seed(seed)
    q, k = (unit(torch.randn(T, H, K, generator=gen).double(), True) for _ in range(2))
    v = torch.randn(T, H, P, generator=gen).double()
    g, b = -torch.rand(T, H, generator=gen).double(), 2 * torch.rand(T, H, generator=gen).double()
    return q, k, v, g, b, torch.randn(H, P, K, generator=gen).double()


def test_recurrence_is_the_product_of_transitions():
    q, k, v, g, b, s0 = draw(1)
    out, state = recurrence(q, k, v, g, b, 0.5, s0)
    eye = torch.eye(5).double()
    for h in range(2):
        s = s0[h]
        for t in range(9):
            kk = k[t, h]
            s = torch.exp(g[t, h]) * s @ (eye - b[t, h] * torch.outer(kk, kk)) + b[t, h] * torch.outer(v[t, h], kk)
            assert torch.allclose(out[t, h], 0.5 * s @ q[t, h], atol=1e-13)
        assert torch.allclose(state[h], s, atol=1e-13)


def test_a_weight_of_one_writes_the_value_under_its_key():
    q, k, v, g, b, s0 = draw(2)
    out, state = recurrence(k, k, v, g, torch.ones_like(b), 1.0, s0)
    assert torch.allclose(out, v, atol=1e-12)
    _, same = recurrence(q, k, v, torch.zeros_like(g), torch.zeros_like(b), 1.0, s0)
    assert torch.equal(same, s0)


def test_one_token_is_the_recurrence_of_one():
    q, k, v, g, b, s0 = draw(3, T=1)
    out, state = recurrence(q, k, v, g, b, 0.7, s0)
    y, s, dy, ds = step_bounds(q, k, v, g, b, 0.7, s0[None])
    assert torch.allclose(y, out, atol=1e-14) and torch.allclose(s[0], state, atol=1e-14)
    assert bool((dy > 0).all() and (ds > 0).all())


def test_bounds_hold_for_rounded_operands():
    """A chunk form whose operands are rounded at random by the errors that the bounds assume stays
    within them, and not by orders of magnitude."""
    gen = torch.Generator().manual_seed(4)
    q, k, v, g, b, s0 = draw(4, T=40, H=2, P=4, K=16)
    want, state = recurrence(q, k, v, g, b, 0.25, s0)
    dout, dstate = bounds(q, k, v, g, b, 0.25, s0, 16, False)

    def off(x, e=U):
        return x * (1 + e * (2 * torch.rand(x.shape, generator=gen).double() - 1))
    s = s0.clone()
    got = torch.empty_like(want)
    for t0 in range(0, 40, 16):
        sl = slice(t0, min(40, t0 + 16))
        qc, kc, vc = (x[sl].transpose(0, 1) for x in (q, k, v))
        c, w = g[sl].t().cumsum(-1), b[sl].t()
        decay = torch.exp(c[:, :, None] - c[:, None, :]).tril()
        T = torch.linalg.inv(torch.eye(c.shape[1]).double() + (w[:, :, None] * (kc @ kc.transpose(1, 2)) * decay).tril(-1)) \
            * w[:, None, :]
        ec = torch.exp(c)[..., None]
        u = off(T, 2.0 ** -16) @ off(vc - ec * (kc @ off(s).transpose(1, 2)))
        got[sl] = (0.25 * ec * (qc @ off(s).transpose(1, 2)) + off((qc @ kc.transpose(1, 2)) * decay * 0.25) @ u).transpose(0, 1)
        s = s * torch.exp(c[:, -1])[:, None, None] + off(torch.exp(c[:, -1:] - c)[..., None] * u).transpose(1, 2) @ kc
    for x, y, d in ((got, want, dout), (s, state, dstate)):
        assert bool(((x - y).abs() <= d).all())
        assert float((x - y).norm() / d.norm()) > 0.005


def test_factors():
    dt, beta = torch.tensor([[-800.0, 0.0, 2.0]]).double(), torch.tensor([[-800.0, 0.0, 1.0]]).double()
    g, b = factors(dt, torch.tensor([-1.0, -2.0, -3.0]).double(), beta, None, True, True)
    assert torch.allclose(g, torch.tensor([[0.0, -1.3862943611198906, -6.3807840330437]]).double(), atol=1e-12)
    assert torch.allclose(b, torch.tensor([[0.0, 0.5, 0.7310585786300049]]).double(), atol=1e-12)
    g, b = factors(dt, torch.ones(3).double(), beta, torch.ones(3).double())
    assert torch.equal(g, dt + 1) and torch.equal(b, beta)
