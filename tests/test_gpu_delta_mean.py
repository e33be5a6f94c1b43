"""The size of the gated delta rule's errors over whole sequences of thousands of tokens, in the norm: what the
header states, so that an operand that loses a part shows, which the worst-case bounds let pass.

Rounding to BF16 is off by e = 0.00166 in the mean (uniform within half a step of 2^-8, over a binade).

F32 states: sums of 64 tokens make about a dozen roundings of 2^-24 a chunk, 0.29 of that each in the mean; over
128 chunks without any forgetting sqrt(12 * 128) * 0.29 * 2^-24 = 7e-7.  At most 2^-20.  (S in two parts where
k reads it: 2^-18 for every token's correction, 1.4e-6 to 3e-6.)

Outputs and BF16 states: their one rounding, e; the operands' 2^-16 are nothing beside it.  (Any operand in one part is a
rounding more of terms of the output's size or half of it: 1.23 e and more.)  The draw is left 5 %.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc

pytestmark = pytest.mark.gpu
E = 0.00166


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


def unit(x):
    x = x.double()
    return x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()


class Long:
    """N sequences of T tokens and what 64 bits make of them, a head a group, on the GPU."""

    def __init__(self, N, T, H, P, K, rate, sigmoid):
        gen = torch.Generator(device="cuda").manual_seed(T + K)

        def rn(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")
        self.q, self.k, self.v = (rn(N, T, H, d).to(torch.bfloat16) for d in (K, K, P))
        self.dt, self.sigmoid = rn(N, T, H), sigmoid
        self.beta = rn(N, T, H) if sigmoid else 1.9 * torch.rand(N, T, H, generator=gen, device="cuda")
        self.A, self.bias = -rate * torch.rand(H, generator=gen, device="cuda"), torch.full((H,), -4.0, device="cuda")
        self.state = (0.3 * rn(N, H, P, K)).to(torch.bfloat16)
        self.init = torch.ones(N, dtype=torch.bool, device="cuda")

    def exact(self, init=True):
        d = torch.nn.functional.softplus(self.dt.double() + self.bias.double())
        decay = torch.exp(d * self.A.double())[..., None, None]
        b = (torch.sigmoid(self.beta.double()) if self.sigmoid else self.beta.double())[..., None]
        q, k, v = unit(self.q)[..., None, :], unit(self.k)[..., None, :], self.v.double()
        s = self.state.double() if init else torch.zeros_like(self.state, dtype=torch.float64)
        out = torch.empty_like(v)
        for t in range(v.shape[1]):
            s = s * decay[:, t]
            u = b[:, t] * (v[:, t] - (s * k[:, t]).sum(-1))
            s = s + u[..., None] * k[:, t]
            out[:, t] = (s * q[:, t]).sum(-1)
        return out * self.q.shape[-1] ** -0.5, s

    def call(self, kind):
        pool = None if kind is None else self.state.to(kind)
        out = dc.gated_delta_scan(self.q, self.k, self.v, self.dt, self.A, self.beta, dt_bias=self.bias, dt_softplus=True,
                                  beta_sigmoid=self.sigmoid, qk_l2norm=True, state=pool,
                                  has_initial_state=None if kind is None else self.init)
        return out, pool


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("N,T,H,P,K,cut", [(1, 4096, 2, 128, 128, True), (1, 2048, 2, 64, 64, True), (1, 2048, 2, 64, 256, True),
                                           (40, 512, 8, 128, 128, False), (1, 640, 300, 32, 64, False),
                                           (1, 320, 260, 64, 200, False)])
@pytest.mark.parametrize("rate,sigmoid", [(8.0, True), (0.02, True), (0.0, True), (0.0, False)])
def test_errors_in_the_mean(N, T, H, P, K, cut, rate, sigmoid):
    case = Long(N, T, H, P, K, rate, sigmoid)
    y, s = case.exact()
    out, pool = case.call(torch.float32)
    assert dc.dcconv_last_kernel().startswith("delta_scan_split") == cut
    most = 1.05 * E
    errors = {"out, F32 states": (off(out, y), most), "F32 states": (off(pool, s), 2.0 ** -20)}
    out, pool = case.call(torch.bfloat16)
    errors["out, BF16 states"], errors["BF16 states"] = (off(out, y), most), (off(pool, s), 1.05 * E)
    y, s = case.exact(init=False)
    errors["out, no states"] = off(case.call(None)[0], y), most
    assert all(v <= most for v, most in errors.values()), errors
