"""The decays and weights of the gated delta rule, over the range of their gates: softplus and sigmoid are
within 2^-21 of themselves in the whole-sequence form and in the one-token form.

A state of ones that one token without weight decays holds exp(softplus(dt) a): with x = softplus(dt) |a|, an
error of 2^-21 of softplus and the roundings of a in base two and of the product (2^-24 each, and 2^-24 for what
the base's own constant is off) move it by x (2^-21 + 2^-22), the exponential and the state's product by 2^-22.
A token of no state with key and value one leaves its weight: 2^-21 and 2^-22 for the products.  In the scan it
passes two matrix products in three BF16 parts, of which a last one, rounded to a multiple of BF16's smallest
step of 2^-133, is off by up to 2^-134 each time: 2^-133 in all, which weights below 2^-110 show.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from delta_reference import softplus

pytestmark = pytest.mark.gpu
N = 4096


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


def one_token(form, dt, A, beta, state, value, **more):
    """The states of N rows behind one token whose key is the first unit vector."""
    one = torch.zeros(N, 1, 8, dtype=torch.bfloat16, device="cuda")
    one[..., 0] = 1.0
    v = torch.full((N, 1, 8), value, dtype=torch.bfloat16, device="cuda")
    args = [one, one, v, dt.cuda()[:, None], A, beta.cuda()[:, None]]
    if form == "update":
        dc.gated_delta_update(*args, state, **more)
    else:
        args = [t[:, None] if t.dim() > 1 else t for t in args]
        dc.gated_delta_scan(*args, state=state, has_initial_state=torch.ones(N, dtype=torch.bool, device="cuda"), **more)
    return state.double().cpu()


@pytest.mark.parametrize("form", ["scan", "update"])
@pytest.mark.parametrize("low,high", [(-80, -70), (-25, -15), (-8, -5), (-4, -3), (-3.5, -3.4), (-2, 0), (0, 1), (1, 8),
                                      (10, 30)])
def test_decays(form, low, high):
    gen = torch.Generator().manual_seed(1)
    dt = low + (high - low) * torch.rand(N, generator=gen)
    d = softplus(dt.double())
    A = (-60.0 / d.max()).float()
    got = one_token(form, dt, A.cuda()[None], torch.zeros(N), torch.ones(N, 1, 8, 8, device="cuda"), 0.0, dt_softplus=True)
    x = -d * A.double()
    err = (got / torch.exp(-x)[:, None, None, None] - 1).abs().amax((1, 2, 3))
    bound = x * (2.0 ** -21 + 2.0 ** -22) + 2.0 ** -22
    assert bool((err <= bound).all()), f"{float((err / bound).max()):.3g} times its bound"


@pytest.mark.parametrize("form", ["scan", "update"])
@pytest.mark.parametrize("low,high", [(-85, -70), (-25, -15), (-8, -5), (-4, 0), (0, 4), (4, 30), (80, 100)])
def test_weights(form, low, high):
    gen = torch.Generator().manual_seed(2)
    beta = low + (high - low) * torch.rand(N, generator=gen)
    got = one_token(form, torch.zeros(N), torch.zeros(1, device="cuda"), beta, torch.zeros(N, 1, 8, 8, device="cuda"), 1.0,
                    beta_sigmoid=True)
    want = torch.sigmoid(beta.double())
    assert not got[..., 1:].any()
    err = (got[..., 0] / want[:, None, None] - 1).abs().amax((1, 2))
    step = 2.0 ** -133 / want if form == "scan" else 0.0
    assert bool((err <= 2.0 ** -21 + 2.0 ** -22 + step).all()), f"off by {float(err.max()):.3g}"


@pytest.mark.parametrize("form", ["scan", "update"])
def test_gates_at_the_ends(form):
    """Infinite logits: weights of zero and one, steps of zero and infinity; a NaN stays one."""
    inf = float("inf")
    ends = torch.tensor([-inf, -200.0, 200.0, inf, float("nan")]).repeat(N // 5 + 1)[:N]
    got = one_token(form, torch.zeros(N), torch.zeros(1, device="cuda"), ends, torch.zeros(N, 1, 8, 8, device="cuda"), 1.0,
                    beta_sigmoid=True)[:5, 0, 0, 0].tolist()
    assert got[:4] == [0.0, 0.0, 1.0, 1.0] and got[4] != got[4]
    got = one_token(form, ends, torch.full((1,), -1.0, device="cuda"), torch.zeros(N),
                    torch.ones(N, 1, 8, 8, device="cuda"), 0.0, dt_softplus=True)[:5, 0, 0, 0].tolist()
    assert got[:4] == [1.0, 1.0, 0.0, 0.0] and got[4] != got[4]
