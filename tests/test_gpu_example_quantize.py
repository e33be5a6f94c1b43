"""The example's quantisation: how far dequantised weights lie from the given ones.

A group's step is its range, zero included, over 15.  Rounding a code costs at most half
a step, and as much at an end of the range, where the rounded zero point may leave half a
step past the last code and the scale, rounded to BF16, 15 * 2^-8 of one: 0.57 steps of a
scale at most 2^-8 larger, below 0.6.  A product with a row of the identity is rounded once."""
import importlib.util
import os

import pytest
import torch

import depthwise_causal_conv1d_amd as dc

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "state_space_layer.py")


@pytest.mark.parametrize("kind", ["normal", "positive", "negative", "constant", "zero", "one"])
@pytest.mark.parametrize("K", [128, 100])
def test_quantize(kind, K):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("state_space_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(24, K, generator=gen, device="cuda")
    if kind == "positive":
        w = 3 + 0.1 * w
    elif kind == "negative":
        w = -3 + 0.1 * w
    elif kind == "constant":
        w = torch.full_like(w, 0.5)
    elif kind == "zero":
        w = torch.zeros_like(w)
    elif kind == "one":
        w = torch.where(torch.arange(K, device="cuda") == 3, w, torch.zeros_like(w))
    q, scales, zeros = module.quantize(w, 64)
    got = dc.w4_matvec(torch.eye(K, device="cuda", dtype=torch.bfloat16), q, scales, zeros, group_size=64).t().float()
    group = torch.arange(K, device="cuda") // 64
    step = torch.stack([(w[:, group == i].amax(1).clamp(min=0) - w[:, group == i].amin(1).clamp(max=0)) / 15
                        for i in range(-(-K // 64))], 1)[:, group]
    assert bool(((got - w).abs() <= 0.6 * step + 2.0 ** -8 * w.abs()).all())
