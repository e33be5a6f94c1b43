"""Products with 4-bit weights at the ends of the value range: what a 32-bit sum of
x * ((code - zero) * scale) holds, the kernel gives.  The bound is ``test_gpu_w4``'s, and
below the least normal number 2^-126 a term may lose as much as 2^-134 a unit of scale
(the least step 2^-149 on sums kept 2^15 below their size)."""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from selective_reference import U
from test_gpu_w4 import Product

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


# a size of x and of the scales whose products are ordinary numbers
@pytest.mark.parametrize("size,scale", [(1e38, 1e-3), (3e37, 1e-38), (1e30, 1e-30), (1e-30, 1e30), (1e-36, 1.0),
                                        (1e-36, 1e36), (1e-3, 3e36)])
@pytest.mark.parametrize("K,gs,zeros,pad", [(256, 128, True, 0), (200, 64, True, 0), (160, 32, False, 3), (700, 256, True, 0)])
def test_sizes_of_x_and_scales(size, scale, K, gs, zeros, pad):
    case = Product(1, 5, 40, K, gs, zeros, False, pad)
    case.x = (case.x.float().clamp(-3, 3) * size).to(torch.bfloat16)
    case.scales = (case.scales.float() * 20 * scale).to(torch.bfloat16)
    got = case.call().double().cpu()
    group = torch.arange(K) // gs
    by = case.scales.double()[group].t()
    w = (case.codes.double() - (8 if case.zeros is None else case.zeros.double()[group].t())) * by
    want, terms = case.x.double() @ w.t(), case.x.double().abs() @ by.t()
    bound = U * want.abs() + 2.0 ** -11 * terms + 2.0 ** -134 * by.sum(1) + 2.0 ** -133
    top = torch.finfo(torch.bfloat16).max
    inside = want.abs() + bound < top          # what rounds to a finite BF16
    assert bool(inside.any())
    assert bool(((got - want).abs() <= bound)[inside].all())
    assert bool((got[want.abs() - bound > top * (1 + U)].abs() == float("inf")).all())


def test_the_largest_values_of_one_sign_in_a_whole_group():
    """128 times the largest BF16 in a row: the sum of a group is past FP32's range, the
    result, by its scales, is not."""
    case = Product(2, 2, 40, 128, 128, True, False)
    top = torch.finfo(torch.bfloat16).max
    case.x[:] = top
    case.scales[:] = 2.0 ** -14
    got = case.call().double().cpu()
    want = top * 2.0 ** -14 * (case.codes.double() - case.zeros.double()[0][:, None]).sum(1)
    assert bool(((got - want).abs() <= U * want.abs() + 2.0 ** -11 * 128 * top * 2.0 ** -14).all())
