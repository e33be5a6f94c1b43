"""The gated delta rule over whole sequences where factors, states or operands leave FP32's range:
what follows is not finite, or right; nothing ahead of it, in another head or sequence changes.
"""
import math

import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from delta_reference import U, bounds, recurrence
from test_gpu_delta import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


def growing(seed, T, H, P, K, state, **more):
    """A case whose log-decays are -dt, of either sign."""
    case = Case(seed, [T], H, P, H, K, state=state, init=None if state is None else [True], logit=False, soft=False,
                f32=True, **more)
    case.A = torch.full((H,), -1.0)
    return case


VARIANTS = [(2, 32, 64, torch.float32), (2, 32, 64, torch.bfloat16), (2, 32, 64, None), (2, 128, 128, torch.float32),
            (3, 40, 200, torch.float32), (3, 40, 200, None), (1, 24, 33, torch.float32)]


@pytest.mark.parametrize("H,P,K,state", VARIANTS)
@pytest.mark.parametrize("fall,rise,back", [(2, 5, 9), (0, 15, 15), (5, 20, 25), (13, 16, 30), (18, 29, 31), (3, 31, 31),
                                            (5, 40, 50), (20, 33, 62), (14, 63, 63), (36, 52, 60), (49, 55, 57), (70, 75, 99)])
def test_decays_that_fall_and_rise(H, P, K, state, fall, rise, back):
    """Every prefix sum of a chunk is moderate, but between two tokens of it a state grows by 2^200: the
    later token's outputs and all behind are not finite, also where decays fall again."""
    T, h = 130, H - 1
    case = growing(70 + fall, T, H, P, K, state)
    case.dt[0, fall, h] = 100 * math.log(2)
    clean = case.call()
    clean_pool = case.pool
    case.dt[0, rise, h] = -200 * math.log(2)
    if back > rise:
        case.dt[0, back, h] = 100 * math.log(2)
    out = case.call()
    assert torch.equal(out[0, :rise], clean[0, :rise]) and torch.equal(out[:, :, :h], clean[:, :, :h])
    assert not torch.isfinite(out[0, rise:, h]).any()
    if state is not None:
        assert torch.equal(case.pool[:, :h], clean_pool[:, :h]) and not torch.isfinite(case.pool[0, h]).any()


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fall,rise,back", [(2, 5, 9), (5, 20, 25), (20, 40, 50), (52, 60, 63)])
def test_decays_that_fall_and_rise_in_blocks_of_128_rows(fall, rise, back, state):
    test_decays_that_fall_and_rise(160, 128, 128, state, fall, rise, back)


@pytest.mark.parametrize("fall,rise,back", [(642, 645, 649), (650, 660, 672), (660, 690, 700), (1590, 1595, 1598)])
def test_decays_that_fall_and_rise_in_cut_sequences(fall, rise, back):
    """In a segment that others follow, whose two matrices carry it on, and in the last one."""
    case = growing(71, 1601, 2, 32, 64, torch.float32)
    case.dt[0, fall, 1] = 100 * math.log(2)
    clean, clean_pool = case.call(), case.pool
    assert dc.dcconv_last_kernel().startswith("delta_scan_split")
    case.dt[0, rise, 1] = -200 * math.log(2)
    case.dt[0, back, 1] = 100 * math.log(2)
    out = case.call()
    assert torch.equal(out[0, :rise], clean[0, :rise]) and torch.equal(out[:, :, 0], clean[:, :, 0])
    assert not torch.isfinite(out[0, rise:, 1]).any()
    assert torch.equal(case.pool[:, 0], clean_pool[:, 0]) and not torch.isfinite(case.pool[0, 1]).any()


@pytest.mark.parametrize("H,P,K,state", VARIANTS)
@pytest.mark.parametrize("first,second", [(2, 9), (5, 20), (20, 31), (5, 40), (33, 62), (50, 53)])
def test_products_of_large_keys_and_weights(H, P, K, state, first, second):
    """Two keys of 1e15 a value, the second with a weight of 1e10: what the second token reads of the
    state, 1e40 and more, is not finite, whatever decays follow."""
    h = H - 1
    case = growing(72, 100, H, P, K, state, l2=False)
    case.k[0, first, h] = 1e15
    clean, clean_pool = case.call(), case.pool
    case.k[0, second, h] = 1e15
    case.beta[0, second, h] = 1e10
    out = case.call()
    assert torch.equal(out[0, :second], clean[0, :second]) and torch.equal(out[:, :, :h], clean[:, :, :h])
    assert not torch.isfinite(out[0, second:, h]).any()
    if state is not None:
        assert torch.equal(case.pool[:, :h], clean_pool[:, :h]) and not torch.isfinite(case.pool[0, h]).any()


@pytest.mark.parametrize("H,P,K,state", [v for v in VARIANTS if v[3] is not torch.bfloat16])
@pytest.mark.parametrize("size", [5, 15, 30, 60])
def test_finite_results_are_right(H, P, K, state, size):
    """Log-decays of either sign: a result that is finite is within the bounds of the exact one, and
    where no two tokens are 2^90 apart all are finite.  (Decays below 2^-126 are taken as zero: a correction
    that has grown by 2^n, from values below 2^3, leaves up to 2^(n + 3 - 126) out.)"""
    for seed in range(4):
        case = growing(73 + seed, 100, H, P, K, state)
        gen = torch.Generator().manual_seed(seed)
        case.dt = torch.randn(case.dt.shape, generator=gen) * size * math.log(2)
        if seed % 2:
            case.dt *= torch.rand(case.dt.shape, generator=gen) < 0.2
        out = case.call()[0].double().cpu()
        cut = case.exact((0, slice(0, 100)))
        s0 = None if state is None else case.state[0].double()
        y, s = recurrence(*cut, s0)
        dy, ds = bounds(*cut, s0, 64 if K <= 128 else 32, state is not None)
        grown, run = torch.zeros(100, H, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
        for t in range(100):
            run = (run + cut[3][t] / math.log(2)).clamp(min=0)
            grown[t] = torch.maximum(grown[t - 1], run) if t else run
        lost = 2.0 ** (grown + 3 - 126)
        fine = torch.isfinite(out)
        assert not (fine & ((out - y).abs() > U * (y.abs() + dy) + dy + lost[..., None])).any()
        assert bool((fine.all(-1) | (grown > 90)).all())
        if state is not None:
            got = case.pool[0].double().cpu()
            fine = torch.isfinite(got)
            assert not (fine & ((got - s).abs() > ds + lost[-1][:, None, None])).any()
            assert bool((fine.all(-1).all(-1) | (grown[-1] > 90)).all())
