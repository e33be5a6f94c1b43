"""Paths of the state-space kernels that only certain sizes take, against the 64-bit form:
the edges of the scan's chunks (32 tokens) and segments, its join where a state's size is
no multiple of four, segments with large states, one-token items of 32 rows several to a
block, and more one-token units than blocks.  Bounds per element are ``selective_reference``'s.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from selective_reference import U, recurrence
from test_gpu_selective import Scan, Update, bf, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [31, 32, 33, 95, 96, 97])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_scan_at_the_edges_of_chunks(T, state):
    Scan(T, [T, T], 3, 64, 1, 128, state=state, init=[False, True]).check()


# p, k, and state elements of a head: odd, or more than 64 and 128 values a row
@pytest.mark.parametrize("P,K,state", [(3, 5, torch.float32), (3, 5, torch.bfloat16), (1, 1, torch.float32),
                                       (64, 128, torch.float32), (64, 128, torch.bfloat16), (32, 200, torch.float32),
                                       (16, 256, torch.bfloat16), (5, 131, torch.float32)])
def test_scan_in_segments(P, K, state):
    Scan(P + K, [1500], 2, P, 1, K, state=state, init=[True]).check()
    assert dc.dcconv_last_kernel().startswith("selective_scan_split")


@pytest.mark.parametrize("off", [-1, 0, 1])
@pytest.mark.parametrize("segments", [4, 7])
def test_scan_at_the_edges_of_segments(off, segments):
    """Two blocks: segments are of 96 tokens, the fewest."""
    T = 96 * segments + off
    Scan(T, [T], 2, 64, 1, 64, state=torch.float32, init=[True]).check()
    assert dc.dcconv_last_kernel().startswith("selective_scan_split")


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [dict(lens=[300], H=4, P=64, G=2, K=128), dict(lens=[1500], H=2, P=64, G=1, K=64),
                                   dict(lens=[200], H=2, P=64, G=1, K=256)])
def test_scan_outputs_in_the_mean(shape, state):
    """The root mean square of the outputs' errors.  One rounding to BF16 errs by at most
    half a unit in the last place, evenly spread: u / sqrt(3) of the value in the root
    mean square at the least mantissa.  A term of y is rounded once (as the state's copy
    that C reads, or as a product of C and B), the x of a 16-bit state once before, and
    the output once.  Errors and terms have random signs, so each adds in quadrature at
    most that share of y: sqrt(3) * u / sqrt(3) = u in all, and a tenth more for the scatter
    of sums over some ten thousand outputs."""
    case = Scan(31, state=state, init=[True], **shape)
    out = case.call()
    x, dt, B, C, z = (f64(t[0]) for t in (case.x, case.dt, case.B, case.C, case.z))
    want = recurrence(x, dt, f64(case.A), B, C, f64(case.D), z, f64(case.bias), True, f64(case.state[0]))[0]
    err = (out[0].double().cpu() - want).square().mean().sqrt() / want.square().mean().sqrt()
    assert float(err) <= 1.1 * U


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("P,K", [(80, 72), (64, 128), (33, 256), (64, 16), (40, 13)])
def test_update_takes_several_items_of_32_rows_a_block(P, K, fused):
    """2048 items of 32 rows and more, F32 states: a block takes the next item's rows ahead."""
    n = 2048 // (24 * -(-P // 32)) + 3
    Update(P * K, n, 24, P, 3, K, torch.float32, fused=fused, slots=n + 4,
           table=[-1 if i % 9 == 4 else n + 3 - i for i in range(n)]).check()


@pytest.mark.parametrize("fused", [False, True])
def test_update_more_units_than_blocks(fused):
    """2^20 + 5 rows of one value: blocks take a second unit, behind a padding row for some."""
    n = (1 << 20) + 5
    gen = torch.Generator().manual_seed(41)
    table = torch.arange(n, dtype=torch.int32)
    table[::7] = -1
    live = table >= 0
    x, dt, state = bf(gen, n, 1, 1), torch.rand(n, 1, generator=gen) * 0.5, torch.randn(n, 1, 1, 1, generator=gen)
    B, C = bf(gen, n, 1, 1), bf(gen, n, 1, 1)
    A = torch.tensor([-1.5])
    pool = state.cuda().clone()
    if fused:
        xbc, conv = torch.cat([x, B, C], 1).squeeze(-1), bf(gen, n, 3, 3)
        weight = bf(gen, 3, 4, scale=0.5)
        history, ws = conv.cuda().clone(), dc.selective_update_workspace(n, 1)
        out = dc.causal_conv1d_selective_update(xbc.cuda(), history, weight.cuda(), None, None, dt.cuda(), A.cuda(), pool,
                                                groups=1, state_indices=table.cuda(), workspace=ws)
        assert not ws.any()
        moved = torch.where(live[:, None, None], torch.cat([conv[:, :, 1:], xbc[:, :, None]], 2), conv)
        assert torch.equal(history.cpu().view(torch.int16), moved.view(torch.int16))
        v = (torch.cat([conv, xbc[:, :, None]], 2).double() * weight.double()).sum(-1)
        va = (torch.cat([conv, xbc[:, :, None]], 2).double() * weight.double()).abs().sum(-1)
    else:
        out = dc.selective_update(x.cuda(), dt.cuda(), A.cuda(), B.cuda(), C.cuda(), pool, state_indices=table.cuda())
        v = torch.cat([x, B, C], 1).squeeze(-1).double()
        va = v.abs()
    d, old = dt[:, 0].double(), state.view(n).double()
    new = old * torch.exp(d * -1.5) + d * v[:, 0] * v[:, 1]
    size = old.abs() * torch.exp(d * -1.5) + d * va[:, 0] * va[:, 1]
    want, bound = new * v[:, 2], 2.0 ** -18 * size * va[:, 2]
    got, kept = out.view(n).double().cpu(), pool.view(n).double().cpu()
    assert not got[~live].any() and torch.equal(kept[~live], old[~live])
    assert bool(((kept - new).abs() <= 2.0 ** -18 * size + 1e-30)[live].all())
    assert bool(((got - want).abs() <= U * want.abs() + bound + 1e-30)[live].all())
