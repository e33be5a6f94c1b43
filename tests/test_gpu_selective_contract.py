"""What the state-space tensor functions promise their callers, on the GPU: refusals and
values at the edges of their ranges."""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from selective_reference import U, close, recurrence
from test_gpu_selective import Scan, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("more", [dict(table=[0, -1]), dict(init=[True, False]), dict(table=[-1, 1], init=[True, True])])
@pytest.mark.parametrize("packed", [False, True])
def test_scan_without_a_pool_refuses_what_selects_from_one(more, packed):
    case = Scan(1, [40, 40], 2, 32, 1, 32, packed=packed, **more)
    for final in (False, True):
        with pytest.raises(ValueError, match="need an ssm_state"):
            case.call(return_final_state=final)


@pytest.mark.parametrize("name", ["x", "B"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,at", [(70, 3), (70, 37), (70, 69), (700, 100), (700, 650)])
def test_scan_is_not_finite_where_the_recurrence_is_not(name, bad, state, tokens, at):
    """An infinity or NaN of x or B is one or the other in the state and the outputs that the
    recurrence takes it to, and every other value is as close as ever."""
    case = Scan(51, [tokens], 2, 64, 1, 64, state=state, init=[True])
    getattr(case, name)[0, at, 0, 5] = bad
    out = case.call()
    cut = [f64(t[0]) for t in (case.x, case.dt, case.B, case.C, case.z)]
    y, ya, h, ha = recurrence(cut[0], cut[1], f64(case.A), cut[2], cut[3], f64(case.D), cut[4], f64(case.bias), True,
                              f64(case.state[0]))
    keep = torch.isfinite(h)
    assert not keep.all() and torch.equal(torch.isfinite(case.pool[0]).cpu(), keep)
    bound = 2.0 ** -17 * ha if state == torch.float32 else U * h.abs() + (U + 2.0 ** -13) * ha
    close(case.pool[0].cpu()[keep], h[keep], bound[keep], "finite states")
    keep = torch.isfinite(y)
    assert not keep.all() and torch.equal(torch.isfinite(out[0]).cpu(), keep)
    close(out[0].cpu()[keep], y[keep], (U * y.abs() + (U + 2.0 ** -13) * ya)[keep], "finite outputs")


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_scan_of_many_packed_sequences_some_of_them_cut(state):
    """More sequences than segments (of 2048 tokens here): places in the workspace go to the cut
    ones alone, several of them one behind the other, ending with the last token.  A value that
    the workspace must not be read or written past lies behind it."""
    gen = torch.Generator().manual_seed(61)
    lens = torch.randint(0, 12, (300,), generator=gen).tolist()
    lens[40:43], lens[150], lens[299] = [2049, 2049, 4097], 2048, 2500
    init = (torch.rand(300, generator=gen) < 0.5).tolist()
    case = Scan(61, lens, 1, 16, 1, 16, state=state, packed=True, slots=303, init=init,
                table=[-1 if i % 50 == 7 else 302 - i for i in range(300)])
    need = dc.dcconv_selective_scan_workspace(300, sum(lens), 1, 16, 1, 16, 1)
    assert 0 < need <= 2 * (sum(lens) // 2048) * 4 * (16 * 16 + 1)
    buf = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    case.check(workspace=buf[:need])
    assert dc.dcconv_last_kernel().startswith("selective_scan_split")
    assert bool((buf[need:] == 0xAB).all())
