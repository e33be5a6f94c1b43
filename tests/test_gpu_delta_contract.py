"""What the gated delta rule's tensor functions promise their callers, on the GPU: refusals, and what a
broken table or a rarer variant leaves alone."""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from test_gpu_delta import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("more", [dict(), dict(table=[-1, -1]), dict(init=[True, False])])
def test_scan_refuses_a_pool_of_no_slots(more, packed):
    case = Case(1, [40, 40], 2, 32, 1, 32, packed=packed, **more)
    case.state = torch.empty(0, 2, 32, 32)
    with pytest.raises(ValueError, match="no slots"):
        case.call()


def test_scan_of_no_sequences_takes_a_pool_of_no_slots():
    case = Case(1, [], 2, 32, 1, 32, packed=True)
    case.state = torch.empty(0, 2, 32, 32)
    assert case.call().shape == (1, 0, 2, 32)
