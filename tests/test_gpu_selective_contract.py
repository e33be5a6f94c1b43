"""What the state-space tensor functions promise their callers, on the GPU: refusals and
values at the edges of their ranges."""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from test_gpu_selective import Scan

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
