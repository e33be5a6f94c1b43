"""Pools of no slots are refused where sequences would leave their final states there."""
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


@pytest.mark.parametrize("packed", [False, True])
def test_selective_scan(packed):
    case = Scan(1, [40, 40], 2, 32, 1, 32, packed=packed)
    case.state = torch.empty(0, 2, 32, 32)
    with pytest.raises(ValueError, match="no slots"):
        case.call()


@pytest.mark.parametrize("indices", [None, [-1, -1]])
def test_causal_conv1d(indices):
    x = torch.zeros(2, 8, 40, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, 4, dtype=torch.bfloat16, device="cuda")
    table = None if indices is None else torch.tensor(indices, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="no slots"):
        dc.causal_conv1d(x, w, conv_state=x.new_empty(0, 8, 3), conv_state_indices=table)
