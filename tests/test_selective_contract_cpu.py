"""What the state-space entry points promise their callers, as far as the host decides
it: no GPU.  Made-up device addresses are never dereferenced, so calls with them run only
where no GPU is visible.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from test_selective_abi_cpu import P, refused, scan

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers are only passed where no GPU exists")


@no_gpu
@pytest.mark.parametrize("over", [dict(state_indices=P[9]), dict(has_initial_state=P[10]),
                                  dict(state_indices=P[9], has_initial_state=P[10])])
@pytest.mark.parametrize("packed", [False, True])
def test_scan_without_a_pool_refuses_what_selects_from_one(over, packed):
    """No slot exists that an index could select: not a call whose sequences are all padding."""
    starts = dict(seq_starts=P[11]) if packed else {}
    refused(scan, dict(ssm_state=None, s=0, **over, **starts), dc.DCCONV_EINVAL, "ssm_state")
