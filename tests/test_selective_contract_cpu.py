"""What the state-space entry points promise their callers, as far as the host decides
it: no GPU.  Made-up device addresses are never dereferenced, so calls with them run only
where no GPU is visible.
"""
import sys

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


def test_a_second_thread_finds_torch_only_with_its_types(monkeypatch):
    """A first call publishes torch in ``_t``, which other threads take as the sign that all
    of the module's names are set: so they are, at every step on the way."""
    from depthwise_causal_conv1d_amd import _binding, selective

    for module, names in ((selective, ("_t", "_BF16", "_F32", "_I32")), (_binding, ("_torch", "stream"))):
        for name in names:
            monkeypatch.setattr(module, name, None)
    rest = ((selective, "_BF16"), (selective, "_F32"), (selective, "_I32"), (_binding, "_torch"), (_binding, "stream"))
    missing = []

    def trace(frame, event, arg):
        frame.f_trace_opcodes = True
        if selective._t is not None:
            missing.extend(name for module, name in rest if getattr(module, name) is None)
        return trace

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        selective._import_torch()
    finally:
        sys.settrace(before)
    assert selective._t is torch and not missing


def test_packed_workspace_grows_with_tokens_not_with_sequences():
    """Only a sequence that is cut into segments has a place in the workspace; as it is longer
    than a segment, t tokens hold at most two segments of cut sequences for each of theirs."""
    heads = (96, 64, 8, 128)
    state = 4 * 96 * (64 * 128 + 1)
    sizes = [dc.dcconv_selective_scan_workspace(n, 65536, *heads, 1) for n in (64, 256, 1024, 65536)]
    assert len(set(sizes)) == 1 and 0 < sizes[0] <= 2 * (65536 // 2048) * state
    assert dc.dcconv_selective_scan_workspace(256, 2100, *heads, 1) <= 2 * state
    assert dc.dcconv_selective_scan_workspace(256, 2000, *heads, 1) == 0
    # few sequences: no more than a place for each segment
    for n in (1, 2, 5):
        few = dc.dcconv_selective_scan_workspace(n, 16381, 24, 64, 2, 128, 1)
        assert 0 < few <= (-(-16381 // 96) + n) * 4 * 24 * (64 * 128 + 1)
