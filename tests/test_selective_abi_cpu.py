"""Refusals of the state-space entry points, and the workspace sizes: host logic, no GPU.

Each call is a valid one with one argument changed; the made-up device addresses are
never dereferenced, so these run only where no GPU is visible.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers are only passed where no GPU exists")

P = [0x10000000 * (k + 1) for k in range(20)]


def update(**over):
    a = dict(x=P[0], n=4, h=6, p=64, xs_n=384, xs_h=64, dt=P[1], dt_dtype=0, ds_n=6, dt_bias=None, dt_softplus=1,
             a=P[2], b=P[3], c=P[4], g=2, k=128, bs_n=256, bs_g=128, cs_n=256, cs_g=128, d_skip=None, z=None, zs_n=0,
             zs_h=0, ssm_state=P[5], state_dtype=1, s=4, ss_s=6 * 64 * 128, state_indices=None, out=P[6], os_n=384,
             os_h=64, dev_status=None, stream=None)
    assert not set(over) - set(a)
    a.update(over)
    return dc.dcconv_selective_update(*a.values())


def fused(**over):
    d = 6 * 64 + 2 * 2 * 128
    a = dict(xbc=P[0], n=4, h=6, p=64, g=2, k=128, xbcs_n=d, conv_state=P[1], l=3, st_s=3 * d, st_d=3, st_l=1,
             weight=P[2], w=4, bias=None, cache_seqlens=None, activation=1, dt=P[3], dt_dtype=0, ds_n=6, dt_bias=None,
             dt_softplus=1, a=P[4], d_skip=None, z=None, zs_n=0, zs_h=0, ssm_state=P[5], state_dtype=1, s=4,
             ss_s=6 * 64 * 128, state_indices=None, out=P[6], os_n=384, os_h=64, workspace=P[7], dev_status=None,
             stream=None)
    assert not set(over) - set(a)
    a.update(over)
    return dc.dcconv_conv_selective_update(*a.values())


def scan(**over):
    a = dict(x=P[0], n=2, t=100, h=6, p=64, xs_n=38400, xs_t=384, xs_h=64, dt=P[1], dt_dtype=0, ds_n=600, ds_t=6,
             dt_bias=None, dt_softplus=1, a=P[2], b=P[3], c=P[4], g=2, k=128, bs_n=25600, bs_t=256, bs_g=128,
             cs_n=25600, cs_t=256, cs_g=128, d_skip=None, z=None, zs_n=0, zs_t=0, zs_h=0, seq_starts=None,
             ssm_state=P[5], state_dtype=1, s=2, ss_s=6 * 64 * 128, state_indices=None, has_initial_state=None,
             out=P[6], os_n=38400, os_t=384, os_h=64, workspace=None, workspace_bytes=0, dev_status=None, stream=None)
    assert not set(over) - set(a)
    a.update(over)
    return dc.dcconv_selective_scan(*a.values())


def w4(**over):
    a = dict(x=P[0], m=4, k=256, xs_m=256, qweight=P[1], n=100, scales=P[2], zeros=None, group_size=128, bias=None,
             out=P[3], os_m=100, stream=None)
    assert not set(over) - set(a)
    a.update(over)
    return dc.dcconv_w4_matvec(*a.values())


SHARED = [  # of the recurrence's three entry points
    (dict(n=-1), dc.DCCONV_EINVAL, "n must"),
    (dict(h=0), dc.DCCONV_EINVAL, ">= 1"),
    (dict(p=0), dc.DCCONV_EINVAL, ">= 1"),
    (dict(k=0), dc.DCCONV_EINVAL, ">= 1"),
    (dict(g=4), dc.DCCONV_EINVAL, "divide"),
    (dict(dt_dtype=2), dc.DCCONV_EINVAL, "dt_dtype"),
    (dict(state_dtype=-1), dc.DCCONV_EINVAL, "state_dtype"),
    (dict(k=257), dc.DCCONV_EUNSUPPORTED, "256"),
    (dict(h=1 << 20, p=1 << 10, g=1), dc.DCCONV_EUNSUPPORTED, "2^26"),
    (dict(s=-1), dc.DCCONV_EINVAL, "s and ss_s"),
    (dict(s=1), dc.DCCONV_EINVAL, "slot"),
    (dict(ss_s=100), dc.DCCONV_EINVAL, "overlap"),
    (dict(ds_n=-1), dc.DCCONV_EINVAL, "non-negative"),
    (dict(os_n=100), dc.DCCONV_EINVAL, "same address"),
    (dict(os_h=32), dc.DCCONV_EINVAL, "same address"),
    (dict(a=None), dc.DCCONV_EINVAL, "non-NULL"),
    (dict(out=None), dc.DCCONV_EINVAL, "non-NULL"),
    (dict(ssm_state=None, state_indices=P[9]), dc.DCCONV_EINVAL, "non-NULL"),
    (dict(out=P[6] + 1), dc.DCCONV_EINVAL, "aligned"),
    (dict(ssm_state=P[5] + 2), dc.DCCONV_EINVAL, "aligned"),
    (dict(dev_status=P[8] + 2), dc.DCCONV_EINVAL, "aligned"),
    (dict(out=P[5] + 64), dc.DCCONV_EINVAL, "overlaps"),
    (dict(state_indices=P[6] + 64), dc.DCCONV_EINVAL, "overlaps"),
    (dict(ss_s=1 << 60), dc.DCCONV_EINVAL, "2^47"),
]


def refused(call, over, code, text):
    assert call(**over) == code
    assert text in dc.dcconv_last_error(), dc.dcconv_last_error()
    assert dc.dcconv_last_kernel() == ""


@no_gpu
@pytest.mark.parametrize("call", [update, fused, scan])
@pytest.mark.parametrize("over,code,text", SHARED)
def test_shared_refusals(call, over, code, text):
    if call is scan and over == dict(os_n=100):
        over = dict(os_n=100, os_t=384)
    refused(call, over, code, text)


@no_gpu
@pytest.mark.parametrize("over,code,text", [
    (dict(xs_h=-64), dc.DCCONV_EINVAL, "non-negative"), (dict(b=None), dc.DCCONV_EINVAL, "non-NULL"),
    (dict(out=P[0] + 64), dc.DCCONV_EINVAL, "overlaps x"), (dict(c=P[5] + 128), dc.DCCONV_EINVAL, "overlaps c"),
    (dict(xs_n=1 << 50), dc.DCCONV_EINVAL, "2^47"), (dict(z=P[6] + 2, zs_n=384, zs_h=64), dc.DCCONV_EINVAL, "overlaps z")])
def test_update_refusals(over, code, text):
    refused(update, over, code, text)


@no_gpu
@pytest.mark.parametrize("over,code,text", [
    (dict(w=3, l=3), dc.DCCONV_EUNSUPPORTED, "w=4"), (dict(l=2), dc.DCCONV_EINVAL, "w-1"),
    (dict(l=70000, st_d=70000, st_s=70000 * 1000), dc.DCCONV_EUNSUPPORTED, "65536"),
    (dict(activation=7), dc.DCCONV_EINVAL, "activation"), (dict(st_d=2), dc.DCCONV_EINVAL, "same address"),
    (dict(workspace=None), dc.DCCONV_EINVAL, "workspace"), (dict(workspace=P[5]), dc.DCCONV_EINVAL, "overlaps"),
    (dict(conv_state=None), dc.DCCONV_EINVAL, "non-NULL"), (dict(weight=P[1] + 8), dc.DCCONV_EINVAL, "overlaps weight"),
    (dict(cache_seqlens=P[8] + 1), dc.DCCONV_EINVAL, "aligned")])
def test_fused_refusals(over, code, text):
    refused(fused, over, code, text)


@no_gpu
@pytest.mark.parametrize("over,code,text", [
    (dict(t=-1), dc.DCCONV_EINVAL, "t (tokens)"), (dict(t=1 << 31), dc.DCCONV_EUNSUPPORTED, "tokens"),
    (dict(ssm_state=None, s=0, has_initial_state=P[9]), dc.DCCONV_EINVAL, "has_initial_state"),
    (dict(seq_starts=P[9] + 2), dc.DCCONV_EINVAL, "aligned"), (dict(seq_starts=P[6]), dc.DCCONV_EINVAL, "overlaps"),
    (dict(workspace_bytes=-1), dc.DCCONV_EINVAL, "non-negative"), (dict(os_t=100), dc.DCCONV_EINVAL, "same address"),
    (dict(n=1, t=100000, s=1), dc.DCCONV_EINVAL, "workspace"),
    (dict(n=1, t=100000, s=1, workspace=P[8], workspace_bytes=1000), dc.DCCONV_EINVAL, "workspace")])
def test_scan_refusals(over, code, text):
    refused(scan, over, code, text)


@no_gpu
@pytest.mark.parametrize("over,code,text", [
    (dict(m=-1), dc.DCCONV_EINVAL, "m must"), (dict(k=0), dc.DCCONV_EINVAL, ">= 1"), (dict(n=0), dc.DCCONV_EINVAL, ">= 1"),
    (dict(n=1 << 25), dc.DCCONV_EUNSUPPORTED, "2^24"), (dict(group_size=0), dc.DCCONV_EINVAL, "group_size"),
    (dict(group_size=48), dc.DCCONV_EUNSUPPORTED, "multiple of 32"), (dict(xs_m=-1), dc.DCCONV_EINVAL, "non-negative"),
    (dict(m=1 << 21), dc.DCCONV_EUNSUPPORTED, "rows"), (dict(x=None), dc.DCCONV_EINVAL, "non-NULL"),
    (dict(os_m=99), dc.DCCONV_EINVAL, "row stride"), (dict(qweight=P[1] + 8), dc.DCCONV_EINVAL, "aligned"),
    (dict(out=P[2]), dc.DCCONV_EINVAL, "overlaps"), (dict(xs_m=1 << 60), dc.DCCONV_EINVAL, "2^47")])
def test_w4_refusals(over, code, text):
    refused(w4, over, code, text)


@no_gpu
def test_pack_refusals():
    assert dc.dcconv_w4_pack(None, 16, 128, P[0], None) == dc.DCCONV_EINVAL
    assert dc.dcconv_w4_pack(P[0], 16, 128, P[0] + 512, None) == dc.DCCONV_EINVAL
    assert dc.dcconv_w4_pack(P[0], 0, 128, P[1], None) == dc.DCCONV_EINVAL


@no_gpu
def test_empty_calls_enqueue_nothing():
    for call, over in ((update, dict(n=0)), (fused, dict(n=0)), (scan, dict(n=0)), (w4, dict(m=0)),
                       (scan, dict(t=0, ssm_state=None, s=0))):
        assert call(**over) == dc.DCCONV_OK, dc.dcconv_last_error()
        assert dc.dcconv_last_kernel() == ""


def test_workspace_sizes():
    """None where no sequence is cut; otherwise a state and a decay a head for each segment."""
    assert dc.dcconv_selective_scan_workspace(8, 2048, 96, 64, 8, 128, 0) == 0
    assert dc.dcconv_selective_scan_workspace(1, 37, 24, 64, 2, 128, 0) == 0
    one = 4 * 24 * (64 * 128 + 1)
    need = dc.dcconv_selective_scan_workspace(1, 16381, 24, 64, 2, 128, 0)
    assert need > 0 and need % one == 0
    packed = dc.dcconv_selective_scan_workspace(5, 16381, 24, 64, 2, 128, 1)
    assert packed % one == 0 and packed >= 5 * one
    for bad in ((0, 100, 1, 1, 1, 1), (1, 0, 1, 1, 1, 1), (1, 100, 3, 1, 2, 1), (1, 100, 1, 1, 1, 300)):
        assert dc.dcconv_selective_scan_workspace(*bad, 0) == 0


def test_tensor_functions_refuse_what_they_cannot_take():
    x = torch.zeros(2, 4, 8, dtype=torch.bfloat16)
    B = torch.zeros(2, 1, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        dc.selective_update(x, torch.zeros(2, 4), torch.zeros(4), B, B, torch.zeros(2, 4, 8, 16))
    with pytest.raises(ValueError, match=r"\[N, H, P\]"):
        dc.selective_update(x[0], torch.zeros(2, 4), torch.zeros(4), B, B, torch.zeros(2, 4, 8, 16))
    with pytest.raises(ValueError, match="GPU"):
        dc.selective_scan(x[None], torch.zeros(1, 2, 4), torch.zeros(4), B[None], B[None])
    with pytest.raises(ValueError, match="GPU"):
        dc.w4_matvec(torch.zeros(1, 32), torch.zeros(1), torch.zeros(1, 16), group_size=32)
    with pytest.raises(ValueError, match="uint8"):
        dc.w4_pack(torch.zeros(4, 32))
