"""Refusals of the gated delta rule's and the norms' entry points, and the workspace sizes: host
logic, no GPU.

Each call is a valid one with one argument changed; the made-up device addresses are never
dereferenced, so these run only where no GPU is visible.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from test_selective_abi_cpu import P, no_gpu, refused

INF, NAN = float("inf"), float("nan")


def update(**over):
    a = dict(q=P[0], key=P[1], v=P[2], n=4, h=6, p=64, g=2, k=128, qs_n=256, qs_g=128, ks_n=256, ks_g=128, vs_n=384,
             vs_h=64, dt=P[3], dt_dtype=0, ds_n=6, dt_bias=None, dt_softplus=1, a=P[4], beta=P[5], beta_dtype=0, es_n=6,
             beta_sigmoid=1, qk_l2norm=1, l2norm_eps=1e-6, scale=0.1, state=P[6], state_dtype=1, s=4, ss_s=6 * 64 * 128,
             state_indices=None, out=P[7], os_n=384, os_h=64, dev_status=None, stream=None)
    assert not set(over) - set(a)
    a.update(over)
    return dc.dcconv_gated_delta_update(*a.values())


def scan(**over):
    a = dict(q=P[0], key=P[1], v=P[2], n=2, t=100, h=6, p=64, g=2, k=128, qs_n=25600, qs_t=256, qs_g=128, ks_n=25600,
             ks_t=256, ks_g=128, vs_n=38400, vs_t=384, vs_h=64, dt=P[3], dt_dtype=0, ds_n=600, ds_t=6, dt_bias=None,
             dt_softplus=1, a=P[4], beta=P[5], beta_dtype=0, es_n=600, es_t=6, beta_sigmoid=1, qk_l2norm=1,
             l2norm_eps=1e-6, scale=0.1, seq_starts=None, state=P[6], state_dtype=1, s=2, ss_s=6 * 64 * 128,
             state_indices=None, has_initial_state=None, out=P[7], os_n=38400, os_t=384, os_h=64, workspace=None,
             workspace_bytes=0, dev_status=None, stream=None)
    assert not set(over) - set(a)
    a.update(over)
    return dc.dcconv_gated_delta_scan(*a.values())


def gated(**over):
    a = dict(x=P[0], n=2, t=5, h=3, d=128, xs_n=1920, xs_t=384, xs_h=128, z=P[1], zs_n=1920, zs_t=384, zs_h=128,
             gate_first=0, weight=P[2], weight_dtype=0, ws_h=0, weight_offset=0.0, eps=1e-6, out=P[3], os_n=1920, os_t=384,
             os_h=128, stream=None)
    assert not set(over) - set(a)
    a.update(over)
    return dc.dcconv_gated_rms_norm(*a.values())


def added(**over):
    a = dict(x=P[0], n=2, t=5, d=512, xs_n=2560, xs_t=512, residual=P[1], residual_dtype=1, rs_n=2560, rs_t=512, gate=P[2],
             gs_n=2560, gs_t=512, residual_scale=1.0, post_weight=P[3], weight=P[4], weight_dtype=0, weight_offset=0.0,
             eps=1e-6, out=P[5], os_n=2560, os_t=512, stream=None)
    assert not set(over) - set(a)
    a.update(over)
    return dc.dcconv_add_rms_norm(*a.values())


SHARED = [  # of the rule's two entry points
    (dict(n=-1), dc.DCCONV_EINVAL, "n must"),
    (dict(h=0), dc.DCCONV_EINVAL, ">= 1"),
    (dict(k=0), dc.DCCONV_EINVAL, ">= 1"),
    (dict(g=4), dc.DCCONV_EINVAL, "divide"),
    (dict(dt_dtype=2), dc.DCCONV_EINVAL, "dt_dtype"),
    (dict(beta_dtype=-1), dc.DCCONV_EINVAL, "beta_dtype"),
    (dict(state_dtype=3), dc.DCCONV_EINVAL, "state_dtype"),
    (dict(l2norm_eps=0.0), dc.DCCONV_EINVAL, "l2norm_eps"),
    (dict(l2norm_eps=NAN), dc.DCCONV_EINVAL, "l2norm_eps"),
    (dict(l2norm_eps=INF), dc.DCCONV_EINVAL, "l2norm_eps"),
    (dict(scale=NAN), dc.DCCONV_EINVAL, "scale"),
    (dict(scale=-INF), dc.DCCONV_EINVAL, "scale"),
    (dict(k=257), dc.DCCONV_EUNSUPPORTED, "256"),
    (dict(h=1 << 20, p=1 << 10, g=1), dc.DCCONV_EUNSUPPORTED, "2^26"),
    (dict(n=(1 << 31) - 5), dc.DCCONV_EUNSUPPORTED, "2^24"),
    (dict(s=-1), dc.DCCONV_EINVAL, "s and ss_s"),
    (dict(s=1), dc.DCCONV_EINVAL, "slot"),
    (dict(ss_s=100), dc.DCCONV_EINVAL, "overlap"),
    (dict(ds_n=-1), dc.DCCONV_EINVAL, "non-negative"),
    (dict(es_n=-6), dc.DCCONV_EINVAL, "non-negative"),
    (dict(os_h=32), dc.DCCONV_EINVAL, "same address"),
    (dict(a=None), dc.DCCONV_EINVAL, "non-NULL"),
    (dict(key=None), dc.DCCONV_EINVAL, "non-NULL"),
    (dict(beta=None), dc.DCCONV_EINVAL, "non-NULL"),
    (dict(out=None), dc.DCCONV_EINVAL, "non-NULL"),
    (dict(state=None, state_indices=P[9]), dc.DCCONV_EINVAL, "non-NULL"),
    (dict(out=P[7] + 1), dc.DCCONV_EINVAL, "aligned"),
    (dict(state=P[6] + 2), dc.DCCONV_EINVAL, "aligned"),
    (dict(dt=P[3] + 2, dt_dtype=1), dc.DCCONV_EINVAL, "aligned"),
    (dict(dev_status=P[8] + 2), dc.DCCONV_EINVAL, "aligned"),
    (dict(out=P[2] + 64), dc.DCCONV_EINVAL, "overlaps v"),
    (dict(state=P[1] + 256), dc.DCCONV_EINVAL, "overlaps key"),
    (dict(out=P[6] + 64), dc.DCCONV_EINVAL, "overlaps"),
    (dict(state_indices=P[7] + 64), dc.DCCONV_EINVAL, "overlaps"),
    (dict(ss_s=1 << 60), dc.DCCONV_EINVAL, "2^47"),
]


@no_gpu
@pytest.mark.parametrize("call", [update, scan])
@pytest.mark.parametrize("over,code,text", SHARED)
def test_shared_refusals(call, over, code, text):
    refused(call, over, code, text)


@no_gpu
@pytest.mark.parametrize("over,code,text", [
    (dict(t=-1), dc.DCCONV_EINVAL, "t (tokens)"), (dict(t=1 << 31), dc.DCCONV_EUNSUPPORTED, "tokens"),
    (dict(state=None, s=0, has_initial_state=P[9]), dc.DCCONV_EINVAL, "has_initial_state"),
    (dict(state=None, s=0, state_indices=P[9]), dc.DCCONV_EINVAL, "state_indices"),
    (dict(seq_starts=P[9] + 2), dc.DCCONV_EINVAL, "aligned"), (dict(seq_starts=P[7]), dc.DCCONV_EINVAL, "overlaps"),
    (dict(workspace_bytes=-1), dc.DCCONV_EINVAL, "non-negative"), (dict(os_t=100), dc.DCCONV_EINVAL, "same address"),
    (dict(qs_t=1 << 50), dc.DCCONV_EINVAL, "2^47"),
    (dict(n=1, t=100000, s=1), dc.DCCONV_EINVAL, "workspace"),
    (dict(n=1, t=100000, s=1, workspace=P[8], workspace_bytes=1000), dc.DCCONV_EINVAL, "workspace"),
    (dict(n=1, t=16381, s=1, workspace=P[8] + 8, workspace_bytes=1 << 40), dc.DCCONV_EINVAL, "aligned"),
    (dict(n=1, t=16381, s=1, workspace=P[6], workspace_bytes=1 << 40), dc.DCCONV_EINVAL, "overlaps")])
def test_scan_refusals(over, code, text):
    refused(scan, over, code, text)


@no_gpu
@pytest.mark.parametrize("call,over,code,text", [
    (gated, dict(n=-1), dc.DCCONV_EINVAL, "n, t and h"), (gated, dict(d=0), dc.DCCONV_EINVAL, "d must"),
    (gated, dict(d=16385), dc.DCCONV_EUNSUPPORTED, "16384"), (gated, dict(weight_dtype=2), dc.DCCONV_EINVAL, "weight_dtype"),
    (gated, dict(eps=-1.0), dc.DCCONV_EINVAL, "eps"), (gated, dict(eps=NAN), dc.DCCONV_EINVAL, "eps"),
    (gated, dict(weight_offset=INF), dc.DCCONV_EINVAL, "weight_offset"), (gated, dict(xs_t=-1), dc.DCCONV_EINVAL, "non-neg"),
    (gated, dict(n=1 << 40, t=1 << 20), dc.DCCONV_EUNSUPPORTED, "2^40"), (gated, dict(x=None), dc.DCCONV_EINVAL, "non-NULL"),
    (gated, dict(os_h=100), dc.DCCONV_EINVAL, "same address"), (gated, dict(out=P[0]), dc.DCCONV_EINVAL, "overlaps x"),
    (gated, dict(out=P[2]), dc.DCCONV_EINVAL, "overlaps"), (gated, dict(z=P[1] + 1), dc.DCCONV_EINVAL, "aligned"),
    (gated, dict(xs_n=1 << 60), dc.DCCONV_EINVAL, "2^47"),
    (added, dict(t=-1), dc.DCCONV_EINVAL, "n, t and h"), (added, dict(d=1 << 20), dc.DCCONV_EUNSUPPORTED, "16384"),
    (added, dict(residual_dtype=7), dc.DCCONV_EINVAL, "residual_dtype"), (added, dict(weight=None), dc.DCCONV_EINVAL, "non-NULL"),
    (added, dict(residual_scale=NAN), dc.DCCONV_EINVAL, "residual_scale"), (added, dict(eps=INF), dc.DCCONV_EINVAL, "eps"),
    (added, dict(rs_t=256), dc.DCCONV_EINVAL, "its own address"), (added, dict(residual=P[0]), dc.DCCONV_EINVAL, "overlaps"),
    (added, dict(out=P[1]), dc.DCCONV_EINVAL, "overlaps"), (added, dict(residual=P[1] + 2), dc.DCCONV_EINVAL, "aligned"),
    (added, dict(gs_n=-1), dc.DCCONV_EINVAL, "non-neg"), (added, dict(gs_t=1 << 50), dc.DCCONV_EINVAL, "2^47")])
def test_norm_refusals(call, over, code, text):
    refused(call, over, code, text)


@no_gpu
def test_empty_calls_enqueue_nothing():
    for call, over in ((update, dict(n=0)), (scan, dict(n=0)), (scan, dict(t=0, state=None, s=0)), (gated, dict(t=0)),
                       (gated, dict(n=0, x=None, out=None)), (gated, dict(h=0)), (added, dict(n=0)), (added, dict(t=0))):
        assert call(**over) == dc.DCCONV_OK, dc.dcconv_last_error()
        assert dc.dcconv_last_kernel() == ""


def test_workspace_sizes():
    """None where no sequence is cut; otherwise what each segment does to a state, [p, k] and [k, k]
    floats a head."""
    size = dc.dcconv_gated_delta_scan_workspace
    assert size(8, 2048, 32, 128, 16, 128, 0) == 0
    assert size(1, 37, 8, 128, 4, 128, 0) == 0
    one = 4 * 16 * (128 + 128) * 128
    need = size(1, 16381, 16, 128, 8, 128, 0)
    assert need >= 2 * one and need % one == 0
    packed = size(3, 16381, 16, 128, 8, 128, 1)
    assert packed >= 3 * one and packed % one == 0
    # grows with the tokens, by no more than a segment of them each
    assert size(1, 1 << 20, 16, 128, 8, 128, 0) <= 64 * one
    for bad in ((0, 100, 1, 1, 1, 1), (1, 0, 1, 1, 1, 1), (1, 100, 3, 1, 2, 1), (1, 100, 1, 1, 1, 300), (1, 100, 0, 1, 1, 1)):
        assert size(*bad, 0) == 0


def test_tensor_functions_refuse_what_they_cannot_take():
    v = torch.zeros(2, 4, 8, dtype=torch.bfloat16)
    k = torch.zeros(2, 1, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        dc.gated_delta_update(k, k, v, torch.zeros(2, 4), torch.zeros(4), torch.zeros(2, 4), torch.zeros(2, 4, 8, 16))
    with pytest.raises(ValueError, match=r"\[N, H, P\]"):
        dc.gated_delta_update(k, k, v[0], torch.zeros(2, 4), torch.zeros(4), torch.zeros(2, 4), torch.zeros(2, 4, 8, 16))
    with pytest.raises(ValueError, match="GPU"):
        dc.gated_delta_scan(k[None], k[None], v[None], torch.zeros(1, 2, 4), torch.zeros(4), torch.zeros(1, 2, 4))
    with pytest.raises(ValueError, match=r"\[N, T, H, P\]"):
        dc.gated_delta_scan(k, k, v, torch.zeros(2, 4), torch.zeros(4), torch.zeros(2, 4))
    with pytest.raises(ValueError, match="GPU"):
        dc.gated_rms_norm(v, v, torch.ones(8))
    with pytest.raises(ValueError, match="dimensions"):
        dc.gated_rms_norm(v[None, None, None], None, None)
    with pytest.raises(ValueError, match="GPU"):
        dc.add_rms_norm(v, v, torch.ones(8))
    with pytest.raises(ValueError, match="dimensions"):
        dc.add_rms_norm(v[None], v[None, None], torch.ones(8))
