"""The gated norm and the residual norm on the GPU against their 64-bit forms.

FP32 sums over at most 16384 squares (a tree over lanes behind at most 64 in a row: under
2^-16 of the sum, half of that in its root), products and SiLU (its exponential and reciprocal
within 2^-21) stay under 2^-15 of a result; where it is stored as BF16 it is rounded once, u =
2^-8 of itself.  A residual in F32 is a sum: 2^-15 of the added term and 2^-23 of the sum; the
norm of a sum is off by what its terms' magnitudes are off.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from delta_reference import U, close, silu

pytestmark = pytest.mark.gpu
E = 2.0 ** -15


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


def bf(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(torch.bfloat16)


def norm(v, eps):
    return v / (v.square().mean(-1, keepdim=True) + eps).sqrt()


def strided(t, pad=8):
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + pad, dtype=t.dtype, device="cuda")
    wide[..., :t.shape[-1]] = t.cuda()
    return wide[..., :t.shape[-1]]


def gated(seed, shape, first=False, z=True, weight="row", kind=torch.bfloat16, offset=0.0, eps=1e-6, scale=1.0,
          place=lambda t: t.cuda(), **more):
    gen = torch.Generator().manual_seed(seed)
    x, zt = bf(gen, *shape, scale=scale), bf(gen, *shape) if z else None
    wshape = shape[-1:] if weight == "row" else shape[-2:]
    w = None if weight is None else (1 + 0.3 * torch.randn(*wshape, generator=gen)).to(kind)
    out = dc.gated_rms_norm(place(x), None if zt is None else place(zt), None if w is None else w.cuda(), eps=eps,
                            gate_first=first, weight_offset=offset, **more)
    gate = silu(zt.double()) if z else 1.0
    v = norm(x.double() * gate, eps) if first else norm(x.double(), eps) * gate
    v = v * (1.0 if w is None else w.double() + offset)
    # an offset that takes a weight near zero leaves its rounding: 2^-23 of the offset
    more_off = 0 if w is None else 2.0 ** -23 * abs(offset) * (v / (w.double() + offset).where(w.double() + offset != 0, torch.ones(()).double())).abs()
    close(out, v, (U + E) * v.abs() + more_off, f"gated norm of {shape}")
    return out


@pytest.mark.parametrize("D", [1, 2, 7, 8, 16, 64, 72, 120, 128, 129, 200, 256, 257, 512, 520, 1000, 1024, 1025, 2048, 4096,
                               4104, 8192, 9000, 16384])
@pytest.mark.parametrize("first", [False, True])
def test_gated_sizes(D, first):
    gated(D, (3, 2, D), first)
    gated(D + 1, (1, D), first)
    gated(D + 2, (D,), first)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("weight", ["row", "heads", None])
def test_gated_options(kind, weight):
    gated(1, (2, 5, 3, 128), weight=weight, kind=kind)
    gated(2, (2, 5, 3, 128), weight=weight, kind=kind, offset=1.0, z=False)
    gated(3, (2, 5, 3, 96), weight=weight, kind=kind, offset=-1.0, first=True, eps=0.1)


def test_gated_views():
    for pad in (8, 3):
        gated(4, (2, 5, 3, 128), place=lambda t: strided(t, pad))
    gated(5, (2, 5, 3, 40), place=lambda t: t.cuda().transpose(1, 2).contiguous().transpose(1, 2))
    buf = torch.full((7, 4, 96), 3.0, dtype=torch.bfloat16, device="cuda")
    gated(6, (7, 2, 80), out=buf[:, 1:3, 8:88])
    assert bool((buf[:, 0] == 3).all() and (buf[:, 3] == 3).all() and (buf[:, :, :8] == 3).all()
                and (buf[:, :, 88:] == 3).all())


def test_gated_many_rows():
    gated(7, (3001, 9, 64))
    gated(8, (1100, 1100))


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30, 3e37])
@pytest.mark.parametrize("D", [64, 512, 4096])
def test_gated_values_of_every_size(scale, D):
    """Squares that leave FP32's range: with eps 0 a norm does not depend on the scale."""
    gated(9, (4, D), scale=scale, eps=0.0)
    gated(10, (4, D), scale=scale, eps=1e-6)


def test_gated_rows_of_zeros_and_what_is_not_finite():
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    assert not dc.gated_rms_norm(x, None, w).any()
    x[1, 3] = float("nan")
    x[2, 3] = float("inf")
    x[3] = 1.0
    out = dc.gated_rms_norm(x, None, w)
    assert not out[0].any() and bool(torch.isnan(out[1]).all()) and bool((out[3] == 1).all())
    assert bool(torch.isnan(out[2, 3])) and int(torch.isnan(out[2]).sum()) == 1


def added(seed, shape, residual=torch.float32, post=False, gate=None, scale=0.75, kind=torch.bfloat16, offset=0.0,
          eps=1e-6, place=lambda t: t.cuda(), **more):
    gen = torch.Generator().manual_seed(seed)
    D = shape[-1]
    x, r = bf(gen, *shape), (2 * torch.randn(*shape, generator=gen)).to(residual)
    g = None if gate is None else bf(gen, *(shape if gate == "each" else (D,)))
    w, pw = ((1 + 0.3 * torch.randn(D, generator=gen)).to(kind) for _ in range(2))
    rd = place(r)
    gd = None if g is None else place(g) if gate == "each" else g.cuda().expand(shape)
    out = dc.add_rms_norm(place(x), rd, w.cuda(), post_weight=pw.cuda() if post else None, gate=gd, residual_scale=scale,
                          eps=eps, weight_offset=offset, **more)
    y = x.double()
    if post:
        y = norm(y, eps) * (pw.double() + offset)
    y = scale * y * (1.0 if g is None else g.double())
    s = r.double() + y
    ds = E * y.abs() + 2.0 ** -23 * s.abs()
    if post:
        ds = ds + 2.0 ** -22 * abs(scale * offset) * (1.0 if g is None else g.double().abs()) * norm(x.double(), eps).abs()
    close(rd, s, ds + (U * (s.abs() + ds) if residual == torch.bfloat16 else 0), f"residual of {shape}")
    wd = w.double() + offset
    root = (s.square().mean(-1, keepdim=True) + eps).sqrt()
    # the sum's own error, and what it moves the root by
    doff = ds / root + (s / root).abs() * (ds.square().mean(-1, keepdim=True).sqrt() / root)
    v = s / root * wd
    bound = (doff + E * (s / root).abs()) * wd.abs() + 2.0 ** -22 * abs(offset) * (s / root).abs()
    close(out, v, bound + U * (v.abs() + bound), f"norm of {shape}")
    return out


@pytest.mark.parametrize("D", [1, 2, 7, 8, 16, 64, 72, 128, 129, 256, 257, 512, 1000, 1024, 1025, 2048, 4096, 4104, 8192,
                               16384])
@pytest.mark.parametrize("residual", [torch.float32, torch.bfloat16])
def test_add_sizes(D, residual):
    added(D, (3, 2, D), residual)
    added(D + 1, (5, D), residual, post=True, gate="each")
    added(D + 2, (D,), residual, post=True)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "each", "shared"])
def test_add_options(kind, residual, post, gate):
    added(1, (3, 5, 320), residual, post, gate, kind=kind)
    added(2, (3, 5, 4096), residual, post, gate, kind=kind, offset=1.0, scale=-1.5, eps=0.01)
    added(3, (2, 1031), residual, post, gate, kind=kind, scale=0.0)


def test_add_views():
    for pad in (8, 3):
        added(4, (3, 5, 96), place=lambda t: strided(t, pad), post=True, gate="each")
        added(5, (3, 5, 96), torch.bfloat16, place=lambda t: strided(t, pad))
    buf = torch.full((7, 96), 3.0, dtype=torch.bfloat16, device="cuda")
    added(6, (7, 80), out=buf[:, 8:88])
    assert bool((buf[:, :8] == 3).all() and (buf[:, 88:] == 3).all())


def test_add_touches_only_its_residual():
    gen = torch.Generator().manual_seed(7)
    wide = torch.full((4, 6, 200), 2.0, device="cuda")
    before = wide.clone()
    x = bf(gen, 4, 3, 128).cuda()
    dc.add_rms_norm(x, wide[:, 1:4, 40:168], torch.ones(128, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(wide[:, 1:4, 40:168], before[:, 1:4, 40:168] + x.float())
    wide[:, 1:4, 40:168] = 2.0
    assert torch.equal(wide, before)


def test_norms_in_a_graph_and_on_another_stream():
    gen = torch.Generator().manual_seed(8)
    x, z = bf(gen, 40, 4, 128).cuda(), bf(gen, 40, 4, 128).cuda()
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    w5 = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    res = torch.randn(40, 512, generator=gen).cuda()
    ref = res.clone()

    def both(r):
        y = dc.gated_rms_norm(x, z, w)
        return y, dc.add_rms_norm(y.flatten(1), r, w5, post_weight=w5)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        mine = both(res.clone())
    torch.cuda.current_stream().wait_stream(stream)
    want = both(res.clone())
    assert all(torch.equal(a, b) for a, b in zip(mine, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(res)
    for _ in range(4):
        want = both(ref)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(ref, res)
