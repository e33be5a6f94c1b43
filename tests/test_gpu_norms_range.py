"""The norms over all sizes of values that FP32 and BF16 hold, subnormal ones among them: with eps 0
a norm does not depend on the scale.  The tolerances are those of ``test_gpu_norms``."""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from delta_reference import U, close, silu
from test_gpu_norms import E, bf, norm

pytestmark = pytest.mark.gpu
SIZES = [1e-44, 1e-42, 1e-40, 1e-38, 1e-30, 1e-25, 1e-20, 1e-15, 1e-12, 1.0, 1e15, 1e20, 1e30, 7e37]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


def check(out, v, w, eps, what):
    """(rows of zeros, as BF16 has for sizes below 2^-134, have no norm)"""
    want = norm(v, eps) * w
    live = v.square().sum(-1) > 0
    close(out[live.to(out.device)], want[live], (U + E) * want[live].abs(), what)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("D", [1, 64, 100, 512, 4096, 16384])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_residuals_of_every_size(size, D, kind):
    """Nothing is added, so that the sum is the residual; then a block's output of that size alone, and a
    first norm of it."""
    gen = torch.Generator().manual_seed(D)
    w = 1 + 0.3 * torch.randn(D, generator=gen)
    r = (torch.randn(5, D, generator=gen).double() * size).to(kind)
    for eps in (0.0, 1e-37, 1e-6):
        rd = r.cuda()
        out = dc.add_rms_norm(torch.zeros(5, D, dtype=torch.bfloat16, device="cuda"), rd, w.cuda(), eps=eps)
        assert torch.equal(rd.cpu(), r)
        check(out, r.double(), w.double(), eps, f"residual of size {size}, eps {eps}")
    x = (torch.randn(5, D, generator=gen).double() * size).to(torch.bfloat16)
    rd = torch.zeros(5, D, device="cuda")
    out = dc.add_rms_norm(x.cuda(), rd, w.cuda(), eps=0.0)
    assert torch.equal(rd.cpu(), x.float())
    check(out, x.double(), w.double(), 0.0, f"sum of size {size}")
    rd = torch.zeros(5, D, device="cuda")
    dc.add_rms_norm(x.cuda(), rd, w.cuda(), post_weight=w.cuda(), eps=0.0)
    live = x.double().square().sum(-1) > 0
    want = (norm(x.double(), 0.0) * w.double())[live]
    close(rd[live.cuda()], want, E * want.abs(), f"first norm of size {size}")


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("D", [64, 512, 4096])
def test_gated_rows_of_every_size(size, D):
    gen = torch.Generator().manual_seed(D)
    x, z = (torch.randn(5, D, generator=gen).double() * size).to(torch.bfloat16), bf(gen, 5, D)
    w = 1 + 0.3 * torch.randn(D, generator=gen)
    for eps in (0.0, 1e-37):
        check(dc.gated_rms_norm(x.cuda(), None, w.cuda(), eps=eps), x.double(), w.double(), eps, f"rows of size {size}")
        check(dc.gated_rms_norm(x.cuda(), z.cuda(), w.cuda(), eps=eps), x.double(), w.double() * silu(z.double()), eps,
              f"gated rows of size {size}")


def test_rows_of_mixed_sizes():
    """A row's small values keep their bits beside large ones, and its mean goes by the large ones."""
    gen = torch.Generator().manual_seed(1)
    sizes = 10.0 ** (torch.rand(64, 512, generator=gen).double() * 30 - 44)
    r = (torch.randn(64, 512, generator=gen).double() * sizes).float()
    w = torch.ones(512)
    out = dc.add_rms_norm(torch.zeros(64, 512, dtype=torch.bfloat16, device="cuda"), r.cuda(), w.cuda(), eps=0.0)
    want = norm(r.double(), 0.0)
    # (subnormal results, below 2^-126, are rounded to multiples of 2^-133)
    close(out, want, (U + E) * want.abs() + 2.0 ** -134, "mixed sizes")


def test_rows_of_zeros_without_eps():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    assert bool(torch.isnan(dc.gated_rms_norm(x, None, w, eps=0.0)).all())
    assert bool(torch.isnan(dc.add_rms_norm(x, torch.zeros(2, 64, device="cuda"), w, eps=0.0)).all())
    assert not dc.add_rms_norm(x, torch.zeros(2, 64, device="cuda"), w, eps=1e-45).any()
