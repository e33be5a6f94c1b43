"""Products with 4-bit weights on the GPU against their 64-bit form.

Bound, per element: the products of BF16 x with 128 + code, their sums over a group
and the offset's removal are FP32 (relative error 2^-24 each) on terms of up to 143
times |x|, at most 16 times the sum of |x (code - zero)| + |x| they stand for; with
groups' and waves' sums of under 2^9 terms added in sequence this is under 2^-11 of
sum |x| scale, and one rounding to BF16: 2^-8 of the result.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from selective_reference import U, close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


class Product:
    def __init__(self, seed, M, N, K, gs, zeros, bias, pad=0):
        gen = torch.Generator().manual_seed(seed)
        self.M, self.N, self.K, self.gs = M, N, K, gs
        groups = -(-K // gs)
        self.x = torch.randn(M, K, generator=gen).to(torch.bfloat16)
        self.codes = torch.randint(0, 16, (N, K), generator=gen, dtype=torch.uint8)
        self.scales = ((0.5 + torch.rand(groups, N, generator=gen)) * 0.05).to(torch.bfloat16)
        self.zeros = torch.randint(0, 16, (groups, N), generator=gen, dtype=torch.uint8) if zeros else None
        self.bias = torch.randn(N, generator=gen).to(torch.bfloat16) if bias else None
        self.pad = pad

    def call(self, out=None):
        wide = torch.full((self.M, self.K + self.pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :self.K] = self.x.cuda()
        return dc.w4_matvec(wide[:, :self.K], dc.w4_pack(self.codes.cuda()), self.scales.cuda(),
                            None if self.zeros is None else self.zeros.cuda(),
                            None if self.bias is None else self.bias.cuda(), group_size=self.gs, out=out)

    def check(self, out=None):
        got = self.call(out)
        group = torch.arange(self.K) // self.gs
        scale = self.scales.double()[group].t()
        w = (self.codes.double() - (8 if self.zeros is None else self.zeros.double()[group].t())) * scale
        want = self.x.double() @ w.t()
        size = self.x.double().abs() @ scale.t()
        if self.bias is not None:
            want = want + self.bias.double()
        close(got, want, U * want.abs() + 2.0 ** -11 * size, f"{self.M} x {self.N} x {self.K}")


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 130])
@pytest.mark.parametrize("N,K", [(48, 256), (33, 160)])
def test_rows(M, N, K):
    Product(M, M, N, K, 32, True, True).check()


@pytest.mark.parametrize("N,K", [(1, 1), (16, 128), (17, 129), (100, 96), (15, 1000), (513, 32), (31, 4096), (4112, 64)])
@pytest.mark.parametrize("gs", [32, 64, 96, 128, 256])
def test_sizes_and_groups(N, K, gs):
    Product(N + K, 3, N, K, gs, True, False).check()
    Product(N + K, 3, N, K, gs, False, True).check()


def test_strided_rows():
    Product(1, 5, 40, 256, 64, True, True, pad=8).check()
    Product(2, 5, 40, 256, 64, True, True, pad=3).check()
    buf = torch.full((5, 60), 7.0, dtype=torch.bfloat16, device="cuda")
    Product(3, 5, 40, 256, 128, True, True).check(out=buf[:, 10:50])
    assert bool((buf[:, :10] == 7).all() and (buf[:, 50:] == 7).all())


def test_no_rows():
    assert Product(4, 0, 40, 128, 128, False, False).call().shape == (0, 40)


def test_pack_lays_out_every_code_once():
    codes = torch.randint(0, 16, (37, 300), dtype=torch.uint8)
    q = dc.w4_pack(codes.cuda()).cpu()
    assert q.shape == (3, 3, 64, 16)
    for n, k in ((0, 0), (36, 299), (5, 130), (16, 128), (20, 77)):
        t = q[n // 16, k // 128]
        j = k % 128
        lane, word, rest = 16 * (j % 32 // 8) + n % 16, j // 32, j % 8
        v, half, u = rest // 4, rest % 4 // 2, rest % 2
        assert int(t[lane, 4 * word + 2 * u + v]) >> (4 * half) & 15 == int(codes[n, k])


def test_a_bad_value_stays_in_its_row():
    case = Product(5, 4, 40, 256, 64, True, True)
    want = case.call().clone()
    case.x[2, 100] = float("nan")
    got = case.call()
    assert bool(torch.isnan(got[2]).all())
    keep = torch.tensor([0, 1, 3], device="cuda")
    assert torch.equal(got[keep], want[keep])


def test_graph_replays_and_another_stream():
    case = Product(6, 2, 64, 512, 128, False, True)
    want = case.call().clone()
    x, q, s, b = case.x.cuda(), dc.w4_pack(case.codes.cuda()), case.scales.cuda(), case.bias.cuda()
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dc.w4_matvec(x, q, s, None, b, group_size=128, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dc.w4_matvec(x, q, s, None, b, group_size=128, out=out)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_offsets_past_32_bits():
    case = Product(7, 2, 40, 128, 128, False, False)
    row = (1 << 31) + 8
    buf = torch.empty(row + 128, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 128), (row, 1))
    x.copy_(case.x)
    got = dc.w4_matvec(x, dc.w4_pack(case.codes.cuda()), case.scales.cuda(), group_size=128)
    assert torch.equal(got, case.call())
