"""The gated delta rule's rarer paths: sequences cut into segments, blocks of 128 rows, many packed
sequences in the order of their lengths, more blocks than a grid's first axis holds, offsets past 4
GiB, workspaces, and calls side by side.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from delta_reference import U, close
from test_gpu_delta import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("H,P,G,K", [(2, 32, 1, 64), (2, 128, 1, 128), (1, 72, 1, 40), (2, 16, 2, 200), (1, 130, 1, 65)])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_cut_sequences(H, P, G, K, state):
    Case(H * P, [1601, 1601], H, P, G, K, state=state, init=[True, False]).check()
    assert dc.dcconv_last_kernel().startswith("delta_scan_split")


def test_cut_sequences_without_decay():
    """All of the state carried through every segment's matrix."""
    case = Case(40, [1500], 1, 32, 1, 64, state=torch.float32, init=[True], rate=0.0)
    case.check()
    assert dc.dcconv_last_kernel().startswith("delta_scan_split")


def test_cut_packed_sequences():
    for state in (torch.float32, torch.bfloat16):
        Case(41, [900, 1, 0, 2200, 640, 257, 1280], 2, 64, 1, 64, state=state, packed=True, slots=9,
             table=[4, 0, 1, 2, -1, 3, 8], init=[True, False, True, True, True, False, True]).check()
        assert dc.dcconv_last_kernel().startswith("delta_scan_split")
    Case(42, [2000, 1500], 2, 40, 1, 33, packed=True).check(return_final_state=True)
    assert dc.dcconv_last_kernel() == "delta_scan_split_scalar"
    Case(43, [1800, 1500], 2, 64, 1, 64, packed=True, state=torch.float32, table=[-1, 0], init=[True, True]).check()


@pytest.mark.parametrize("what", ["q", "k", "v", "beta", "dt"])
def test_cut_sequences_not_finite(what):
    """A NaN in the middle of a segment reaches what is behind it, and no earlier token, other head or
    channel of v, through the segments' matrices either."""
    t0 = 700
    case = Case(45, [1601], 2, 32, 2, 64, state=torch.float32, init=[True], logit=False, soft=False, f32=True)
    clean = case.call()
    assert dc.dcconv_last_kernel().startswith("delta_scan_split")
    clean_pool = case.pool
    at = {"q": (0, t0, 1, 5), "k": (0, t0, 1, 5), "v": (0, t0, 1, 7), "beta": (0, t0, 1), "dt": (0, t0, 1)}[what]
    getattr(case, what)[at] = float("nan")
    out, pool = case.call(), case.pool
    fine = torch.isfinite(out)
    assert torch.equal(out[0, :, 0], clean[0, :, 0]) and torch.equal(out[0, :t0], clean[0, :t0])
    assert torch.equal(pool[0, 0], clean_pool[0, 0])
    if what == "q":
        assert not fine[0, t0, 1].any() and torch.equal(out[0, t0 + 1:], clean[0, t0 + 1:])
        assert torch.equal(pool, clean_pool)
        return
    if what == "v":
        others = [p for p in range(32) if p != 7]
        assert not fine[0, t0:, 1, 7].any() and torch.equal(out[..., others], clean[..., others])
        assert not torch.isfinite(pool[0, 1, 7]).any() and torch.equal(pool[:, :, others], clean_pool[:, :, others])
        return
    assert not fine[0, t0:, 1].any() and not torch.isfinite(pool[0, 1]).any()


def test_cut_sequences_do_not_read_the_workspace_before_they_write_it():
    case = Case(44, [1601], 2, 64, 1, 64, state=torch.float32, init=[True])
    need = dc.dcconv_gated_delta_scan_workspace(1, 1601, 2, 64, 1, 64, 0)
    assert need > 0
    buf = torch.full((need // 4 + 64,), float("nan"), device="cuda")
    first = case.call(workspace=buf[:need // 4].view(torch.uint8))
    state = case.pool
    assert bool(torch.isnan(buf[need // 4:]).all()), "written past the workspace's end"
    buf.fill_(3.0e38)
    assert torch.equal(first, case.call(workspace=buf.view(torch.uint8))) and torch.equal(state, case.pool)
    case.check()


def test_cut_sequences_in_two_graphs_that_share_a_workspace():
    """Replayed one after the other on a stream: each call writes all that it reads of it."""
    cases = [Case(45 + i, [1300 + 100 * i], 2, 64, 1, 64, state=torch.float32, init=[True]) for i in range(2)]
    need = max(dc.dcconv_gated_delta_scan_workspace(1, c.lens[0], 2, 64, 1, 64, 0) for c in cases)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    init = torch.ones(1, dtype=torch.bool, device="cuda")
    graphs = []
    for c in cases:
        args = [t.cuda() for t in (c.q, c.k, c.v, c.dt, c.A, c.beta)]
        more = dict(dt_bias=c.bias.cuda(), dt_softplus=True, beta_sigmoid=True, qk_l2norm=True, has_initial_state=init)
        pool, ref, out = c.state.cuda(), c.state.cuda(), torch.empty_like(args[2])
        dc.gated_delta_scan(*args, state=pool.clone(), out=out, workspace=work, **more)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dc.gated_delta_scan(*args, state=pool, out=out, workspace=work, **more)
        graphs.append((graph, args, more, pool, ref, out))
    for _ in range(3):
        for graph, args, more, pool, ref, out in graphs:
            graph.replay()
        for graph, args, more, pool, ref, out in graphs:
            want = dc.gated_delta_scan(*args, state=ref, **more)
            torch.cuda.synchronize()
            assert torch.equal(want, out) and torch.equal(pool, ref)


@pytest.mark.parametrize("P,K", [(128, 128), (200, 64), (72, 128)])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_blocks_of_128_rows(P, K, state):
    """Enough heads for a block of 128 rows a CU."""
    Case(P + K, [70] * 2, 128 if P <= 128 else 64, P, 16, K, state=state, init=[True, False]).check()


@pytest.mark.parametrize("n", [63, 64, 65, 150])
def test_many_packed_sequences(n):
    """In the order of their lengths up to 64 of them; the same lengths, empty and padding ones among
    them, and tokens that are whole chunks in all."""
    gen = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 40, (n,), generator=gen).tolist()
    lens[3] = lens[7] = 100
    lens[n - 1] = 0
    lens[5] = 64 - (sum(lens) - lens[5]) % 64
    table = torch.randperm(n + 4, generator=gen)[:n].tolist()
    table[2] = table[7] = -1
    Case(n, lens, 2, 32, 1, 64, state=torch.float32, packed=True, slots=n + 4, table=table,
         init=[i % 3 > 0 for i in range(n)]).check()


def one_token(n, H, P, K, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, k = (torch.randn(n, 1, K, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    v = torch.randn(n, H, P, generator=gen, device="cuda").to(torch.bfloat16)
    beta = torch.rand(n, H, generator=gen, device="cuda")
    want = beta[..., None].double() * v.double() * (q.double() * k.double()).sum(-1, keepdim=True)
    bound = beta[..., None].double() * v.double().abs() * (q.double() * k.double()).abs().sum(-1, keepdim=True)
    return q, k, v, beta, want.cpu(), bound.cpu()


def test_more_blocks_than_a_grid_axis():
    """Every sequence a token from no state: out = scale b (k.q) v.  (P's products are rounded, and U's.)"""
    n = (1 << 20) + 300
    q, k, v, beta, want, bound = one_token(n, 1, 8, 8, 50)
    A = torch.full((1,), -1.0, device="cuda")
    out = dc.gated_delta_scan(q[:, None], k[:, None], v[:, None], torch.zeros(n, 1, 1, device="cuda"), A, beta[:, None],
                              scale=1.0)
    close(out[:, 0], want, U * want.abs() + (U + 2.0 ** -14) * bound * (1 + U), "scan")
    table = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    table[n - 1] = 0
    state = torch.zeros(1, 1, 8, 8, device="cuda")
    out = dc.gated_delta_update(q, k, v, torch.zeros(n, 1, device="cuda"), A, beta, state, scale=1.0, state_indices=table)
    assert not out[:-1].any()
    close(out[-1:], want[-1:], U * want[-1:].abs() + 2.0 ** -17 * bound[-1:], "update")


def test_state_offsets_past_4_gib():
    """Slots more than 2^31 bytes apart, in a pool of 12 GiB."""
    far = (1 << 30) + 24
    pool = torch.empty(2 * far + 2 * 32 * 64, device="cuda").as_strided((3, 2, 32, 64), (far, 32 * 64, 64, 1))
    case = Case(51, [70, 33], 2, 32, 1, 64, state=torch.float32, packed=True, table=[2, 1], slots=3, init=[True, True])
    step = Case(52, None, 2, 32, 1, 64, state=torch.float32, rows=2, table=[2, 1], slots=3)
    for c in (case, step):
        pool.copy_(c.state)
        out = c.call()
        args = [t.cuda() for t in (c.q, c.k, c.v, c.dt, c.A, c.beta)]
        more = dict(dt_bias=c.bias.cuda(), dt_softplus=True, beta_sigmoid=True, qk_l2norm=True,
                    state_indices=torch.tensor([2, 1], dtype=torch.int32, device="cuda"))
        if c is case:
            got = dc.gated_delta_scan(*args, state=pool, has_initial_state=torch.ones(2, dtype=torch.bool, device="cuda"),
                                      seq_starts=torch.tensor([0, 70, 103], dtype=torch.int32, device="cuda"), **more)
        else:
            got = dc.gated_delta_update(*args, pool, **more)
        assert torch.equal(got, out) and torch.equal(pool, c.pool)


@pytest.mark.parametrize("stride", [(1 << 22) + 8, (1 << 23) + 8, (1 << 22) + 3])
def test_token_offsets_past_4_gib(stride):
    """Tokens megabytes apart: the last starts 5 GiB behind the first."""
    T = 5 * (1 << 30) // (2 * stride) + 2
    case = Case(53, [T], 1, 16, 1, 16, state=torch.float32, init=[True])
    want = case.call()
    flat = torch.empty((T - 1) * stride + 64, dtype=torch.bfloat16, device="cuda")
    views = []
    for i, t in enumerate((case.q, case.k, case.v)):
        view = flat[16 * i:].as_strided((1, T, 1, 16), (T * stride, stride, 16, 1))
        view.copy_(t)
        views.append(view)
    out = flat[48:].as_strided((1, T, 1, 16), (T * stride, stride, 16, 1))
    pool = case.state.cuda()
    # (operands and the output share their tokens' rows: rows of the output lie between the others', which
    # the call refuses, so it writes elsewhere)
    with pytest.raises(ValueError, match="overlaps"):
        dc.gated_delta_scan(*views, case.dt.cuda(), case.A.cuda(), case.beta.cuda(), state=pool, out=out)
    got = dc.gated_delta_scan(*views, case.dt.cuda(), case.A.cuda(), case.beta.cuda(), dt_bias=case.bias.cuda(),
                              dt_softplus=True, beta_sigmoid=True, qk_l2norm=True, state=pool,
                              has_initial_state=torch.ones(1, dtype=torch.bool, device="cuda"))
    assert torch.equal(got, want) and torch.equal(pool, case.pool)
    del flat, views, out


def test_output_offsets_past_4_gib():
    stride = (1 << 22) + 8
    T = 5 * (1 << 30) // (2 * stride) + 2
    case = Case(54, [T], 1, 16, 1, 16)
    want = case.call()
    flat = torch.empty((T - 1) * stride + 16, dtype=torch.bfloat16, device="cuda")
    out = flat.as_strided((1, T, 1, 16), (T * stride, stride, 16, 1))
    assert torch.equal(case.call(out=out), want)


def test_calls_on_two_streams_at_once():
    cases = [Case(55 + i, [1400], 2, 64, 1, 64, state=torch.float32, init=[True]) for i in range(2)]
    want = []
    for c in cases:
        want.append((c.call(), c.pool))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append((c.call(), c.pool))
        torch.cuda.synchronize()
        for (o, p), (x, y) in zip(want, got):
            assert torch.equal(o, x) and torch.equal(p, y)


@pytest.mark.parametrize("big", [1e4, 1e8])
def test_large_values_and_states(big):
    """Channels scale: values and states of another size give outputs of that size."""
    case = Case(60, [100], 2, 32, 1, 64, state=torch.float32, init=[True])
    case.v = (case.v.float() * big).to(torch.bfloat16)
    case.state = case.state * big
    case.check()


def test_refuses_tensors_that_require_gradients():
    case = Case(61, None, 2, 32, 1, 64, state=torch.float32, rows=2)
    case.v = case.v.cuda().requires_grad_()
    with pytest.raises(NotImplementedError, match="training"):
        case.call()
    x = torch.ones(2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    with pytest.raises(NotImplementedError, match="training"):
        dc.gated_rms_norm(x, x, w)
    with pytest.raises(NotImplementedError, match="training"):
        dc.add_rms_norm(x, torch.ones(2, 64, device="cuda", requires_grad=True), w.detach())
