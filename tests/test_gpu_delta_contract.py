"""What the gated delta rule's tensor functions promise their callers, on the GPU: refusals, and what a
broken table or a rarer variant leaves alone."""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from delta_reference import U, bounds, close, recurrence
from test_gpu_delta import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("more", [dict(), dict(table=[-1, -1]), dict(init=[True, False])])
def test_scan_refuses_a_pool_of_no_slots(more, packed):
    case = Case(1, [40, 40], 2, 32, 1, 32, packed=packed, **more)
    case.state = torch.empty(0, 2, 32, 32)
    with pytest.raises(ValueError, match="no slots"):
        case.call()


def test_scan_of_no_sequences_takes_a_pool_of_no_slots():
    case = Case(1, [], 2, 32, 1, 32, packed=True)
    case.state = torch.empty(0, 2, 32, 32)
    assert case.call().shape == (1, 0, 2, 32)


# blocks of 64 and of 128 rows, chunks of 64 and of 32 tokens, rows of whole 16 bytes and others
VARIANTS = [(2, 32, 64, torch.bfloat16), (2, 32, 64, None), (160, 128, 128, torch.float32), (160, 128, 128, torch.bfloat16),
            (160, 72, 40, None), (2, 24, 200, torch.float32), (2, 24, 200, torch.bfloat16), (2, 24, 200, None),
            (2, 9, 33, torch.float32), (2, 9, 33, None)]


@pytest.mark.parametrize("H,P,K,state", VARIANTS)
@pytest.mark.parametrize("what", ["q", "k", "v", "beta", "dt"])
@pytest.mark.parametrize("t0,value", [(5, float("nan")), (20, float("inf")), (37, float("nan")), (63, float("inf")),
                                      (70, float("nan"))])
def test_scan_not_finite_in_every_variant(H, P, K, state, what, t0, value):
    """What is not finite reaches the outputs and states behind it that the recurrence takes it to, and no
    earlier token, other channel of v, or other head."""
    h = H - 1
    case = Case(2, [100], H, P, H, K, state=state, init=None if state is None else [True], logit=False, soft=False, f32=True)
    if what == "dt" and value > 0:
        case.A[h] = 1.0  # a decay that is infinite
    clean, clean_pool = case.call(), case.pool
    at = {"q": (0, t0, h, 5), "k": (0, t0, h, 5), "v": (0, t0, h, 7), "beta": (0, t0, h), "dt": (0, t0, h)}[what]
    getattr(case, what)[at] = value
    out, pool = case.call(), case.pool
    fine = torch.isfinite(out)
    assert torch.equal(out[:, :, :h], clean[:, :, :h]) and torch.equal(out[:, :t0], clean[:, :t0])
    if what == "q":
        assert not fine[0, t0, h].any() and torch.equal(out[0, t0 + 1:], clean[0, t0 + 1:])
        assert state is None or torch.equal(pool, clean_pool)
        return
    if state is not None:
        assert torch.equal(pool[:, :h], clean_pool[:, :h])
    if what == "v":
        others = [p for p in range(P) if p != 7]
        assert not fine[0, t0:, h, 7].any() and torch.equal(out[..., others], clean[..., others])
        if state is not None:
            assert not torch.isfinite(pool[0, h, 7]).any() and torch.equal(pool[:, :, others], clean_pool[:, :, others])
        return
    assert not fine[0, t0:, h].any()
    assert state is None or not torch.isfinite(pool[0, h]).any()


@pytest.mark.parametrize("state", [torch.bfloat16, None])
@pytest.mark.parametrize("K", [64, 128, 200])
@pytest.mark.parametrize("repeated", [False, True])
@pytest.mark.parametrize("logit", [False, True])
def test_scan_without_decay(state, K, repeated, logit):
    """All of a state kept, keys that are one and the same, and weights up to 1.9, with states in BF16 or none."""
    case = Case(3, [150], 2, 64, 1, K, state=state, init=None if state is None else [True], rate=0.0, logit=logit)
    if repeated:
        case.k = case.k[:, :1].expand_as(case.k).contiguous()
    case.check()


def guarded(shape, dtype, value):
    """A tensor between 4096 elements of `value` on either side, and what says whether those are left."""
    size = 1
    for n in shape:
        size *= n
    flat = torch.full((size + 8192,), value, dtype=dtype, device="cuda")
    inner = flat[4096:4096 + size].view(shape)
    return inner, lambda: bool((flat[:4096] == value).all() and (flat[4096 + size:] == value).all())


BROKEN = [[0, 30, 10, 100], [0, 30, 120, 100], [0, -5, 50, 100], [5, 30, 50, 90], [0, 30, 50, 1 << 30],
          [0, 30, 50, -(1 << 31)], [(1 << 31) - 1, 0, 100, 100], [100, 50, 30, 0]]


@pytest.mark.parametrize("bad", BROKEN)
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_scan_of_a_broken_table(bad, state):
    """Few sequences, not cut: those of a broken table that are ordered and inside the tokens are right, the
    others' slots are left, and nothing is written outside."""
    case = Case(4, [30, 20, 50], 2, 32, 1, 32, state=state, packed=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool, pool_kept = guarded(case.state.shape, state, 5.0)
    pool.copy_(case.state)
    out, out_kept = guarded(case.v.shape, torch.bfloat16, 7.0)
    out.fill_(3.0)
    args = [t.cuda() for t in (case.q, case.k, case.v, case.dt, case.A, case.beta)]
    dc.gated_delta_scan(*args, dt_bias=case.bias.cuda(), dt_softplus=True, qk_l2norm=True, beta_sigmoid=True, state=pool,
                        out=out, dev_status=status, seq_starts=torch.tensor(bad, dtype=torch.int32, device="cuda"))
    assert int(status) == dc.DCCONV_DEV_BAD_SEQ and pool_kept() and out_kept()
    live = [i for i in range(3) if 0 <= bad[i] <= bad[i + 1] <= 100]
    alone = [i for i in live if all(j == i or bad[j + 1] <= bad[i] or bad[j] >= bad[i + 1] for j in live)]
    for i in range(3):
        if i not in live:
            assert torch.equal(pool[i].cpu(), case.state[i])
    for i in alone:
        cut = case.exact((0, slice(bad[i], bad[i + 1])))
        y, s = recurrence(*cut)
        f32 = state == torch.float32
        dy, ds = bounds(*cut, None, 64, f32)
        close(out[0, bad[i]:bad[i + 1]], y, U * (y.abs() + dy) + dy, f"out of sequence {i}")
        close(pool[i], s, ds if f32 else ds + U * (s.abs() + ds), f"state of sequence {i}")
    inside = torch.zeros(100, dtype=torch.bool)
    for i in live:
        inside[bad[i]:bad[i + 1]] = True
    assert bool((out[0, ~inside.cuda()] == 3.0).all())


@pytest.mark.parametrize("n", [3, 70])
@pytest.mark.parametrize("seed", range(4))
def test_scan_of_a_broken_table_of_cut_or_many_sequences(n, seed):
    """Nothing is written outside the operands and the workspace, whatever the table says."""
    t = 3000 if n == 3 else 700
    gen = torch.Generator().manual_seed(seed)
    table = torch.randint(-t, 2 * t, (n + 1,), generator=gen)
    if seed % 2:
        table = table.clamp(0, t)
        table[1::3] = table[1::3].sort().values
    case = Case(5, [t], 1, 32, 1, 32, state=torch.float32, packed=True, slots=n)
    pool, pool_kept = guarded(case.state.shape, torch.float32, 5.0)
    pool.copy_(case.state)
    out, out_kept = guarded(case.v.shape, torch.bfloat16, 7.0)
    need = dc.dcconv_gated_delta_scan_workspace(n, t, 1, 32, 1, 32, 1)
    assert (need > 0) == (n == 3)
    work, work_kept = guarded((need,), torch.uint8, 9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [x.cuda() for x in (case.q, case.k, case.v, case.dt, case.A, case.beta)]
    dc.gated_delta_scan(*args, qk_l2norm=True, beta_sigmoid=True, state=pool, out=out, workspace=work, dev_status=status,
                        has_initial_state=torch.ones(n, dtype=torch.bool, device="cuda"),
                        seq_starts=table.to(torch.int32).cuda())
    assert int(status) == dc.DCCONV_DEV_BAD_SEQ and pool_kept() and out_kept() and work_kept()


@pytest.mark.parametrize("sizes", [(0, 8, 1, 8), (2, 0, 1, 8), (2, 8, 0, 8), (2, 8, 1, 0)])
def test_sizes_of_zero_are_refused(sizes):
    """Heads, channels, groups and keys: as any other size that the entry points refuse."""
    H, P, G, K = sizes
    z = torch.zeros(2, 3, 8, 8, dtype=torch.bfloat16, device="cuda")
    k, v = z[:, :, :G, :K], z[:, :, :H, :P]
    A, state = torch.zeros(H, device="cuda"), torch.zeros(2, H, P, K, device="cuda")
    dt = torch.zeros(2, 3, H, device="cuda")
    with pytest.raises(ValueError, match=">= 1"):
        dc.gated_delta_scan(k, k, v, dt, A, dt)
    with pytest.raises(ValueError, match=">= 1"):
        dc.gated_delta_update(k[:, 0], k[:, 0], v[:, 0], dt[:, 0], A, dt[:, 0], state)
