"""The gated delta rule on the GPU against its 64-bit form: whole sequences and one token.

Sizes sit at and around the kernels' edges (chunks of 64 tokens, 32 where keys are long,
tiles of 16 values), with strided views, padding and rejected rows, empty sequences and
both state types.  The bounds are derived in ``delta_reference``.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from delta_reference import U, bounds, close, factors, recurrence, step_bounds, unit

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dc._load()
    yield
    torch.cuda.synchronize()


def bf(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(torch.bfloat16)


def strided(t, pad=8):
    """The same values on the device in rows `pad` elements longer."""
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + pad, dtype=t.dtype, device="cuda")
    wide[..., :t.shape[-1]] = t.cuda()
    return wide[..., :t.shape[-1]]


def dev(t):
    return None if t is None else t.cuda()


class Case:
    """One call's inputs from the seed.  lens: tokens of each sequence; None: one token of
    `rows` rows."""

    def __init__(self, seed, lens, H, P, G, K, state=None, packed=False, table=None, slots=None, init=None, l2=True,
                 soft=True, logit=True, f32=False, scale=None, rows=None, place=dev, rate=8.0, spread=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.P, self.G, self.K, self.packed = lens, H, P, G, K, packed
        n = rows if lens is None else len(lens)
        lead = (n,) if lens is None else (1, sum(lens)) if packed else (n, lens[0])
        self.q, self.k, self.v = (bf(gen, *lead, *s, scale=spread) for s in ((G, K), (G, K), (H, P)))
        if not l2:  # no longer than one, also once rounded
            self.q, self.k = (x / (x.norm(dim=-1, keepdim=True) * 1.01) for x in (self.q.float(), self.k.float()))
            self.q, self.k = self.q.to(torch.bfloat16), self.k.to(torch.bfloat16)
        self.dt, self.beta = torch.randn(*lead, H, generator=gen), torch.randn(*lead, H, generator=gen)
        self.bias = -4.0 + 2.0 * torch.rand(H, generator=gen)
        self.A = -rate * torch.rand(H, generator=gen)
        if not soft:
            self.dt, self.bias = self.dt.abs() * 0.1, None
        if not logit:
            self.beta = torch.rand(*lead, H, generator=gen) * 1.9  # up to where the state's sign along k turns
        if not f32:
            self.dt, self.beta = self.dt.to(torch.bfloat16), self.beta.to(torch.bfloat16)
        self.l2, self.soft, self.logit, self.scale = l2, soft, logit, scale
        self.table, self.init, self.state, self.place = table, init, None, place
        if state is not None:
            self.state = (torch.randn(slots or n, H, P, K, generator=gen) * 0.3).to(state)
        self.group = torch.arange(H) // (H // G)

    def call(self, **more):
        self.pool = None if self.state is None else dev(self.state).clone()
        table = None if self.table is None else torch.tensor(self.table, dtype=torch.int32).cuda()
        args = [self.place(t) for t in (self.q, self.k, self.v, self.dt)] + [dev(self.A), self.place(self.beta)]
        more = dict(dt_bias=dev(self.bias), dt_softplus=self.soft, beta_sigmoid=self.logit, qk_l2norm=self.l2,
                    scale=self.scale, state_indices=table, **more)
        if self.lens is None:
            return dc.gated_delta_update(*args, self.pool, **more)
        starts = torch.tensor([0] + self.lens).cumsum(0).to(torch.int32).cuda() if self.packed else None
        init = None if self.init is None else torch.tensor(self.init, dtype=torch.bool).cuda()
        return dc.gated_delta_scan(*args, state=self.pool, has_initial_state=init, seq_starts=starts, **more)

    def exact(self, at):
        """q, k, v, log-decay and weight of the tokens `at`, by heads, float64."""
        q, k, v = (t[at].double() for t in (self.q, self.k, self.v))
        q, k = (unit(t, self.l2)[..., self.group, :] for t in (q, k))
        bias = None if self.bias is None else self.bias.double()
        g, b = factors(self.dt[at].double(), self.A.double(), self.beta[at].double(), bias, self.soft, self.logit)
        return q, k, v, g, b, self.K ** -0.5 if self.scale is None else self.scale

    def check(self, dead=(), **more):
        out = self.call(**more)
        if self.lens is None:
            return self.check_step(out, dead)
        final = None
        if isinstance(out, tuple):
            out, final = out
        want = bound = None
        if self.state is not None:
            want = self.state.double()
            bound = torch.zeros_like(want)
        at = 0
        for i, L in enumerate(self.lens):
            row, lo = (0, at) if self.packed else (i, 0)
            at += L if self.packed else 0
            got = out[row, lo:lo + L]
            slot = i if self.table is None else self.table[i]
            if slot < 0 or i in dead:
                assert not got.any(), f"sequence {i}: padding must be zeros"
                continue
            s0 = self.state[slot].double() if self.init is not None and self.init[i] else None
            cut = self.exact((row, slice(lo, lo + L)))
            y, s = recurrence(*cut, s0)
            f32 = final is not None or (self.state is not None and self.state.dtype == torch.float32)
            dy, ds = bounds(*cut, s0, 64 if self.K <= 128 else 32, f32)
            close(got, y, U * (y.abs() + dy) + dy, f"out of sequence {i}")
            if self.state is not None:
                want[slot], bound[slot] = s, ds if f32 else ds + U * (s.abs() + ds)
            elif final is not None:
                close(final[i], s, ds, f"final state of sequence {i}")
        if self.state is not None:
            close(self.pool, want, bound, "states")

    def check_step(self, out, dead):
        n = len(self.v)
        want, bound = self.state.double(), torch.zeros_like(self.state.double())
        slots = list(range(n)) if self.table is None else self.table
        live = [i for i in range(n) if slots[i] >= 0 and i not in dead]
        for i in range(n):
            assert i in live or not out[i].any(), f"row {i}: padding must be zeros"
        if live:
            q, k, v, g, b, scale = self.exact(live)
            y, s, dy, ds = step_bounds(q, k, v, g, b, scale, want[[slots[i] for i in live]])
            close(out[live], y, U * (y.abs() + dy) + dy, "out")
            to = [slots[i] for i in live]
            want[to], bound[to] = s, ds if self.state.dtype == torch.float32 else ds + U * (s.abs() + ds)
        close(self.pool, want, bound, "states")


LAYOUTS = [(1, 64, 1, 128), (3, 32, 1, 16), (5, 80, 5, 72), (4, 128, 2, 64), (2, 16, 1, 256), (6, 96, 2, 32),
           (9, 8, 3, 8), (2, 64, 2, 1), (3, 1, 1, 5), (2, 33, 1, 130), (7, 64, 1, 200), (1, 200, 1, 65), (2, 256, 2, 128)]


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 129, 200])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_scan_lengths(T, state):
    Case(T, [T, T], 4, 128, 2, 128, state=state, init=[True, False]).check()


@pytest.mark.parametrize("H,P,G,K", LAYOUTS)
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_scan_head_layouts(H, P, G, K, state):
    Case(H * P + K, [70], H, P, G, K, state=state, init=[True]).check()
    Case(H * P + K, [70], H, P, G, K, state=state, init=[True], l2=False, logit=False).check()


@pytest.mark.parametrize("l2,soft,logit,f32,scale", [(False, True, True, False, None), (True, False, True, True, 1.0),
                                                     (True, True, False, True, -0.5), (False, False, False, False, 0.0)])
def test_scan_options(l2, soft, logit, f32, scale):
    more = dict(l2=l2, soft=soft, logit=logit, f32=f32, scale=scale)
    Case(3, [90], 3, 64, 1, 64, **more).check()
    Case(4, [90], 3, 64, 1, 64, **more).check(return_final_state=True)


def test_scan_packed_with_pool():
    lens = [0, 1, 70, 64, 0, 300, 3, 5]
    for state in (torch.float32, torch.bfloat16):
        Case(5, lens, 4, 64, 2, 128, state=state, packed=True, slots=12, table=[3, 0, -1, 7, 11, 2, -1, 9],
             init=[True, True, True, False, False, True, False, True]).check()


def test_scan_long_sequence():
    Case(6, [1500], 2, 32, 1, 64, state=torch.float32, init=[True]).check()
    Case(7, [900, 1, 0, 1200, 256, 257], 2, 128, 1, 128, state=torch.bfloat16, packed=True,
         table=[4, 0, 1, 2, -1, 3], slots=5, init=[True, False, True, True, True, False]).check()


def test_scan_without_decay_and_with_repeated_keys():
    """A of zeros keeps all of the state; one and the same key makes the triangular matrix as
    far from the unit matrix as it gets."""
    case = Case(8, [150], 2, 64, 1, 128, state=torch.float32, init=[True], rate=0.0)
    case.check()
    for logit in (True, False):
        case = Case(9, [150], 2, 64, 1, 128, state=torch.float32, init=[True], rate=0.0, logit=logit)
        case.k = case.k[:, :1].expand_as(case.k).contiguous()
        case.check()


def test_scan_of_steps_that_forget_everything():
    """Decays far below what FP32 holds, also an infinite one: what lies behind such a token is
    forgotten, and the decays between later tokens keep their bits."""
    for big in (1e3, 1e6, float("inf")):
        case = Case(10, [100], 2, 64, 1, 64, state=torch.float32, init=[True], soft=False, f32=True)
        case.A = torch.tensor([-1.0, -0.5])
        case.dt[0, 10] = big
        case.dt[0, 70] = big
        out = case.call()
        cut = case.exact((0, slice(0, 100)))
        y, s = recurrence(*cut, case.state[0].double())
        # the same bounds, with a finite stand-in whose decay is zero in 64 bits too
        dy, ds = bounds(*cut[:3], cut[3].clamp(min=-800.0), *cut[4:], case.state[0].double(), 64, True)
        close(out[0], y, U * (y.abs() + dy) + dy, f"out behind a step of {big}")
        close(case.pool[0], s, ds, f"state behind a step of {big}")


def test_scan_of_strided_and_unaligned_views():
    Case(11, [100], 4, 64, 2, 128, state=torch.float32, place=strided).check()
    Case(12, [100], 4, 64, 2, 128, state=torch.float32, place=lambda t: strided(t, 3)).check()

    def off(t):  # a base two bytes past 16
        flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten().cuda()
        return flat[1:].view(t.shape)
    Case(13, [100], 4, 64, 2, 128, state=torch.bfloat16, place=off).check()


def test_scan_of_head_major_and_broadcast_operands():
    """Heads further apart than tokens, so that a row past the end is another head's; and rows
    that are one and the same."""
    def head_major(t):
        t = t.cuda()
        return t.transpose(1, 2).contiguous().transpose(1, 2) if t.dim() == 4 else t
    case = Case(14, [75, 75], 6, 64, 2, 64, state=torch.float32, place=head_major)
    buf = torch.full((2, 6, 90, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    case.check(out=buf[:, :, 5:80].transpose(1, 2))
    assert bool((buf[:, :, :5] == 7).all() and (buf[:, :, 80:] == 7).all())
    case = Case(15, [75, 75], 4, 32, 1, 64, state=torch.float32)
    for t in (case.q, case.k, case.v):
        t.copy_(t[:1, :1].expand_as(t).clone())
    case.place = lambda t: t[:1, :1].cuda().expand(t.shape) if t.dim() == 4 else t.cuda()
    case.check()


def test_scan_writes_only_its_output():
    case = Case(16, [77, 77], 3, 40, 1, 24, state=torch.float32)
    buf = torch.full((2, 77, 5, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :, 1:4, 8:48]
    case.check(out=out)
    assert bool((buf[:, :, 0] == 7).all() and (buf[:, :, 4] == 7).all() and (buf[..., :8] == 7).all())


def test_scan_leaves_the_rest_of_a_pool():
    """Slots further apart than their states, and slots that no sequence selects."""
    case = Case(17, [40, 80], 2, 32, 1, 40, state=torch.float32, packed=True, table=[4, 1], slots=6, init=[True, True])
    wide = torch.full((6, 2 * 32 * 40 + 24), 5.0, device="cuda")
    pool = wide[:, :2 * 32 * 40].view(6, 2, 32, 40)
    pool.copy_(case.state)
    first = pool.clone()
    case.call()
    out = dc.gated_delta_scan(*[t.cuda() for t in (case.q, case.k, case.v, case.dt, case.A, case.beta)],
                              dt_bias=case.bias.cuda(), dt_softplus=True, beta_sigmoid=True, qk_l2norm=True, state=pool,
                              state_indices=torch.tensor([4, 1], dtype=torch.int32, device="cuda"),
                              has_initial_state=torch.tensor([True, True], device="cuda"),
                              seq_starts=torch.tensor([0, 40, 120], dtype=torch.int32, device="cuda"))
    assert torch.equal(pool, case.pool) and bool((wide[:, 2 * 32 * 40:] == 5).all()) and bool(out.any())
    assert all(torch.equal(pool[i], first[i]) for i in (0, 2, 3, 5))


def test_scan_bad_and_duplicate_indices():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Case(18, [20] * 5, 2, 32, 1, 32, state=torch.float32, slots=6, table=[6, -1, 2, 4, 4]).check(
        dead=(0, 3, 4), dev_status=status)
    assert int(status) == dc.DCCONV_DEV_BAD_INDEX | dc.DCCONV_DEV_DUP_INDEX


def test_scan_broken_table_reads_nothing_outside():
    """Sequences of a table that is not ordered are left out; the others are right."""
    case = Case(19, [30, 20, 50], 2, 32, 1, 32, state=torch.float32, packed=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [t.cuda() for t in (case.q, case.k, case.v, case.dt, case.A, case.beta)]
    for bad in ([0, 30, 10, 100], [0, 30, 120, 100], [0, -5, 50, 100], [5, 30, 50, 90], [0, 30, 50, 1 << 30]):
        status.zero_()
        pool = case.state.cuda().clone()
        dc.gated_delta_scan(*args, qk_l2norm=True, beta_sigmoid=True, state=pool, dev_status=status,
                            seq_starts=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert int(status) == dc.DCCONV_DEV_BAD_SEQ, bad


def test_scan_of_no_tokens():
    """Every sequence empty: initial states stay, the others become zeros."""
    z = torch.zeros(2, 0, 1, 16, dtype=torch.bfloat16, device="cuda")
    pool = torch.ones(2, 1, 16, 16, device="cuda")
    dc.gated_delta_scan(z, z, z, z[..., 0], torch.zeros(1, device="cuda"), z[..., 0], state=pool,
                        has_initial_state=torch.tensor([True, False], device="cuda"))
    assert bool((pool[0] == 1).all()) and not pool[1].any()


@pytest.mark.parametrize("what", ["q", "k", "v", "beta", "dt"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_scan_not_finite(what, value):
    """What is not finite reaches the outputs and states behind it that the recurrence takes it
    to, and no earlier token, other channel of v, other head or other sequence."""
    t0 = 37
    case = Case(20, [100, 100], 2, 32, 2, 64, state=torch.float32, logit=False, soft=False, f32=True)
    clean = case.call()
    clean_pool = case.pool
    at = {"q": (0, t0, 1, 5), "k": (0, t0, 1, 5), "v": (0, t0, 1, 7), "beta": (0, t0, 1), "dt": (0, t0, 1)}[what]
    if what == "dt" and value > 0:
        case.A = torch.tensor([-1.0, 1.0])  # a decay that is infinite
        clean = case.call()
        clean_pool = case.pool
    getattr(case, what)[at] = value
    out = case.call()
    torch.cuda.synchronize()
    fine = torch.isfinite(out)
    assert bool(fine[1].all() and fine[0, :, 0].all() and fine[0, :t0].all())
    assert torch.equal(out[1], clean[1]) and torch.equal(out[0, :, 0], clean[0, :, 0])
    assert torch.equal(out[0, :t0], clean[0, :t0])
    pool = case.pool
    assert torch.equal(pool[1], clean_pool[1]) and torch.equal(pool[0, 0], clean_pool[0, 0])
    if what == "q":
        assert not fine[0, t0, 1].any() and bool(fine[0, t0 + 1:].all()) and torch.equal(pool, clean_pool)
        return
    if what == "v":
        others = [p for p in range(32) if p != 7]
        assert not fine[0, t0:, 1, 7].any() and torch.equal(out[..., others], clean[..., others])
        assert not torch.isfinite(pool[0, 1, 7]).any() and torch.equal(pool[:, :, others], clean_pool[:, :, others])
        return
    assert not fine[0, t0:, 1].any() and not torch.isfinite(pool[0, 1]).any()


def test_scan_of_a_state_that_is_not_finite():
    case = Case(21, [70], 2, 32, 1, 64, state=torch.float32, init=[True])
    clean = case.call()
    case.state[0, 1, 3, 9] = float("nan")
    out = case.call()
    others = [p for p in range(32) if p != 3]
    assert not torch.isfinite(out[0, :, 1, 3]).any() and not torch.isfinite(case.pool[0, 1, 3]).any()
    assert torch.equal(out[0, :, 0], clean[0, :, 0]) and torch.equal(out[0, :, 1, others], clean[0, :, 1, others])


def test_scan_continues_where_it_left_off():
    """A prompt in two calls is the prompt in one, within both's bounds (the same FP32 state
    ahead of the second call, whose chunks start elsewhere)."""
    whole = Case(22, [150], 4, 64, 2, 128, state=torch.float32, init=[True])
    whole.check()
    case = Case(22, [150], 4, 64, 2, 128, state=torch.float32, init=[True])
    out = []
    pool = case.state.cuda()
    for lo, hi in ((0, 50), (50, 150)):
        args = [t[:, lo:hi].cuda() for t in (case.q, case.k, case.v, case.dt)] + [case.A.cuda(), case.beta[:, lo:hi].cuda()]
        out.append(dc.gated_delta_scan(*args, dt_bias=case.bias.cuda(), dt_softplus=True, beta_sigmoid=True,
                                       qk_l2norm=True, state=pool, has_initial_state=torch.ones(1, dtype=torch.bool,
                                                                                              device="cuda")))
    cut = case.exact((0, slice(0, 150)))
    s0 = case.state[0].double()
    y, s = recurrence(*cut, s0)
    dy, ds = bounds(*cut, s0, 64, True)
    first = [t[:50] for t in cut[:5]]
    y1, s1 = recurrence(*first, cut[5], s0)
    d1, e1 = bounds(*first, cut[5], s0, 64, True)
    d2, e2 = bounds(*[t[50:] for t in cut[:5]], cut[5], s1, 64, True)
    got = torch.cat(out, 1)[0]
    close(got[:50], y[:50], U * (y[:50].abs() + d1) + d1, "first call")
    # the first call's error of a row shrinks on its way: its whole norm is an upper bound
    d2 = d2 + e1[..., 0] * cut[0][50:].norm(dim=-1)[..., None] * abs(cut[5])
    close(got[50:], y[50:], U * (y[50:].abs() + d2) + d2, "second call")
    close(pool[0], s, e1 + e2, "state")


def test_scan_is_the_same_on_every_run_and_on_another_stream():
    case = Case(23, [300, 300], 4, 128, 2, 128, state=torch.bfloat16, init=[True, True])
    first = case.call()
    state = case.pool
    stream = torch.cuda.Stream()
    for _ in range(3):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            again = case.call()
        torch.cuda.current_stream().wait_stream(stream)
        assert torch.equal(first, again) and torch.equal(state, case.pool)


def test_calls_in_a_graph():
    """Captured and replayed several times with eager work in between: the states advance as
    in eager calls."""
    scan = Case(24, [90, 90], 4, 64, 2, 128, state=torch.float32, init=[True, True])
    step = Case(25, None, 4, 64, 2, 128, state=torch.float32, rows=2)
    args = [t.cuda() for t in (scan.q, scan.k, scan.v, scan.dt, scan.A, scan.beta)]
    tok = [t.cuda() for t in (step.q, step.k, step.v, step.dt, step.A, step.beta)]
    init = torch.ones(2, dtype=torch.bool, device="cuda")
    more = dict(dt_softplus=True, beta_sigmoid=True, qk_l2norm=True)
    pool, ref = scan.state.cuda(), scan.state.cuda()
    out, tout = torch.empty_like(args[2]), torch.empty_like(tok[2])

    def both(state, o, t):
        dc.gated_delta_scan(*args, state=state, has_initial_state=init, out=o, **more)
        dc.gated_delta_update(*tok, state, out=t, **more)
    both(pool.clone(), out, tout)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(pool, out, tout)
    for _ in range(4):
        want, twant = torch.empty_like(out), torch.empty_like(tout)
        both(ref, want, twant)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out) and torch.equal(twant, tout) and torch.equal(ref, pool)


@pytest.mark.parametrize("rows,H,P,G,K", [(1,) + s for s in LAYOUTS] + [(5, 4, 128, 2, 128), (61, 9, 80, 3, 72),
                                                                        (70, 32, 64, 4, 64), (3, 2, 24, 1, 12)])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_update_layouts(rows, H, P, G, K, state):
    Case(rows * H + P + K, None, H, P, G, K, state=state, rows=rows).check()


@pytest.mark.parametrize("l2,soft,logit,f32,scale", [(False, True, True, False, None), (True, False, True, True, 1.0),
                                                     (True, True, False, True, -0.5), (False, False, False, False, 0.0)])
def test_update_options(l2, soft, logit, f32, scale):
    Case(30, None, 6, 64, 2, 128, state=torch.float32, rows=7, l2=l2, soft=soft, logit=logit, f32=f32, scale=scale).check()


def test_update_routes_pads_and_rejects():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Case(31, None, 4, 64, 2, 128, state=torch.float32, rows=6, slots=9, table=[3, -1, 9, 5, 0, 5]).check(
        dead=(2, 3, 5), dev_status=status)
    assert int(status) == dc.DCCONV_DEV_BAD_INDEX | dc.DCCONV_DEV_DUP_INDEX
    Case(32, None, 4, 64, 2, 128, state=torch.bfloat16, rows=3, slots=9, table=[-1, -1, -1]).check()


def test_update_of_strided_views():
    Case(33, None, 4, 64, 2, 128, state=torch.float32, rows=5, place=strided).check()
    Case(34, None, 4, 64, 2, 128, state=torch.bfloat16, rows=5, place=lambda t: strided(t, 3)).check()
    case = Case(35, None, 3, 40, 1, 24, state=torch.float32, rows=5)
    buf = torch.full((5, 5, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    case.check(out=buf[:, 1:4, 8:48])
    assert bool((buf[:, 0] == 7).all() and (buf[:, 4] == 7).all() and (buf[..., :8] == 7).all())


def test_update_keeps_what_is_not_finite_to_its_row():
    case = Case(36, None, 2, 32, 2, 64, state=torch.float32, rows=2)
    clean = case.call()
    case.v[1, 1, 4] = float("inf")
    out = case.call()
    assert not torch.isfinite(out[1, 1, 4]) and int((~torch.isfinite(out)).sum()) == 1
    assert not torch.isfinite(case.pool[1, 1, 4]).any()
    out[1, 1, 4] = clean[1, 1, 4]
    assert torch.equal(out, clean)


def test_tokens_continue_a_prompt():
    """A prompt's last tokens one by one: the same outputs within both forms' bounds."""
    case = Case(37, [72], 4, 64, 2, 128, state=torch.float32, init=[True])
    args = [t.cuda() for t in (case.q, case.k, case.v, case.dt)] + [case.A.cuda(), case.beta.cuda()]
    more = dict(dt_bias=case.bias.cuda(), dt_softplus=True, beta_sigmoid=True, qk_l2norm=True)
    pool = case.state.cuda()
    cut = [a[:, :64] if a.dim() > 1 else a for a in args]
    dc.gated_delta_scan(*cut, state=pool, has_initial_state=torch.ones(1, dtype=torch.bool, device="cuda"), **more)
    got = [dc.gated_delta_update(*[a[:, t] if a.dim() > 1 else a for a in args], pool, **more) for t in range(64, 72)]
    exact = case.exact((0, slice(0, 72)))
    y, s = recurrence(*exact, case.state[0].double())
    dy, ds = bounds(*exact, case.state[0].double(), 64, True)
    close(torch.cat(got), y[64:], U * (y[64:].abs() + dy[64:]) + dy[64:], "tokens")
    close(pool[0], s, ds, "state")
