"""The state-space recurrence on the GPU against its 64-bit form: whole sequences, one
token, and one token with the convolution ahead of it.

Sizes sit at and around the kernels' edges (chunks of 32 tokens, tiles of 16 state
values and 32 channels, segments of long sequences, more units than blocks), with
strided views, padding and rejected rows, empty sequences and both state types.  The
bounds are derived in ``selective_reference``.
"""
import pytest
import torch

import depthwise_causal_conv1d_amd as dc
from selective_reference import U, close, convolve, recurrence

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


def params(gen, H):
    """Rates of -1 to -8 and steps of at most about 0.3."""
    A = -1.0 - 7.0 * torch.rand(H, generator=gen)
    bias = -4.0 + 2.0 * torch.rand(H, generator=gen)
    return A, torch.randn(H, generator=gen), bias


def f64(t):
    return None if t is None else t.double()


def strided(t, pad=8):
    """The same values on the device in rows `pad` elements longer."""
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + pad, dtype=t.dtype, device="cuda")
    wide[..., :t.shape[-1]] = t.cuda()
    return wide[..., :t.shape[-1]]


class Scan:
    """One call of selective_scan: inputs from the seed, the call, its check."""

    def __init__(self, seed, lens, H, P, G, K, state=None, packed=False, table=None, slots=None, init=None, z=True,
                 skip=True, soft=True, dt_f32=False, place=lambda t: t.cuda()):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.P, self.G, self.K, self.packed = lens, H, P, G, K, packed
        n = len(lens)
        rows, T = (1, sum(lens)) if packed else (n, lens[0])
        self.x, self.z = bf(gen, rows, T, H, P), bf(gen, rows, T, H, P) if z else None
        self.B, self.C = bf(gen, rows, T, G, K), bf(gen, rows, T, G, K)
        self.dt = torch.randn(rows, T, H, generator=gen) * 0.7
        if not soft:
            self.dt = self.dt.abs() * 0.2
        if not dt_f32:
            self.dt = self.dt.to(torch.bfloat16)
        self.A, self.D, self.bias = params(gen, H)
        if not skip:
            self.D = None
        if not soft:
            self.bias = None
        self.soft, self.table, self.init, self.state = soft, table, init, None
        if state is not None:
            slots = slots or n
            self.state = torch.randn(slots, H, P, K, generator=gen).to(state)
        self.place = place

    def call(self, **more):
        def dev(t):
            return None if t is None else t.cuda()
        self.pool = None if self.state is None else dev(self.state).clone()
        starts = torch.tensor([0] + self.lens).cumsum(0).to(torch.int32).cuda() if self.packed else None
        table = None if self.table is None else torch.tensor(self.table, dtype=torch.int32).cuda()
        init = None if self.init is None else torch.tensor(self.init, dtype=torch.bool).cuda()
        return dc.selective_scan(self.place(self.x), self.place(self.dt), dev(self.A), self.place(self.B),
                                 self.place(self.C), D=dev(self.D), z=None if self.z is None else self.place(self.z),
                                 dt_bias=dev(self.bias), dt_softplus=self.soft, ssm_state=self.pool,
                                 state_indices=table, has_initial_state=init, seq_starts=starts, **more)

    def check(self, dead=(), **more):
        out = self.call(**more)
        final = None
        if isinstance(out, tuple):
            out, final = out
        want_state = None if self.state is None else self.state.double()
        bound_state = None if self.state is None else torch.zeros_like(want_state)
        at = 0
        for i, L in enumerate(self.lens):
            row, lo = (0, at) if self.packed else (i, 0)
            at += L if self.packed else 0
            got = out[row, lo:lo + L]
            slot = i if self.table is None else self.table[i]
            if slot < 0 or i in dead:
                assert not got.any(), f"sequence {i}: padding must be zeros"
                continue
            h0 = self.state[slot].double() if self.init is not None and self.init[i] else None
            cut = [f64(t[row, lo:lo + L]) if t is not None else None for t in (self.x, self.dt, self.B, self.C, self.z)]
            y, ya, h, ha = recurrence(cut[0], cut[1], f64(self.A), cut[2], cut[3], f64(self.D), cut[4], f64(self.bias),
                                      self.soft, h0)
            close(got, y, U * y.abs() + (U + 2.0 ** -13) * ya, f"out of sequence {i}")
            if self.state is not None:
                want_state[slot] = h
                exact = self.state.dtype == torch.float32
                bound_state[slot] = 2.0 ** -17 * ha if exact else U * h.abs() + (U + 2.0 ** -13) * ha
            elif final is not None:
                close(final[i], h, 2.0 ** -17 * ha, f"final state of sequence {i}")
        if self.state is not None:
            close(self.pool, want_state, bound_state, "states")


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 129, 200])
def test_scan_lengths(T):
    Scan(T, [T, T], 4, 64, 2, 128, state=torch.float32, init=[True, False]).check()


@pytest.mark.parametrize("H,P,G,K", [(1, 64, 1, 128), (3, 32, 1, 16), (5, 80, 5, 72), (4, 128, 2, 64), (2, 16, 1, 256),
                                     (6, 96, 2, 32), (9, 8, 3, 8), (2, 64, 2, 1), (3, 1, 1, 5), (2, 33, 1, 130),
                                     (7, 64, 1, 200), (1, 200, 1, 65)])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_scan_head_layouts(H, P, G, K, state):
    Scan(H * P + K, [70], H, P, G, K, state=state, init=[True]).check()


@pytest.mark.parametrize("z,skip,soft,dt_f32", [(False, True, True, False), (True, False, True, True),
                                                (True, True, False, True), (False, False, False, False)])
def test_scan_options(z, skip, soft, dt_f32):
    Scan(3, [90], 3, 64, 1, 64, z=z, skip=skip, soft=soft, dt_f32=dt_f32).check()
    Scan(4, [90], 3, 64, 1, 64, z=z, skip=skip, soft=soft, dt_f32=dt_f32).check(return_final_state=True)


def test_scan_packed_with_pool():
    lens = [0, 1, 70, 64, 0, 300, 3, 5]
    Scan(5, lens, 4, 64, 2, 128, state=torch.float32, packed=True, slots=12, table=[3, 0, -1, 7, 11, 2, -1, 9],
         init=[True, True, True, False, False, True, False, True]).check()


def test_scan_long_sequences_are_split_and_joined():
    """Few blocks and many tokens: segments, with a pool slot read ahead and written behind."""
    case = Scan(6, [1500], 2, 32, 1, 64, state=torch.float32, init=[True])
    case.check()
    assert dc.dcconv_last_kernel().startswith("selective_scan_split")
    case = Scan(7, [900, 1, 0, 1200, 256, 257], 2, 32, 1, 64, state=torch.bfloat16, packed=True,
                table=[4, 0, 1, 2, -1, 3], slots=5, init=[True, False, True, True, True, False])
    case.check()
    assert dc.dcconv_last_kernel().startswith("selective_scan_split")
    Scan(8, [700, 700], 3, 40, 1, 33).check(return_final_state=True)


def test_scan_of_strided_and_unaligned_views():
    Scan(9, [100], 4, 64, 2, 128, state=torch.float32, place=strided).check()
    Scan(10, [100], 4, 64, 2, 128, state=torch.float32, place=lambda t: strided(t, 3)).check()
    assert dc.dcconv_last_kernel() == "selective_scan_scalar"

    def off(t):  # a base two bytes past 16
        flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten().cuda()
        return flat[1:].view(t.shape)
    Scan(11, [100], 4, 64, 2, 128, state=torch.bfloat16, place=off).check()


def test_scan_of_head_major_and_broadcast_operands():
    """Heads further apart than tokens, so that a row past the end is another head's; and
    rows that are one and the same."""
    def head_major(t):
        t = t.cuda()
        return t.transpose(1, 2).contiguous().transpose(1, 2) if t.dim() == 4 else t
    case = Scan(18, [75, 75], 6, 64, 2, 64, state=torch.float32, place=head_major)
    buf = torch.full((2, 6, 90, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    case.check(out=buf[:, :, 5:80].transpose(1, 2))
    assert bool((buf[:, :, :5] == 7).all() and (buf[:, :, 80:] == 7).all())
    case = Scan(19, [75, 75], 4, 32, 1, 64, state=torch.float32)
    for t in (case.x, case.z, case.B, case.C):
        t.copy_(t[:1, :1].expand_as(t).clone())
    case.place = lambda t: t[:1, :1].cuda().expand(t.shape) if t.dim() == 4 else t.cuda()
    case.check()


def test_scan_writes_only_its_output():
    case = Scan(12, [77, 77], 3, 40, 1, 24, state=torch.float32)
    buf = torch.full((2, 77, 5, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :, 1:4, 8:48]
    case.check(out=out)
    assert bool((buf[:, :, 0] == 7).all() and (buf[:, :, 4] == 7).all() and (buf[..., :8] == 7).all())


def test_scan_bad_and_duplicate_indices():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Scan(13, [20] * 5, 2, 32, 1, 32, state=torch.float32, slots=6, table=[6, -1, 2, 4, 4]).check(
        dead=(0, 3, 4), dev_status=status)
    assert int(status) == dc.DCCONV_DEV_BAD_INDEX | dc.DCCONV_DEV_DUP_INDEX


@pytest.mark.parametrize("starts", [[0, 50, 40, 100], [1, 40, 60, 100], [0, 40, 60, 90], [0, -5, 60, 100],
                                    [0, 40, 2000, 100]])
def test_scan_reports_a_broken_sequence_table(starts):
    case = Scan(14, [100], 2, 32, 1, 32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    buf = torch.full((3, 100, 2, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    dc.selective_scan(case.x.cuda(), case.dt.cuda(), case.A.cuda(), case.B.cuda(), case.C.cuda(), out=buf[1:2],
                      seq_starts=torch.tensor(starts, dtype=torch.int32).cuda(), dev_status=status)
    assert int(status) & dc.DCCONV_DEV_BAD_SEQ
    assert bool((buf[0] == 7).all() and (buf[2] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scan_keeps_bad_values_where_the_recurrence_takes_them(bad):
    """A NaN or infinity in x, B or C of one token leaves every earlier token, every other
    sequence and, for x, every other channel as they were."""
    clean = Scan(15, [60, 100, 30], 2, 64, 1, 64, state=torch.float32, packed=True)
    want, states = clean.call(), None
    states = clean.pool.clone()
    for name in ("x", "B", "C"):
        case = Scan(15, [60, 100, 30], 2, 64, 1, 64, state=torch.float32, packed=True)
        getattr(case, name)[0, 60 + 37, 0, 5] = bad
        out = case.call()
        assert torch.equal(out[0, :97], want[0, :97]) and torch.equal(out[0, 160:], want[0, 160:]), name
        assert torch.equal(case.pool[0], states[0]) and torch.equal(case.pool[2], states[2]), name
        assert not torch.isfinite(out[0, 97, 0, 5]), name
        if name == "x":
            keep = torch.arange(64, device="cuda") != 5
            assert torch.equal(out[0, :, 0, keep], want[0, :, 0, keep]) and torch.equal(out[0, :, 1], want[0, :, 1])
        if name == "C":
            assert torch.equal(case.pool, states) and torch.equal(out[0, 98:], want[0, 98:])


@pytest.mark.parametrize("step", [300.0, 1e6, 3e37])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_scan_after_a_step_that_decays_everything(step, state):
    """A step whose decay is zero leaves the decays between the tokens behind it as exact as
    any others, though a chunk's sum of dt A has grown to the size of that step's."""
    case = Scan(21, [70], 3, 64, 1, 64, state=state, init=[True], soft=False, dt_f32=True)
    case.x[0, 40] *= 1.0 / step
    case.dt[0, 40] = step
    case.check()


def test_scan_more_units_than_blocks():
    n = (1 << 20) + 5
    x = torch.randn(n, 1, 1, 2, device="cuda").to(torch.bfloat16)
    one = torch.ones(n, 1, 1, 1, device="cuda").to(torch.bfloat16)
    dt = torch.rand(n, 1, 1, device="cuda")
    out = dc.selective_scan(x, dt, torch.zeros(1, device="cuda"), one, one)
    want = dt[..., None].double() * x.double()
    assert bool(((out.double() - want).abs() <= 2.1 * U * want.abs()).all())


class Update:
    """One call of selective_update, or of its fused form."""

    def __init__(self, seed, N, H, P, G, K, state, table=None, slots=None, z=True, skip=True, soft=True, dt_f32=False,
                 fused=False, L=3, layout="compact", bias=True, act="silu", seen=None, place=lambda t: t.cuda()):
        gen = torch.Generator().manual_seed(seed)
        self.N, self.H, self.P, self.G, self.K, self.L = N, H, P, G, K, L
        S = slots or N
        self.x, self.z = bf(gen, N, H, P), bf(gen, N, H, P) if z else None
        self.B, self.C = bf(gen, N, G, K), bf(gen, N, G, K)
        self.dt = torch.randn(N, H, generator=gen) * (0.7 if soft else 0.1)
        if not dt_f32:
            self.dt = self.dt.to(torch.bfloat16)
        self.A, self.D, self.bias = params(gen, H)
        self.D, self.bias = self.D if skip else None, self.bias if soft else None
        self.soft, self.table, self.place, self.fused, self.act, self.seen = soft, table, place, fused, act, seen
        self.state = torch.randn(S, H, P, K, generator=gen).to(state)
        Dc = H * P + 2 * G * K
        self.xbc = bf(gen, N, Dc)
        self.conv = bf(gen, S, Dc, L)
        self.weight, self.cbias = bf(gen, Dc, 4, scale=0.5), bf(gen, Dc, scale=0.1) if bias else None
        self.layout = layout

    def call(self, **more):
        def dev(t):
            return None if t is None else t.cuda()
        self.pool = dev(self.state).clone()
        table = None if self.table is None else torch.tensor(self.table, dtype=torch.int32).cuda()
        z = None if self.z is None else self.place(self.z)
        rest = dict(D=dev(self.D), z=z, dt_bias=dev(self.bias), dt_softplus=self.soft, state_indices=table, **more)
        if not self.fused:
            return dc.selective_update(self.place(self.x), self.place(self.dt), dev(self.A), self.place(self.B),
                                       self.place(self.C), self.pool, **rest)
        if self.layout == "compact":
            self.history = self.conv.cuda().clone()
        else:
            self.history = self.conv.permute(0, 2, 1).contiguous().cuda().permute(0, 2, 1)
        seen = None if self.seen is None else torch.tensor(self.seen, dtype=torch.int32).cuda()
        return dc.causal_conv1d_selective_update(self.place(self.xbc), self.history, dev(self.weight), dev(self.cbias),
                                                 self.act, self.place(self.dt), dev(self.A), self.pool, groups=self.G,
                                                 cache_seqlens=seen, **rest)

    def check(self, dead=(), **more):
        out = self.call(**more)
        state, bound = self.state.double(), torch.zeros(self.state.shape, dtype=torch.float64)
        conv = self.conv.clone()
        H, P, G, K, L = self.H, self.P, self.G, self.K, self.L
        for i in range(self.N):
            slot = i if self.table is None else self.table[i]
            if slot < 0 or i in dead:
                assert not out[i].any(), f"row {i}: padding must be zeros"
                continue
            x, B, C = (f64(t[i]) for t in (self.x, self.B, self.C))
            if self.fused:
                at = [L - 3 + j for j in range(3)] if self.seen is None else [(self.seen[i] - 3 + j) % L for j in range(3)]
                v = convolve(f64(self.conv[slot][:, at]), f64(self.xbc[i]), f64(self.weight), f64(self.cbias), self.act)
                x, B, C = v[:H * P].view(H, P), v[H * P:H * P + G * K].view(G, K), v[H * P + G * K:].view(G, K)
                if self.seen is None:
                    conv[slot] = torch.cat([self.conv[slot][:, 1:], self.xbc[i][:, None]], 1)
                else:
                    conv[slot][:, self.seen[i] % L] = self.xbc[i]
            z = None if self.z is None else f64(self.z[i])[None]
            y, ya, h, ha = recurrence(x[None], f64(self.dt[i])[None], f64(self.A), B[None], C[None], f64(self.D), z,
                                      f64(self.bias), self.soft, f64(self.state[slot]))
            # the convolution's own sum: five terms of up to 2^4 around results near 2^-4 at the least
            wide = 2.0 ** -15 if self.fused else 2.0 ** -18
            close(out[i], y[0], U * y[0].abs() + wide * ya[0] + (1e-5 if self.fused else 0.0), f"out of row {i}")
            state[slot] = h
            bound[slot] = wide * ha + (1e-5 if self.fused else 0.0)
            if self.state.dtype == torch.bfloat16:
                bound[slot] += U * h.abs()
        close(self.pool, state, bound, "states")
        if self.fused:
            assert torch.equal(self.history.cpu().contiguous().view(torch.int16), conv.contiguous().view(torch.int16))


LAYOUTS = [(1, 64, 1, 128), (3, 32, 1, 16), (5, 80, 5, 72), (4, 128, 2, 64), (2, 16, 1, 256), (6, 96, 2, 32),
           (9, 8, 3, 8), (2, 64, 2, 1), (3, 1, 1, 5), (2, 33, 1, 130), (1, 200, 1, 65)]


@pytest.mark.parametrize("H,P,G,K", LAYOUTS)
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fused", [False, True])
def test_update_head_layouts(H, P, G, K, state, fused):
    Update(H * P + K, 3, H, P, G, K, state, fused=fused).check()


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("z,skip,soft,dt_f32", [(False, True, True, False), (True, False, True, True),
                                                (True, True, False, True), (False, False, False, False)])
def test_update_options(z, skip, soft, dt_f32, fused):
    Update(3, 4, 3, 64, 1, 64, torch.float32, z=z, skip=skip, soft=soft, dt_f32=dt_f32, fused=fused).check()


@pytest.mark.parametrize("fused", [False, True])
def test_update_routing(fused):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Update(4, 6, 2, 64, 1, 128, torch.float32, slots=9, table=[8, -1, 9, 3, 0, 3], fused=fused).check(
        dead=(2, 3, 5), dev_status=status)
    assert int(status) == dc.DCCONV_DEV_BAD_INDEX | dc.DCCONV_DEV_DUP_INDEX


@pytest.mark.parametrize("fused", [False, True])
def test_update_large_grid_takes_more_rows_a_block(fused):
    """Enough heads that a block takes 64 rows of the state instead of 16."""
    case = Update(5, 70, 30, 80, 3, 72, torch.bfloat16, fused=fused)
    case.check()


@pytest.mark.parametrize("fused", [False, True])
def test_update_of_strided_views(fused):
    Update(6, 4, 3, 40, 1, 24, torch.float32, fused=fused, place=lambda t: strided(t, 3)).check()
    case = Update(7, 4, 3, 40, 1, 24, torch.float32, fused=fused)
    buf = torch.full((4, 5, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    case.check(out=buf[:, 1:4])
    assert bool((buf[:, 0] == 7).all() and (buf[:, 4] == 7).all())


@pytest.mark.parametrize("L", [3, 4, 5, 9])
@pytest.mark.parametrize("layout", ["compact", "channel_last"])
@pytest.mark.parametrize("ring", [False, True])
def test_fused_histories(L, layout, ring):
    seen = [0, 1, 7, 4095] if ring else None
    Update(L, 4, 4, 64, 2, 128, torch.float32, fused=True, L=L, layout=layout, seen=seen, bias=False, act=None).check()


def test_fused_negative_count_is_padding():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Update(8, 3, 2, 64, 1, 128, torch.float32, fused=True, L=4, seen=[5, -1, 2]).check(dead=(1,), dev_status=status)
    assert int(status) == dc.DCCONV_DEV_BAD_SEQLEN


def test_fused_workspace_is_left_zero_and_serves_again():
    case = Update(9, 5, 6, 64, 3, 128, torch.float32, fused=True, slots=7, table=[3, -1, 0, 6, 2])
    ws = dc.selective_update_workspace(5, 3)
    for _ in range(3):
        case.check(workspace=ws)
        assert not ws.any()


def test_fused_steps_continue_a_prompt():
    """conv prefill + scan over T tokens, then steps, against the scan over all of them."""
    N, T, more, H, P, G, K = 2, 100, 5, 4, 64, 2, 128
    Dc = H * P + 2 * G * K
    gen = torch.Generator().manual_seed(10)
    xbc, z, dt = bf(gen, N, T + more, Dc), bf(gen, N, T + more, H, P), bf(gen, N, T + more, H)
    w, b = bf(gen, Dc, 4, scale=0.5).cuda(), bf(gen, Dc, scale=0.1).cuda()
    A, D, bias = (v.cuda() for v in params(gen, H))
    xbc, z, dt = xbc.cuda(), z.cuda(), dt.cuda()

    def prompt(t):
        y, conv = dc.causal_conv1d(xbc[:, :t].permute(0, 2, 1), w, b, "silu", return_final_state=True)
        y = y.permute(0, 2, 1)
        x, B, C = y[..., :H * P], y[..., H * P:H * P + G * K], y[..., H * P + G * K:]
        out, state = dc.selective_scan(x.unflatten(-1, (H, P)), dt[:, :t], A, B.unflatten(-1, (G, K)),
                                       C.unflatten(-1, (G, K)), D=D, z=z[:, :t], dt_bias=bias, dt_softplus=True,
                                       return_final_state=True)
        return out, conv, state

    whole, _, last = prompt(T + more)
    out, conv, state = prompt(T)
    assert torch.equal(out[:, :64], whole[:, :64])
    for i in range(more):
        y = dc.causal_conv1d_selective_update(xbc[:, T + i], conv, w, b, "silu", dt[:, T + i], A, state, groups=G, D=D,
                                              z=z[:, T + i], dt_bias=bias, dt_softplus=True)
        # the prompt's x, B and C are rounded to BF16, and its products once more
        scale = whole[:, T + i].float().square().mean().sqrt()
        assert float((y.float() - whole[:, T + i].float()).abs().max()) <= 0.05 * float(scale) + 0.02
    assert float((state - last).norm() / last.norm()) < 4 * U


def test_calls_on_another_stream_and_in_a_graph():
    case = Update(11, 4, 4, 64, 2, 128, torch.float32, fused=True)
    want = case.call().clone()
    state, history = case.pool.clone(), case.history.clone()
    scan = Scan(12, [1500], 2, 32, 1, 64, state=torch.float32)
    want_scan = scan.call().clone()
    args = [t.cuda() for t in (case.xbc, case.weight, case.cbias, case.dt, case.A, case.D, case.z, case.bias)]
    sargs = [t.cuda() for t in (scan.x, scan.dt, scan.A, scan.B, scan.C, scan.D, scan.z, scan.bias)]
    pool, conv, spool = case.state.cuda(), case.conv.cuda(), scan.state.cuda()
    ws = dc.selective_update_workspace(4, 2)
    out, sout = torch.empty(4, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty_like(want_scan)
    need = dc.dcconv_selective_scan_workspace(1, 1500, 2, 32, 1, 64, 0)
    sws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def both():
        dc.causal_conv1d_selective_update(args[0], conv, args[1], args[2], "silu", args[3], args[4], pool, groups=2,
                                          D=args[5], z=args[6], dt_bias=args[7], dt_softplus=True, workspace=ws, out=out)
        dc.selective_scan(sargs[0], sargs[1], sargs[2], sargs[3], sargs[4], D=sargs[5], z=sargs[6], dt_bias=sargs[7],
                          dt_softplus=True, ssm_state=spool, workspace=sws, out=sout)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(pool, state) and torch.equal(conv, history)
    assert torch.equal(sout, want_scan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(4):
        pool.copy_(case.state)
        conv.copy_(case.conv)
        spool.copy_(scan.state)
        out.zero_(), sout.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool, state) and torch.equal(conv, history)
        assert torch.equal(sout, want_scan)


def test_results_do_not_depend_on_the_run():
    case = Scan(16, [1500, 20], 4, 64, 2, 128, state=torch.float32, packed=True)
    first, state = case.call().clone(), case.pool.clone()
    for _ in range(3):
        assert torch.equal(case.call(), first) and torch.equal(case.pool, state)


def test_offsets_past_32_bits():
    """Slots and rows more than 2^32 bytes apart."""
    H, P, K = 2, 32, 64
    gen = torch.Generator().manual_seed(17)
    slot = (1 << 30) + 8
    pool = torch.empty(slot + H * P * K + 64, dtype=torch.float32, device="cuda")
    view = pool.as_strided((2, H, P, K), (slot, P * K, K, 1))
    start = torch.randn(2, H, P, K, generator=gen)
    view.copy_(start)
    row = (1 << 31) + 8
    xbuf = torch.empty(row + H * P, dtype=torch.bfloat16, device="cuda")
    x = xbuf.as_strided((2, H, P), (row, P, 1))
    xs = bf(gen, 2, H, P)
    x.copy_(xs)
    B, C, dt = bf(gen, 2, 1, K), bf(gen, 2, 1, K), torch.rand(2, H, generator=gen) * 0.2
    A, _, _ = params(gen, H)
    for scan in (False, True):
        view.copy_(start)
        if scan:
            out = dc.selective_scan(x[:, None], dt.cuda()[:, None], A.cuda(), B.cuda()[:, None], C.cuda()[:, None],
                                    ssm_state=view, has_initial_state=torch.ones(2, dtype=torch.bool, device="cuda"))[:, 0]
        else:
            out = dc.selective_update(x, dt.cuda(), A.cuda(), B.cuda(), C.cuda(), view)
        for i in range(2):
            y, ya, h, ha = recurrence(f64(xs[i])[None], f64(dt[i])[None], f64(A), f64(B[i])[None], f64(C[i])[None],
                                      h0=f64(start[i]))
            close(out[i], y[0], U * y[0].abs() + (U + 2.0 ** -13) * ya[0], "out")
            close(view[i], h, 2.0 ** -17 * ha, "state")


def test_scan_heads_past_32_bits():
    """Heads 2^31 elements apart, read and written element by element."""
    apart, T, H, P = (1 << 31) + 8, 40, 2, 32
    case = Scan(21, [T], H, P, 1, 64, state=torch.float32, z=False)
    buf = torch.empty(apart + 2 * T * P, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((1, T, H, P), (0, P, apart, 1))
    x.copy_(case.x)
    want = case.call()
    state = case.pool.clone()
    case.place = lambda t: x if t is case.x else t.cuda()
    big = torch.empty(apart + T * P, dtype=torch.bfloat16, device="cuda")
    out = big.as_strided((1, T, H, P), (0, P, apart, 1))
    got = case.call(out=out)
    assert torch.equal(got, want) and torch.equal(case.pool, state)


def test_refusals():
    case = Update(20, 3, 4, 64, 2, 128, torch.float32)
    x, dt, A, B, C, state = (t.cuda() for t in (case.x, case.dt, case.A, case.B, case.C, case.state))

    def update(**over):
        a = dict(x=x, dt=dt, A=A, B=B, C=C, ssm_state=state)
        a.update(over)
        return dc.selective_update(a.pop("x"), a.pop("dt"), a.pop("A"), a.pop("B"), a.pop("C"), a.pop("ssm_state"), **a)
    for over, what in ((dict(x=x.float()), "bfloat16"), (dict(dt=dt.half()), "dt must be"), (dict(A=A.bfloat16()), "A must"),
                       (dict(A=None), "A must"), (dict(B=B[:, :, :64]), "C must"), (dict(C=C[:2]), "C must"),
                       (dict(ssm_state=state.half()), "ssm_state"), (dict(ssm_state=state[:, :, :, ::2]), "ssm_state"),
                       (dict(ssm_state=state.transpose(1, 2).contiguous().transpose(1, 2)), "dense"),
                       (dict(x=x.transpose(1, 2).contiguous().transpose(1, 2)), "unit stride"),
                       (dict(z=x[:, :2]), "z must"), (dict(D=A[:2]), "D must"), (dict(out=x), "overlap"),
                       (dict(state_indices=torch.zeros(3, dtype=torch.int64, device="cuda")), "int32"),
                       (dict(ssm_state=state[:2]), "slot"), (dict(dt=dt.cpu()), "on cpu")):
        before = state.clone()
        with pytest.raises(ValueError, match=what):
            update(**over)
        assert torch.equal(state, before)
    with pytest.raises(NotImplementedError, match="training"):
        update(x=x.clone().requires_grad_())
    big = torch.zeros(3, 2, 300, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(NotImplementedError, match="256"):
        update(B=big, C=big, ssm_state=torch.zeros(3, 4, 64, 300, device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        dc.causal_conv1d_selective_update(torch.zeros(3, 768, dtype=torch.bfloat16, device="cuda"),
                                          torch.zeros(3, 768, 3, dtype=torch.bfloat16, device="cuda"),
                                          torch.zeros(768, 4, dtype=torch.bfloat16, device="cuda"), None, None, dt, A, state,
                                          groups=2, workspace=torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="packed"):
        dc.selective_scan(x[:, None], dt[:, None], A, B[:, None], C[:, None],
                          seq_starts=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="need an ssm_state"):
        dc.selective_scan(x[:, None], dt[:, None], A, B[:, None], C[:, None], return_final_state=True,
                          has_initial_state=torch.ones(3, dtype=torch.bool, device="cuda"))
