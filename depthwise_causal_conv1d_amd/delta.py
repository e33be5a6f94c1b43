"""The gated delta rule behind the convolution, and the norms of its layer: Python binding.

``gated_delta_scan`` runs whole prompts and ``gated_delta_update`` one token a row.  Per
head, with d = softplus(dt + dt_bias), b = sigmoid(beta) and the head's group holding q and
k::

    state = exp(d * A) * state
    u     = b * (v - state k)
    state = state + u k^T
    out   = scale * state q

``gated_rms_norm`` norms the recurrence's output head by head and gates it;
``add_rms_norm`` adds a block's output to the residual stream and norms that for the next
block.

The ``dcconv_*`` functions mirror the C entry points of ``include/dcconv.h`` one to one; the
tensor functions check shapes and types, pass strides and the current stream, and allocate
the output.
"""
from __future__ import annotations

import ctypes

from . import _binding as _b
from . import selective as _s

__all__ = [
    "dcconv_gated_delta_update", "dcconv_gated_delta_scan", "dcconv_gated_delta_scan_workspace",
    "dcconv_gated_rms_norm", "dcconv_add_rms_norm",
    "gated_delta_scan", "gated_delta_update", "gated_rms_norm", "add_rms_norm",
]


def declare(lib: ctypes.CDLL) -> None:
    """The argument types of this module's C entry points."""
    i64, vp, i32, f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.dcconv_gated_delta_update.restype = i32
    lib.dcconv_gated_delta_update.argtypes = (
        [vp, vp, vp] + [i64] * 5                      # q, key, v, n, h, p, g, k
        + [i64] * 6                                   # qs_n, qs_g, ks_n, ks_g, vs_n, vs_h
        + [vp, i32, i64, vp, i32, vp]                 # dt, dt_dtype, ds_n, dt_bias, dt_softplus, a
        + [vp, i32, i64, i32]                         # beta, beta_dtype, es_n, beta_sigmoid
        + [i32, f32, f32]                             # qk_l2norm, l2norm_eps, scale
        + [vp, i32, i64, i64, vp]                     # state, state_dtype, s, ss_s, state_indices
        + [vp, i64, i64, vp, vp])                     # out, os_n, os_h, dev_status, stream
    lib.dcconv_gated_delta_scan.restype = i32
    lib.dcconv_gated_delta_scan.argtypes = (
        [vp, vp, vp] + [i64] * 6                      # q, key, v, n, t, h, p, g, k
        + [i64] * 9                                   # strides of q, key and v
        + [vp, i32, i64, i64, vp, i32, vp]            # dt, dt_dtype, ds_n, ds_t, dt_bias, dt_softplus, a
        + [vp, i32, i64, i64, i32]                    # beta, beta_dtype, es_n, es_t, beta_sigmoid
        + [i32, f32, f32, vp]                         # qk_l2norm, l2norm_eps, scale, seq_starts
        + [vp, i32, i64, i64, vp, vp]                 # state, state_dtype, s, ss_s, state_indices, has_initial_state
        + [vp, i64, i64, i64, vp, i64, vp, vp])       # out, os_n, os_t, os_h, workspace, bytes, dev_status, stream
    lib.dcconv_gated_delta_scan_workspace.restype = i64
    lib.dcconv_gated_delta_scan_workspace.argtypes = [i64] * 6 + [i32]
    lib.dcconv_gated_rms_norm.restype = i32
    lib.dcconv_gated_rms_norm.argtypes = (
        [vp] + [i64] * 7                              # x, n, t, h, d, xs_n, xs_t, xs_h
        + [vp, i64, i64, i64, i32]                    # z, zs_n, zs_t, zs_h, gate_first
        + [vp, i32, i64, f32, f32]                    # weight, weight_dtype, ws_h, weight_offset, eps
        + [vp, i64, i64, i64, vp])                    # out, os_n, os_t, os_h, stream
    lib.dcconv_add_rms_norm.restype = i32
    lib.dcconv_add_rms_norm.argtypes = (
        [vp] + [i64] * 5                              # x, n, t, d, xs_n, xs_t
        + [vp, i32, i64, i64]                         # residual, residual_dtype, rs_n, rs_t
        + [vp, i64, i64, f32]                         # gate, gs_n, gs_t, residual_scale
        + [vp, vp, i32, f32, f32]                     # post_weight, weight, weight_dtype, weight_offset, eps
        + [vp, i64, i64, vp])                         # out, os_n, os_t, stream


# ----------------------------------------------------------------- raw C ABI


def dcconv_gated_delta_update(*args) -> int:
    """The one-token C entry point, one to one (pointers as ints, 0/None = NULL)."""
    return _b.load().dcconv_gated_delta_update(*args)


def dcconv_gated_delta_scan(*args) -> int:
    """The whole-sequence C entry point, one to one (pointers as ints)."""
    return _b.load().dcconv_gated_delta_scan(*args)


def dcconv_gated_delta_scan_workspace(n, t, h, p, g, k, packed) -> int:
    """Bytes of workspace a scan of these sizes needs, one to one."""
    return _b.load().dcconv_gated_delta_scan_workspace(n, t, h, p, g, k, packed)


def dcconv_gated_rms_norm(*args) -> int:
    """The gated norm's C entry point, one to one (pointers as ints)."""
    return _b.load().dcconv_gated_rms_norm(*args)


def dcconv_add_rms_norm(*args) -> int:
    """The residual norm's C entry point, one to one (pointers as ints)."""
    return _b.load().dcconv_add_rms_norm(*args)


# ------------------------------------------------------------ tensor front end


def _like(t):
    """A new contiguous tensor of t's shape and type (the shorter of torch's ways: 0.5 to 1 us a call)."""
    return _s._t.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _per_head(name, t, shape, dev):
    """(address, dtype code, strides) of dt or beta."""
    code = _s._dtype(name, t)
    if t.shape != shape or t.get_device() != dev or t.requires_grad:
        _s._refuse(name, t, None, shape, dev)
    stride = t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride along its heads")
    return t.data_ptr(), code, stride


def _pool(state, H, P, K, dev):
    """(dtype code, S, slot stride) of a state [S, H, P, K]."""
    if state.dim() != 4:
        raise ValueError(f"state must be [S, H, P, K], got shape {tuple(state.shape)}")
    code = _s._dtype("state", state)
    shape = state.shape
    if shape[1:] != (H, P, K) or state.get_device() != dev or state.requires_grad:
        _s._refuse("state", state, None, (shape[0], H, P, K), dev)
    S, stride = shape[0], state.stride()
    if stride[1:] != (P * K, K, 1) and S > 0 and not state[0].is_contiguous():
        raise ValueError("state must be dense inside a slot")
    return code, S, (stride[0] if S > 1 else H * P * K)


def gated_delta_update(q, k, v, dt, A, beta, state, *, dt_bias=None, dt_softplus=False, beta_sigmoid=False,
                       qk_l2norm=False, l2norm_eps=1e-6, scale=None, state_indices=None, out=None, dev_status=None):
    """One token of N rows: ``state`` is updated in place and the output [N, H, P] returned.

    q, k: bf16 [N, G, K] (H a multiple of G); v: bf16 [N, H, P]; dt, beta: bf16 or float32
    [N, H]; A, dt_bias: float32 [H]; state: bf16 or float32 [S, H, P, K].  Any strides with
    dense last dimensions.  The decay is exp(d * A) with d = dt + dt_bias, through softplus
    if ``dt_softplus`` (a log-decay that is at hand goes in as dt, with A of ones).
    ``beta_sigmoid``: beta is a logit.  ``qk_l2norm``: q and k are divided by the root of
    their sum of squares + ``l2norm_eps``.  ``scale``: K ** -0.5 if None.
    ``state_indices`` (int32 [N]) routes rows to slots, -1 being a padding row (zero
    output, no state moves)."""
    lib = _s._lib()
    if v.dim() != 3 or k.dim() != 3:
        raise ValueError(f"v must be [N, H, P] and k [N, G, K], got {tuple(v.shape)} and {tuple(k.shape)}")
    dev = _s._gpu(v)
    N, H, P = rows = v.shape
    _, G, K = keys = (N, *k.shape[1:])
    vs = _s._bf16("v", v, rows, dev)
    qs, ks = _s._bf16("q", q, keys, dev), _s._bf16("k", k, keys, dev)
    code, S, slot = _pool(state, H, P, K, dev)
    dt_at, dt_code, ds = _per_head("dt", dt, (N, H), dev)
    beta_at, beta_code, es = _per_head("beta", beta, (N, H), dev)
    if A is None:
        raise ValueError("A must be given")
    if out is None:
        out, os_ = _like(v), (H * P, P)
    else:
        os_ = _s._bf16("out", out, rows, dev)
    with _b.on(dev):
        rc = lib.dcconv_gated_delta_update(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), N, H, P, G, K, qs[0], qs[1], ks[0], ks[1], vs[0], vs[1],
            dt_at, dt_code, ds[0], _s._vector("dt_bias", dt_bias, _s._F32, H, dev), int(bool(dt_softplus)),
            _s._vector("A", A, _s._F32, H, dev), beta_at, beta_code, es[0], int(bool(beta_sigmoid)),
            int(bool(qk_l2norm)), l2norm_eps, max(K, 1) ** -0.5 if scale is None else scale, state.data_ptr(), code, S, slot,
            _s._vector("state_indices", state_indices, _s._I32, N, dev), out.data_ptr(), os_[0], os_[1],
            _s._status(dev_status, dev), _b.stream(dev))
    _b.raise_for(rc)
    return out


def gated_delta_scan(q, k, v, dt, A, beta, *, dt_bias=None, dt_softplus=False, beta_sigmoid=False, qk_l2norm=False,
                     l2norm_eps=1e-6, scale=None, state=None, state_indices=None, has_initial_state=None,
                     seq_starts=None, return_final_state=False, workspace=None, out=None, dev_status=None):
    """The recurrence over whole sequences; returns the output [N, T, H, P].

    q, k: bf16 [N, T, G, K]; v: bf16 [N, T, H, P]; dt, beta: bf16 or float32 [N, T, H]; A,
    dt_bias: float32 [H].  With ``seq_starts`` (int32 [n+1] on the device) N is 1 and the T
    axis holds n packed sequences.
    state: bf16 or float32 [S, H, P, K] pool; sequences that ``has_initial_state`` (bool/uint8
    [n]) marks start from their slot's state, and every sequence leaves its final state there;
    ``state_indices`` (int32 [n]) routes sequences to slots, -1 being padding.
    return_final_state: without ``state``, returns ``(out, state)`` with a new float32
    [n, H, P, K] state.  ``workspace``: a uint8 buffer of ``dcconv_gated_delta_scan_workspace``
    bytes (allocated here if None).  The rest as for ``gated_delta_update``.

    Sums and states are 32 bits, the operands of the matrix products keep 16 bits or more, and
    the output (and a bf16 state) is rounded once."""
    lib = _s._lib()
    if v.dim() != 4 or k.dim() != 4:
        raise ValueError(f"v must be [N, T, H, P] and k [N, T, G, K], got {tuple(v.shape)} and {tuple(k.shape)}")
    dev = _s._gpu(v)
    N, T, H, P = rows = v.shape
    _, _, G, K = keys = (N, T, *k.shape[2:])
    vs = _s._bf16("v", v, rows, dev)
    qs, ks = _s._bf16("q", q, keys, dev), _s._bf16("k", k, keys, dev)
    dt_at, dt_code, ds = _per_head("dt", dt, (N, T, H), dev)
    beta_at, beta_code, es = _per_head("beta", beta, (N, T, H), dev)
    if A is None:
        raise ValueError("A must be given")
    n = N
    if seq_starts is not None:
        if N != 1:
            raise ValueError("with seq_starts, v must be [1, total_T, H, P] (packed sequences)")
        if seq_starts.dim() != 1 or seq_starts.shape[0] < 1:
            raise ValueError("seq_starts must be a contiguous int32 [n+1] tensor")
        n = seq_starts.shape[0] - 1
    starts = _s._vector("seq_starts", seq_starts, _s._I32, n + 1, dev)
    init = None
    if has_initial_state is not None:
        if has_initial_state.dtype not in (_s._t.bool, _s._t.uint8):
            raise ValueError("has_initial_state must be a contiguous bool/uint8 [n] tensor")
        init = _s._vector("has_initial_state", has_initial_state, has_initial_state.dtype, n, dev)
    final = None
    if state is None and (has_initial_state is not None or state_indices is not None):
        raise ValueError("has_initial_state and state_indices need a state")
    if state is None and return_final_state:
        state = final = _s._t.empty(n, H, P, K, dtype=_s._F32, device=v.device)
    code, S, slot, pool = _s.DCCONV_DTYPE_F32, 0, 0, None
    if state is not None:
        code, S, slot = _pool(state, H, P, K, dev)
        if S == 0 and n > 0:  # (its address is NULL, which would mean no state)
            raise ValueError(f"state has no slots for {n} sequences")
        pool = state.data_ptr()
    if out is None:
        out, os_ = _like(v), (T * H * P, H * P, P)
    else:
        os_ = _s._bf16("out", out, rows, dev)
    need = lib.dcconv_gated_delta_scan_workspace(n, T, H, P, G, K, int(starts is not None))
    if workspace is None:
        workspace = _s._t.empty(need, dtype=_s._t.uint8, device=v.device) if need else None
    elif workspace.dtype is not _s._t.uint8 or not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be a contiguous uint8 tensor on v's device")
    with _b.on(dev):
        rc = lib.dcconv_gated_delta_scan(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), n, T, H, P, G, K, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2],
            vs[0], vs[1], vs[2], dt_at, dt_code, ds[0], ds[1], _s._vector("dt_bias", dt_bias, _s._F32, H, dev),
            int(bool(dt_softplus)), _s._vector("A", A, _s._F32, H, dev), beta_at, beta_code, es[0], es[1],
            int(bool(beta_sigmoid)), int(bool(qk_l2norm)), l2norm_eps, max(K, 1) ** -0.5 if scale is None else scale, starts,
            pool, code, S, slot, _s._vector("state_indices", state_indices, _s._I32, n, dev), init, out.data_ptr(),
            os_[0], os_[1], os_[2], None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel(), _s._status(dev_status, dev), _b.stream(dev))
    _b.raise_for(rc)
    return (out, final) if final is not None else out


def _weight(name, t, shapes, dev):
    """(address, dtype code) of a contiguous weight of one of `shapes`."""
    code = _s._dtype(name, t)
    if t.shape not in shapes or t.get_device() != dev or t.requires_grad:
        _s._refuse(name, t, None, shapes[0], dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), code


def gated_rms_norm(x, z, weight, *, eps=1e-6, gate_first=False, weight_offset=0.0, out=None):
    """Rows of x divided by their root mean square, times weight and silu(z); returns bf16
    of x's shape.

    x: bf16 [..., D] with one to four dimensions, z: likewise or None (no gate), any strides
    with a dense last dimension; weight: bf16 or float32 [D], or [H, D] with H the size of x's
    second last dimension, or None (ones).  ``weight_offset`` is added to every weight.
    ``gate_first``: x * silu(z) is normed, instead of x."""
    lib = _s._lib()
    if not 1 <= x.dim() <= 4:
        raise ValueError(f"x must have one to four dimensions, got shape {tuple(x.shape)}")
    dev = _s._gpu(x)
    shape = x.shape
    D = shape[-1]
    xs = _s._bf16("x", x, shape, dev)
    pad, lead = (0,) * (4 - len(shape)), (1,) * (4 - len(shape))
    zs = _s._bf16("z", z, shape, dev) if z is not None else (0,) * len(shape)
    weight_at, code, pitch = None, 0, 0
    if weight is not None:
        per_row = (shape[-2], D) if len(shape) > 1 else (D,)
        weight_at, code = _weight("weight", weight, ((D,), per_row), dev)
        pitch = D if weight.dim() > 1 else 0
    if out is None:
        out = _like(x)
        os_ = out.stride()
    else:
        os_ = _s._bf16("out", out, shape, dev)
    n, t, h, _ = lead + tuple(shape)
    xs, zs, os_ = pad + xs, pad + zs, pad + os_
    with _b.on(dev):
        rc = lib.dcconv_gated_rms_norm(
            x.data_ptr(), n, t, h, D, xs[0], xs[1], xs[2], None if z is None else z.data_ptr(), zs[0], zs[1], zs[2],
            int(bool(gate_first)), weight_at, code, pitch, weight_offset, eps, out.data_ptr(), os_[0], os_[1], os_[2],
            _b.stream(dev))
    _b.raise_for(rc)
    return out


def add_rms_norm(x, residual, weight, *, post_weight=None, gate=None, residual_scale=1.0, eps=1e-6, weight_offset=0.0,
                 out=None):
    """Adds a block's output x to ``residual`` in place and returns the norm of the sum, bf16
    of x's shape:

        y        = x, or x / rms(x) * post_weight
        residual = residual + residual_scale * y * gate
        out      = residual / rms(residual) * weight

    x: bf16 [..., D] with one to three dimensions; residual: bf16 or float32 likewise; gate:
    bf16 of x's shape (strides of 0 share a row) or None; any strides with dense last
    dimensions; weight, post_weight: bf16 or float32 (both the same) [D].  ``weight_offset``
    is added to every weight.  The sum is normed before it is rounded to a bf16 residual."""
    lib = _s._lib()
    if not 1 <= x.dim() <= 3:
        raise ValueError(f"x must have one to three dimensions, got shape {tuple(x.shape)}")
    dev = _s._gpu(x)
    shape = x.shape
    D = shape[-1]
    xs = _s._bf16("x", x, shape, dev)
    residual_at, residual_code, rs = _per_head("residual", residual, shape, dev)
    gs = _s._bf16("gate", gate, shape, dev) if gate is not None else (0,) * len(shape)
    if weight is None:
        raise ValueError("weight must be given")
    weight_at, code = _weight("weight", weight, ((D,),), dev)
    post_at = None
    if post_weight is not None:
        post_at, post_code = _weight("post_weight", post_weight, ((D,),), dev)
        if post_code != code:
            raise ValueError(f"post_weight must be {weight.dtype} as weight, got {post_weight.dtype}")
    if out is None:
        out = _like(x)
        os_ = out.stride()
    else:
        os_ = _s._bf16("out", out, shape, dev)
    pad = (0,) * (3 - len(shape))
    n, t, _ = (1,) * (3 - len(shape)) + tuple(shape)
    xs, rs, gs, os_ = pad + xs, pad + rs, pad + gs, pad + os_
    with _b.on(dev):
        rc = lib.dcconv_add_rms_norm(
            x.data_ptr(), n, t, D, xs[0], xs[1], residual_at, residual_code, rs[0], rs[1],
            None if gate is None else gate.data_ptr(), gs[0], gs[1], residual_scale, post_at, weight_at, code,
            weight_offset, eps, out.data_ptr(), os_[0], os_[1], _b.stream(dev))
    _b.raise_for(rc)
    return out
