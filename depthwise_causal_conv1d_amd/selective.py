"""The state-space recurrence behind the convolution: Python binding.

``selective_scan`` runs whole prompts, ``selective_update`` one token a row, and
``causal_conv1d_selective_update`` one token through the short convolution and the
recurrence in one launch; ``w4_matvec`` multiplies a few rows with 4-bit weights, as a
decoding layer's projections.  Per head, with d = softplus(dt + dt_bias) and the head's
group holding B and C::

    state = exp(d * A) * state + d * x B^T
    out   = (state C + D x) * silu(z)

The ``dcconv_*`` functions mirror the C entry points of ``include/dcconv.h`` one to
one; the tensor functions check shapes and types, pass strides and the current
stream, and allocate the output (and, for prompts, the workspace).
"""
from __future__ import annotations

import ctypes

from . import _binding as _b

__all__ = [
    "DCCONV_DTYPE_BF16", "DCCONV_DTYPE_F32",
    "dcconv_selective_update", "dcconv_conv_selective_update", "dcconv_selective_scan",
    "dcconv_selective_scan_workspace", "selective_scan", "selective_update",
    "causal_conv1d_selective_update", "selective_update_workspace",
    "dcconv_w4_matvec", "dcconv_w4_pack", "w4_matvec", "w4_pack",
]

DCCONV_DTYPE_BF16, DCCONV_DTYPE_F32 = 0, 1

_t = _BF16 = _F32 = _I32 = None  # torch and three of its types, from the first call on


def _lib():
    """The loaded library, and torch in ``_t``."""
    if _t is None:
        _import_torch()
    return _b.load()


def _import_torch():
    global _t, _BF16, _F32, _I32
    import torch

    _b.bind_torch(torch)
    _BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
    _t = torch  # last: another thread's first call goes by it


def declare(lib: ctypes.CDLL) -> None:
    """The argument types of this module's C entry points."""
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.dcconv_selective_update.restype = i32
    lib.dcconv_selective_update.argtypes = (
        [vp, i64, i64, i64, i64, i64]                 # x, n, h, p, xs_n, xs_h
        + [vp, i32, i64, vp, i32]                     # dt, dt_dtype, ds_n, dt_bias, dt_softplus
        + [vp, vp, vp, i64, i64]                      # a, b, c, g, k
        + [i64] * 4                                   # bs_n, bs_g, cs_n, cs_g
        + [vp, vp, i64, i64]                          # d_skip, z, zs_n, zs_h
        + [vp, i32, i64, i64, vp]                     # ssm_state, state_dtype, s, ss_s, state_indices
        + [vp, i64, i64, vp, vp])                     # out, os_n, os_h, dev_status, stream
    lib.dcconv_conv_selective_update.restype = i32
    lib.dcconv_conv_selective_update.argtypes = (
        [vp, i64, i64, i64, i64, i64, i64]            # xbc, n, h, p, g, k, xbcs_n
        + [vp, i64, i64, i64, i64]                    # conv_state, l, st_s, st_d, st_l
        + [vp, i64, vp, vp, i32]                      # weight, w, bias, cache_seqlens, activation
        + [vp, i32, i64, vp, i32]                     # dt, dt_dtype, ds_n, dt_bias, dt_softplus
        + [vp, vp, vp, i64, i64]                      # a, d_skip, z, zs_n, zs_h
        + [vp, i32, i64, i64, vp]                     # ssm_state, state_dtype, s, ss_s, state_indices
        + [vp, i64, i64, vp, vp, vp])                 # out, os_n, os_h, workspace, dev_status, stream
    lib.dcconv_selective_scan.restype = i32
    lib.dcconv_selective_scan.argtypes = (
        [vp, i64, i64, i64, i64, i64, i64, i64]       # x, n, t, h, p, xs_n, xs_t, xs_h
        + [vp, i32, i64, i64, vp, i32]                # dt, dt_dtype, ds_n, ds_t, dt_bias, dt_softplus
        + [vp, vp, vp, i64, i64]                      # a, b, c, g, k
        + [i64] * 6                                   # bs_n, bs_t, bs_g, cs_n, cs_t, cs_g
        + [vp, vp, i64, i64, i64]                     # d_skip, z, zs_n, zs_t, zs_h
        + [vp, vp, i32, i64, i64, vp, vp]             # seq_starts, ssm_state, dtype, s, ss_s, indices, has_init
        + [vp, i64, i64, i64, vp, i64, vp, vp])       # out, os_n, os_t, os_h, workspace, bytes, status, stream
    lib.dcconv_selective_scan_workspace.restype = i64
    lib.dcconv_selective_scan_workspace.argtypes = [i64] * 6 + [i32]
    lib.dcconv_w4_matvec.restype = i32
    lib.dcconv_w4_matvec.argtypes = [vp, i64, i64, i64, vp, i64,       # x, m, k, xs_m, qweight, n
                                     vp, vp, i64, vp, vp, i64, vp]     # scales, zeros, group, bias, out, os_m, stream
    lib.dcconv_w4_pack.restype = i32
    lib.dcconv_w4_pack.argtypes = [vp, i64, i64, vp, vp]               # codes, n, k, qweight, stream


# ----------------------------------------------------------------- raw C ABI


def dcconv_selective_update(*args) -> int:
    """The one-token C entry point, one to one (pointers as ints, 0/None = NULL)."""
    return _b.load().dcconv_selective_update(*args)


def dcconv_conv_selective_update(*args) -> int:
    """The fused one-token C entry point, one to one (pointers as ints)."""
    return _b.load().dcconv_conv_selective_update(*args)


def dcconv_selective_scan(*args) -> int:
    """The whole-sequence C entry point, one to one (pointers as ints)."""
    return _b.load().dcconv_selective_scan(*args)


def dcconv_selective_scan_workspace(n, t, h, p, g, k, packed) -> int:
    """Bytes of workspace a scan of these sizes needs, one to one."""
    return _b.load().dcconv_selective_scan_workspace(n, t, h, p, g, k, packed)


def dcconv_w4_matvec(*args) -> int:
    """The 4-bit matrix-vector C entry point, one to one (pointers as ints)."""
    return _b.load().dcconv_w4_matvec(*args)


def dcconv_w4_pack(*args) -> int:
    """The packing C entry point, one to one (pointers as ints)."""
    return _b.load().dcconv_w4_pack(*args)


# ------------------------------------------------------------ tensor front end


# A call's checks cost more than its launch if written carelessly: each of these reads an
# attribute once, compares the device by its index, and leaves the wording to _refuse.


def _bf16(name, t, shape, dev):
    """``t`` as a BF16 operand of ``shape`` whose last dimension is dense; its strides."""
    if t.dtype is not _BF16 or t.shape != shape or t.get_device() != dev or t.requires_grad:
        _refuse(name, t, _BF16, shape, dev)
    stride = t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return stride


def _vector(name, t, kind, n, dev):
    """The address of a contiguous [n] operand, None for None."""
    if t is None:
        return None
    if t.dtype is not kind or t.shape != (n,) or t.get_device() != dev or t.requires_grad or not t.is_contiguous():
        _refuse(name, t, kind, (n,), dev)
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _refuse(name, t, kind, shape, dev):
    if kind is not None and t.dtype is not kind:
        raise ValueError(f"{name} must be {str(kind)[6:]}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the rest on GPU {dev}")
    if t.requires_grad:
        raise NotImplementedError(f"inference only: {name} requires grad (training is not served)")


def _dtype(name, t):
    kind = t.dtype
    if kind is _BF16:
        return DCCONV_DTYPE_BF16
    if kind is _F32:
        return DCCONV_DTYPE_F32
    raise ValueError(f"{name} must be bfloat16 or float32, got {kind}")


def _steps(dt, shape, dev):
    """(dtype code, strides) of dt."""
    code = _dtype("dt", dt)
    if dt.shape != shape or dt.get_device() != dev or dt.requires_grad:
        _refuse("dt", dt, None, shape, dev)
    stride = dt.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError("dt must have unit stride along its heads")
    return code, stride


def _pool(state, H, P, K, dev):
    """(dtype code, S, slot stride) of an ssm_state [S, H, P, K]."""
    code = _dtype("ssm_state", state)
    shape = state.shape
    if shape[1:] != (H, P, K) or state.get_device() != dev or state.requires_grad:
        _refuse("ssm_state", state, None, (shape[0], H, P, K), dev)
    S, stride = shape[0], state.stride()
    if stride[1:] != (P * K, K, 1) and S > 0 and not state[0].is_contiguous():
        raise ValueError("ssm_state must be dense inside a slot")
    return code, S, (stride[0] if S > 1 else H * P * K)


def _status(dev_status, dev):
    if dev_status is None:
        return None
    if dev_status.dtype is not _I32 or dev_status.get_device() != dev or dev_status.numel() < 1:
        raise ValueError("dev_status must be an int32 tensor on the operands' device")
    return dev_status.data_ptr()


def _gpu(t):
    """The index of the GPU that holds ``t``."""
    if not t.is_cuda:
        raise ValueError(f"tensors must be on a GPU, got {t.device}")
    return t.get_device()


def selective_update(x, dt, A, B, C, ssm_state, *, D=None, z=None, dt_bias=None, dt_softplus=False,
                     state_indices=None, out=None, dev_status=None):
    """One token of N rows: ``ssm_state`` is updated in place and the output [N, H, P]
    returned.

    x, z: bf16 [N, H, P]; B, C: bf16 [N, G, K] (H a multiple of G); dt: bf16 or float32
    [N, H]; A, D, dt_bias: float32 [H]; ssm_state: bf16 or float32 [S, H, P, K].  Any
    strides with dense last dimensions.  ``state_indices`` (int32 [N]) routes rows to
    slots, -1 being a padding row (zero output, no state moves)."""
    lib = _lib()
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError(f"x must be [N, H, P] and B [N, G, K], got {tuple(x.shape)} and {tuple(B.shape)}")
    dev = _gpu(x)
    N, H, P = rows = x.shape
    _, G, K = B.shape
    xs = _bf16("x", x, rows, dev)
    bs, cs = _bf16("B", B, (N, G, K), dev), _bf16("C", C, (N, G, K), dev)
    if ssm_state.dim() != 4:
        raise ValueError(f"ssm_state must be [S, H, P, K], got shape {tuple(ssm_state.shape)}")
    code, S, slot = _pool(ssm_state, H, P, K, dev)
    dt_code, ds = _steps(dt, (N, H), dev)
    if A is None:
        raise ValueError("A must be given")
    zs = _bf16("z", z, rows, dev) if z is not None else (0, 0)
    if out is None:
        out, os_ = _t.empty(rows, dtype=_BF16, device=x.device), (H * P, P)
    else:
        os_ = _bf16("out", out, rows, dev)
    with _b.on(dev):
        rc = lib.dcconv_selective_update(
            x.data_ptr(), N, H, P, xs[0], xs[1], dt.data_ptr(), dt_code, ds[0],
            _vector("dt_bias", dt_bias, _F32, H, dev), int(bool(dt_softplus)), _vector("A", A, _F32, H, dev),
            B.data_ptr(), C.data_ptr(), G, K, bs[0], bs[1], cs[0], cs[1], _vector("D", D, _F32, H, dev),
            None if z is None else z.data_ptr(), zs[0], zs[1], ssm_state.data_ptr(), code, S, slot,
            _vector("state_indices", state_indices, _I32, N, dev), out.data_ptr(), os_[0], os_[1],
            _status(dev_status, dev), _b.stream(dev))
    _b.raise_for(rc)
    return out


def selective_update_workspace(rows, groups, device=None):
    """The zeroed int32 [rows * groups] counters of ``causal_conv1d_selective_update``,
    which leaves them zero: one buffer serves any number of successive calls."""
    _lib()
    return _t.zeros(rows * groups, dtype=_I32, device="cuda" if device is None else device)


def causal_conv1d_selective_update(xbc, conv_state, weight, bias, activation, dt, A, ssm_state, *, groups,
                                   D=None, z=None, dt_bias=None, dt_softplus=False, state_indices=None,
                                   cache_seqlens=None, workspace=None, out=None, dev_status=None):
    """One token of N rows through the causal convolution and the recurrence, both
    states updated in place; returns the output [N, H, P].

    xbc: bf16 [N, Dc], the channels of x, B and C one after the other (Dc = H*P +
    2*groups*K); conv_state: bf16 [S, Dc, L]; weight: bf16 [Dc, 4], bias: bf16 [Dc] or
    None; activation and cache_seqlens as for ``causal_conv1d_update``.  The convolved
    channels are not rounded before the recurrence reads them.  ``workspace`` comes
    from ``selective_update_workspace`` (allocated and zeroed here if None).  The rest
    as for ``selective_update``."""
    lib = _lib()
    if xbc.dim() != 2 or ssm_state.dim() != 4 or conv_state.dim() != 3 or weight.dim() != 2:
        raise ValueError(f"xbc must be [N, Dc], conv_state [S, Dc, L], weight [Dc, W] and ssm_state [S, H, P, K], got "
                         f"{tuple(xbc.shape)}, {tuple(conv_state.shape)}, {tuple(weight.shape)}, "
                         f"{tuple(ssm_state.shape)}")
    dev = _gpu(xbc)
    N = xbc.shape[0]
    _, H, P, K = ssm_state.shape
    code, S, slot = _pool(ssm_state, H, P, K, dev)
    Dc = H * P + 2 * groups * K
    xs = _bf16("xbc", xbc, (N, Dc), dev)
    L, W = conv_state.shape[2], weight.shape[1]
    if conv_state.dtype is not _BF16 or conv_state.shape != (S, Dc, L) or conv_state.get_device() != dev \
            or conv_state.requires_grad:
        _refuse("conv_state", conv_state, _BF16, (S, Dc, L), dev)
    if _bf16("weight", weight, (Dc, W), dev)[0] != W and Dc > 1:
        raise ValueError("weight must be contiguous [Dc, W]")
    if bias is not None:
        _bf16("bias", bias, (Dc,), dev)
    if activation not in _b.ACTIVATIONS:
        raise ValueError(f"activation must be None, 'identity', 'silu' or 'swish', got {activation!r}")
    dt_code, ds = _steps(dt, (N, H), dev)
    if A is None:
        raise ValueError("A must be given")
    zs = _bf16("z", z, (N, H, P), dev) if z is not None else (0, 0)
    if workspace is None:
        workspace = selective_update_workspace(N, groups, xbc.device)
    elif workspace.dtype is not _I32 or not workspace.is_contiguous() or workspace.get_device() != dev \
            or workspace.numel() < N * groups:
        raise ValueError(f"workspace must be a contiguous int32 tensor of at least {N * groups} zeros")
    if out is None:
        out, os_ = _t.empty(N, H, P, dtype=_BF16, device=xbc.device), (H * P, P)
    else:
        os_ = _bf16("out", out, (N, H, P), dev)
    st = conv_state.stride()
    with _b.on(dev):
        rc = lib.dcconv_conv_selective_update(
            xbc.data_ptr(), N, H, P, groups, K, xs[0], conv_state.data_ptr(), L, st[0],
            st[1], st[2], weight.data_ptr(), W, None if bias is None else bias.data_ptr(),
            _vector("cache_seqlens", cache_seqlens, _I32, N, dev), _b.ACTIVATIONS[activation], dt.data_ptr(), dt_code,
            ds[0], _vector("dt_bias", dt_bias, _F32, H, dev), int(bool(dt_softplus)),
            _vector("A", A, _F32, H, dev), _vector("D", D, _F32, H, dev), None if z is None else z.data_ptr(), zs[0],
            zs[1], ssm_state.data_ptr(), code, S, slot, _vector("state_indices", state_indices, _I32, N, dev),
            out.data_ptr(), os_[0], os_[1], workspace.data_ptr(), _status(dev_status, dev), _b.stream(dev))
    _b.raise_for(rc)
    return out


def selective_scan(x, dt, A, B, C, *, D=None, z=None, dt_bias=None, dt_softplus=False, ssm_state=None,
                   state_indices=None, has_initial_state=None, seq_starts=None, return_final_state=False,
                   workspace=None, out=None, dev_status=None):
    """The recurrence over whole sequences; returns the output [N, T, H, P].

    x, z: bf16 [N, T, H, P]; dt: bf16 or float32 [N, T, H]; B, C: bf16 [N, T, G, K];
    A, D, dt_bias: float32 [H].  With ``seq_starts`` (int32 [n+1] on the device) N is 1
    and the T axis holds n packed sequences.
    ssm_state: bf16 or float32 [S, H, P, K] pool; sequences that ``has_initial_state``
    (bool/uint8 [n]) marks start from their slot's state, and every sequence leaves its
    final state there; ``state_indices`` (int32 [n]) routes sequences to slots, -1 being
    padding.  return_final_state: without ``ssm_state``, returns ``(out, state)`` with
    a new float32 [n, H, P, K] state.  ``workspace``: a uint8 buffer of
    ``dcconv_selective_scan_workspace`` bytes (allocated here if None).

    Sums and states are 32 bits; operands of the matrix products are rounded to bf16 (the
    copy of the state that C reads, the products of C and B, and, unless ``ssm_state`` is
    float32 or a final state is returned, the scaled x that enters the state)."""
    lib = _lib()
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError(f"x must be [N, T, H, P] and B [N, T, G, K], got {tuple(x.shape)} and {tuple(B.shape)}")
    dev = _gpu(x)
    N, T, H, P = rows = x.shape
    _, _, G, K = B.shape
    xs = _bf16("x", x, rows, dev)
    bs, cs = _bf16("B", B, (N, T, G, K), dev), _bf16("C", C, (N, T, G, K), dev)
    dt_code, ds = _steps(dt, (N, T, H), dev)
    if A is None:
        raise ValueError("A must be given")
    zs = _bf16("z", z, rows, dev) if z is not None else (0, 0, 0)
    n = N
    if seq_starts is not None:
        if N != 1:
            raise ValueError("with seq_starts, x must be [1, total_T, H, P] (packed sequences)")
        if seq_starts.dim() != 1 or seq_starts.shape[0] < 1:
            raise ValueError("seq_starts must be a contiguous int32 [n+1] tensor")
        n = seq_starts.shape[0] - 1
    starts = _vector("seq_starts", seq_starts, _I32, n + 1, dev)
    init = None
    if has_initial_state is not None:
        if has_initial_state.dtype not in (_t.bool, _t.uint8):
            raise ValueError("has_initial_state must be a contiguous bool/uint8 [n] tensor")
        init = _vector("has_initial_state", has_initial_state, has_initial_state.dtype, n, dev)
    final = None
    if ssm_state is None and (has_initial_state is not None or state_indices is not None):
        raise ValueError("has_initial_state and state_indices need an ssm_state")
    if ssm_state is None and return_final_state:
        ssm_state = final = _t.empty(n, H, P, K, dtype=_F32, device=x.device)
    code, S, slot, pool = DCCONV_DTYPE_F32, 0, 0, None
    if ssm_state is not None:
        if ssm_state.dim() != 4:
            raise ValueError(f"ssm_state must be [S, H, P, K], got shape {tuple(ssm_state.shape)}")
        code, S, slot = _pool(ssm_state, H, P, K, dev)
        pool = ssm_state.data_ptr()
    if out is None:
        out, os_ = _t.empty(rows, dtype=_BF16, device=x.device), (T * H * P, H * P, P)
    else:
        os_ = _bf16("out", out, rows, dev)
    need = lib.dcconv_selective_scan_workspace(n, T, H, P, G, K, int(starts is not None))
    if workspace is None:
        workspace = _t.empty(need, dtype=_t.uint8, device=x.device) if need else None
    elif workspace.dtype is not _t.uint8 or not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be a contiguous uint8 tensor on x's device")
    with _b.on(dev):
        rc = lib.dcconv_selective_scan(
            x.data_ptr(), n, T, H, P, xs[0], xs[1], xs[2], dt.data_ptr(), dt_code, ds[0], ds[1],
            _vector("dt_bias", dt_bias, _F32, H, dev), int(bool(dt_softplus)), _vector("A", A, _F32, H, dev),
            B.data_ptr(), C.data_ptr(), G, K, bs[0], bs[1], bs[2], cs[0], cs[1], cs[2],
            _vector("D", D, _F32, H, dev), None if z is None else z.data_ptr(), zs[0], zs[1], zs[2], starts, pool, code,
            S, slot, _vector("state_indices", state_indices, _I32, n, dev), init, out.data_ptr(), os_[0], os_[1],
            os_[2], None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel(), _status(dev_status, dev), _b.stream(dev))
    _b.raise_for(rc)
    return (out, final) if final is not None else out


def w4_pack(codes):
    """Lay out the codes (uint8 [N, K], values 0 to 15) of a 4-bit weight matrix for
    ``w4_matvec``: uint8 [ceil(N/16), ceil(K/128), 64, 16]."""
    lib = _lib()
    if codes.dim() != 2 or codes.dtype is not _t.uint8 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous uint8 [N, K] tensor")
    dev = _gpu(codes)
    N, K = codes.shape
    q = _t.empty(-(-N // 16), -(-K // 128), 64, 16, dtype=_t.uint8, device=codes.device)
    with _b.on(dev):
        rc = lib.dcconv_w4_pack(codes.data_ptr(), N, K, q.data_ptr(), _b.stream(dev))
    _b.raise_for(rc)
    return q


def w4_matvec(x, qweight, scales, zeros=None, bias=None, *, group_size, out=None):
    """x [M, K] (bf16) times a 4-bit weight matrix: out [M, N], with
    out[m, n] = sum_k x[m, k] * (code[n, k] - zeros[k // group_size, n]) * scales[k // group_size, n] + bias[n].

    qweight: ``w4_pack``'s tiles; scales: bf16 [ceil(K / group_size), N]; zeros: uint8 of
    that shape or None (8); bias: bf16 [N] or None; group_size: a multiple of 32."""
    lib = _lib()
    if x.dim() != 2 or scales.dim() != 2:
        raise ValueError(f"x must be [M, K] and scales [groups, N], got {tuple(x.shape)} and {tuple(scales.shape)}")
    dev = _gpu(x)
    M, K = x.shape
    N = scales.shape[1]
    groups = -(-K // group_size) if group_size > 0 else 0
    xs = _bf16("x", x, (M, K), dev)
    if _bf16("scales", scales, (groups, N), dev)[0] != N and groups > 1:
        raise ValueError("scales must be contiguous")
    shape = (-(-N // 16), -(-K // 128), 64, 16)
    if qweight.dtype is not _t.uint8 or qweight.shape != shape or qweight.get_device() != dev:
        _refuse("qweight", qweight, _t.uint8, shape, dev)
    if not qweight.is_contiguous():
        raise ValueError("qweight must be contiguous")
    if zeros is not None:
        if zeros.dtype is not _t.uint8 or zeros.shape != (groups, N) or zeros.get_device() != dev:
            _refuse("zeros", zeros, _t.uint8, (groups, N), dev)
        if not zeros.is_contiguous():
            raise ValueError("zeros must be contiguous")
    if bias is not None:
        _bf16("bias", bias, (N,), dev)
    if out is None:
        out, pitch = _t.empty(M, N, dtype=_BF16, device=x.device), N
    else:
        pitch = _bf16("out", out, (M, N), dev)[0]
        if M <= 1:
            pitch = N
    with _b.on(dev):
        rc = lib.dcconv_w4_matvec(
            x.data_ptr(), M, K, xs[0], qweight.data_ptr(), N, scales.data_ptr(),
            None if zeros is None else zeros.data_ptr(), group_size, None if bias is None else bias.data_ptr(),
            out.data_ptr(), pitch, _b.stream(dev))
    _b.raise_for(rc)
    return out
