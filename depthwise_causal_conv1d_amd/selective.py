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

_t = None  # torch, from the first call on


def _lib():
    """The loaded library, and torch in ``_t``."""
    global _t
    lib = _b.load()
    if _t is None:
        import torch

        _b.bind_torch(torch)
        _t = torch
    return lib



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


def _bf16(name, t, shape, dev):
    """``t`` as a BF16 operand of ``shape`` whose last dimension is dense; its strides."""
    if t.dtype is not _t.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if t.shape != shape or t.device != dev or t.requires_grad:
        _refuse(name, t, shape, dev)
    stride = t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return stride


def _shaped(name, t, shape, dev):
    if t.shape != shape or t.device != dev or t.requires_grad:
        _refuse(name, t, shape, dev)


def _refuse(name, t, shape, dev):
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the rest on {dev}")
    raise NotImplementedError(f"inference only: {name} requires grad (training is not served)")


def _f32_vector(name, t, n, dev):
    if t is None:
        return None
    if t.dtype is not _t.float32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 [{n}] tensor")
    _shaped(name, t, (n,), dev)
    return t.data_ptr()


def _i32_vector(name, t, n, dev):
    if t is None:
        return None
    if t.dtype is not _t.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor")
    _shaped(name, t, (n,), dev)
    return t.data_ptr()


def _dtype(name, t):
    if t.dtype is _t.bfloat16:
        return DCCONV_DTYPE_BF16
    if t.dtype is _t.float32:
        return DCCONV_DTYPE_F32
    raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _steps(dt, shape, dev):
    code = _dtype("dt", dt)
    _shaped("dt", dt, shape, dev)
    if dt.stride(-1) != 1 and dt.shape[-1] > 1:
        raise ValueError("dt must have unit stride along its heads")
    return code


def _pool(state, H, P, dev, K=None):
    """(dtype code, S, slot stride, K) of an ssm_state [S, H, P, K]."""
    code = _dtype("ssm_state", state)
    if state.dim() != 4:
        raise ValueError(f"ssm_state must be [S, H, P, K], got shape {tuple(state.shape)}")
    S, K = state.shape[0], state.shape[3] if K is None else K
    _shaped("ssm_state", state, (S, H, P, K), dev)
    if S > 0 and not state[0].is_contiguous():
        raise ValueError("ssm_state must be dense inside a slot")
    return code, S, (state.stride(0) if S > 1 else H * P * K), K


def _status(dev_status, dev):
    if dev_status is None:
        return None
    if dev_status.dtype is not _t.int32 or dev_status.device != dev or dev_status.numel() < 1:
        raise ValueError("dev_status must be an int32 tensor on the operands' device")
    return dev_status.data_ptr()


def _gpu(t):
    if t.device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {t.device}")
    return t.device


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
    code, S, slot, _ = _pool(ssm_state, H, P, dev, K)
    dt_code = _steps(dt, (N, H), dev)
    if A is None:
        raise ValueError("A must be given")
    zs = _bf16("z", z, rows, dev) if z is not None else (0, 0)
    if out is None:
        out = _t.empty(rows, dtype=_t.bfloat16, device=dev)
    os_ = _bf16("out", out, rows, dev)
    with _b.on(dev) as stream:
        rc = lib.dcconv_selective_update(
            x.data_ptr(), N, H, P, xs[0], xs[1], dt.data_ptr(), dt_code, dt.stride(0),
            _f32_vector("dt_bias", dt_bias, H, dev), int(bool(dt_softplus)), _f32_vector("A", A, H, dev),
            B.data_ptr(), C.data_ptr(), G, K, bs[0], bs[1], cs[0], cs[1], _f32_vector("D", D, H, dev),
            None if z is None else z.data_ptr(), zs[0], zs[1], ssm_state.data_ptr(), code, S, slot,
            _i32_vector("state_indices", state_indices, N, dev), out.data_ptr(), os_[0], os_[1],
            _status(dev_status, dev), stream)
    _b.raise_for(rc)
    return out


def selective_update_workspace(rows, groups, device=None):
    """The zeroed int32 [rows * groups] counters of ``causal_conv1d_selective_update``,
    which leaves them zero: one buffer serves any number of successive calls."""
    _lib()
    return _t.zeros(rows * groups, dtype=_t.int32, device="cuda" if device is None else device)


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
    code, S, slot, _ = _pool(ssm_state, H, P, dev)
    Dc = H * P + 2 * groups * K
    _bf16("xbc", xbc, (N, Dc), dev)
    if conv_state.dtype is not _t.bfloat16:
        raise ValueError(f"conv_state must be bfloat16, got {conv_state.dtype}")
    _shaped("conv_state", conv_state, (S, Dc, conv_state.shape[2]), dev)
    _bf16("weight", weight, (Dc, weight.shape[1]), dev)
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous [Dc, W]")
    if bias is not None:
        _bf16("bias", bias, (Dc,), dev)
    if activation not in _b.ACTIVATIONS:
        raise ValueError(f"activation must be None, 'identity', 'silu' or 'swish', got {activation!r}")
    dt_code = _steps(dt, (N, H), dev)
    if A is None:
        raise ValueError("A must be given")
    zs = _bf16("z", z, (N, H, P), dev) if z is not None else (0, 0)
    if workspace is None:
        workspace = selective_update_workspace(N, groups, dev)
    elif workspace.dtype is not _t.int32 or not workspace.is_contiguous() or workspace.device != dev \
            or workspace.numel() < N * groups:
        raise ValueError(f"workspace must be a contiguous int32 tensor of at least {N * groups} zeros")
    if out is None:
        out = _t.empty(N, H, P, dtype=_t.bfloat16, device=dev)
    os_ = _bf16("out", out, (N, H, P), dev)
    st = conv_state.stride()
    with _b.on(dev) as stream:
        rc = lib.dcconv_conv_selective_update(
            xbc.data_ptr(), N, H, P, groups, K, xbc.stride(0), conv_state.data_ptr(), conv_state.shape[2], st[0],
            st[1], st[2], weight.data_ptr(), weight.shape[1], None if bias is None else bias.data_ptr(),
            _i32_vector("cache_seqlens", cache_seqlens, N, dev), _b.ACTIVATIONS[activation], dt.data_ptr(), dt_code,
            dt.stride(0), _f32_vector("dt_bias", dt_bias, H, dev), int(bool(dt_softplus)),
            _f32_vector("A", A, H, dev), _f32_vector("D", D, H, dev), None if z is None else z.data_ptr(), zs[0],
            zs[1], ssm_state.data_ptr(), code, S, slot, _i32_vector("state_indices", state_indices, N, dev),
            out.data_ptr(), os_[0], os_[1], workspace.data_ptr(), _status(dev_status, dev), stream)
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
    ``dcconv_selective_scan_workspace`` bytes (allocated here if None)."""
    lib = _lib()
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError(f"x must be [N, T, H, P] and B [N, T, G, K], got {tuple(x.shape)} and {tuple(B.shape)}")
    dev = _gpu(x)
    N, T, H, P = rows = x.shape
    _, _, G, K = B.shape
    xs = _bf16("x", x, rows, dev)
    bs, cs = _bf16("B", B, (N, T, G, K), dev), _bf16("C", C, (N, T, G, K), dev)
    dt_code = _steps(dt, (N, T, H), dev)
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
    starts = _i32_vector("seq_starts", seq_starts, n + 1, dev)
    init = None
    if has_initial_state is not None:
        if has_initial_state.dtype not in (_t.bool, _t.uint8) or not has_initial_state.is_contiguous():
            raise ValueError("has_initial_state must be a contiguous bool/uint8 [n] tensor")
        _shaped("has_initial_state", has_initial_state, (n,), dev)
        init = has_initial_state.data_ptr()
    final = None
    if ssm_state is None and return_final_state:
        if has_initial_state is not None or state_indices is not None:
            raise ValueError("has_initial_state and state_indices need an ssm_state")
        ssm_state = final = _t.empty(n, H, P, K, dtype=_t.float32, device=dev)
    code, S, slot, pool = DCCONV_DTYPE_F32, 0, 0, None
    if ssm_state is not None:
        code, S, slot, _ = _pool(ssm_state, H, P, dev, K)
        pool = ssm_state.data_ptr()
    if out is None:
        out = _t.empty(rows, dtype=_t.bfloat16, device=dev)
    os_ = _bf16("out", out, rows, dev)
    need = lib.dcconv_selective_scan_workspace(n, T, H, P, G, K, int(starts is not None))
    if workspace is None:
        workspace = _t.empty(need, dtype=_t.uint8, device=dev) if need else None
    elif workspace.dtype is not _t.uint8 or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be a contiguous uint8 tensor on x's device")
    ds = dt.stride()
    with _b.on(dev) as stream:
        rc = lib.dcconv_selective_scan(
            x.data_ptr(), n, T, H, P, xs[0], xs[1], xs[2], dt.data_ptr(), dt_code, ds[0], ds[1],
            _f32_vector("dt_bias", dt_bias, H, dev), int(bool(dt_softplus)), _f32_vector("A", A, H, dev),
            B.data_ptr(), C.data_ptr(), G, K, bs[0], bs[1], bs[2], cs[0], cs[1], cs[2],
            _f32_vector("D", D, H, dev), None if z is None else z.data_ptr(), zs[0], zs[1], zs[2], starts, pool, code,
            S, slot, _i32_vector("state_indices", state_indices, n, dev), init, out.data_ptr(), os_[0], os_[1],
            os_[2], None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel(), _status(dev_status, dev), stream)
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
    q = _t.empty(-(-N // 16), -(-K // 128), 64, 16, dtype=_t.uint8, device=dev)
    with _b.on(dev) as stream:
        rc = lib.dcconv_w4_pack(codes.data_ptr(), N, K, q.data_ptr(), stream)
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
    _bf16("x", x, (M, K), dev)
    _bf16("scales", scales, (groups, N), dev)
    if not scales.is_contiguous():
        raise ValueError("scales must be contiguous")
    if qweight.dtype is not _t.uint8 or not qweight.is_contiguous():
        raise ValueError("qweight must be a contiguous uint8 tensor")
    _shaped("qweight", qweight, (-(-N // 16), -(-K // 128), 64, 16), dev)
    if zeros is not None:
        if zeros.dtype is not _t.uint8 or not zeros.is_contiguous():
            raise ValueError("zeros must be a contiguous uint8 tensor")
        _shaped("zeros", zeros, (groups, N), dev)
    if bias is not None:
        _bf16("bias", bias, (N,), dev)
    if out is None:
        out = _t.empty(M, N, dtype=_t.bfloat16, device=dev)
    else:
        _bf16("out", out, (M, N), dev)
    with _b.on(dev) as stream:
        rc = lib.dcconv_w4_matvec(
            x.data_ptr(), M, K, x.stride(0), qweight.data_ptr(), N, scales.data_ptr(),
            None if zeros is None else zeros.data_ptr(), group_size, None if bias is None else bias.data_ptr(),
            out.data_ptr(), out.stride(0) if M > 1 else N, stream)
    _b.raise_for(rc)
    return out
