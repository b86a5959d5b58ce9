"""Norm of every query and key head with the position rotation in the same pass, and its gradient.

    q, k = qk_norm_rope_forward(q, k, q_gain, k_gain, cos, sin, positions=positions)
    O, LSE = attention_forward(q, k, v, is_causal=True)

Tensors are [B, H, N, D] views with any strides (the head dim contiguous), so
the heads of one packed projection [B, N, heads, D] are passed as they lie
(``packed[:, :, :Hq].transpose(1, 2)``); outputs are contiguous [B, H, N, D],
the layout attention_forward takes, unless the caller passes views.
"""
from __future__ import annotations

import ctypes
import struct

from .binding import Fa2Error  # noqa: F401  (what these calls raise)
from .binding import _check, _dtype_code_of, library
from .streams import device_guard, empty_on, scratch_for, stream_handle

# the strides a call passes, as the C side reads them (bytes are passed by address)
_FWD_STRIDES = struct.Struct("=14q").pack
_BWD_STRIDES = struct.Struct("=20q").pack
_NO_VIEW = (0, 0, 0)
_bwd_bytes = {}


def fa2_qk_norm_rope_bwd_workspace_bytes(D: int) -> int:
    n = ctypes.c_size_t(0)
    _check(library().fa2_qk_norm_rope_bwd_workspace_bytes(int(D), ctypes.byref(n)),
           "fa2_qk_norm_rope_bwd_workspace_bytes")
    return n.value


def _check_view(name, t, B, H, N, D, dt, dev):
    """(batch, head, token) strides of a [B, H, N, D] view, which has the dtype and device of the call."""
    if t.shape != (B, H, N, D):
        raise ValueError(f"{name} must have the shape {[B, H, N, D]}")
    if t.dtype != dt or t.get_device() != dev:
        raise ValueError(f"{name} must have the dtype and device of q and k")
    sb, sh, sn, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return sb, sh, sn


def _check_sides(q, k):
    """(like, Hq, Hkv, B, N, D, dtype, device index, q's strides, k's strides); `like` is the present one of q and k."""
    like = q if q is not None else k
    if like is None:
        raise ValueError("at least one of q and k is needed")
    dev = like.get_device()
    if like.dim() != 4 or dev < 0:
        raise ValueError("q and k must be CUDA tensors [B, H, N, D]")
    B, Hq, N, D = like.shape
    dt = like.dtype
    Hkv = 0
    qs = ks = _NO_VIEW
    if q is not None:
        qs = _check_view("q", q, B, Hq, N, D, dt, dev)
    else:
        Hq = 0
    if k is not None:
        if k.dim() != 4:
            raise ValueError("q and k must be CUDA tensors [B, H, N, D]")
        Hkv = k.shape[1]
        ks = _check_view("k", k, B, Hkv, N, D, dt, dev)
    return like, Hq, Hkv, B, N, D, dt, dev, qs, ks


def _check_gains(q_gain, k_gain, D, dt, dev):
    """Nonzero when the gains are float32. Both have one dtype: float32 or that of q and k."""
    import torch
    kind = None
    for w in (q_gain, k_gain):
        if w is None:
            continue
        wt = w.dtype
        if w.shape != (D,) or not w.is_contiguous() or w.get_device() != dev:
            raise ValueError(f"a gain must be a contiguous [{D}] tensor on the device of q and k")
        if wt != torch.float32 and wt != dt:
            raise ValueError("a gain must be float32 or of the dtype of q and k")
        if kind is not None and wt != kind:
            raise ValueError("q_gain and k_gain must share one dtype")
        kind = wt
    return 1 if kind == torch.float32 else 0


def _check_tables(cos, sin, positions, B, N, dev):
    """(rot, table rows, positions are int64, strides of positions)."""
    import torch
    if cos is None or sin is None:
        if cos is not sin:
            raise ValueError("cos and sin must be given together")
        if positions is not None:
            raise ValueError("positions need cos and sin")
        return 0, 0, 0, 0, 0
    shape = cos.shape
    if len(shape) != 2 or sin.shape != shape:
        raise ValueError("cos and sin must share one shape [rows, rot / 2]")
    f32 = torch.float32
    if cos.dtype != f32 or sin.dtype != f32 or not cos.is_contiguous() or not sin.is_contiguous() or \
            cos.get_device() != dev or sin.get_device() != dev:
        raise ValueError("cos and sin must be contiguous float32 tensors on the device of q and k")
    rows, half = shape
    if positions is None:
        if rows < N:
            raise ValueError(f"the tables have {rows} rows; without positions {N} are needed")
        return 2 * half, rows, 0, 0, 0
    pt = positions.dtype
    if (pt != torch.int64 and pt != torch.int32) or positions.get_device() != dev:
        raise ValueError("positions must be int32 or int64 on the device of q and k")
    if positions.shape == (B, N):
        pb, pn = positions.stride()
    elif positions.shape == (N,):
        pb, pn = 0, positions.stride(0)
    else:
        raise ValueError(f"positions must be [{B}, {N}] or [{N}]")
    return 2 * half, rows, 1 if pt == torch.int64 else 0, pb, pn


def qk_norm_rope_forward(q, k, q_gain=None, k_gain=None, cos=None, sin=None, positions=None, eps: float = 1e-6,
                         interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of each head of q and k, times its gain, then the position rotation; returns (q', k').

    q, k: CUDA tensors [B, Hq, N, D] and [B, Hkv, N, D] (fp16/bf16) with any
    strides whose last dimension is contiguous; one of them may be None (and
    its result is None): a decoder that cached its normed keys passes only q.
    q_gain, k_gain: [D], float32 or q's dtype, or None for ones.
    cos, sin: float32 tables [rows, rot / 2]; rot, a multiple of 16 up to D, is
    how many leading elements of a head are rotated (None: no rotation).
    positions: the tables' row for each token, int32/int64 [B, N] or [N]
    (default 0 .. N-1). A position outside the tables gives NaN in the
    rotated elements of its rows.
    interleaved: rotated pairs are (2i, 2i+1) instead of (i, i + rot/2).
    q_out, k_out: views to write to (a cache slot, say); each may be exactly
    its own input. Contiguous tensors are allocated otherwise.
    Runs on `stream` (a torch.cuda.Stream) or the current stream.
    """
    like, Hq, Hkv, B, N, D, dt, dev, qs, ks = _check_sides(q, k)
    gain_f32 = _check_gains(q_gain, k_gain, D, dt, dev)
    rot, rows, p64, pb, pn = _check_tables(cos, sin, positions, B, N, dev)
    dtc = _dtype_code_of(dt)
    handle = stream_handle(dev, stream, (q, k, q_gain, k_gain, cos, sin, positions, q_out, k_out))
    qos = kos = _NO_VIEW
    if q is None:
        if q_out is not None:
            raise ValueError("q_out was given without q")
    elif q_out is None:
        q_out = empty_on(stream, (B, Hq, N, D), dt, like.device)
        qos = (Hq * N * D, N * D, D)
    else:
        qos = _check_view("q_out", q_out, B, Hq, N, D, dt, dev)
    if k is None:
        if k_out is not None:
            raise ValueError("k_out was given without k")
    elif k_out is None:
        k_out = empty_on(stream, (B, Hkv, N, D), dt, like.device)
        kos = (Hkv * N * D, N * D, D)
    else:
        kos = _check_view("k_out", k_out, B, Hkv, N, D, dt, dev)
    strides = _FWD_STRIDES(*qs, *ks, *qos, *kos, pb, pn)
    with device_guard(dev):
        code = library().fa2_qk_norm_rope_fwd(
            q.data_ptr() if q is not None else None, k.data_ptr() if k is not None else None,
            q_gain.data_ptr() if q_gain is not None else None, k_gain.data_ptr() if k_gain is not None else None,
            cos.data_ptr() if rot else None, sin.data_ptr() if rot else None,
            positions.data_ptr() if positions is not None else None, q_out.data_ptr() if q is not None else None,
            k_out.data_ptr() if k is not None else None, strides, B, Hq, Hkv, N, D, rot, rows, eps,
            1 if interleaved else 0, gain_f32, p64, dtc, handle)
    if code:
        _check(code, "fa2_qk_norm_rope_fwd")
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_gain=None, k_gain=None, cos=None, sin=None, positions=None,
                          eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, workspace=None,
                          stream=None):
    """Gradient of qk_norm_rope_forward for upstream gradients dq_out, dk_out of its results.

    q, k and the arguments after them are the forward's. Returns (dq, dk,
    dq_gain, dk_gain): dq, dk like q, k (None where the input is), the gains'
    gradients [D] in the gains' dtype (None without a gain).
    dq, dk: views to write to, for instance the parts of a packed projection's
    gradient; each may be exactly its upstream gradient or its input.
    workspace: optional uint8 CUDA tensor of at least
    fa2_qk_norm_rope_bwd_workspace_bytes(D) bytes (by default one is kept for
    each device, head dim, current stream and host thread; a captured call, and
    one that names its stream, gets its own).
    """
    like, Hq, Hkv, B, N, D, dt, dev, qs, ks = _check_sides(q, k)
    gain_f32 = _check_gains(q_gain, k_gain, D, dt, dev)
    rot, rows, p64, pb, pn = _check_tables(cos, sin, positions, B, N, dev)
    dtc = _dtype_code_of(dt)
    handle = stream_handle(dev, stream, (dq_out, dk_out, q, k, q_gain, k_gain, cos, sin, positions, dq, dk, workspace))
    device = like.device
    gqs = gks = dqs = dks = _NO_VIEW
    dq_gain = dk_gain = None
    if q is None:
        if dq_out is not None or dq is not None or q_gain is not None:
            raise ValueError("dq_out, dq and q_gain need q")
    else:
        if dq_out is None:
            raise ValueError("dq_out is needed with q")
        gqs = _check_view("dq_out", dq_out, B, Hq, N, D, dt, dev)
        if dq is None:
            dq = empty_on(stream, (B, Hq, N, D), dt, device)
        dqs = _check_view("dq", dq, B, Hq, N, D, dt, dev)
        if q_gain is not None:
            dq_gain = empty_on(stream, (D,), q_gain.dtype, device)
    if k is None:
        if dk_out is not None or dk is not None or k_gain is not None:
            raise ValueError("dk_out, dk and k_gain need k")
    else:
        if dk_out is None:
            raise ValueError("dk_out is needed with k")
        gks = _check_view("dk_out", dk_out, B, Hkv, N, D, dt, dev)
        if dk is None:
            dk = empty_on(stream, (B, Hkv, N, D), dt, device)
        dks = _check_view("dk", dk, B, Hkv, N, D, dt, dev)
        if k_gain is not None:
            dk_gain = empty_on(stream, (D,), k_gain.dtype, device)
    need = 0
    if q_gain is not None or k_gain is not None:
        need = _bwd_bytes.get(D)
        if need is None:
            need = _bwd_bytes[D] = fa2_qk_norm_rope_bwd_workspace_bytes(D)
        if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous() or
                                      workspace.nbytes < need):
            raise ValueError(f"workspace must be a contiguous CUDA tensor of at least {need} bytes on q's device")
    strides = _BWD_STRIDES(*gqs, *gks, *qs, *ks, *dqs, *dks, pb, pn)
    has_q, has_k = q is not None, k is not None
    with device_guard(dev):
        if need and workspace is None:
            workspace = scratch_for("norm_rope_bwd", need, device, dev, handle, stream)
        code = library().fa2_qk_norm_rope_bwd(
            dq_out.data_ptr() if has_q else None, dk_out.data_ptr() if has_k else None,
            q.data_ptr() if has_q else None, k.data_ptr() if has_k else None,
            q_gain.data_ptr() if q_gain is not None else None, k_gain.data_ptr() if k_gain is not None else None,
            cos.data_ptr() if rot else None, sin.data_ptr() if rot else None,
            positions.data_ptr() if positions is not None else None, dq.data_ptr() if has_q else None,
            dk.data_ptr() if has_k else None, dq_gain.data_ptr() if q_gain is not None else None,
            dk_gain.data_ptr() if k_gain is not None else None, strides, B, Hq, Hkv, N, D, rot, rows, eps,
            1 if interleaved else 0, gain_f32, p64, dtc, workspace.data_ptr() if need else None,
            workspace.nbytes if need else 0, handle)
    if code:
        _check(code, "fa2_qk_norm_rope_bwd")
    return dq, dk, dq_gain, dk_gain
