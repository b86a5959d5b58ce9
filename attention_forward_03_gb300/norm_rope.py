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

from .binding import Fa2Error  # noqa: F401  (what these calls raise)
from .binding import _check, _dtype_code_of, library
from .streams import empty_on, launch_stream

_F_ARGS = ctypes.c_longlong * 14
_B_ARGS = ctypes.c_longlong * 20


def fa2_qk_norm_rope_bwd_workspace_bytes(D: int) -> int:
    n = ctypes.c_size_t(0)
    _check(library().fa2_qk_norm_rope_bwd_workspace_bytes(int(D), ctypes.byref(n)),
           "fa2_qk_norm_rope_bwd_workspace_bytes")
    return n.value


def _strides(t):
    """(batch, head, token) strides of a view, for the C call."""
    if t is None:
        return 0, 0, 0
    s = t.stride()
    return s[0], s[1], s[2]


def _check_view(name, t, like, shape):
    if t.dim() != 4 or t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    if t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must have the dtype and device of q and k")
    if t.stride(3) != 1 and shape[3] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _check_sides(q, k):
    """The present one of q and k (for device, dtype and sizes), the head counts, and B, N, D."""
    like = q if q is not None else k
    if like is None:
        raise ValueError("at least one of q and k is needed")
    if like.dim() != 4 or not like.is_cuda:
        raise ValueError("q and k must be CUDA tensors [B, H, N, D]")
    B, _, N, D = like.shape
    heads = []
    for name, t in (("q", q), ("k", k)):
        if t is None:
            heads.append(0)
            continue
        if t.dim() != 4:
            raise ValueError("q and k must be CUDA tensors [B, H, N, D]")
        _check_view(name, t, like, (B, t.shape[1], N, D))
        heads.append(t.shape[1])
    return like, heads[0], heads[1], B, N, D


def _check_gains(q_gain, k_gain, like, D):
    """Nonzero when the gains are float32. Both have one dtype: float32 or that of q and k."""
    import torch
    kind = None
    for name, w in (("q_gain", q_gain), ("k_gain", k_gain)):
        if w is None:
            continue
        if w.shape != (D,) or not w.is_contiguous() or w.device != like.device:
            raise ValueError(f"{name} must be a contiguous [{D}] tensor on the device of q and k")
        if w.dtype != torch.float32 and w.dtype != like.dtype:
            raise ValueError(f"{name} must be float32 or of the dtype of q and k")
        if kind is not None and w.dtype != kind:
            raise ValueError("q_gain and k_gain must share one dtype")
        kind = w.dtype
    return int(kind == torch.float32)


def _check_tables(cos, sin, positions, like, B, N):
    """(rot, table rows, positions are int64, strides of positions)."""
    import torch
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin must be given together")
    if cos is None:
        if positions is not None:
            raise ValueError("positions need cos and sin")
        return 0, 0, 0, 0, 0
    for name, t in (("cos", cos), ("sin", sin)):
        if t.dim() != 2 or t.dtype != torch.float32 or not t.is_contiguous() or t.device != like.device:
            raise ValueError(f"{name} must be a contiguous float32 [rows, rot / 2] tensor on the device of q and k")
    if cos.shape != sin.shape:
        raise ValueError("cos and sin must share one shape")
    rows, half = cos.shape
    if positions is None:
        if rows < N:
            raise ValueError(f"the tables have {rows} rows; without positions {N} are needed")
        return 2 * half, rows, 0, 0, 0
    if positions.dtype not in (torch.int32, torch.int64) or positions.device != like.device:
        raise ValueError("positions must be int32 or int64 on the device of q and k")
    if positions.shape == (N,):
        strides = 0, positions.stride(0)
    elif positions.shape == (B, N):
        strides = positions.stride()
    else:
        raise ValueError(f"positions must be [{B}, {N}] or [{N}]")
    return 2 * half, rows, int(positions.dtype == torch.int64), strides[0], strides[1]


def _ptr(t):
    return None if t is None else t.data_ptr()


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
    import torch
    like, Hq, Hkv, B, N, D = _check_sides(q, k)
    gain_f32 = _check_gains(q_gain, k_gain, like, D)
    rot, rows, p64, pb, pn = _check_tables(cos, sin, positions, like, B, N)
    dtc = _dtype_code_of(like.dtype)
    dev = like.device
    s = launch_stream(dev, stream, (q, k, q_gain, k_gain, cos, sin, positions, q_out, k_out))
    outs = []
    for name, x, out in (("q_out", q, q_out), ("k_out", k, k_out)):
        if x is None:
            if out is not None:
                raise ValueError(f"{name} was given without its input")
        elif out is None:
            out = empty_on(s, stream, x.shape, x.dtype, dev)
        else:
            _check_view(name, out, like, x.shape)
        outs.append(out)
    strides = _F_ARGS(*_strides(q), *_strides(k), *_strides(outs[0]), *_strides(outs[1]), pb, pn)
    with torch.cuda.device(dev):
        code = library().fa2_qk_norm_rope_fwd(_ptr(q), _ptr(k), _ptr(q_gain), _ptr(k_gain), _ptr(cos), _ptr(sin),
                                              _ptr(positions), _ptr(outs[0]), _ptr(outs[1]), strides, B, Hq, Hkv, N,
                                              D, rot, rows, eps, 1 if interleaved else 0, gain_f32, p64, dtc,
                                              s.cuda_stream)
    if code:
        _check(code, "fa2_qk_norm_rope_fwd")
    return outs[0], outs[1]


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
    fa2_qk_norm_rope_bwd_workspace_bytes(D) bytes (allocated per call otherwise).
    """
    import torch
    like, Hq, Hkv, B, N, D = _check_sides(q, k)
    gain_f32 = _check_gains(q_gain, k_gain, like, D)
    rot, rows, p64, pb, pn = _check_tables(cos, sin, positions, like, B, N)
    dtc = _dtype_code_of(like.dtype)
    dev = like.device
    s = launch_stream(dev, stream, (dq_out, dk_out, q, k, q_gain, k_gain, cos, sin, positions, dq, dk, workspace))
    outs, gains = [], []
    for i, x, g, out, w in (("q", q, dq_out, dq, q_gain), ("k", k, dk_out, dk, k_gain)):
        if x is None:
            if g is not None or out is not None or w is not None:
                raise ValueError(f"d{i}_out, d{i} and {i}_gain need {i}")
        else:
            if g is None:
                raise ValueError(f"d{i}_out is needed with {i}")
            _check_view(f"d{i}_out", g, like, x.shape)
            if out is None:
                out = empty_on(s, stream, x.shape, x.dtype, dev)
            else:
                _check_view(f"d{i}", out, like, x.shape)
        outs.append(out)
        gains.append(None if w is None else empty_on(s, stream, (D,), w.dtype, dev))
    if q_gain is None and k_gain is None:
        need = 0
    else:
        need = fa2_qk_norm_rope_bwd_workspace_bytes(D)
        if workspace is None:
            workspace = empty_on(s, stream, (need,), torch.uint8, dev)
        elif workspace.device != dev or not workspace.is_contiguous() or \
                workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace must be a contiguous CUDA tensor of at least {need} bytes on q's device")
    ws_ptr, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if need else (None, 0)
    strides = _B_ARGS(*_strides(dq_out), *_strides(dk_out), *_strides(q), *_strides(k), *_strides(outs[0]),
                      *_strides(outs[1]), pb, pn)
    with torch.cuda.device(dev):
        code = library().fa2_qk_norm_rope_bwd(_ptr(dq_out), _ptr(dk_out), _ptr(q), _ptr(k), _ptr(q_gain),
                                              _ptr(k_gain), _ptr(cos), _ptr(sin), _ptr(positions), _ptr(outs[0]),
                                              _ptr(outs[1]), _ptr(gains[0]), _ptr(gains[1]), strides, B, Hq, Hkv, N,
                                              D, rot, rows, eps, 1 if interleaved else 0, gain_f32, p64, dtc, ws_ptr,
                                              ws_bytes, s.cuda_stream)
    if code:
        _check(code, "fa2_qk_norm_rope_bwd")
    return outs[0], outs[1], gains[0], gains[1]
