"""Cross attention: queries of one sequence over the keys and values of another, of another length.

    O, LSE = cross_attention_forward(q, k, v, key_lengths=lengths)
    dQ, dK, dV = cross_attention_backward(q, k, v, O, LSE, dO, key_lengths=lengths)

q is [B, Hq, Nq, D]; k and v are [B, Hkv, Nk, D] with Hq a multiple of Hkv;
lengths [B] says how many of the Nk keys each batch entry has.
"""
from __future__ import annotations

import ctypes
import math

from .binding import FA2_OK, _check, _dtype_code_of, library
from .streams import device_guard, empty_on, scratch_for, stream_handle

_fwd_bytes = {}


def fa2_cross_fwd_workspace_bytes(D: int) -> int:
    n = ctypes.c_size_t(0)
    _check(library().fa2_cross_fwd_workspace_bytes(int(D), ctypes.byref(n)), "fa2_cross_fwd_workspace_bytes")
    return n.value


def fa2_cross_bwd_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, D: int) -> int:
    n = ctypes.c_size_t(0)
    _check(library().fa2_cross_bwd_workspace_bytes(int(B), int(Hq), int(Hkv), int(Nq), int(Nk), int(D),
                                                   ctypes.byref(n)), "fa2_cross_bwd_workspace_bytes")
    return n.value


def _check_inputs(q, k, v, key_lengths):
    """(B, Hq, Hkv, Nq, Nk, D, device index) of a call, after the checks the C ABI cannot make."""
    dev = q.get_device()
    if dev < 0 or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k, v must be CUDA tensors on one device")
    ks = k.shape
    if q.dim() != 4 or len(ks) != 4 or v.shape != ks:
        raise ValueError("q must be [B, Hq, Nq, D], and k, v of one shape [B, Hkv, Nk, D]")
    B, Hq, Nq, D = q.shape
    _, Hkv, Nk, _ = ks
    if ks[0] != B or ks[3] != D:
        raise ValueError("q, k, v must share B and D")
    if Hkv == 0 or Hq % Hkv:
        raise ValueError(f"the {Hq} query heads must be a multiple of the {Hkv} key heads")
    dt = q.dtype
    if k.dtype != dt or v.dtype != dt:
        raise ValueError("q, k, v must share one dtype")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous")
    if key_lengths is not None:
        import torch
        if key_lengths.shape != (B,) or key_lengths.dtype != torch.int32 or not key_lengths.is_contiguous() or \
                key_lengths.get_device() != dev:
            raise ValueError(f"key_lengths must be a contiguous int32 [{B}] tensor on q's device")
    return B, Hq, Hkv, Nq, Nk, D, dev


def _like(name, t, shape, dtype, dev):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on q's device")
    return t


def _check_workspace(workspace, need, dev):
    if workspace.get_device() != dev or not workspace.is_contiguous() or workspace.nbytes < need:
        raise ValueError(f"workspace must be a contiguous CUDA tensor of at least {need} bytes on q's device")


def cross_attention_forward(q, k, v, scale: float | None = None, key_lengths=None, out=None, lse=None,
                            workspace=None, stream=None):
    """Attention of q [B, Hq, Nq, D] over k, v [B, Hkv, Nk, D]; returns (O, LSE).

    O is like q, LSE float32 [B, Hq, Nq]. Query head h reads key head
    h // (Hq // Hkv). key_lengths: int32 [B], the keys each batch entry has
    (default: all Nk); what lies behind them is never used. A row without any
    key gives O = 0 and LSE = +inf (not the -inf of an empty sum: merging two
    attentions by their LSE, replace it); one with a NaN or +inf score gives NaN.
    out, lse: caller-owned outputs. workspace: a uint8 CUDA tensor of at least
    fa2_cross_fwd_workspace_bytes(D) bytes (by default one is kept for each
    device, head dim, current stream and host thread; a captured call, and one
    that names its stream, gets its own).
    Runs on `stream` (a torch.cuda.Stream) or the current stream.
    """
    import torch
    B, Hq, Hkv, Nq, Nk, D, dev = _check_inputs(q, k, v, key_lengths)
    dt = q.dtype
    dtc = _dtype_code_of(dt)
    if out is not None:
        _like("out", out, q.shape, dt, dev)
    if lse is not None:
        _like("lse", lse, (B, Hq, Nq), torch.float32, dev)
    handle = stream_handle(dev, stream, (q, k, v, key_lengths, out, lse, workspace))
    if out is None:
        out = empty_on(stream, q.shape, dt, q.device)
    if lse is None:
        lse = empty_on(stream, (B, Hq, Nq), torch.float32, q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with device_guard(dev):
        need = _fwd_bytes.get((dev, D))
        if need is None:
            need = _fwd_bytes[(dev, D)] = fa2_cross_fwd_workspace_bytes(D)
        if workspace is None:
            workspace = scratch_for("cross_fwd", need, q.device, dev, handle, stream)
        else:
            _check_workspace(workspace, need, dev)
        code = library().fa2_cross_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                       None if key_lengths is None else key_lengths.data_ptr(), B, Hq, Hkv, Nq, Nk,
                                       D, scale, dtc, workspace.data_ptr(), workspace.nbytes, handle)
    if code != FA2_OK:
        _check(code, "fa2_cross_fwd")
    return out, lse


def cross_attention_backward(q, k, v, o, lse, do, scale: float | None = None, key_lengths=None, dq=None, dk=None,
                             dv=None, workspace=None, stream=None):
    """Gradient of cross_attention_forward w.r.t. q, k, v for an upstream gradient `do` of O; returns (dQ, dK, dV).

    q, k, v, scale, key_lengths are the forward's, o and lse its outputs for
    them, or the merged ones of a softmax that k and v are a part of (then dQ
    is the part's share). dQ is like q; dK and dV are like k, summed over the query heads of
    each key head, with zeros behind the key lengths.
    dq, dk, dv: caller-owned outputs. workspace: a uint8 CUDA tensor of at
    least fa2_cross_bwd_workspace_bytes(B, Hq, Hkv, Nq, Nk, D) bytes
    (allocated per call otherwise).
    """
    import torch
    B, Hq, Hkv, Nq, Nk, D, dev = _check_inputs(q, k, v, key_lengths)
    dt = q.dtype
    dtc = _dtype_code_of(dt)
    _like("o", o, q.shape, dt, dev)
    _like("do", do, q.shape, dt, dev)
    _like("lse", lse, (B, Hq, Nq), torch.float32, dev)
    for name, t, x in (("dq", dq, q), ("dk", dk, k), ("dv", dv, k)):
        if t is not None:
            _like(name, t, x.shape, dt, dev)
    handle = stream_handle(dev, stream, (q, k, v, o, lse, do, key_lengths, dq, dk, dv, workspace))
    if dq is None:
        dq = empty_on(stream, q.shape, dt, q.device)
    if dk is None:
        dk = empty_on(stream, k.shape, dt, q.device)
    if dv is None:
        dv = empty_on(stream, k.shape, dt, q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    need = fa2_cross_bwd_workspace_bytes(B, Hq, Hkv, Nq, Nk, D)
    if workspace is None:  # as large as the queries: a call's own
        workspace = empty_on(stream, max(need, 1), torch.uint8, q.device)
    else:
        _check_workspace(workspace, need, dev)
    with device_guard(dev):
        code = library().fa2_cross_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                                       lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                       None if key_lengths is None else key_lengths.data_ptr(), B, Hq, Hkv, Nq, Nk,
                                       D, scale, dtc, workspace.data_ptr(), workspace.nbytes, handle)
    if code != FA2_OK:
        _check(code, "fa2_cross_bwd")
    return dq, dk, dv
