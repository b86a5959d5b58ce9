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
from .streams import empty_on, launch_stream

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
    """(B, Hq, Hkv, Nq, Nk, D) of a call, after the checks the C ABI cannot make."""
    import torch
    if not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise ValueError("q, k, v must be CUDA tensors")
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape:
        raise ValueError("q must be [B, Hq, Nq, D], and k, v of one shape [B, Hkv, Nk, D]")
    B, Hq, Nq, D = q.shape
    if k.shape[0] != B or k.shape[3] != D:
        raise ValueError("q, k, v must share B and D")
    Hkv, Nk = k.shape[1], k.shape[2]
    if Hkv == 0 or Hq % Hkv:
        raise ValueError(f"the {Hq} query heads must be a multiple of the {Hkv} key heads")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share one dtype")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous")
    if k.device != q.device or v.device != q.device:
        raise ValueError("q, k, v must be on one device")
    if key_lengths is not None and (key_lengths.shape != (B,) or key_lengths.dtype != torch.int32 or
                                    not key_lengths.is_contiguous() or key_lengths.device != q.device):
        raise ValueError(f"key_lengths must be a contiguous int32 [{B}] tensor on q's device")
    return B, Hq, Hkv, Nq, Nk, D


def _like(name, t, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on q's device")
    return t


def _workspace(workspace, need, s, stream, device):
    import torch
    if workspace is None:
        return empty_on(s, stream, (max(need, 1),), torch.uint8, device)
    if workspace.device != device or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a contiguous CUDA tensor of at least {need} bytes on q's device")
    return workspace


def cross_attention_forward(q, k, v, scale: float | None = None, key_lengths=None, out=None, lse=None,
                            workspace=None, stream=None):
    """Attention of q [B, Hq, Nq, D] over k, v [B, Hkv, Nk, D]; returns (O, LSE).

    O is like q, LSE float32 [B, Hq, Nq]. Query head h reads key head
    h // (Hq // Hkv). key_lengths: int32 [B], the keys each batch entry has
    (default: all Nk); what lies behind them is never used. A row without any
    key gives O = 0 and LSE = +inf.
    out, lse: caller-owned outputs. workspace: a uint8 CUDA tensor of at least
    fa2_cross_fwd_workspace_bytes(D) bytes (allocated per call otherwise).
    Runs on `stream` (a torch.cuda.Stream) or the current stream.
    """
    import torch
    B, Hq, Hkv, Nq, Nk, D = _check_inputs(q, k, v, key_lengths)
    dtc = _dtype_code_of(q.dtype)
    dev = q.device
    s = launch_stream(dev, stream, (q, k, v, key_lengths, out, lse, workspace))
    out = empty_on(s, stream, q.shape, q.dtype, dev) if out is None else _like("out", out, q.shape, q.dtype, dev)
    lse_shape = (B, Hq, Nq)
    lse = empty_on(s, stream, lse_shape, torch.float32, dev) if lse is None else \
        _like("lse", lse, lse_shape, torch.float32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(dev):
        need = _fwd_bytes.get((dev.index, D))
        if need is None:
            need = _fwd_bytes[(dev.index, D)] = fa2_cross_fwd_workspace_bytes(D)
        ws = _workspace(workspace, need, s, stream, dev)
        code = library().fa2_cross_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                       None if key_lengths is None else key_lengths.data_ptr(), B, Hq, Hkv, Nq, Nk,
                                       D, scale, dtc, ws.data_ptr(), ws.numel() * ws.element_size(), s.cuda_stream)
    if code != FA2_OK:
        _check(code, "fa2_cross_fwd")
    return out, lse


def cross_attention_backward(q, k, v, o, lse, do, scale: float | None = None, key_lengths=None, dq=None, dk=None,
                             dv=None, workspace=None, stream=None):
    """Gradient of cross_attention_forward w.r.t. q, k, v for an upstream gradient `do` of O; returns (dQ, dK, dV).

    q, k, v, scale, key_lengths are the forward's, o and lse its outputs for
    them. dQ is like q; dK and dV are like k, summed over the query heads of
    each key head, with zeros behind the key lengths.
    dq, dk, dv: caller-owned outputs. workspace: a uint8 CUDA tensor of at
    least fa2_cross_bwd_workspace_bytes(B, Hq, Hkv, Nq, Nk, D) bytes
    (allocated per call otherwise).
    """
    import torch
    B, Hq, Hkv, Nq, Nk, D = _check_inputs(q, k, v, key_lengths)
    dtc = _dtype_code_of(q.dtype)
    dev = q.device
    for name, t in (("o", o), ("do", do)):
        _like(name, t, q.shape, q.dtype, dev)
    _like("lse", lse, (B, Hq, Nq), torch.float32, dev)
    s = launch_stream(dev, stream, (q, k, v, o, lse, do, key_lengths, dq, dk, dv, workspace))
    outs = []
    for name, t, x in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        outs.append(empty_on(s, stream, x.shape, x.dtype, dev) if t is None else _like(name, t, x.shape, x.dtype, dev))
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    ws = _workspace(workspace, fa2_cross_bwd_workspace_bytes(B, Hq, Hkv, Nq, Nk, D), s, stream, dev)
    with torch.cuda.device(dev):
        code = library().fa2_cross_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                                       lse.data_ptr(), outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(),
                                       None if key_lengths is None else key_lengths.data_ptr(), B, Hq, Hkv, Nq, Nk,
                                       D, scale, dtc, ws.data_ptr(), ws.numel() * ws.element_size(), s.cuda_stream)
    if code != FA2_OK:
        _check(code, "fa2_cross_bwd")
    return tuple(outs)
