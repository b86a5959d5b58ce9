"""A key/value cache in pages, and what a serving program runs on it.

    paged_cache_append(k, v, k_cache, v_cache, table, lengths)            # a step's new tokens into the cache
    O, LSE = paged_attention_forward(q, k_cache, v_cache, table, lengths)  # their attention over it
    weights = paged_key_weights(q, LSE, k_cache, table, lengths, weights=weights)  # what each cached key weighs
    lengths, kept = paged_cache_evict(k_cache, v_cache, weights, table, lengths, new_table, keep)

A cache is [pages, Hkv, page size, D] with any strides (the head dim
contiguous), so [pages, page size, Hkv, D] is passed as
``cache.transpose(1, 2)`` and one buffer [pages, 2, Hkv, page size, D] as its
two halves. Page sizes are 16, 32, 64, 128 and 256. table [B, max_pages] int32
holds each sequence's pages in order, lengths [B] int32 its positions, the
call's new tokens included; entries behind a sequence's last page are not read.

The new tokens are packed, [T, heads, D]. Sequence b's are the rows
query_starts[b] to query_starts[b + 1] (int32 [B + 1], ascending) and stand at
its last positions; without query_starts every sequence has T / B of them.
Single tokens, chunks of prompts and whole prompts may be mixed.
"""
from __future__ import annotations

import ctypes
import math
import struct

from .binding import FA2_OK, _check, _dtype_code_of, library
from .streams import device_guard, empty_on, scratch_for, stream_handle

# the strides a call passes, as the C side reads them (bytes are passed by address)
_STRIDES11 = struct.Struct("=11q").pack
_STRIDES9 = struct.Struct("=9q").pack
_STRIDES8 = struct.Struct("=8q").pack
_STRIDES6 = struct.Struct("=6q").pack
_fwd_bytes = {}
_weights_bytes = {}


def fa2_paged_fwd_workspace_bytes(D: int) -> int:
    n = ctypes.c_size_t(0)
    _check(library().fa2_paged_fwd_workspace_bytes(int(D), ctypes.byref(n)), "fa2_paged_fwd_workspace_bytes")
    return n.value


def fa2_paged_key_weights_workspace_bytes() -> int:
    n = ctypes.c_size_t(0)
    _check(library().fa2_paged_key_weights_workspace_bytes(ctypes.byref(n)), "fa2_paged_key_weights_workspace_bytes")
    return n.value


# The checks of a small call cost more than its kernel (measured on one of 4
# sequences: 20 us, of which the library's own share is 5), so each tensor is
# asked for each of its properties once.
def _check_cache(name, c, dt, dev, shape=None):
    """(shape, page, head and slot strides) of a cache, which has the dtype and device of the call."""
    s = c.shape
    if (s != shape if shape is not None else len(s) != 4):
        raise ValueError(f"{name} must be [pages, Hkv, page size, D]" + ("" if shape is None else " like k_cache"))
    if c.dtype is not dt or c.get_device() != dev:
        raise ValueError(f"{name} must have the dtype and device of the other tensors")
    strides = c.stride()
    if strides[3] != 1 and s[3] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return s, strides[:3]


def _check_tokens(name, t, T, heads, D, dt, dev):
    """(token, head) strides of a [T, heads, D] view."""
    if t.shape != (T, heads, D):
        raise ValueError(f"{name} must have the shape {[T, heads, D]}")
    if t.dtype is not dt or t.get_device() != dev:
        raise ValueError(f"{name} must have the dtype and device of the other tensors")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return st, sh


def _check_table(name, table, dev, B=None):
    """(rows, entries per row, row stride) of a page table."""
    import torch
    shape = table.shape
    if len(shape) != 2 or table.dtype is not torch.int32 or table.get_device() != dev:
        raise ValueError(f"{name} must be an int32 [B, pages] tensor on the caches' device")
    rows, width = shape
    row, column = table.stride()
    if column != 1 and width > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    if B is not None and rows != B:
        raise ValueError(f"{name} must have {B} rows")
    return rows, width, row


def _check_ints(name, t, n, dev):
    import torch
    if t.shape != (n,) or t.dtype is not torch.int32 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor on the caches' device")
    return t.data_ptr()


def _check_batch(table, key_lengths, query_starts, T, dev):
    """(B, max_pages, table stride, pointers of the table, lengths and starts)."""
    B, width, row = _check_table("block_table", table, dev)
    lengths = _check_ints("key_lengths", key_lengths, B, dev)
    starts = None
    if query_starts is not None:
        starts = _check_ints("query_starts", query_starts, B + 1, dev)
    elif T and (B == 0 or T % B):
        raise ValueError(f"without query_starts the {T} tokens must be a multiple of the {B} sequences")
    return B, width, row, table.data_ptr(), lengths, starts


def _check_pool(name, t, shape, dev):
    import torch
    if t.shape != shape[:3] or t.dtype != torch.float32 or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous float32 {list(shape[:3])} tensor on the caches' device")
    return t.data_ptr()


def _like(name, t, shape, dtype, dev):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on the caches' device")


def _check_workspace(workspace, need, dev):
    if workspace.get_device() != dev or not workspace.is_contiguous() or workspace.nbytes < need:
        raise ValueError(f"workspace must be a contiguous CUDA tensor of at least {need} bytes on q's device")


def _device_of(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("the tensors must be CUDA tensors")
    return dev


def _group(Hq, Hkv):
    if Hkv == 0 or Hq % Hkv:
        raise ValueError(f"the {Hq} query heads must be a multiple of the {Hkv} key heads")


def paged_cache_append(k, v, k_cache, v_cache, block_table, key_lengths, query_starts=None, weights=None,
                       stream=None):
    """Writes new tokens' k, v [T, Hkv, D] to their positions in the caches (in place); returns (k_cache, v_cache).

    k, v: views with any strides, the head dim contiguous (parts of a packed
    projection, or what qk_norm_rope_forward wrote). block_table, key_lengths,
    query_starts: see the module; key_lengths count the new tokens already.
    weights: float32 [pages, Hkv, page size] for paged_key_weights; the written
    positions' are set to 0. Tokens without a position, or whose page number is
    not one of the cache's, are not written. No two tokens share a position.
    Runs on `stream` (a torch.cuda.Stream) or the current stream.
    """
    dev = _device_of(k_cache)
    dt = k_cache.dtype
    dtc = _dtype_code_of(dt)
    shape, ks = _check_cache("k_cache", k_cache, dt, dev)
    vs = _check_cache("v_cache", v_cache, dt, dev, shape)[1]
    pages, Hkv, page, D = shape
    T = k.shape[0]
    kt = _check_tokens("k", k, T, Hkv, D, dt, dev)
    vt = _check_tokens("v", v, T, Hkv, D, dt, dev)
    B, width, row, table, lengths, starts = _check_batch(block_table, key_lengths, query_starts, T, dev)
    w = None if weights is None else _check_pool("weights", weights, shape, dev)
    handle = stream_handle(dev, stream, (k, v, k_cache, v_cache, block_table, key_lengths, query_starts, weights))
    with device_guard(dev):
        code = library().fa2_paged_append(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), w,
                                          table, lengths, starts, _STRIDES11(*kt, *vt, *ks, *vs, row),
                                          T, B, Hkv, D, pages, page, width, dtc, handle)
    if code != FA2_OK:
        _check(code, "fa2_paged_append")
    return k_cache, v_cache


def paged_attention_forward(q, k_cache, v_cache, block_table, key_lengths, query_starts=None,
                            scale: float | None = None, is_causal: bool = True, max_query_length: int | None = None,
                            out=None, lse=None, workspace=None, stream=None):
    """Attention of the new tokens q [T, Hq, D] over their sequences' positions; returns (O, LSE).

    O is contiguous [T, Hq, D], LSE float32 [T, Hq]. Query head h reads key
    head h // (Hq // Hkv). A token sees its own position and the earlier ones
    (is_causal=False: all of its sequence's). A row without any position gives
    O = 0 and LSE = +inf, as in cross_attention_forward; rows of O and LSE that
    are no sequence's tokens are left as they were. What the caches hold
    elsewhere is never used. A page number outside the cache makes the rows
    that see its positions NaN.
    q: a view with any strides, the head dim contiguous.
    max_query_length: the most new tokens that a sequence has, where the caller
    knows (the call chooses its kernels by it: a wrong one costs time, and O
    and LSE may differ in their last bits).
    out, lse: caller-owned outputs. workspace: a uint8 CUDA tensor of at least
    fa2_paged_fwd_workspace_bytes(D) bytes (by default one is kept for each
    device, head dim, current stream and host thread; a captured call, and one
    that names its stream, gets its own).
    Runs on `stream` (a torch.cuda.Stream) or the current stream.
    """
    import torch
    dev = _device_of(q)
    dt = q.dtype
    dtc = _dtype_code_of(dt)
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, D]")
    T, Hq, D = q.shape
    shape, ks = _check_cache("k_cache", k_cache, dt, dev)
    vs = _check_cache("v_cache", v_cache, dt, dev, shape)[1]
    pages, Hkv, page, _ = shape
    _group(Hq, Hkv)
    qs = _check_tokens("q", q, T, Hq, shape[3], dt, dev)
    B, width, row, table, lengths, starts = _check_batch(block_table, key_lengths, query_starts, T, dev)
    if out is not None:
        _like("out", out, q.shape, dt, dev)
    if lse is not None:
        _like("lse", lse, (T, Hq), torch.float32, dev)
    handle = stream_handle(dev, stream, (q, k_cache, v_cache, block_table, key_lengths, query_starts, out, lse,
                                         workspace))
    if out is None:
        out = empty_on(stream, (T, Hq, D), dt, q.device)
    if lse is None:
        lse = empty_on(stream, (T, Hq), torch.float32, q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with device_guard(dev):
        need = _fwd_bytes.get((dev, D))
        if need is None:
            need = _fwd_bytes[(dev, D)] = fa2_paged_fwd_workspace_bytes(D)
        if workspace is None:
            workspace = scratch_for("paged_fwd", need, q.device, dev, handle, stream)
        else:
            _check_workspace(workspace, need, dev)
        code = library().fa2_paged_fwd(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
                                       lse.data_ptr(), table, lengths, starts,
                                       _STRIDES9(*qs, *ks, *vs, row), T, B, Hq, Hkv, D, pages, page, width,
                                       T if max_query_length is None else max_query_length, scale,
                                       1 if is_causal else 0, dtc, workspace.data_ptr(), workspace.nbytes, handle)
    if code != FA2_OK:
        _check(code, "fa2_paged_fwd")
    return out, lse


def paged_key_weights(q, lse, k_cache, block_table, key_lengths, query_starts=None, scale: float | None = None,
                      is_causal: bool = True, max_query_length: int | None = None, weights=None, out=None,
                      workspace=None, stream=None):
    """What every cached key weighs in the new tokens' softmax rows, added to `weights`; returns out.

    out[slot] = weights[slot] + sum of exp(scale <q_i, k> - LSE_i) over the
    rows i (tokens that see the position, query heads of its key head): the
    column sums of the attention that paged_attention_forward(q, ...) = (O,
    lse) computed with the same arguments. Both are float32 [pages, Hkv, page
    size]; weights=None stands for zeros. out may be `weights` itself, and is
    where it is not given (without either, a new tensor of zeros). Every
    position of every sequence is written, nothing else is; two sequences share
    no position. The sums have a fixed order. A row whose lse is NaN (it sees a
    page number outside the cache, say) makes all that it sees NaN, and
    paged_cache_evict keeps these first.
    max_query_length: as for paged_attention_forward. workspace: a uint8 CUDA
    tensor of at least fa2_paged_key_weights_workspace_bytes() bytes (kept by
    default, as paged_attention_forward's is).
    Runs on `stream` (a torch.cuda.Stream) or the current stream.
    """
    import torch
    dev = _device_of(q)
    dt = q.dtype
    dtc = _dtype_code_of(dt)
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, D]")
    T, Hq, D = q.shape
    shape, ks = _check_cache("k_cache", k_cache, dt, dev)
    pages, Hkv, page, _ = shape
    _group(Hq, Hkv)
    qs = _check_tokens("q", q, T, Hq, shape[3], dt, dev)
    _like("lse", lse, (T, Hq), torch.float32, dev)
    B, width, row, table, lengths, starts = _check_batch(block_table, key_lengths, query_starts, T, dev)
    w = None if weights is None else _check_pool("weights", weights, shape, dev)
    if out is None:
        out = weights
    elif out is not weights:
        _check_pool("out", out, shape, dev)
    handle = stream_handle(dev, stream, (q, lse, k_cache, block_table, key_lengths, query_starts, weights, out,
                                         workspace))
    if out is None:
        out = empty_on(stream, shape[:3], torch.float32, q.device)
        if stream is None:
            out.zero_()
        else:
            with torch.cuda.stream(stream):
                out.zero_()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with device_guard(dev):
        need = _weights_bytes.get(dev)
        if need is None:
            need = _weights_bytes[dev] = fa2_paged_key_weights_workspace_bytes()
        if workspace is None:
            workspace = scratch_for("paged_key_weights", need, q.device, dev, handle, stream)
        else:
            _check_workspace(workspace, need, dev)
        code = library().fa2_paged_key_weights(q.data_ptr(), lse.data_ptr(), k_cache.data_ptr(), w, out.data_ptr(),
                                               table, lengths, starts, _STRIDES6(*qs, *ks, row), T, B,
                                               Hq, Hkv, D, pages, page, width,
                                               T if max_query_length is None else max_query_length, scale,
                                               1 if is_causal else 0, dtc, workspace.data_ptr(), workspace.nbytes,
                                               handle)
    if code != FA2_OK:
        _check(code, "fa2_paged_key_weights")
    return out


def paged_cache_evict(k_cache, v_cache, weights, block_table, key_lengths, new_table, keep: int, recent: int = 0,
                      new_lengths=None, kept=None, stream=None):
    """Cuts every sequence down to `keep` positions of its key heads, those of the greatest weight; returns (new_lengths, kept).

    Kept are, for each key head on its own, the last `recent` positions and,
    of the others, the keep - recent of the greatest weight (of equal ones the
    earlier; NaN counts as above +inf); a sequence of at most `keep` positions
    keeps all. Their keys, values and weights are copied in order to the
    positions 0, 1, ... of the pages in new_table [B, pages] int32 (room for
    `keep` positions; none of them may be a page that a sequence still has
    positions in, nor occur twice). The old pages keep what they hold and may
    be given away once the call has run.
    new_lengths: int32 [B], min(key_lengths, keep), the lengths for the calls
    that follow with new_table. kept: int32 [B, Hkv, keep], the positions that
    were kept, ascending, -1 behind them. A position whose page number is not
    one of the cache's counts as the least weight and is copied as zeros.
    Runs on `stream` (a torch.cuda.Stream) or the current stream.
    """
    import torch
    dev = _device_of(k_cache)
    dt = k_cache.dtype
    dtc = _dtype_code_of(dt)
    shape, ks = _check_cache("k_cache", k_cache, dt, dev)
    vs = _check_cache("v_cache", v_cache, dt, dev, shape)[1]
    pages, Hkv, page, D = shape
    w = _check_pool("weights", weights, shape, dev)
    B, width, row = _check_table("block_table", block_table, dev)
    new_width, new_row = _check_table("new_table", new_table, dev, B)[1:]
    lengths = _check_ints("key_lengths", key_lengths, B, dev)
    if not 0 <= recent <= keep or keep > new_width * page:
        raise ValueError(f"0 <= recent <= keep <= {new_width * page} (the room in new_table) is needed")
    if new_lengths is not None:
        _check_ints("new_lengths", new_lengths, B, dev)
    if kept is not None:
        _like("kept", kept, (B, Hkv, keep), torch.int32, dev)
    handle = stream_handle(dev, stream, (k_cache, v_cache, weights, block_table, key_lengths, new_table, new_lengths,
                                         kept))
    if new_lengths is None:
        new_lengths = empty_on(stream, (B,), torch.int32, k_cache.device)
    if kept is None:
        kept = empty_on(stream, (B, Hkv, keep), torch.int32, k_cache.device)
    with device_guard(dev):
        code = library().fa2_paged_evict(k_cache.data_ptr(), v_cache.data_ptr(), w, block_table.data_ptr(), lengths,
                                         new_table.data_ptr(), new_lengths.data_ptr(), kept.data_ptr(),
                                         _STRIDES8(*ks, *vs, row, new_row), B, Hkv, D, pages, page, width, new_width,
                                         keep, recent, dtc, handle)
    if code != FA2_OK:
        _check(code, "fa2_paged_evict")
    return new_lengths, kept
