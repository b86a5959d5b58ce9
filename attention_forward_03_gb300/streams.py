"""The stream and device a call runs on, and the tensors that are made for it.

torch's allocator hands a freed block to later work of the stream that the
block was allocated on. A call on another stream than the current one
therefore tells the allocator about its inputs (record_stream), and makes its
outputs and scratch on the stream that writes them.

The checks of a small call cost more than its kernel, so these helpers stay
with the cheap queries: device indices instead of torch.device objects, the
current stream's handle instead of a Stream object, and the device switched
only where it is not the current one (measured on a call of 12 heads: 26 us
before, of which the library's own share is 5 us).
"""
from __future__ import annotations

import threading


def stream_handle(index: int, stream, tensors) -> int:
    """The handle of `stream`, or of the current stream of device `index`; records `tensors` (None skipped) on a given one."""
    if stream is None:
        return current_handle(index)
    if stream.device_index != index:
        raise ValueError(f"stream is on device {stream.device_index}, the tensors on {index}")
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)
    return stream.cuda_stream


def current_handle(index: int) -> int:
    """The handle of the current stream of device `index`, by torch's query for it alone where there is one."""
    global current_handle
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    current_handle = raw if raw is not None else (lambda i: torch.cuda.current_stream(i).cuda_stream)
    return current_handle(index)


def empty_on(stream, shape, dtype, device):
    """An uninitialised tensor that belongs to the call's stream (`stream`: the caller's argument)."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_scratch = threading.local()  # .kept: the workspaces of this host thread


def scratch_for(kind, need, device, index, handle, stream):
    """A workspace of `need` bytes for a call on stream `handle` of device `index`.

    To be called with that device current. One per kind, size, current stream
    and host thread is kept: the calls of a thread on one stream are ordered,
    so they may share it. Those of two threads are not, where a call is more
    than one kernel: theirs could alternate. A call that names its stream, and
    one that is being captured (two graphs may be replayed at once), gets its
    own.
    """
    import torch
    if stream is not None or torch.cuda.is_current_stream_capturing():
        return empty_on(stream, max(need, 1), torch.uint8, device)
    try:
        kept = _scratch.kept
    except AttributeError:
        kept = _scratch.kept = {}
    key = (kind, need, index, handle)
    ws = kept.get(key)
    if ws is None:
        ws = kept[key] = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    return ws


class _Here:
    """A guard that has nothing to do."""

    __slots__ = ()

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_here = _Here()


def device_guard(index: int):
    """`with device_guard(i):` makes device i current (nothing happens where it already is)."""
    import torch
    return _here if torch.cuda.current_device() == index else torch.cuda.device(index)
