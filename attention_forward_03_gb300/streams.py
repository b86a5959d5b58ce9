"""The stream a call runs on, and the tensors that are made for it.

torch's allocator hands a freed block to later work of the stream that the
block was allocated on. A call on another stream than the current one
therefore tells the allocator about its inputs (record_stream), and makes its
outputs and scratch on the stream that writes them.
"""
from __future__ import annotations


def launch_stream(device, stream, tensors):
    """`stream`, or the current stream of `device`; records `tensors` (None skipped) on a stream that is not current."""
    import torch
    cur = torch.cuda.current_stream(device)
    if stream is None or stream == cur:
        return cur
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)
    return stream


def empty_on(s, stream, shape, dtype, device):
    """An uninitialised tensor that belongs to the call's stream `s` (`stream`: the caller's argument)."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=device)
