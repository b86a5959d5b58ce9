"""The scratch that the binding keeps for small calls, on the CPU: who shares it and who does not."""
from __future__ import annotations

import threading

import pytest
import torch

from attention_forward_03_gb300 import streams


@pytest.fixture
def scratch(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return lambda handle=0, kind="k", need=64: streams.scratch_for(kind, need, "cpu", 0, handle, None)


def test_calls_of_one_thread_and_stream_share(scratch):
    a = scratch()
    assert scratch() is a and a.nbytes == 64
    assert scratch(handle=8) is not a and scratch(kind="other") is not a and scratch(need=128) is not a
    assert scratch() is a


def test_two_host_threads_do_not_share(scratch):
    # both on one stream: a call of two kernels could be cut in two by the other thread's
    got, both = {}, threading.Barrier(2)

    def call(i):
        both.wait()
        got[i] = [scratch() for _ in range(3)]
        both.wait()

    threads = [threading.Thread(target=call, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert got[0][0] is got[0][2] and got[1][0] is got[1][2]
    assert got[0][0].data_ptr() != got[1][0].data_ptr() and scratch() is not got[0][0]


def test_a_captured_call_gets_its_own(scratch, monkeypatch):
    a = scratch()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    assert scratch() is not a and scratch() is not scratch()
