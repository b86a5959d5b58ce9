"""Two host threads that call on one stream at once: the calls of more than one kernel keep their scratch apart."""
from __future__ import annotations

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_head_norm_gradients_of_two_threads():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_forward_03_gb300 import build
    build.build()
    import attention_forward_03_gb300 as fa2
    dev = torch.device("cuda")
    sets = []
    for seed in range(2):
        g = torch.Generator(device=dev).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731, B023
        q, k, gq, gk = (r(1, h, 40, 64).half() for h in (4, 2, 4, 2))
        sets.append((gq, gk, q, k, 1 + 0.3 * r(64), 1 + 0.3 * r(64)))
    want = [fa2.qk_norm_rope_backward(*s) for s in sets]
    torch.cuda.synchronize()
    wrong, both = [], threading.Barrier(2)

    def call(i):
        both.wait()
        for _ in range(100):
            got = [fa2.qk_norm_rope_backward(*sets[i]) for _ in range(5)]
            torch.cuda.current_stream().synchronize()
            wrong.extend(i for g in got if not all(torch.equal(a, b) for a, b in zip(g, want[i])))

    threads = [threading.Thread(target=call, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
