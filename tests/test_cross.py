"""Cross attention on the CPU: the oracle against differences and against attention over equal lengths, and the C
entry points' refusals. No kernel runs here."""
from __future__ import annotations

import pytest
import torch

from oracle import cross as ref


@pytest.fixture(scope="module")
def lib():
    from attention_forward_03_gb300 import build
    build.build()
    from attention_forward_03_gb300 import binding
    return binding


def rnd(g, *s):
    return torch.randn(*s, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("lengths", [None, [5, 0], [7, 3]])
def test_oracle_gradient_against_differences(lengths):
    g = torch.Generator().manual_seed(0)
    q, k, v, up = rnd(g, 2, 4, 3, 8), rnd(g, 2, 2, 7, 8), rnd(g, 2, 2, 7, 8), rnd(g, 2, 4, 3, 8)
    o, lse, _ = ref.forward(q, k, v, 0.4, lengths)
    grads = ref.backward(q, k, v, o, lse, up, 0.4, lengths)
    loss = lambda q, k, v: float((ref.forward(q, k, v, 0.4, lengths)[0] * up).sum())  # noqa: E731
    for _ in range(4):
        d, e = [rnd(g, *t.shape) for t in (q, k, v)], 1e-6
        num = (loss(*(t + e * x for t, x in zip((q, k, v), d))) - loss(*(t - e * x for t, x in zip((q, k, v), d)))) / (2 * e)
        ana = sum(float((grads[n][0] * x).sum()) for n, x in zip(("dq", "dk", "dv"), d))
        assert abs(num - ana) <= 1e-7 * float(up.abs().sum())


def test_oracle_ignores_what_lies_behind_the_keys():
    g = torch.Generator().manual_seed(1)
    q, k, v = rnd(g, 1, 2, 3, 8), rnd(g, 1, 1, 6, 8), rnd(g, 1, 1, 6, 8)
    a = ref.forward(q, k[:, :, :4], v[:, :, :4], 0.3)
    k[:, :, 4:], v[:, :, 4:] = float("nan"), float("inf")
    b = ref.forward(q, k, v, 0.3, [4])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert ref.forward(q, k, v, 0.3, [0])[1].isinf().all()


A = 0x1000000
FWD = dict(Q=A, K=A * 2, V=A * 3, O=A * 4, LSE=A * 5, n=None, B=2, Hq=4, Hkv=2, Nq=8, Nk=20, D=64, scale=0.125,
           dtype=0, ws=None, wsb=0, stream=None)


def fwd(lib, **over):
    return lib.library().fa2_cross_fwd(*dict(FWD, **over).values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -1), (dict(Hq=-4), -1), (dict(Hkv=-1), -1), (dict(Nq=-1), -1), (dict(Nk=-1), -1),
    (dict(D=48), -2), (dict(D=256), -2), (dict(D=0), -2), (dict(dtype=3), -2),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(Hq=5), -1), (dict(Hkv=0), -1), (dict(Hkv=3), -1),
    (dict(Q=None), -1), (dict(K=None), -1), (dict(V=None), -1), (dict(O=None), -1), (dict(LSE=None), -1),
    (dict(Q=A + 8), -3), (dict(K=A * 2 + 2), -3), (dict(LSE=A * 5 + 4), -3), (dict(n=A * 6 + 2), -3),
    (dict(ws=A * 7 + 8, wsb=1 << 20), -3),
    (dict(O=A + 128), -1), (dict(O=A), -1), (dict(LSE=A * 4 + 64), -1), (dict(O=A * 2), -1), (dict(LSE=A * 3), -1),
    (dict(n=A * 4 + 16), -1), (dict(n=A * 5), -1),
    (dict(ws=A * 4, wsb=1 << 16), -1), (dict(ws=A, wsb=1 << 16), -1), (dict(n=A * 7, ws=A * 7, wsb=1 << 16), -1),
    (dict(Nq=1 << 30), -1), (dict(Nk=(1 << 30) + 1), -1), (dict(B=1 << 20, Hq=1 << 14, Hkv=1 << 14), -1),
    (dict(B=1 << 24, Nq=1 << 20), -1),
])
def test_forward_refusals(lib, over, code):
    assert fwd(lib, **over) == code


def test_forward_of_nothing_is_nothing(lib):
    for over in (dict(B=0), dict(Hq=0), dict(Nq=0), dict(Hq=0, Hkv=0)):
        assert fwd(lib, Q=None, K=None, V=None, O=None, LSE=None, **over) == 0


BWD = dict(Q=A, K=A * 2, V=A * 3, O=A * 4, dO=A * 8, LSE=A * 5, dQ=A * 9, dK=A * 10, dV=A * 11, n=None, B=2, Hq=4,
           Hkv=2, Nq=8, Nk=20, D=64, scale=0.125, dtype=0, ws=A * 12, wsb=1 << 24, stream=None)


def bwd(lib, **over):
    return lib.library().fa2_cross_bwd(*dict(BWD, **over).values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -1), (dict(Nk=-2), -1), (dict(D=256), -2), (dict(D=48), -2), (dict(dtype=2), -2), (dict(scale=0.0), -1),
    (dict(Hq=3), -1), (dict(Hkv=0), -1), (dict(dO=None), -1), (dict(O=None), -1), (dict(LSE=None), -1),
    (dict(dV=None), -1), (dict(dQ=None), -1), (dict(K=None), -1), (dict(ws=None), -1), (dict(wsb=1 << 10), -1),
    (dict(ws=A * 12 + 128), -3), (dict(dQ=A * 9 + 4), -3), (dict(n=A * 6 + 1), -3),
    (dict(dQ=A), -1), (dict(dK=A * 2), -1), (dict(dK=A * 11), -1), (dict(dQ=A * 4 + 64), -1), (dict(dV=A * 5), -1),
    (dict(ws=A), -1), (dict(ws=A * 9), -1), (dict(n=A * 12), -1), (dict(n=A * 10), -1),
    (dict(Nq=1 << 30), -1), (dict(B=1 << 20, Hq=1 << 14, Hkv=1 << 14), -1),
])
def test_backward_refusals(lib, over, code):
    assert bwd(lib, **over) == code


def test_workspace_size_arguments(lib):
    import ctypes
    f = lib.library().fa2_cross_fwd_workspace_bytes
    assert f(64, None) == -1
    f, n = lib.library().fa2_cross_bwd_workspace_bytes, ctypes.c_size_t(0)
    assert f(2, 4, 2, 8, 20, 64, None) == -1 and f(2, 4, 2, 8, 20, 65, ctypes.byref(n)) == -2
    assert f(2, 4, 3, 8, 20, 64, ctypes.byref(n)) == -1 and f(2, 4, 2, -8, 20, 64, ctypes.byref(n)) == -1
    # 4 key heads of 16 rows: dQ, two statistics padded to a 128-row step, 160 partials of 2 x 128 x 64, 160 flags
    assert f(2, 4, 2, 8, 20, 64, ctypes.byref(n)) == 0
    assert n.value == 4 * 16 * 64 * 4 + 2 * 4 * 128 * 4 + 160 * 2 * 64 * 128 * 4 + 160 * 8
    assert f(2, 4, 2, 8, 10 ** 6, 64, ctypes.byref(n)) == 0 and n.value < 1 << 24  # not by the keys' length


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    from attention_forward_03_gb300 import cross_attention_forward
    x = torch.zeros(1, 1, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        cross_attention_forward(x, x, x)
