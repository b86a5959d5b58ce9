"""The head norm with position rotation on the CPU: the oracle's gradient
against differences, and the C entry points' refusals. No kernel runs here."""
from __future__ import annotations

import ctypes

import pytest
import torch

from oracle import norm_rope as ref


@pytest.fixture(scope="module")
def lib():
    from attention_forward_03_gb300 import build
    build.build()
    from attention_forward_03_gb300 import binding
    return binding


def tables(rows, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f[None]
    return a.cos().float(), a.sin().float()


@pytest.mark.parametrize("rot,interleaved", [(0, False), (32, False), (32, True), (16, False), (16, True)])
def test_oracle_gradient_against_differences(rot, interleaved):
    g = torch.Generator().manual_seed(rot + interleaved)
    B, H, N, D = 2, 2, 3, 32
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, up, gain = rnd(B, H, N, D), rnd(B, H, N, D), rnd(D)
    cos, sin = tables(8, rot) if rot else (None, None)
    pos = torch.tensor([[1, 5, 7], [0, 2, 3]])
    loss = lambda x, w: float((ref.forward(x, w, cos, sin, pos if rot else None, 1e-5, interleaved)[0] * up).sum())  # noqa: E731
    dx, _, dw, _ = ref.backward(up, x, gain, cos, sin, pos if rot else None, 1e-5, interleaved)
    for _ in range(4):
        d, dg = rnd(*x.shape), rnd(D)
        e = 1e-6
        num = (loss(x + e * d, gain + e * dg) - loss(x - e * d, gain - e * dg)) / (2 * e)
        ana = float((dx * d).sum() + (dw * dg).sum())
        # differences of step 1e-6 in 64 bits: ~1e-16 / 1e-6 relative to the loss's terms
        assert abs(num - ana) <= 1e-7 * float(up.abs().sum())


def test_oracle_rotation_keeps_lengths_and_relative_angles():
    # <R(m) a, R(n) b> depends on m - n only
    g = torch.Generator().manual_seed(0)
    a, b = (torch.randn(1, 1, 1, 64, generator=g, dtype=torch.float64) for _ in range(2))
    cos, sin = tables(64, 64)
    for inter in (False, True):
        at = lambda t, p: ref.forward(t, None, cos, sin, torch.tensor([[p]]), 0.0, inter)[0].flatten()  # noqa: E731
        assert abs(float(at(a, 9) @ at(b, 4) - at(a, 45) @ at(b, 40))) < 1e-4  # fp32 tables
        assert abs(float(at(a, 9).norm() ** 2) - 64) < 1e-4


A = 0x100000  # fake aligned addresses, never dereferenced
FWD = dict(q=A, k=A * 2, qw=A * 3, kw=A * 4, cos=A * 5, sin=A * 6, pos=None, qo=A * 7, ko=A * 8, strides=None, B=1,
           Hq=2, Hkv=1, N=8, D=64, rot=64, rows=8, eps=1e-6, inter=0, gain_f32=1, p64=0, dtype=0, stream=None)


def fwd(lib, **over):
    a = dict(FWD, **over)
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_longlong * 14)(*a["strides"])
    return lib.library().fa2_qk_norm_rope_fwd(*a.values())


# contiguous strides of FWD's views, positions
S = [1024, 512, 64, 512, 512, 64, 1024, 512, 64, 512, 512, 64, 8, 1]


def s_with(**at):
    s = list(S)
    for i, v in at.items():
        s[int(i[1:])] = v
    return s


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -1), (dict(Hq=-1), -1), (dict(Hkv=-2), -1), (dict(N=-1), -1), (dict(rot=-16), -1),
    (dict(rows=-1), -1),
    (dict(D=48), -2), (dict(D=0), -2), (dict(D=2048), -2), (dict(dtype=2), -2), (dict(rot=24), -2), (dict(rot=8), -2),
    (dict(rot=80), -1), (dict(eps=-1e-6), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1), (dict(ko=None), -1), (dict(cos=None), -1),
    (dict(sin=None), -1), (dict(rows=7), -1),
    (dict(qw=A * 3 + 8), -3), (dict(kw=A * 4 + 2), -3), (dict(pos=A * 9 + 2), -3), (dict(pos=A * 9 + 4, p64=1), -3),
    (dict(q=A + 8), -3), (dict(ko=A * 8 + 2), -3), (dict(cos=A * 5 + 4), -3), (dict(sin=A * 6 + 8), -3),
    (dict(qo=A + 64), -1),                    # q_out meets q, not exactly
    (dict(qo=A * 2), -1),                     # q_out meets k
    (dict(ko=A), -1),                         # k_out meets q
    (dict(ko=A * 7 + 1024), -1),              # outputs meet each other
    (dict(qo=A * 5), -1),                     # q_out meets the tables
    (dict(qo=A * 3 - 1024), -1),              # q_out reaches into q_gain
    (dict(pos=A * 7 + 16), -1),               # positions inside q_out
    (dict(strides=s_with(_0=-8)), -1), (dict(strides=s_with(_7=1 << 45)), -1), (dict(strides=s_with(_12=-1), pos=A * 9), -1),
    (dict(strides=s_with(_1=516)), -3),       # a head stride off the 16-byte grid
    (dict(strides=s_with(_7=0)), -1), (dict(strides=s_with(_8=32)), -1),  # rows of q_out overlap one another
    (dict(B=1 << 20, N=1 << 20, rows=1 << 20), -1),
])
def test_forward_refusals(lib, over, code):
    assert fwd(lib, **over) == code


def test_forward_of_nothing_is_nothing(lib):
    for over in (dict(B=0), dict(N=0), dict(Hq=0, Hkv=0)):
        assert fwd(lib, q=None, k=None, qo=None, ko=None, **over) == 0


def test_forward_accepts_in_place_and_interleaved_views(lib):
    # past every argument check: what is left is the missing GPU here
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only where no kernel can start")
    good = fwd(lib)
    assert good not in (0, -1, -3)
    assert fwd(lib, qo=A, ko=A * 2) == good                               # in place
    # heads of one packed [B, N, 4, D] buffer, read and written in place
    packed = [8 * 256, 64, 256, 8 * 256, 64, 256] * 2 + [8, 1]
    assert fwd(lib, q=A, k=A + 2 * 128, qo=A, ko=A + 2 * 128, strides=packed) == good
    assert fwd(lib, q=A, k=A + 2 * 128, qo=A, ko=A + 128, strides=packed) == -1   # k_out on a q head
    # the two halves of a [B, 2, H, N, D] buffer
    halves = [2048, 512, 64, 512, 512, 64, 2048, 512, 64, 2048, 512, 64, 8, 1]
    assert fwd(lib, B=2, Hq=2, Hkv=2, qo=A * 7, ko=A * 7 + 2048, strides=halves) == good
    assert fwd(lib, B=2, Hq=2, Hkv=2, qo=A * 7, ko=A * 7 + 1024, strides=halves) == -1


BWD = dict(dqo=A * 10, dko=A * 11, q=A, k=A * 2, qw=A * 3, kw=A * 4, cos=A * 5, sin=A * 6, pos=None, dq=A * 7,
           dk=A * 8, dqw=A * 12, dkw=A * 13, strides=None, B=1, Hq=2, Hkv=1, N=8, D=64, rot=64, rows=8, eps=1e-6,
           inter=0, gain_f32=1, p64=0, dtype=0, ws=A * 20, wsb=1280 * 64 * 4, stream=None)


def bwd(lib, **over):
    a = dict(BWD, **over)
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_longlong * 20)(*a["strides"])
    return lib.library().fa2_qk_norm_rope_bwd(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -1), (dict(D=40), -2), (dict(dtype=7), -2), (dict(rot=40), -2), (dict(rot=96), -1),
    (dict(dqo=None), -1), (dict(dk=None), -1), (dict(dqw=None), -1), (dict(qw=None), -1), (dict(kw=None), -1),
    (dict(ws=None), -1), (dict(wsb=1280 * 64 * 4 - 4), -1), (dict(ws=A * 20 + 8), -3), (dict(dq=A * 7 + 2), -3),
    (dict(dqw=A * 12 + 4), -3), (dict(dqw=A * 5 + 64), -1), (dict(ws=A * 6), -1), (dict(ws=A * 4), -1),
    (dict(pos=A * 20 + 64), -1), (dict(pos=A * 13), -1),
    (dict(B=1 << 16, N=1 << 14, rows=1 << 14, strides=[1 << 40, 64, 64] * 6 + [1, 1]), -1),
    (dict(dq=A + 128), -1), (dict(dq=A * 10 + 128), -1), (dict(dq=A * 11), -1), (dict(dk=A * 7), -1),
    (dict(ws=A * 7), -1), (dict(ws=A), -1), (dict(dqw=A * 12, dkw=A * 12 + 64), -1), (dict(dqw=A * 20 + 256), -1),
    (dict(dqw=A * 3), -1), (dict(dqw=A * 7 + 64), -1), (dict(rows=4), -1),
])
def test_backward_refusals(lib, over, code):
    assert bwd(lib, **over) == code


def test_backward_workspace_size(lib):
    n = ctypes.c_size_t(0)
    f = lib.library().fa2_qk_norm_rope_bwd_workspace_bytes
    assert f(128, ctypes.byref(n)) == 0 and n.value == 1280 * 128 * 4
    assert f(100, ctypes.byref(n)) == -2 and f(64, None) == -1


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    from attention_forward_03_gb300 import qk_norm_rope_backward, qk_norm_rope_forward
    x = torch.zeros(1, 1, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        qk_norm_rope_forward(x, x)
    with pytest.raises(ValueError):
        qk_norm_rope_forward(None, None)
    with pytest.raises(ValueError):
        qk_norm_rope_backward(x, x, x, x)
