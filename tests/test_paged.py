"""Host-side checks of the paged calls' C ABI: what is refused before anything touches a GPU."""
from __future__ import annotations

import struct

import pytest

A = 1 << 32  # fake addresses, 4 GB apart; never dereferenced by these tests
TOKENS = (512, 64)              # token, head
CACHE = (8 * 16 * 64, 16 * 64, 64)  # page, head, slot


@pytest.fixture(scope="module")
def lib():
    from attention_forward_03_gb300 import build
    build.build()
    from attention_forward_03_gb300 import binding
    return binding


SIZES = dict(T=4, B=4, Hkv=8, D=64, pages=100, page=16, width=10)
GOOD = {
    "append": dict(SIZES, K=A, V=2 * A, kc=3 * A, vc=4 * A, w=None, table=5 * A, lengths=6 * A, starts=7 * A,
                   strides=(*TOKENS, *TOKENS, *CACHE, *CACHE, 10), dtype=0),
    "fwd": dict(SIZES, Hq=8, Q=A, kc=3 * A, vc=4 * A, O=8 * A, LSE=9 * A, table=5 * A, lengths=6 * A, starts=7 * A,
                strides=(*TOKENS, *CACHE, *CACHE, 10), most=4, scale=0.125, causal=1, dtype=0, ws=10 * A, wsb=1 << 30),
    "weights": dict(SIZES, Hq=8, Q=A, LSE=9 * A, kc=3 * A, w=11 * A, out=12 * A, table=5 * A, lengths=6 * A,
                    starts=7 * A, strides=(*TOKENS, *CACHE, 10), most=4, scale=0.125, causal=1, dtype=0, ws=10 * A,
                    wsb=1 << 30),
    "evict": dict(SIZES, kc=3 * A, vc=4 * A, w=11 * A, table=5 * A, lengths=6 * A, new=7 * A, new_lengths=8 * A,
                  kept=9 * A, strides=(*CACHE, *CACHE, 10, 4), new_width=4, keep=50, recent=8, dtype=0),
}


def call(lib, op, **over):
    a = dict(GOOD[op], **over)
    c = lib.library()
    strides = a["strides"]
    if strides is not None:
        strides = struct.pack(f"={len(strides)}q", *strides)
    tail = (a["pages"], a["page"], a["width"])
    if op == "append":
        return c.fa2_paged_append(a["K"], a["V"], a["kc"], a["vc"], a["w"], a["table"], a["lengths"], a["starts"],
                                  strides, a["T"], a["B"], a["Hkv"], a["D"], *tail, a["dtype"], None)
    if op == "fwd":
        return c.fa2_paged_fwd(a["Q"], a["kc"], a["vc"], a["O"], a["LSE"], a["table"], a["lengths"], a["starts"],
                               strides, a["T"], a["B"], a["Hq"], a["Hkv"], a["D"], *tail, a["most"], a["scale"],
                               a["causal"], a["dtype"], a["ws"], a["wsb"], None)
    if op == "weights":
        return c.fa2_paged_key_weights(a["Q"], a["LSE"], a["kc"], a["w"], a["out"], a["table"], a["lengths"],
                                       a["starts"], strides, a["T"], a["B"], a["Hq"], a["Hkv"], a["D"], *tail,
                                       a["most"], a["scale"], a["causal"], a["dtype"], a["ws"], a["wsb"], None)
    return c.fa2_paged_evict(a["kc"], a["vc"], a["w"], a["table"], a["lengths"], a["new"], a["new_lengths"], a["kept"],
                             strides, a["B"], a["Hkv"], a["D"], *tail, a["new_width"], a["keep"], a["recent"],
                             a["dtype"], None)


INVALID, UNSUPPORTED, ALIGN = -1, -2, -3
COMMON = [
    (dict(B=-1), INVALID), (dict(Hkv=-1), INVALID), (dict(pages=-1), INVALID), (dict(width=-1), INVALID),
    (dict(D=48), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(D=0), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(page=0), UNSUPPORTED),
    (dict(width=1 << 27), INVALID), (dict(kc=None), INVALID), (dict(table=None), INVALID), (dict(lengths=None), INVALID),
    (dict(strides=None), INVALID), (dict(kc=3 * A + 8), ALIGN), (dict(table=5 * A + 2), ALIGN), (dict(lengths=6 * A + 1), ALIGN),
]
TOKEN_CALLS = [(dict(T=-1), INVALID), (dict(T=(1 << 30) + 1), INVALID), (dict(T=5, starts=None), INVALID),
               (dict(starts=7 * A + 2), ALIGN)]
ATTENDING = [(dict(Hq=12), INVALID), (dict(Hq=-8), INVALID), (dict(most=-1), INVALID), (dict(scale=0.0), INVALID),
             (dict(scale=float("inf")), INVALID), (dict(Q=None), INVALID), (dict(LSE=None), INVALID), (dict(Q=A + 4), ALIGN),
             (dict(LSE=9 * A + 2), ALIGN)]


def strided(op, at, value):
    s = list(GOOD[op]["strides"])
    s[at] = value
    return dict(strides=tuple(s))


CASES = [(op, o, c) for op in GOOD for o, c in COMMON]
CASES += [(op, o, c) for op in ("append", "fwd", "weights") for o, c in TOKEN_CALLS]
CASES += [(op, o, c) for op in ("fwd", "weights") for o, c in ATTENDING]
CASES += [
    ("append", dict(K=None), INVALID), ("append", dict(V=2 * A + 2), ALIGN), ("append", dict(w=11 * A + 1), ALIGN),
    ("append", dict(K=3 * A + 4096), INVALID), ("append", dict(w=A), INVALID), ("append", dict(vc=5 * A), INVALID),
    ("append", strided("append", 0, 4), INVALID), ("append", strided("append", 2, -8), INVALID),
    ("append", strided("append", 4, 0), INVALID), ("append", strided("append", 9, 12), INVALID),
    ("append", strided("append", 7, 1 << 39), INVALID), ("append", strided("append", 10, -1), INVALID),
    ("fwd", dict(vc=None), INVALID), ("fwd", dict(O=None), INVALID), ("fwd", dict(ws=None), INVALID),
    ("fwd", dict(O=8 * A + 8), ALIGN), ("fwd", dict(ws=10 * A + 8), ALIGN), ("fwd", dict(O=A), INVALID),
    ("fwd", dict(LSE=8 * A + 64), INVALID), ("fwd", dict(O=3 * A + 1024), INVALID), ("fwd", dict(ws=5 * A), INVALID),
    ("fwd", dict(pages=0), INVALID), ("fwd", dict(width=0), INVALID), ("fwd", dict(Hkv=0), INVALID),
    ("fwd", strided("fwd", 0, 20), INVALID), ("fwd", strided("fwd", 2, 1 << 45), INVALID),
    ("weights", dict(out=None), INVALID), ("weights", dict(ws=None), INVALID), ("weights", dict(ws=10 * A + 8), ALIGN),
    ("weights", dict(ws=12 * A), INVALID), ("weights", dict(out=3 * A), INVALID), ("weights", dict(out=11 * A + 64), INVALID),
    ("weights", dict(out=9 * A), INVALID), ("weights", dict(out=12 * A + 2), ALIGN), ("weights", strided("weights", 4, 4), INVALID),
    ("evict", dict(w=None), INVALID), ("evict", dict(new=None), INVALID), ("evict", dict(kept=None), INVALID),
    ("evict", dict(new_lengths=None), INVALID), ("evict", dict(new=5 * A), INVALID), ("evict", dict(keep=65), INVALID),
    ("evict", dict(recent=51), INVALID), ("evict", dict(recent=-1), INVALID), ("evict", dict(keep=-1, recent=-1), INVALID),
    ("evict", dict(kept=5 * A), INVALID), ("evict", dict(new_lengths=6 * A), INVALID), ("evict", dict(new=7 * A + 2), ALIGN),
    ("evict", strided("evict", 3, 0), INVALID), ("evict", strided("evict", 7, -4), INVALID), ("evict", dict(pages=0), INVALID),
]


@pytest.mark.parametrize("op,over,code", CASES, ids=lambda x: str(x)[:60])
def test_refused(lib, op, over, code):
    assert call(lib, op, **over) == code


@pytest.mark.parametrize("op,over", [("append", dict(T=0)), ("append", dict(B=0)), ("append", dict(pages=0)),
                                     ("fwd", dict(T=0)), ("fwd", dict(B=0)), ("weights", dict(B=0)),
                                     ("weights", dict(pages=0)), ("evict", dict(B=0))], ids=str)
def test_nothing_to_do(lib, op, over):
    assert call(lib, op, **over) == 0


def test_workspace_query(lib):
    import ctypes
    n = ctypes.c_size_t(0)
    assert lib.library().fa2_paged_fwd_workspace_bytes(64, None) == INVALID
    assert lib.library().fa2_paged_fwd_workspace_bytes(80, ctypes.byref(n)) == UNSUPPORTED
