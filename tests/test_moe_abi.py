"""The C ABI of include/lk_moe.h and include/lk_sample.h on the host: every declared
entry point is exported and bound, and bad arguments are refused before any
launch (the pointers are never dereferenced).  No GPU."""
import ctypes
import os
import re

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")

from q8_quantized_gemv_gb300 import build, lk  # noqa: E402

FAKE = 0x7F0000000000
BIG = 1 << 28  # bytes between buffers that must not overlap


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lk._load()


def P(v):
    return None if v is None else ctypes.c_void_p(v)


@pytest.mark.parametrize("header,symbols", [("lk_moe.h", lk.moe_symbols), ("lk_sample.h", lk.sample_symbols)])
def test_symbols(lib, header, symbols):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lk_[a-z0-9_]+)\s*\(", src)))
    assert sorted(symbols()) == names
    for n in names:
        assert hasattr(lib, n), n


def test_route_refusals(lib):
    def call(l=FAKE, b=None, M=2, E=16, score=0, ng=1, tg=1, gs=1, k=4, renorm=1, scale=1.0, ids=FAKE + BIG,
             w=FAKE + 2 * BIG, cfg=None):
        return lib.lk_moe_route(P(l), P(b), M, E, score, ng, tg, gs, k, renorm, scale, P(ids), P(w), lk._cfg(cfg), None)
    assert call(score=2) == -1 and call(score=-1) == -1 and call(scale=float("inf")) == -1 and call(scale=float("nan")) == -1
    for bad in (dict(M=-1), dict(M=65), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(E=64, k=33), dict(ng=0),
                dict(ng=3), dict(ng=33, E=66), dict(tg=0), dict(ng=4, tg=5), dict(gs=0), dict(gs=3)):
        assert call(**bad) == -3, bad
    assert call(l=None) == -1 and call(ids=None) == -1 and call(w=None) == -1
    assert call(l=FAKE + 1) == -2 and call(b=FAKE + BIG // 2 + 2) == -2 and call(ids=FAKE + BIG + 2) == -2 and \
        call(w=FAKE + 1) == -2
    assert call(ids=FAKE) == -1 and call(w=FAKE + BIG + 28) == -1 and call(w=FAKE + 100) == -1 and \
        call(b=FAKE + BIG + 4) == -1
    assert call(cfg=lk.launch_cfg(pdl=2)) == -1
    assert call(M=0, l=None) == 0


def glu_args(**over):
    a = dict(wg=1, wsg=2, wu=3, wsu=4, E=4, F=128, K=256, mode=2, x=None, xq=5, xl=6, xs=7, M=2, ids=8, k=2, h=9, hq=10,
             hl=11, hs=12, cnt=13, cfg=None)
    a.update(over)
    return a


def down_args(**over):
    a = dict(wd=1, wsd=2, E=4, N=128, F=256, mode=2, h=None, hq=5, hl=6, hs=7, M=2, ids=8, w=9, k=2, y=10, cfg=None)
    a.update(over)
    return a


def buf(v):
    """Small numbers are buffers far apart, the others addresses as they are."""
    return P(v if v is None or v > 1000 else FAKE + v * BIG)


def glu(lib, **over):
    a = glu_args(**over)
    return lib.lk_moe_glu_q8(*(buf(a[n]) for n in ("wg", "wsg", "wu", "wsu")), a["E"], a["F"], a["K"], a["mode"],
                             *(buf(a[n]) for n in ("x", "xq", "xl", "xs")), a["M"], buf(a["ids"]), a["k"],
                             *(buf(a[n]) for n in ("h", "hq", "hl", "hs", "cnt")), lk._cfg(a["cfg"]), None)


def down(lib, **over):
    a = down_args(**over)
    return lib.lk_moe_down_q8(buf(a["wd"]), buf(a["wsd"]), a["E"], a["N"], a["F"], a["mode"],
                              *(buf(a[n]) for n in ("h", "hq", "hl", "hs")), a["M"], buf(a["ids"]), buf(a["w"]), a["k"],
                              buf(a["y"]), lk._cfg(a["cfg"]), None)


SHAPES = [dict(E=0), dict(E=1025), dict(M=-1), dict(M=65), dict(k=0), dict(k=33), dict(F=0), dict(F=64), dict(F=192),
          dict(F=-128), dict(E=1024, F=1 << 22)]


def test_glu_refusals(lib):
    assert glu(lib, mode=3) == -1 and glu(lib, mode=-1) == -1 and glu(lib, cfg=lk.launch_cfg(pdl=2)) == -1
    for bad in SHAPES + [dict(K=0), dict(K=64), dict(K=160), dict(K=-256)]:
        assert glu(lib, **bad) == -3, bad
    for n in ("wg", "wsg", "wu", "wsu", "xq", "xl", "xs", "ids", "h", "hl", "hs", "cnt"):
        assert glu(lib, **{n: None}) == -1, n
    assert glu(lib, mode=0, x=None) == -1
    for n, i in (("wg", 1), ("wsg", 2), ("wu", 3), ("wsu", 4), ("xq", 5), ("xl", 6), ("xs", 7), ("h", 9), ("hq", 10),
                 ("hl", 11), ("hs", 12)):
        assert glu(lib, **{n: FAKE + i * BIG + 8}) == -2, n
    assert glu(lib, ids=FAKE + 8 * BIG + 2) == -2 and glu(lib, cnt=FAKE + 13 * BIG + 2) == -2
    assert glu(lib, mode=0, x=FAKE + 4) == -2
    # what is written over what is read, or over each other
    for n in ("h", "hq", "hl", "hs", "cnt"):
        for m in (1, 2, 3, 4, 5, 6, 7, 8):
            assert glu(lib, **{n: m}) == -1, (n, m)
    assert glu(lib, hq=9) == -1 and glu(lib, hs=FAKE + 10 * BIG + 496) == -1 and glu(lib, cnt=12) == -1
    assert glu(lib, E=1, k=1, F=1 << 29) == -3 and glu(lib, E=1, k=2, F=1 << 28) == -3
    assert glu(lib, M=0, wg=None) == 0


def test_down_refusals(lib):
    assert down(lib, mode=3) == -1 and down(lib, cfg=lk.launch_cfg(pdl=2)) == -1
    for bad in SHAPES[:6] + [dict(N=n) for n in (0, 64, 192, -128)] + [dict(F=n) for n in (0, 64, 160, -256)]:
        assert down(lib, **bad) == -3, bad
    for n in ("wd", "wsd", "hq", "hl", "hs", "ids", "w", "y"):
        assert down(lib, **{n: None}) == -1, n
    assert down(lib, mode=0, h=None) == -1
    for n, i in (("wd", 1), ("wsd", 2), ("hq", 5), ("hl", 6), ("hs", 7), ("y", 10)):
        assert down(lib, **{n: FAKE + i * BIG + 8}) == -2, n
    assert down(lib, ids=FAKE + 8 * BIG + 1) == -2 and down(lib, w=FAKE + 9 * BIG + 2) == -2
    for m in (1, 2, 5, 6, 7, 8, 9):
        assert down(lib, y=m) == -1, m
    assert down(lib, M=0, wd=None) == 0


def test_sample_refusals(lib):
    names = ("temperature", "top_k", "top_p", "min_p", "u")

    def call(logits=1, M=2, N=1000, temperature=2, top_k=3, top_p=4, min_p=5, u=6, idx=7, prob=8, cfg=None):
        return lib.lk_sample(buf(logits), M, N, *(buf(v) for v in (temperature, top_k, top_p, min_p, u, idx, prob)),
                             lk._cfg(cfg), None)
    for bad in (dict(M=-1), dict(M=65), dict(N=0), dict(N=-5), dict(N=(1 << 21) + 1)):
        assert call(**bad) == -3, bad
    assert call(logits=None) == -1 and call(u=None) == -1 and call(idx=None) == -1
    for i, n in enumerate(("logits", *names, "idx", "prob")):
        assert call(**{n: FAKE + (i + 1) * BIG + 2}) == -2, n
    for n in ("idx", "prob"):
        for m in range(1, 7):
            assert call(**{n: m}) == -1, (n, m)
    assert call(prob=7) == -1 and call(cfg=lk.launch_cfg(pdl=3)) == -1
    assert call(M=0, logits=None) == 0


def test_binding_refuses(lib):
    """Argument checks of the Python layer that need no device."""
    q = torch.zeros((2, 128, 128), dtype=torch.int8)
    s = torch.zeros((2, 128, 4), dtype=torch.float16)
    with pytest.raises(ValueError):
        lk.Experts()
    with pytest.raises(ValueError):
        lk.Experts(gate=(q, s))
    with pytest.raises(ValueError):
        lk.Experts(down=(q, s))  # not on a CUDA device
    with pytest.raises(TypeError):
        lk.Experts(down=(q.float(), s))
    with pytest.raises(ValueError):
        lk.Experts(down=(q, s[:1]))
