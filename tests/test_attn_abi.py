"""The attention step's C ABI (include/lk_attn.h) on the host: every declared
entry point is exported and bound, and bad arguments are refused before any
launch (the pointers are never dereferenced).  No GPU."""
import ctypes
import math
import os
import re

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")

from q8_quantized_gemv_gb300 import build, lk  # noqa: E402

FAKE = 0x7F0000000000
BIG = 1 << 24  # bytes between buffers that must not overlap


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lk._load()


def P(v):
    return None if v is None else ctypes.c_void_p(v)


def cache(type=0, n_kv=2, head_dim=128, page=16, n_pages=4, k=FAKE, v=FAKE, ks=None, vs=None):
    return ctypes.byref(lk.LkKvCache(k, v, ks, vs, type, n_kv, head_dim, page, n_pages, 0))


BAD_CACHES = [(dict(type=3), -1), (dict(type=-1), -1), (dict(head_dim=96), -3), (dict(head_dim=256), -3),
              (dict(page=8), -3), (dict(page=24), -3), (dict(page=2048), -3), (dict(n_kv=0), -3), (dict(n_kv=3), -3),
              (dict(n_pages=0), -3), (dict(k=None), -1), (dict(v=None), -1), (dict(type=2), -1),
              (dict(type=2, ks=FAKE), -1), (dict(k=FAKE + 8), -2), (dict(v=FAKE + 4), -2),
              (dict(type=2, ks=FAKE + 2, vs=FAKE), -2)]


def test_symbols(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "lk_attn.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lk_[a-z0-9_]+)\s*\(", src)))
    assert sorted(lk.attn_symbols()) == names
    for n in names:
        assert hasattr(lib, n), n
    assert ctypes.sizeof(lk.LkKvCache) == 4 * 8 + 6 * 4


def test_append_refusals(lib):
    def call(c=None, q=FAKE, k=FAKE + 1024, v=FAKE + 2048, ld=1024, n_q=4, table=FAKE, tw=4, lens=FAKE, B=2, R=2,
             p0=0, cos=FAKE, sin=FAKE, n_pos=100, rot=128, qr=FAKE + BIG, qg=None, kg=None, cfg=None, **kw):
        return lib.lk_kv_append(c or cache(**kw), P(q), P(k), P(v), ld, n_q, P(table), tw, P(lens), B, R, p0, P(cos),
                                P(sin), n_pos, rot, 0, P(qg), P(kg), 1e-6, P(qr), lk._cfg(cfg), None)

    for bad, st in BAD_CACHES:
        assert call(**bad) == st, bad
    assert lib.lk_kv_append(None, *[None] * 3, 0, 4, None, 0, None, 1, 1, 0, None, None, 0, 0, 0, None, None, 1e-6,
                            None, None, None) == -1
    assert call(n_q=3) == -3 and call(n_q=0) == -3 and call(n_q=8192) == -3
    assert call(B=65, R=1) == -3 and call(B=8, R=9) == -3 and call(B=-1) == -3 and call(R=-1) == -3
    assert call(tw=-1) == -3 and call(tw=1 << 30) == -3
    assert call(rot=32) == -3 and call(rot=256) == -3 and call(head_dim=64, rot=128) == -3 and call(p0=-1) == -3
    assert call(n_pos=-1) == -3
    assert call(ld=508) == -3
    for name in ("q", "k", "v", "qr", "lens", "table", "cos", "sin"):
        assert call(**{name: None}) == -1, name
    assert call(q=FAKE + 4) == -2 and call(k=FAKE + 1028) == -2 and call(qr=FAKE + BIG + 8) == -2
    assert call(ld=1026) == -2 and call(lens=FAKE + 2) == -2 and call(cos=FAKE + 1) == -2 and call(qg=FAKE + 3) == -2
    # qr over the rows of q, k or v
    assert call(qr=FAKE) == -1 and call(qr=FAKE + 1024) == -1 and call(qr=FAKE + 3 * 4096 + 1024) == -1
    assert call(cfg=lk.launch_cfg(pdl=2)) == -1
    assert call(B=0) == 0 and call(R=0) == 0


def test_attn_refusals(lib):
    need = lk.lk_attn_workspace_bytes(4, 2, 128, 2, 2, True)

    def call(c=None, q=FAKE, n_q=4, pt=FAKE, pw=4, pl=50, table=FAKE, tw=4, lens=FAKE, B=2, R=2, scale=0.1, mode=0,
             out=FAKE, hq=FAKE, hl=FAKE, hs=FAKE, ws=FAKE, wsb=need, cfg=None, **kw):
        return lib.lk_attn_shared(c or cache(**kw), P(q), n_q, P(pt), pw, pl, P(table), tw, P(lens), B, R, scale, mode,
                                  P(out), P(hq), P(hl), P(hs), P(ws), wsb, lk._cfg(cfg), None)

    for bad, st in BAD_CACHES:
        assert call(**bad) == st, bad
    assert call(n_q=5) == -3
    assert call(B=64, R=2) == -3 and call(B=-1) == -3 and call(tw=-1) == -3
    assert call(pl=-1) == -3 and call(pl=65) == -3 and call(pw=-1) == -3 and call(pw=1 << 30) == -3
    assert call(tw=1 << 26, B=64, R=1, wsb=1 << 40) == -3     # more key units than 32 bits
    assert call(scale=math.inf) == -1 and call(scale=math.nan) == -1
    assert call(mode=3) == -1 and call(mode=-1) == -1
    for name in ("q", "pt", "table", "lens"):
        assert call(**{name: None}) == -1, name
    assert call(out=None) == -1                    # Dequant needs the f32 rows
    assert call(mode=1, hq=None) == -1 and call(mode=1, hs=None) == -1 and call(mode=2, hl=None) == -1
    assert call(q=FAKE + 4) == -2 and call(pt=FAKE + 2) == -2 and call(out=FAKE + 2) == -2
    assert call(mode=1, hs=FAKE + 2) == -2 and call(ws=FAKE + 8) == -2
    assert call(ws=None) == -4 and call(wsb=need - 1) == -4
    assert call(cfg=lk.launch_cfg(pdl=-1)) == -1
    assert call(B=0) == 0 and call(R=0) == 0
    # lk_attn shares the checks
    a = [P(FAKE), 4, P(FAKE), 4, P(FAKE), 2, 2, 0.1, 0, P(FAKE), None, None, None, P(FAKE)]
    assert lib.lk_attn(cache(page=12), *a, need, None, None) == -3
    assert lib.lk_attn(cache(), *a, 16, None, None) == -4


def test_workspace_bytes(lib):
    f = lk.lk_attn_workspace_bytes
    assert f(4, 2, 96, 1) == 0 and f(4, 3, 64, 1) == 0 and f(4, 0, 64, 1) == 0 and f(2, 4, 64, 1) == 0
    assert f(4, 2, 64, 65) == 0 and f(4, 2, 64, 8, 9) == 0 and f(4, 2, 64, -1) == 0
    assert 0 < f(32, 8, 128, 1) <= f(32, 8, 128, 64) < f(32, 8, 128, 64, 1, True)
    assert f(32, 8, 64, 4) < f(32, 8, 128, 4)


def test_launches(lib):
    f, much = lib.lk_attn_launches, 1 << 20
    assert f(0, 32, 8, 128, 1, 1, 0, much) == 2                 # streaming, join
    assert f(0, 32, 8, 128, 1, 64, 0, 1000) == 2                # tile, join
    assert f(1, 32, 8, 128, 64, 1, 32768, 1000) == 3            # tile (prefix), streaming (own), join
    assert f(1, 32, 8, 128, 64, 1, 100, 1000) == 2              # a short prefix streams too
    assert f(2, 32, 8, 64, 4, 8, 0, much) == 2 and f(2, 32, 8, 64, 4, 9, 50000, much) == 2
    assert f(0, 32, 8, 128, 1, 1, 0, 1024) == 1                 # clusters
    assert f(0, 32, 8, 128, 1, 1, 10, 1024) == 1 and f(0, 32, 8, 128, 1, 1, 20000, 1024) == 2
    assert f(0, 32, 8, 128, 64, 1, 0, 1024) == 2
    assert f(3, 32, 8, 128, 1, 1, 0, 1) == 0 and f(0, 32, 5, 128, 1, 1, 0, 1) == 0
    assert f(0, 32, 8, 128, 65, 1, 0, 1) == 0 and f(0, 32, 8, 128, 0, 1, 0, 1) == 0
    assert f(0, 32, 8, 128, 1, 1, -1, 1) == 0 and f(0, 32, 8, 128, 1, 1, 0, -1) == 0


def test_binding_refusals():
    k = torch.zeros((4, 2, 16, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        lk.KvCache(k, k)  # not on a GPU
    with pytest.raises(TypeError):
        lk.KvCache(k.float(), k.float())
    with pytest.raises(ValueError):
        lk.KvCache(k[0], k[0])
