"""Attention refuses buffers that it writes over others (paths differ in when
they read and write, so what would come out would depend on the path).  The
pointers are never dereferenced.  No GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from q8_quantized_gemv_gb300 import build, lk  # noqa: E402

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: only where nothing can be launched")

# B 2, R 2, 4 query heads on 2 of 128, 5 pages of 16: bytes of each argument
N, M = 4 * 128, 4
SIZES = dict(q=M * N * 4, out=M * N * 4, hq=M * N, hl=M * N, hs=M * N // 8, ws=None, k=5 * 2 * 16 * 128, v=5 * 2 * 16 * 128,
             ks=5 * 2 * 16 * 8, vs=5 * 2 * 16 * 8, table=2 * 3 * 4, lens=2 * 4, pt=4 * 4)
WRITTEN = ["out", "hq", "hl", "hs", "ws"]
ALIGN = dict(hq=1, hl=1, out=4, hs=4, table=4, lens=4, pt=4)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lk._load()


def call(lib, at, mode=2):
    P = ctypes.c_void_p
    c = lk.LkKvCache(at["k"], at["v"], at["ks"], at["vs"], 2, 2, 128, 16, 5, 0)
    return lib.lk_attn_shared(ctypes.byref(c), P(at["q"]), 4, P(at["pt"]), 4, 50, P(at["table"]), 3, P(at["lens"]), 2, 2,
                              0.1, mode, P(at["out"]), P(at["hq"]), P(at["hl"]), P(at["hs"]), P(at["ws"]), SIZES["ws"],
                              None, None)


def places():
    """The arguments one behind the other, without a byte between them but for alignment."""
    SIZES["ws"] = lk.lk_attn_workspace_bytes(4, 2, 128, 2, 2, True)
    at, p = {}, 0x7F0000000000
    for name, n in SIZES.items():
        p = -(-p // 16) * 16
        at[name] = p
        p += n
    return at


def test_neighbours_are_no_overlap(lib):
    at = places()
    assert call(lib, at) not in (-1, -2, -3, -4)  # as far as the device, which is not there
    assert call(lib, dict(at, out=at["q"])) not in (-1, -2, -3, -4)
    # what a mode does not write may be anything
    assert call(lib, dict(at, hq=at["q"], hl=at["q"], hs=at["q"]), mode=0) not in (-1, -2, -3, -4)
    assert call(lib, dict(at, hl=at["hq"]), mode=1) not in (-1, -2, -3, -4)


@pytest.mark.parametrize("name", WRITTEN)
@pytest.mark.parametrize("other", list(SIZES))
def test_overlap_is_refused(lib, name, other):
    if name == other:
        return
    at, a = places(), ALIGN.get(name, 16)
    # the last bytes of the other, its first, and all of it (exactly in place: out on q is allowed)
    ends = [(at[other] + SIZES[other] - 1) // a * a, -(-(at[other] - SIZES[name] + 1) // a) * a]
    if (name, other) != ("out", "q"):
        ends.append(at[other])
    for p in ends:
        if p == at[other] and (name, other) == ("out", "q"):
            continue
        moved = dict(at)
        moved[name] = p
        assert call(lib, moved) == -1, p - at[other]
