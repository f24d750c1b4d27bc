"""Rows too long for a kernel of the experts' products are refused whatever their
length: the bytes of a row pass 32 bits long before the length does.  On the host:
the refusals come before the device is looked at.  No GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from q8_quantized_gemv_gb300 import build, lk  # noqa: E402

SHAPE = -3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lk._load()


def at(i):
    """Buffers a terabyte apart: none reaches the next."""
    return ctypes.c_void_p((i + 1) << 40)


def glu(lib, mode, K, path=0):
    x = (at(4), None, None, None) if mode == 0 else (None, at(4), at(5), at(6))
    return lib.lk_moe_glu_q8(at(0), at(1), at(2), at(3), 1, 128, K, mode, *x, 1, at(7), 1, at(8), None, None, None, None,
                             lk._cfg(lk.launch_cfg(path=path)), None)


def down(lib, mode, F, path=0):
    h = (at(2), None, None, None) if mode == 0 else (None, at(2), at(3), at(4))
    return lib.lk_moe_down_q8(at(0), at(1), 1, 128, F, mode, *h, 1, at(5), at(6), 1, at(7),
                              lk._cfg(lk.launch_cfg(path=path)), None)


@pytest.mark.parametrize("call", [glu, down])
@pytest.mark.parametrize("K", [51200, 1 << 20, (1 << 30) - 128, 1 << 30, (1 << 30) + 128, (1 << 30) + 12800,
                               (1 << 30) + 51200, 3 << 29, (1 << 31) - 128])
def test_rows_past_shared_memory(lib, call, K):
    """4 K bytes of f32 wrap to next to nothing from 2^30 on, K and more of words near 2^31."""
    assert call(lib, 0, K) == SHAPE
    assert call(lib, 1, 4 * K if 4 * K < 1 << 31 else K, 2) == SHAPE
    assert call(lib, 2, 2 * K if 2 * K < 1 << 31 else K, 2) == SHAPE


@pytest.mark.parametrize("call", [glu, down])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("path", [0, 3])
def test_lengths_that_slices_of_it_would_pass(lib, call, mode, path):
    """The tensor-core kernel takes rows in slices, whose number is rounded up from the length."""
    for K in ((1 << 30) + 128, (1 << 31) - 384, (1 << 31) - 128):
        assert call(lib, mode, K, path) == SHAPE


@pytest.mark.parametrize("call", [glu, down])
@pytest.mark.parametrize("mode,K", [(1, 180000 // 128 * 128), (1, 196608), (2, 102400), (2, 1 << 20), (1, 1 << 20)])
def test_the_library_takes_them_to_the_kernel_that_holds_none(lib, call, mode, K):
    """Quantized rows of any length are taken by the library's own choice: the
    shape is not what a call without a device fails for."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are of no memory")
    assert call(lib, mode, K, 0) != SHAPE
    assert (call(lib, mode, K, 2) == SHAPE) == (mode * K + K // 8 > 200000)
