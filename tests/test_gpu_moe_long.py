"""The experts' products (include/lk_moe.h) on rows longer than a block's shared
memory holds, on the GPU."""
import math

import pytest

torch = pytest.importorskip("torch")

from moehelp import acts_of, as_h, down_ref, experts, glu_ref, quantize  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def lk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_gemv_gb300 import build, lk
    build.build()
    yield lk
    assert lk.lk_device_error(reset=True) == 0


def rows(n, K, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn((n, K), generator=g, device=DEV)


@pytest.mark.parametrize("mode", ["int8act", "twopass"])
@pytest.mark.parametrize("M", [1, 6])
def test_down_where_the_activations_do_not_fit(lk, mode, M):
    """k rows of 24576: the library's choice takes the kernel that holds none of
    them, for one row as for many."""
    E, k, N, F, m = 16, 8, 256, 24576, lk.MODES[mode]
    down = experts(E, N, F, 1, DEV)
    ids = torch.stack([torch.randperm(E, device=DEV)[:k] for _ in range(M)]).to(torch.int32)
    acts, w = quantize(rows(M * k, F, 2), m), torch.rand((M, k), device=DEV)
    got = []
    for path in (0, 3):
        y = torch.full((M, N), math.nan, device=DEV)
        lk.lk_moe_down_q8(lk.Experts(down=down), m, ids, w, y, cfg=lk.launch_cfg(path=path), **as_h(acts))
        got.append(y)
    want, tol = down_ref(down, acts, m, ids, w, E)
    assert torch.equal(*got) and bool(((got[0].double() - want).abs() <= tol).all())
    with pytest.raises(lk.LkError) as err:
        lk.lk_moe_down_q8(lk.Experts(down=down), m, ids, w, got[0], cfg=lk.launch_cfg(path=2), **as_h(acts))
    assert err.value.status == -3


@pytest.mark.parametrize("mode", ["int8act", "twopass"])
def test_gate_up_where_the_row_does_not_fit(lk, mode):
    M, E, k, F, K, m = 1, 3, 2, 128, 196608, lk.MODES[mode]
    gate, up = experts(E, F, K, 1, DEV), experts(E, F, K, 2, DEV)
    acts, ids = acts_of(rows(M, K, 3), m), torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    h = torch.full((M * k, F), math.nan, device=DEV)
    lk.lk_moe_glu_q8(lk.Experts(gate=gate, up=up), m, ids, h, **acts)
    want, tol = glu_ref(gate, up, acts, m, ids, E)
    assert bool(((h.double() - want).abs() <= tol).all())


def test_dequant_sums_over_many_slices(lk):
    """Equal products, so that every slice's sum is the same and rounds the same way when
    it is added: 4 x, 8 x and a lane's sums of them, and those of the lanes, are exact in
    f32, the sum over the 98 slices is not (plain f32: 25 half steps off).  One rounding
    is left where its rest is kept."""
    F, N = 49920, 128
    x = 0x29CBF8 * 2.0 ** -21
    h = torch.full((1, F), x, device=DEV)
    down = (torch.ones((1, N, F), dtype=torch.int8, device=DEV), torch.ones((1, N, F // 32), dtype=torch.float16, device=DEV))
    ids, w, y = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones((1, 1), device=DEV), torch.empty((1, N), device=DEV)
    lk.lk_moe_down_q8(lk.Experts(down=down), "dequant", ids, w, y, h=h)
    assert float((y.double() / (F * x) - 1).abs().max()) <= 2 * 2.0 ** -24
    gate = (torch.ones((1, N, F), dtype=torch.int8, device=DEV), down[1])
    hh = torch.empty((1, N), device=DEV)
    lk.lk_moe_glu_q8(lk.Experts(gate=gate, up=gate), "dequant", ids, hh, x=h * 2.0 ** -17)
    g = torch.tensor(F * x * 2.0 ** -17, dtype=torch.float64)
    want = float(g * torch.sigmoid(g) * g)
    # (the two products, an exponential of 2 units, three operations)
    assert float((hh.double() / want - 1).abs().max()) <= 12 * 2.0 ** -24


@pytest.mark.parametrize("K", [4224, 8192, 16384, 24704, 32768, 40064, 49920])
def test_dequant_of_one_sign(lk, K):
    """Products of one sign, where roundings add up: within 1e-5 of the sum, as lk_gemv_q8's."""
    E, k, R = 2, 1, 256
    gate, up, down = (experts(E, R, K, s, DEV) for s in (1, 2, 3))
    for q, s in (gate, up, down):
        q.abs_()
    ids, w = torch.tensor([[1]], dtype=torch.int32, device=DEV), torch.ones((1, 1), device=DEV)
    x = rows(1, K, K).abs()
    h, y = torch.empty((1, R), device=DEV), torch.empty((1, R), device=DEV)
    lk.lk_moe_glu_q8(lk.Experts(gate=gate, up=up), "dequant", ids, h, x=x)
    want, tol = glu_ref(gate, up, {"x": x}, lk.LK_DEQUANT, ids, E)
    assert bool(((h.double() - want).abs() <= tol).all())
    lk.lk_moe_down_q8(lk.Experts(down=down), "dequant", ids, w, y, h=x)
    want, tol = down_ref(down, {"x": x}, lk.LK_DEQUANT, ids, w, E)
    assert bool(((y.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("K", [1024, 8192])
def test_dequant_past_f32(lk, K):
    """Sums that pass f32's range are infinite, whether a row is one slice or several."""
    q = torch.ones((1, 128, K), dtype=torch.int8, device=DEV)
    s = torch.ones((1, 128, K // 32), dtype=torch.float16, device=DEV)
    ids, w, y = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones((1, 1), device=DEV), torch.empty((1, 128), device=DEV)
    h = torch.full((1, K), 1e36, device=DEV)
    lk.lk_moe_down_q8(lk.Experts(down=(q, s)), "dequant", ids, w, y, h=h)
    assert bool((y == math.inf).all())
    lk.lk_moe_down_q8(lk.Experts(down=(q, s)), "dequant", ids, w, y, h=-h)
    assert bool((y == -math.inf).all())
