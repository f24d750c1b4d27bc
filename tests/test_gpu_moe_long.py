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
