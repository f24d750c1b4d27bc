"""Routing (lk_moe_route) on the GPU where f32's errors are as large as they get: the
choices are those of the scores in 64 bits all the same."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moehelp import route_ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def lk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_gemv_gb300 import build, lk
    build.build()
    yield lk
    assert lk.lk_device_error(reset=True) == 0


def route(lk, logits, bias, k, **kw):
    M = logits.shape[0]
    ids = torch.full((M, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((M, k), math.nan, device=DEV)
    lk.lk_moe_route(torch.from_numpy(logits).to(DEV), ids, w,
                    bias=None if bias is None else torch.from_numpy(bias).to(DEV), **kw)
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("where", [0.97, 0.98, 0.99])
def test_softmax_whose_sum_loses_the_most(lk, where):
    """1024 experts: one with e = 1, and others whose e or whose lanes' sums are just under half
    a step of what they are added to, each time (31 in a lane, 5 between lanes).  The sum
    is off by nearly 36 half steps, and s + bias of two experts is rounded towards each
    other's place."""
    E, t = 1024, U * (1 - 2.0 ** -10)
    l = np.full((1, E), -80.0, np.float32)
    l[0, 0] = 0
    l[0, 32::32] = math.log(t)
    l[0, [2, 4, 8, 16]] = math.log(t)
    l[0, 1] = math.log(t / 2)
    l[0, 3] = math.log(0.49 * U)
    C = round(where * 2.0 ** 24) * U
    bias = np.full(E, -5.0, np.float32)
    bias[0] = C + 0.5625 * U - 1  # 1 + bias: rounded up to C + U
    bias[3] = C - 35 * U        # s + bias: rounded down to it
    s = np.exp(l[0].astype(np.float64))
    s /= s.sum()
    c = s + bias
    assert 0 < c[3] - c[0] < 1.5 * U  # f32 has it 36 half steps the other way round
    want, ww, gap = route_ref(l, bias, "softmax", 1, 1, 1, 2, True, 1.0)
    assert want[0].tolist() == [3, 0] and gap > 1e-9
    for k in (1, 2):
        ids, _ = route(lk, l, bias, k)
        assert ids[0].tolist() == want[0, :k].tolist()


def test_group_sums_of_biases_of_both_signs(lk):
    """A group's value is small, what it is the sum of is not: s + bias is rounded at the
    bias's size."""
    # equal scores, 2^-10 each; 1 + 2^-11 and odd half steps more: rounded down, rounded up
    E = 1024
    l, bias = np.zeros((1, E), np.float32), np.full(E, -5.0, np.float32)
    b = -round(0.99 * 2.0 ** 24) * U
    bias[[0, 1]] = 1 - 2.0 ** -11 + U, b + 3 * U
    bias[[512, 513]] = 1 - 2.0 ** -11 + 3 * U, b
    s = 2.0 ** -10 + bias.astype(np.float64)
    assert s[0] + s[1] == s[512] + s[513] + U
    ids, _ = route(lk, l, bias, 2, n_group=2, top_group=1, group_sum=2)
    assert ids[0].tolist() == [0, 1]
    # sigmoids; the f32 sums (a step of 100 is 2^-17) are off by more than they differ
    for l in ([-0.33351847529411316, -0.1987764537334442, 0.09946588426828384, -0.6499243974685669],
              [1.0161256790161133, 0.02421480044722557, -0.8853384852409363, 2.907092809677124],
              [-0.3497023582458496, 0.5829254984855652, 0.22258533537387848, -0.0008985933382064104]):
        l, bias = np.array([l], np.float32), np.float32([100, -100, 100, -100])
        want, _, gap = route_ref(l, bias, "sigmoid", 2, 1, 2, 2, True, 1.0)
        assert gap > 1e-9 and want[0].tolist() == [0, 1]
        ids, _ = route(lk, l, bias, 2, score="sigmoid", n_group=2, top_group=1, group_sum=2)
        assert ids[0].tolist() == [0, 1]
