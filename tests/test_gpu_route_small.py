"""Routing weights (lk_moe_route) on the GPU of scores far below 1."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

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


def route(lk, logits, k, **kw):
    M = logits.shape[0]
    ids = torch.full((M, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((M, k), math.nan, device=DEV)
    lk.lk_moe_route(torch.from_numpy(logits).to(DEV), ids, w, **kw)
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def near(got, want):
    """Within 2^-15 relatively, 2^-126 below f32's normal range."""
    return np.all(np.abs(got - want) <= 2.0 ** -15 * np.abs(want) + 2.0 ** -126)


@pytest.mark.parametrize("top", [-30.0, -90.0, -150.0, -700.0, -707.5])
def test_sigmoids_over_their_sum(lk, top):
    """Of the k chosen, by their logits' differences: exp(l) / (1 + exp(l)) is as good as exp(l)
    there, and its quotients need no range."""
    r = np.random.default_rng(1)
    logits = (top - 3 * np.arange(24)[None] - r.random((5, 24))).astype(np.float32)
    logits = r.permuted(logits, axis=1)
    for k in (1, 8, 24):
        ids, w = route(lk, logits, k, score="sigmoid", scale=2.5)
        for t in range(5):
            order = np.argsort(-logits[t], kind="stable")[:k]
            assert ids[t].tolist() == order.tolist()
            l = logits[t, order].astype(np.float64)
            e = np.exp(l - l[0]) / (1 + np.exp(l))
            # (of logits below -708 alone: zeros, see the next test)
            assert near(w[t], 2.5 * e / e.sum() if l[0] >= -708 else 0 * e), (t, k)


def test_sigmoids_below_64_bits(lk):
    """Where the range of 64 bits holds none of the chosen sigmoids, they count as zeros."""
    logits = np.float32([[-709, -720, -1000, np.finfo(np.float32).min]])
    ids, w = route(lk, logits, 3, score="sigmoid")
    assert ids[0].tolist() == [0, 1, 2] and w[0].tolist() == [0, 0, 0]
    logits[0, 3] = -700  # (one that it holds)
    ids, w = route(lk, logits, 3, score="sigmoid")
    e = np.exp(np.float64([0, -9, -20]))
    assert ids[0].tolist() == [3, 0, 1] and near(w[0], e / e.sum())


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("scale", [1.0, 2.5, 1e10, -1e20, 1e30])
def test_scores_below_32_bits_times_a_scale(lk, score, renorm, scale):
    """scale brings scores that f32 does not hold back into its range."""
    logits = np.float32([[1.0, -60.0, -86.0, -88.0, -92.0, -100.0, -120.0, -145.0, -1e4, np.finfo(np.float32).min]])
    l = logits[0].astype(np.float64)
    if score == "softmax":
        s = np.exp(l - l.max())
        s /= s.sum()
    else:
        s = np.array([1 / (1 + math.exp(-x)) if x > -700 else 0.0 for x in l])
    if renorm:
        s /= s.sum()
    ids, w = route(lk, logits, 10, score=score, renorm=renorm, scale=scale)
    assert ids[0].tolist() == list(range(10))
    assert near(w[0], float(np.float32(scale)) * s)
