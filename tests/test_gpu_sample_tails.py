"""Draws from tails that lk_sample (include/lk_sample.h) must not lose, on the GPU: many
tokens far below the largest, whose sum counts though none of them does."""
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


def near(N):
    """How near to a border either side of it may be drawn, as the header says."""
    return 2.0 ** -27 if N <= 1 << 18 else 2.0 ** -26


def shares(logits):
    """Running sums of the weights in 64 bits, the first of them 0."""
    l = logits.astype(np.float64)
    c = np.concatenate([[0.0], np.cumsum(np.exp(l - l.max()))])
    return c


def draw(lk, logits, u, **kept):
    M = logits.shape[0]
    idx, prob = torch.full((M,), -7, dtype=torch.int32, device=DEV), torch.full((M,), math.nan, device=DEV)
    lk.lk_sample(logits, torch.from_numpy(np.asarray(u, np.float32)).to(DEV), idx, prob=prob, **kept)
    return idx.cpu().numpy(), prob.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("N", [5003, 151936, 262144, 1 << 21])
@pytest.mark.parametrize("bits", [20.5, 33.0, 38.9, 40.9, 41.02, 41.2, 42.6, 44.0, 46.9, 48.3, 60.0])
@pytest.mark.parametrize("peak", ["first", "last"])
def test_a_peak_and_a_flat_tail(lk, N, bits, peak):
    """One logit 0, all others 2^-bits below: u just above (below) the peak's share."""
    x = np.full(N, -bits * math.log(2), np.float32)
    at = 0 if peak == "first" else N - 1
    x[at] = 0
    c = shares(x)
    total, tol = c[-1], near(N)
    tail = (N - 1) * float(np.exp(np.float64(x[1])))
    logits = torch.from_numpy(x).to(DEV)[None]
    one = torch.ones((1,), device=DEV)
    us = [1 - 2.0 ** -24, 1 - 2.0 ** -23, 1 - 2.0 ** -22, 1 - 2.0 ** -20, 1 - 2.0 ** -12] if at == 0 else \
        [tail * f / total for f in (0.0, 0.01, 0.3, 0.7, 0.99, 1.01, 2.0)]
    for u in np.float32(us):
        for kept in ({}, dict(min_p=one * 2.0 ** -60), dict(top_k=(one * (N - 1)).int()), dict(top_p=one * (1 - 2.0 ** -24))):
            # (top_k, top_p: some of the tail's last tokens are not kept; what that moves is
            # below the tail's own part that they take)
            cut = tail / (N - 1) if "top_k" in kept else min(tail, 2.0 ** -24 * total) if "top_p" in kept else 0.0
            i, p = draw(lk, logits, [u], **kept)
            i = int(i[0])
            want = min(float(u), 1 - 2.0 ** -24) * total  # (1 and above: as just below it)
            assert c[i] - tol * total - cut <= want <= c[i + 1] + tol * total + cut, (u, kept, i)
            e = 1.0 if i == at else tail / (N - 1)
            assert abs(float(p[0]) / (e / total) - 1) <= 2.0 ** -22 + cut / total, (u, kept, i)


@pytest.mark.parametrize("M,N", [(1, 151936), (64, 151936), (3, 1 << 21)])
def test_draws_up_to_the_last_token(lk, M, N):
    """u of 1 and above: the last token that counts, those aside that come to less than
    the error of the sums together."""
    r = np.random.default_rng(N)
    x = (r.standard_normal((M, N)) * 3 - 20).astype(np.float32)
    x[:, 100] = 0
    for u in (1.0, 2.0, math.inf):
        idx, prob = draw(lk, torch.from_numpy(x).to(DEV), np.full(M, u))
        for t in range(M):
            c = shares(x[t])
            i = int(idx[t])
            assert c[i + 1] >= c[-1] * (1 - near(N)), (t, i)
            assert abs(prob[t] * c[-1] / np.exp(np.float64(x[t, i])) - 1) <= 2.0 ** -22


@pytest.mark.parametrize("N", [151936, 1 << 21])
def test_top_p_ends_in_the_tail(lk, N):
    """top_p just below 1: the shortest beginning ends among equal tokens of the tail,
    whose sum is many times 1 - top_p."""
    x = np.full(N, -30.0 * math.log(2), np.float32)
    x[0] = 0
    c = shares(x)
    logits, one = torch.from_numpy(x).to(DEV)[None], torch.ones((1,), device=DEV)
    for short in (2.0 ** -24, 2.0 ** -20, 2.0 ** -17, 2.0 ** -14):
        p = 1 - short
        if p * c[-1] <= 1:
            continue
        i, _ = draw(lk, logits, [1.0], top_p=one * p)
        # the last token kept
        want = int(np.searchsorted(c, p * c[-1], "left")) - 1
        assert abs(c[int(i[0]) + 1] - c[want + 1]) <= 2 * near(N) * c[-1], (short, int(i[0]), want)
