"""Sums of many small weights in lk_sample (include/lk_sample.h) on the GPU: a peak
and as much again in a flat tail far below it, whose weights are alike, so that what
their sum leaves out does not average out."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moehelp import sample_ref  # noqa: E402

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


@pytest.mark.parametrize("M,N", [(64, 151936), (1, 151936), (2, 1 << 21), (64, 32003)])
@pytest.mark.parametrize("weight", [0.98 * 2.0 ** -16, 0.77 * 2.0 ** -17, 0.93 * 2.0 ** -20, 2.0 ** -10.3])
def test_probabilities_over_a_flat_tail(lk, M, N, weight):
    """prob is within 2^-22 (its own roundings; those of e and of the sum are below 2^-27):
    of the peak, drawn at u 0, and of a token of the tail."""
    logits = torch.full((M, N), float(np.float32(np.log(weight))), device=DEV)
    logits[:, 0] = 0
    w = np.exp(np.float64(np.float32(np.log(weight))))
    total = 1 + (N - 1) * w
    one = torch.ones((M,), device=DEV)
    for kept in ({}, dict(min_p=one * (0.5 * weight)), dict(top_p=one * 2), dict(top_k=(one * (N - 1)).int()),
                 dict(top_p=one * 0.75)):
        z = total - (w if "top_k" in kept else 0)
        if kept.get("top_p") is not None and float(kept["top_p"][0]) < 1:
            # the peak and as many of the tail as reach it: to a token or two by their sum's error
            n = max(0.0, np.ceil((0.75 * total - 1) / w))
            z = 1 + n * w
        room = 2.0 ** -22 + (2 * w / z if "top_p" in kept else 0)
        for u, p in ((0.0, 1 / z), (0.999, w / z)):
            if u > 0 and 0.999 * z < 1:
                continue  # (the peak's too)
            idx, prob = torch.zeros((M,), dtype=torch.int32, device=DEV), torch.zeros((M,), device=DEV)
            lk.lk_sample(logits, one * u, idx, prob=prob, **kept)
            assert bool((idx == 0).all()) == (u == 0), kept
            assert float((prob.double() / p - 1).abs().max()) <= room, (u, kept)


@pytest.mark.parametrize("M,N", [(64, 151936), (1, 151936), (2, 1 << 21)])
def test_sums_beside_a_border(lk, M, N):
    """The same tail above a border that lies among other tokens still: its sum is taken
    in one piece, without being sorted."""
    r = np.random.default_rng(N)
    x = np.empty((M, N), np.float32)
    x[:, ::2] = np.log(0.98 * 2.0 ** -16)
    x[:, 1::2] = -np.log(2) * r.uniform(25, 40, (M, N // 2))
    x[:, 0] = 0
    logits, one = torch.from_numpy(x).to(DEV), torch.ones((M,), device=DEV)
    w = -np.sort(-np.exp(x.astype(np.float64)), 1)
    c = np.cumsum(w, 1)
    for kept in (dict(top_k=(one * (N // 2 + N // 4)).int()), dict(top_p=one * (1 - 2.0 ** -16)),
                 dict(top_p=one * (1 - 2.0 ** -16), min_p=one * 2.0 ** -17)):
        idx, prob = torch.zeros((M,), dtype=torch.int32, device=DEV), torch.zeros((M,), device=DEV)
        lk.lk_sample(logits, one * 0, idx, prob=prob, **kept)
        assert bool((idx == 0).all())
        for t in range(M):
            n = N // 2 + N // 4
            if "top_p" in kept:
                n = int(np.searchsorted(c[t], (1 - 2.0 ** -16) * c[t, -1], "left")) + 1
                assert N // 2 < n < N
            if "min_p" in kept:
                n = N // 2
            # (a token at top_p's border more or less is 2^-25)
            assert abs(float(prob[t]) * c[t, n - 1] - 1) <= 2.0 ** -22


@pytest.mark.parametrize("M,N", [(1, 151936), (64, 32003), (17, 5003), (64, 151936)])
def test_min_p_at_every_place_of_the_order(lk, M, N):
    """min_p's border before top_k's and top_p's, behind them, and beside them, where the
    bins of the order do not tell them apart; at a token's own weight too."""
    r = np.random.default_rng(M + N)
    x = (3 * r.standard_normal((M, N))).astype(np.float32)
    logits, order = torch.from_numpy(x).to(DEV), np.argsort(-x, 1, kind="stable")
    f = lambda v: torch.from_numpy(np.asarray(v, np.float32)).to(DEV)  # noqa: E731
    u = r.random(M).astype(np.float32)
    e = np.exp(x.astype(np.float64) - x.max(1, keepdims=True).astype(np.float64))
    k = np.full(M, min(3000, N // 2), np.int32)
    p = np.full(M, 0.97, np.float32)
    near = np.stack([e[t, order[t, k[t] - 1]] for t in range(M)])
    c = np.cumsum(np.take_along_axis(e, order, 1), 1)
    last = np.array([np.searchsorted(c[t], 0.97 * c[t, -1]) for t in range(M)])
    at_p = np.stack([e[t, order[t, last[t]]] for t in range(M)])
    undecided = drawn = 0
    for least in (near, near * (1 - 1e-3), near * (1 + 1e-3), near * 1.02, at_p, at_p * (1 + 2e-4), at_p * 0.98, 0 * at_p + 1e-9,
                  0 * at_p + 0.3, 0 * at_p + 1, np.sqrt(near), near * near):
        for kept in (dict(top_k=k), dict(top_p=p), dict(top_k=k, top_p=p), {}):
            least = least.astype(np.float32)
            idx, prob = torch.zeros((M,), dtype=torch.int32, device=DEV), torch.zeros((M,), device=DEV)
            lk.lk_sample(logits, f(u), idx, prob=prob, min_p=f(least), **{n: torch.from_numpy(v).to(DEV) for n, v in kept.items()})
            for t in range(0, M, max(1, M // 8)):
                i, q, margin = sample_ref(x[t], 1.0, int(k[t]) if "top_k" in kept else 0, float(p[t]) if "top_p" in kept else 1.0,
                                          float(least[t]), float(u[t]))
                drawn += 1
                if margin < 2.0 ** -27:
                    undecided += 1
                    continue
                assert int(idx[t]) == i and abs(float(prob[t]) - q) <= 2.0 ** -22 * q, (t, list(kept), float(least[t]))
    # (min_p at a token's weight rounded to f32 is 2^-25 from it on the mean, one case in four within
    # the margin: of the six pairs of twelve that are such, and hardly any other)
    assert undecided < drawn / 4


@pytest.mark.parametrize("M", [1, 64])
def test_the_largest_sums(lk, M):
    """2^21 equal logits, whose sum is the most that whole numbers of 64 bits are asked
    to hold, in many blocks and in as few as there are: the token is u's share of the row, exactly."""
    N = 1 << 21
    logits = torch.full((M, N), 2.5, device=DEV)
    logits[::2] = -7
    idx, prob = torch.zeros((M,), dtype=torch.int32, device=DEV), torch.zeros((M,), device=DEV)
    for r in range(3):
        u = (torch.arange(M, device=DEV, dtype=torch.float64) * 0.0153 + 0.31 * r).float()
        u[-1] = (0.0, 0.5, 1 - 2.0 ** -24)[r]
        lk.lk_sample(logits, u, idx, prob=prob)
        assert torch.equal(idx.long(), (u.double() * N).floor().long().clamp(max=N - 1))
        assert float((prob.double() * N - 1).abs().max()) <= 2.0 ** -22
