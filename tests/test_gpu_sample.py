"""The drawn token (include/lk_sample.h) on the GPU, against its definition in
64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moehelp import U, sample_ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
# sums of whole numbers of 2^-39 of at most 2^18 terms, e to 2^-32: a border this near may go either way
NEAR = 2.0 ** -28


@pytest.fixture(scope="module")
def lk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_gemv_gb300 import build, lk
    build.build()
    yield lk
    assert lk.lk_device_error(reset=True) == 0


def draw(lk, logits, u, cfg=None, **settings):
    M = logits.shape[0]
    idx = torch.full((M,), -7, dtype=torch.int32, device=DEV)
    prob = torch.full((M,), math.nan, device=DEV)
    d = {k: torch.from_numpy(np.asarray(v)).to(DEV) for k, v in settings.items()}
    lk.lk_sample(torch.from_numpy(logits).to(DEV), torch.from_numpy(u).to(DEV), idx, prob=prob, cfg=cfg, **d)
    return idx.cpu().numpy(), prob.cpu().numpy().astype(np.float64)


def check(lk, logits, u, near=0, **s):
    """near: how many rows may have a border within NEAR (either side is then right)."""
    M = logits.shape[0]
    u = np.asarray(u, np.float32)
    s = {k: np.asarray(v, np.int32 if k == "top_k" else np.float32) for k, v in s.items()}
    idx, prob = draw(lk, logits, u, **s)
    for t in range(M):
        g = lambda n, off: s[n][t].item() if n in s else off  # noqa: E731
        i, p, margin = sample_ref(logits[t], g("temperature", 1.0), g("top_k", 0), g("top_p", 1.0), g("min_p", 0.0),
                                  float(u[t]))
        if margin < NEAR:
            near -= 1
            assert near >= 0, f"row {t}: the case itself is undecided ({margin})"
            continue
        assert idx[t] == i, (t, idx[t], i, p, prob[t])
        assert abs(prob[t] - p) <= 2.0 ** -22 * p, (t, prob[t], p)


def vocab(M, N, seed, spread=1.0):
    r = np.random.default_rng(seed)
    rank = np.argsort(r.random((M, N)), 1) + 1.0
    return (spread * (r.standard_normal((M, N)) - 1.1 * np.log(rank)) + 12).astype(np.float32)


@pytest.mark.parametrize("N", [1, 2, 31, 33, 1000, 1024, 4097, 32003, 151936])
@pytest.mark.parametrize("M", [1, 5, 64])
def test_settings(lk, M, N):
    M = min(M, max(5, (1 << 21) // N))
    logits = vocab(M, N, N + M)
    r = np.random.default_rng(N)
    u = r.random(M).astype(np.float32)
    one = np.ones(M)
    check(lk, logits, u)
    check(lk, logits, u, temperature=0.3 + r.random(M))
    check(lk, logits, u, top_k=r.integers(0, 60, M))
    check(lk, logits, u, top_k=(N // 3) * one, temperature=2 * one)
    check(lk, logits, u, top_p=r.random(M))
    check(lk, logits, u, near=1, top_p=0.999 * one, temperature=1.5 * one)
    check(lk, logits, u, min_p=0.3 * r.random(M))
    check(lk, logits, u, temperature=0.2 + 2 * r.random(M), top_k=r.integers(0, 3000, M), top_p=r.random(M) * 1.1,
          min_p=0.1 * r.random(M))


def test_flat_and_narrow(lk):
    """Nearly equal logits: every token counts, and the borders lie in the middle
    of a crowd; logits that only their last bits tell apart."""
    M, N = 8, 50000
    r = np.random.default_rng(5)
    u = r.random(M).astype(np.float32)
    flat = (0.01 * r.standard_normal((M, N))).astype(np.float32)
    narrow = (np.float32(3.0) + np.float32(2.0 ** -22) * r.integers(0, 5, (M, N)).astype(np.float32)).astype(np.float32)
    for x in (flat, narrow, vocab(M, N, 6, spread=0.2)):
        check(lk, x, u, near=1)
        check(lk, x, u, near=1, top_k=r.integers(1, N, M))
        check(lk, x, u, near=2, top_p=0.1 + 0.85 * r.random(M))
        check(lk, x, u, near=2, top_k=r.integers(20000, N, M), top_p=0.1 + 0.85 * r.random(M))


@pytest.mark.parametrize("N", [7, 5000, 131072])
def test_equal_logits(lk, N):
    """All equal: what top_k and top_p keep is a beginning of the vocabulary."""
    M = 6
    logits = np.full((M, N), -3.25, np.float32)
    u = np.float32([0, 0.123, 0.5, 0.777, 0.9999, 0.25])
    idx, prob = draw(lk, logits, u)
    for t in range(M):  # exactly: the weights are equal
        assert idx[t] == int(np.float64(u[t]) * N) and abs(prob[t] * N - 1) < 2.0 ** -22
    k = np.minimum([1, 2, 3, 1000, 4097, N], N)
    check(lk, logits, u, near=6, top_k=k)
    idx, prob = draw(lk, logits, u, top_k=k.astype(np.int32))
    for t in range(M):
        assert idx[t] == int(np.float64(u[t]) * k[t]) and abs(prob[t] * k[t] - 1) < 2.0 ** -22
    idx, _ = draw(lk, logits, u, top_p=np.full(M, 0.6, np.float32))
    kept = math.ceil(float(np.float32(0.6)) * N)
    assert [int(v) for v in idx] == [int(np.float64(v) * kept) for v in u]


def test_edges(lk):
    inf, nan, low = np.inf, np.nan, np.finfo(np.float32).min
    N = 300
    base = np.random.default_rng(1).standard_normal(N).astype(np.float32)
    rows = []

    def row(**at):
        x = base.copy()
        for k, v in at.items():
            x[int(k[1:])] = v
        rows.append(x)
    row()
    rows.append(np.full(N, -inf, np.float32))            # nothing to draw
    rows.append(np.full(N, nan, np.float32))
    row(i5=inf)                                          # the largest f32
    row(i5=inf, i9=inf)
    x = np.full(N, -inf, np.float32)
    x[17] = -3
    rows.append(x)                                       # one token
    rows.append(np.full(N, low, np.float32))             # the type's lowest value
    x = base.copy()
    x[::2], x[1::4] = -inf, nan
    rows.append(x)
    x = base.copy()
    x[100:] = low
    rows.append(x)
    x = np.full(N, 0.0, np.float32)
    x[::3] = -0.0
    rows.append(x)
    logits = np.stack(rows)
    M = len(rows)
    one = np.ones(M)
    u = np.linspace(0.02, 0.97, M)
    for s in ({}, dict(top_k=3 * one), dict(top_p=0.5 * one), dict(min_p=0.2 * one), dict(min_p=one), dict(min_p=7 * one),
              dict(top_k=N * one), dict(top_k=-1 * one), dict(top_k=one), dict(top_p=0 * one), dict(top_p=1e-12 * one),
              dict(top_p=-1 * one), dict(top_p=one), dict(top_p=5 * one), dict(temperature=0 * one),
              dict(temperature=-1 * one), dict(temperature=nan * one), dict(temperature=1e-30 * one),
              dict(temperature=1e-4 * one), dict(temperature=1e4 * one), dict(top_p=nan * one), dict(min_p=nan * one)):
        if "top_p" in s and np.isnan(s["top_p"]).all() or "min_p" in s and np.isnan(s["min_p"]).all():
            assert np.array_equal(draw(lk, logits, np.float32(u), **{k: np.float32(v) for k, v in s.items()})[0],
                                  draw(lk, logits, np.float32(u))[0])  # off
            continue
        check(lk, logits, u, near=3, **s)
    for v in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0):
        check(lk, logits, np.full(M, v), near=M if v == 1.0 - 2.0 ** -24 else 0)
    assert np.array_equal(draw(lk, logits, np.full(M, nan, np.float32))[0], draw(lk, logits, np.zeros(M, np.float32))[0])


def test_shares(lk):
    """As many draws as there are probabilities for: evenly spaced u give each
    token its share, to one draw."""
    N, M = 8, 64
    x = np.tile(np.float32([0, 1, 2, -1, 0.5, -5, 1.5, 0.25]), (M, 1))
    p = np.exp(x[0].astype(np.float64))
    p /= p.sum()
    n = 64 * M
    count = np.zeros(N)
    for r in range(64):
        u = (np.arange(r * M, (r + 1) * M) + 0.5) / n
        idx, prob = draw(lk, x, u.astype(np.float32))
        assert np.all(np.abs(prob / p[idx] - 1) < 2.0 ** -22)
        count += np.bincount(idx, minlength=N)
    assert np.all(np.abs(count - n * p) <= 1 + 1e-6)


@pytest.mark.parametrize("M", [1, 9, 17, 19, 33, 40])
def test_rows_of_any_alignment(lk, M):
    """Row counts that take clusters of every size, rows that begin at any
    multiple of 4 bytes, and tokens masked with -inf and the type's lowest value."""
    N = 20001
    r = np.random.default_rng(M)
    flat = np.concatenate([np.float32([7]), vocab(1, M * N, M)[0]])
    flat[r.integers(0, flat.size, flat.size // 4)] = -np.inf
    flat[r.integers(0, flat.size, flat.size // 8)] = np.finfo(np.float32).min
    u = r.random(M).astype(np.float32)
    for shift in (0, 1):
        logits = flat[shift:shift + M * N].reshape(M, N)
        x = torch.from_numpy(flat).to(DEV)[shift:shift + M * N].view(M, N)
        idx, tp = torch.zeros((M,), dtype=torch.int32, device=DEV), torch.full((M,), 0.9, device=DEV)
        lk.lk_sample(x, torch.from_numpy(u).to(DEV), idx, top_p=tp)
        near = 0
        for t in range(M):
            i, _, margin = sample_ref(logits[t], 1.0, 0, float(np.float32(0.9)), 0.0, float(u[t]))
            near += margin < NEAR
            assert margin < NEAR or int(idx[t]) == i
        assert near <= 1


@pytest.mark.parametrize("N", [32767, 32768, 50001, 98305, 600011])
@pytest.mark.parametrize("M", [1, 3])
def test_few_rows_in_many_blocks(lk, M, N):
    """Rows that most blocks share, from the fewest tokens a block to the most warps."""
    logits = vocab(M, N, N)
    logits[:, ::5] = np.round(logits[:, ::5])
    r = np.random.default_rng(N)
    u, one = r.random(M), np.ones(M)
    check(lk, logits, u, near=1)
    check(lk, logits, u, near=1, top_k=40 * one, top_p=0.9 * one)
    check(lk, logits, u, near=1, top_k=(N // 2) * one, min_p=1e-4 * one)
    check(lk, logits, u, near=1, top_p=0.97 * one, temperature=1.3 * one)


def test_largest_row(lk):
    """As many logits as a row may have, and tokens a bin too many to count."""
    N = 1 << 21
    x = torch.full((2, N), -2.0, device=DEV)
    x[0, 5::7] = 1.0
    x[1, 11] = 30.0
    x[1, N - 1] = 30.0
    idx, prob = torch.zeros((2,), dtype=torch.int32, device=DEV), torch.zeros((2,), device=DEV)
    u = torch.tensor([0.5, 0.75], device=DEV)
    lk.lk_sample(x, u, idx, prob=prob, top_k=torch.tensor([100000, 0], dtype=torch.int32, device=DEV),
                 top_p=torch.tensor([0.5, 0.9], device=DEV))
    # row 0: the first 100000 of the equal largest, of these 50000, of these the one at half
    assert idx.tolist() == [5 + 7 * 25000, N - 1]
    assert abs(float(prob[0]) * 50000 - 1) < 2.0 ** -22 and abs(float(prob[1]) * 2 - 1) < 2.0 ** -22
    with pytest.raises(lk.LkError) as err:
        lk.lk_sample(torch.zeros((1, N + 1), device=DEV), u[:1], idx[:1])
    assert err.value.status == -3


def test_two_streams_at_once(lk):
    M, N = 12, 30011
    sets = [(torch.from_numpy(vocab(M, N, s)).to(DEV), torch.rand((M,), device=DEV), torch.zeros((M,), dtype=torch.int32, device=DEV))
            for s in range(2)]
    tk = torch.full((M,), 80, dtype=torch.int32, device=DEV)
    want = []
    for x, u, idx in sets:
        lk.lk_sample(x, u, idx, top_k=tk)
        want.append(idx.clone())
        idx.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for st, (x, u, idx) in zip(streams, sets):
            lk.lk_sample(x, u, idx, top_k=tk, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(idx, w) for (_, _, idx), w in zip(sets, want))


def test_captured(lk):
    """A captured call behind the launch that writes its logits, dependent, its
    inputs changed between replays; the same bits as a call alone."""
    M, N = 7, 20011
    src = torch.zeros((M, N), device=DEV)
    logits, u = torch.zeros((M, N), device=DEV), torch.zeros((M,), device=DEV)
    idx, prob = torch.zeros((M,), dtype=torch.int32, device=DEV), torch.zeros((M,), device=DEV)
    tk = torch.full((M,), 50, dtype=torch.int32, device=DEV)
    tp = torch.full((M,), 0.9, device=DEV)
    cfg = lk.launch_cfg(pdl=1)

    def step():
        torch.add(src, 0.0, out=logits)
        lk.lk_sample(logits, u, idx, prob=prob, top_k=tk, top_p=tp, cfg=cfg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(3):
                step()
        for seed in range(10):
            x = vocab(M, N, 50 + seed)
            r = np.random.default_rng(seed).random(M).astype(np.float32)
            src.copy_(torch.from_numpy(x))
            u.copy_(torch.from_numpy(r))
            graph.replay()
            got, p = idx.clone(), prob.clone()
            side.synchronize()
            want, wp = draw(lk, x, r, top_k=np.full(M, 50, np.int32), top_p=np.full(M, 0.9, np.float32))
            assert got.tolist() == want.tolist() and p.cpu().numpy().astype(np.float64).tolist() == wp.tolist()
    torch.cuda.current_stream().wait_stream(side)
