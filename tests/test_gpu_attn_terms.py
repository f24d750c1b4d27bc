"""The third bf16 terms of the streaming kernel (queries always, weights where there
is room for few keys): two tokens of one non-zero value each, so that every
product and sum is exact but for what is counted here, and queries picked so
that the third term alone moves the result by far more than that.

Units: x = RN32(q * c), c = scale * log2 e, is what the kernel splits; hi, lo its
bf16 terms, third = x - hi - lo (up to 2^-17 for x in [1, 2)).

Queries.  Keys kappa e_0 and kappa e_1 with kappa = 128, values +1 and -1, so out =
tanh((s0 - s1) / 2) with scores s near 128 to 192 in log2 units, |s0 - s1| < 0.75.
Errors of s0 - s1 (log2 units): x to f32, 2 * 192 * 2^-24 < 2^-15; an MMA that truncates at
2^-22 of its sum, 2 * 192 * 2^-22 < 2^-13 (its products and sums of one value are
exact, so this is generous); the sums of the terms and the difference to the
maximum, 4 * 192 * 2^-24 < 2^-14.  Together below 2^-12 * 0.8; out moves by ln 2 / 2 of it
at most, 6.8e-5, the weights' two terms add 2^-16 and ex2 2^-21: below 2^-13 * 0.72.  Tolerance 2^-13.
The third terms move s0 - s1 by at least 128 * 2^-16.5, out by 2^-9.5 * ln 2 / 2 * (1 - out^2) > 3 tolerances.

Weights.  Keys 0 and -e_0, values 0 and 1: out = p / (1 + p), p = 2^-x, x in (0, 1).
Errors relative to out: ex2.approx 2^-22 and its argument 2^-24 * 2, the weights' sum and the
quotient 2^-24 each, three terms 2^-24: below 2^-21.  Tolerance 2^-20.  Without the third
term the sum of the values lacks at least 2^-18 of p."""
import math

import pytest

torch = pytest.importorskip("torch")

from q8_quantized_gemv_gb300 import build, lk  # noqa: E402

DEV = "cuda"
SCALE = 0.125


def terms(x):
    """bf16 terms hi, lo of f32 values and what they leave, in 64 bits."""
    hi = x.to(torch.bfloat16).float()
    lo = (x - hi).to(torch.bfloat16).float()
    return hi.double(), lo.double(), (x - hi - lo).double()


def split_of(q):
    c = torch.tensor(SCALE, dtype=torch.float32) * torch.tensor(1.44269504088896340736, dtype=torch.float32)
    return q * c


def query_pairs(n, seed):
    """q0, q1 (f32 [n]) and the exact outputs, picked by their third terms."""
    g = torch.Generator()
    g.manual_seed(seed)
    a = (1.05 + 0.4 * torch.rand((400 * n,), generator=g)) / split_of(torch.ones(1))
    b = a * (1 + 0.003 * (2 * torch.rand(a.shape, generator=g) - 1))
    xa, xb = split_of(a), split_of(b)
    (ha, la, ta), (hb, lb, tb) = terms(xa), terms(xb)
    t = ta - tb
    ok = (t.abs() >= 2.0 ** -16.5) & (xa > 1.0) & (xa < 1.5) & (xb > 1.0) & (xb < 1.5)
    a, b = a[ok][:n], b[ok][:n]
    assert a.numel() == n
    want = torch.tanh((a.double() - b.double()) * SCALE * 128 / 2)
    two = torch.tanh(((ha + la) - (hb + lb))[ok][:n] * 128 * math.log(2) / 2)
    assert ((want - two).abs() > 3 * 2.0 ** -13).all()  # a kernel of two terms fails
    return a, b, want


def weight_queries(n, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    a = (0.05 + 0.9 * torch.rand((400 * n,), generator=g)) / split_of(torch.ones(1))
    p = torch.exp2(-split_of(a).double())
    t = terms(p.float())[2] / p
    a = a[t.abs() >= 2.0 ** -18 + 2.0 ** -21][:n]
    assert a.numel() == n
    p = torch.exp(-a.double() * SCALE)
    return a, p / (1 + p)


def test_the_picks():
    """(on the CPU: the picked queries are what the bounds above need)"""
    for seed in range(3):
        query_pairs(76, seed)
        weight_queries(76, seed)


# clusters; the streaming kernel with little room (152 items: no clusters) and with much
PATHS = [("clusters", 4, 1, 1), ("clusters", 40, 1, 1), ("streaming", 76, 2, 1), ("streaming, long", 8, 1, 300)]


def attend(D, n_kv, B, width, q, keys, values):
    """keys, values: [(index, value) or None] of two tokens."""
    page = 64
    k, v = (torch.zeros((1, n_kv, page, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for i in range(2):
        if keys[i]:
            k[0, :, i, keys[i][0]] = keys[i][1]
        v[0, :, i] = values[i]
    cache = lk.KvCache(k, v)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[:, 0] = 0
    lens = torch.full((B,), 2, dtype=torch.int32, device=DEV)
    ws = torch.empty((lk.lk_attn_workspace_bytes(n_kv, n_kv, D, B),), dtype=torch.uint8, device=DEV)
    out = torch.empty((B, n_kv * D), device=DEV)
    lk.lk_attn(cache, q.view(B, -1), table, lens, ws, scale=SCALE, out=out)
    torch.cuda.synchronize()
    launches = lk.lk_attn_launches(cache, n_kv, B, width)
    assert lk.lk_device_error(reset=True) == 0
    return out.view(B, n_kv, D).cpu().double(), launches


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


@pytest.mark.gpu
@pytest.mark.parametrize("path,n_kv,B,width", PATHS)
@pytest.mark.parametrize("D", [64, 128])
def test_third_term_of_the_queries(lib, path, n_kv, B, width, D):
    for i0, i1 in ((0, 1), (9, 30), (D - 1, 33)):
        a, b, want = query_pairs(B * n_kv, 100 + i0)
        q = torch.zeros((B, n_kv, D), device=DEV)
        q[:, :, i0], q[:, :, i1] = a.view(B, n_kv).to(DEV), b.view(B, n_kv).to(DEV)
        out, launches = attend(D, n_kv, B, width, q, [(i0, 128.0), (i1, 128.0)], [1.0, -1.0])
        assert launches == (1 if path == "clusters" else 2)
        err = (out - want.view(B, n_kv, 1)).abs().max().item()
        assert err <= 2.0 ** -13, err


@pytest.mark.gpu
@pytest.mark.parametrize("path,n_kv,B,width", PATHS[:3])
@pytest.mark.parametrize("D", [64, 128])
def test_third_term_of_the_weights(lib, path, n_kv, B, width, D):
    a, want = weight_queries(B * n_kv, 7 + D)
    q = torch.zeros((B, n_kv, D), device=DEV)
    q[:, :, 5] = a.view(B, n_kv).to(DEV)
    out, launches = attend(D, n_kv, B, width, q, [None, (5, -1.0)], [0.0, 1.0])
    assert launches == (1 if path == "clusters" else 2)
    err = ((out / want.view(B, n_kv, 1)) - 1).abs().max().item()
    assert err <= 2.0 ** -20, err
