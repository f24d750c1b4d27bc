"""Routing and the experts' products (include/lk_moe.h) on the GPU, against their
definitions in 64 bits, and bit for bit against lk_gemv_q8's products."""
import itertools
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moehelp import U, acts_of, as_h, down_ref, experts, glu_ref, quantize, route_ref  # noqa: E402

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


# ---- routing -----------------------------------------------------------------------

def route(lk, logits, bias, k, **kw):
    M = logits.shape[0]
    ids = torch.full((M, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((M, k), math.nan, device=DEV)
    lk.lk_moe_route(torch.from_numpy(logits).to(DEV), ids, w,
                    bias=None if bias is None else torch.from_numpy(bias).to(DEV), **kw)
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def check_route(lk, logits, bias, k, score="softmax", n_group=1, top_group=1, group_sum=1, renorm=True, scale=1.0):
    ids, w = route(lk, logits, bias, k, score=score, n_group=n_group, top_group=top_group, group_sum=group_sum,
                   renorm=renorm, scale=scale)
    want, ww, gap = route_ref(logits, bias, score, n_group, top_group, group_sum, k, renorm, scale)
    # two f64 evaluations of a value may differ by a few of its last places
    assert gap > 1e-13, "the case itself is undecided"
    assert np.array_equal(ids, want)
    assert np.all(np.abs(w - ww) <= 2.0 ** -15 * np.abs(ww) + 2.0 ** -120)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("M,E,k,groups", [(1, 1, 1, (1, 1, 1)), (1, 128, 8, (1, 1, 1)), (64, 256, 8, (8, 4, 2)),
                                          (33, 60, 4, (1, 1, 1)), (5, 160, 6, (8, 3, 1)), (7, 257, 32, (1, 1, 1)),
                                          (3, 1024, 17, (32, 5, 2)), (2, 33, 32, (3, 2, 2)), (64, 8, 2, (4, 2, 1)),
                                          (4, 96, 8, (1, 1, 2))])
def test_route(lk, score, with_bias, M, E, k, groups):
    r = np.random.default_rng(E * 64 + M)
    logits = (1.5 * r.standard_normal((M, E))).astype(np.float32)
    bias = (0.1 * r.standard_normal(E)).astype(np.float32) if with_bias else None
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        check_route(lk, logits, bias, k, score, *groups, renorm=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_decided_in_f64(lk, score):
    """s + bias of all experts within 2^-24 of each other: f32 cannot tell."""
    r = np.random.default_rng(3)
    E = 128
    logits = r.standard_normal((1, E)).astype(np.float32)
    l = logits[0].astype(np.float64)
    s = np.exp(l - l.max()) / np.exp(l - l.max()).sum() if score == "softmax" else 1 / (1 + np.exp(-l))
    bias = (0.5 - s).astype(np.float32)
    c = s + bias.astype(np.float64)
    assert np.ptp(c) < 2.0 ** -23 and np.ptp(c) > 0
    check_route(lk, logits, bias, 8, score)
    check_route(lk, logits, bias, 4, score, 4, 2, 2)
    check_route(lk, np.repeat(logits, 64, 0), bias, 16, score, 8, 3, 1)


def test_route_group_sums_decided_in_f64(lk):
    """Without a bias: groups whose two largest scores sum to nearly the same."""
    a = np.float32(1.0)
    logits = np.full((1, 32), -20, np.float32)
    near = np.nextafter(a, np.float32(2))
    logits[0, [0, 1]] = [a, a]
    logits[0, [8, 9]] = [near, a]
    logits[0, [16, 17]] = [near, near]
    logits[0, [24, 25]] = [a, np.float32(0.5)]
    for top in (1, 2, 3):
        check_route(lk, logits, None, 4, "softmax", 4, top, 2)
        check_route(lk, logits, None, 4, "sigmoid", 4, top, 2)


def test_route_ties_and_missing(lk):
    r = np.random.default_rng(4)
    logits = np.round(2 * r.standard_normal((9, 64))).astype(np.float32)  # many equal ones
    check_route(lk, logits, None, 8)
    check_route(lk, logits, np.zeros(64, np.float32), 8, "sigmoid")
    check_route(lk, logits, None, 8, "softmax", 8, 3, 1)
    logits[0] = -np.inf                       # no expert at all
    logits[1, 3:] = -np.inf                   # fewer than k
    logits[2, ::2] = np.nan
    logits[3, 5] = np.inf
    logits[4] = 0
    logits[5] = np.finfo(np.float32).min      # the type's lowest value, everywhere
    logits[6, 10:] = np.finfo(np.float32).min
    logits[7, :56] = -np.inf                  # one group only
    logits[8] = -0.0
    logits[8, 7] = 0.0
    bias = (0.1 * r.standard_normal(64)).astype(np.float32)
    for renorm in (True, False):
        check_route(lk, logits, None, 8, renorm=renorm)
        check_route(lk, logits, None, 8, "sigmoid", 8, 2, 1, renorm=renorm)
        check_route(lk, logits, None, 8, "sigmoid", 8, 2, 2, renorm=renorm)
        check_route(lk, logits, bias, 8, "softmax", 8, 2, 2, renorm=renorm)
    bias[::3] = np.inf
    bias[1::6] = np.nan
    check_route(lk, logits, bias, 8, "sigmoid")


def test_route_small_scores(lk):
    """Scores far below the row's largest, which is in no group that stays;
    sigmoids below f32's range."""
    logits = np.full((1, 16), -90, np.float32)
    logits[0, :4] = [3, -100, -100, -100]
    logits[0, 8:12] = [-88, -89, -89.5, -91]
    bias = np.zeros(16, np.float32)
    bias[8:12] = 1e3
    check_route(lk, logits, bias, 4, "softmax", 4, 1, 1)
    check_route(lk, logits - 10, None, 4, "sigmoid", 4, 4, 1)


# ---- the experts' products -----------------------------------------------------------

def make_ids(M, E, k, seed, padding=True):
    r = np.random.default_rng(seed)
    ids = np.stack([r.permutation(max(E, k))[:k] for _ in range(M)]).astype(np.int32)
    if padding:
        ids[ids >= E] = -1
        if M > 2:
            ids[1] = -1                     # a row without experts
            ids[2, k // 2:] = E             # pairs that are not there
        if k > 1:
            ids[0, 1] = ids[0, 0]           # the same expert twice
    return torch.from_numpy(ids).to(DEV)


def x_rows(n, K, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((n, K), generator=g, device=DEV)
    x[:, ::97] *= 20
    x[:, 32:64] = 0
    return x


def bits(t):
    return t.contiguous().view(torch.int32)


CASES = [  # M, E, k, F, K
    (1, 4, 1, 128, 128), (1, 16, 8, 256, 1024), (2, 5, 3, 384, 640), (3, 8, 2, 128, 1408), (9, 6, 4, 256, 384),
    (17, 3, 2, 128, 512), (64, 16, 4, 128, 256), (64, 2, 2, 128, 128), (5, 40, 32, 128, 128), (1, 3, 2, 1152, 5120),
    (33, 1, 1, 256, 768), (64, 1024, 8, 128, 128),
]


@pytest.mark.parametrize("mode", ["dequant", "int8act", "twopass"])
@pytest.mark.parametrize("M,E,k,F,K", CASES)
def test_glu(lk, mode, M, E, k, F, K):
    mode = lk.MODES[mode]
    gate, up = experts(E, F, K, 1, DEV), experts(E, F, K, 2, DEV)
    acts = acts_of(x_rows(M, K, 3), mode)
    ids = make_ids(M, E, k, 4)
    h = torch.full((M * k, F), 77.0, device=DEV)
    ex = lk.Experts(gate=gate, up=up)
    lk.lk_moe_glu_q8(ex, mode, ids, h, **acts)
    want, tol = glu_ref(gate, up, acts, mode, ids, E)
    there = ((ids >= 0) & (ids < E)).flatten()
    assert bool((h[~there] == 77).all())
    assert bool(((h.double() - want).abs() <= tol)[there].all())
    if mode == lk.LK_DEQUANT:
        return
    # bit for bit the products of lk_gemv_q8 and the SwiGLU and quantizer of lk_swiglu_quant
    n = M * k
    words = dict(hq=torch.full((n, F), 55, dtype=torch.int8, device=DEV),
                 hl=torch.full((n, F), 55, dtype=torch.int8, device=DEV),
                 hs=torch.full((n, F // 32), 55.0, device=DEV))
    cnt = torch.zeros((n * F // 32,), dtype=torch.int32, device=DEV)
    h2 = torch.full((n, F), 77.0, device=DEV)
    for _ in range(2):  # the counters are left as they were found
        lk.lk_moe_glu_q8(ex, mode, ids, h2, cnt=cnt, **words, **acts)
    assert torch.equal(bits(h2), bits(h)) and not bool(cnt.any())
    q = quantize(h, mode)
    for name, of in (("hq", "xq"), ("hs", "xs"), *((("hl", "xl"),) if mode == lk.LK_TWOPASS else ())):
        assert torch.equal(words[name][there], q[of][there]), name
        assert bool((words[name][~there] == 55).all()), name
    g, u = torch.empty((1, F), device=DEV), torch.empty((1, F), device=DEV)
    one = torch.empty((1, F), device=DEV)
    for p in [int(v) for v in there.nonzero()[:: max(1, n // 24)]]:
        e, t = int(ids.flatten()[p]), p // k
        row = {a: v[t:t + 1] for a, v in acts.items()}
        lk.lk_gemv_q8(gate[0][e], gate[1][e], mode, g, **row)
        lk.lk_gemv_q8(up[0][e], up[1][e], mode, u, **row)
        lk.lk_swiglu_quant(g, u, mode, h=one, hq=torch.empty((1, F), dtype=torch.int8, device=DEV),
                           hl=torch.empty((1, F), dtype=torch.int8, device=DEV), hs=torch.empty((1, F // 32), device=DEV))
        assert torch.equal(bits(one[0]), bits(h[p])), p


@pytest.mark.parametrize("mode", ["dequant", "int8act", "twopass"])
@pytest.mark.parametrize("M,E,k,N,F", CASES)
def test_down(lk, mode, M, E, k, N, F):
    mode = lk.MODES[mode]
    down = experts(E, N, F, 5, DEV)
    acts = acts_of(x_rows(M * k, F, 6), mode)
    ids = make_ids(M, E, k, 7)
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    w = torch.randn((M, k), generator=g, device=DEV)
    # what belongs to absent pairs is not looked at
    there = (ids >= 0) & (ids < E)
    w[~there] = math.nan
    for t in acts.values():
        t[~there.flatten()] = 99 if t.dtype == torch.int8 else math.nan
    y = torch.full((M, N), math.nan, device=DEV)
    lk.lk_moe_down_q8(lk.Experts(down=down), mode, ids, w, y, **as_h(acts))
    want, tol = down_ref(down, acts, mode, ids, w, E)
    assert bool(((y.double() - want).abs() <= tol).all())
    assert bool((y[~there.any(1)] == 0).all())
    if mode == lk.LK_DEQUANT:
        return
    # the products of lk_gemv_q8, added in ascending j
    d = torch.empty((1, N), device=DEV)
    for t in range(0, M, max(1, M // 8)):
        acc = torch.zeros((N,), device=DEV)
        for j in range(k):
            if not bool(there[t, j]):
                continue
            row = {a: v[t * k + j:t * k + j + 1] for a, v in acts.items()}
            e = int(ids[t, j])
            lk.lk_gemv_q8(down[0][e], down[1][e], mode, d, **row)
            acc = (w[t, j].double() * d[0].double() + acc.double()).float()
        assert torch.equal(bits(acc), bits(y[t])), t


def test_step_together(lk):
    """Routing, gate/up and down as a decoder's step runs them: words handed
    on, dependent launches, in a captured graph whose inputs change between
    replays, on a stream of its own."""
    M, E, k, H, F, mode = 6, 16, 4, 512, 384, lk.LK_TWOPASS
    gate, up, down = experts(E, F, H, 1, DEV), experts(E, F, H, 2, DEV), experts(E, H, F, 3, DEV)
    ex = lk.Experts(gate=gate, up=up, down=down)
    n, i8 = M * k, dict(dtype=torch.int8, device=DEV)
    x, logits = torch.zeros((M, H), device=DEV), torch.zeros((M, E), device=DEV)
    xq, xl, xs = torch.zeros((M, H), **i8), torch.zeros((M, H), **i8), torch.zeros((M, H // 32), device=DEV)
    ids, w = torch.zeros((M, k), dtype=torch.int32, device=DEV), torch.zeros((M, k), device=DEV)
    h, y = torch.zeros((n, F), device=DEV), torch.zeros((M, H), device=DEV)
    hq, hl, hs = torch.zeros((n, F), **i8), torch.zeros((n, F), **i8), torch.zeros((n, F // 32), device=DEV)
    cnt = torch.zeros((n * F // 32,), dtype=torch.int32, device=DEV)
    cfg = lk.launch_cfg(pdl=1)

    def step():
        lk.lk_quantize_act(x, mode, xq, xl, xs, cfg=cfg)
        lk.lk_moe_route(logits, ids, w, cfg=cfg)
        lk.lk_moe_glu_q8(ex, mode, ids, h, xq=xq, xl=xl, xs=xs, hq=hq, hl=hl, hs=hs, cnt=cnt, cfg=cfg)
        lk.lk_moe_down_q8(ex, mode, ids, w, y, hq=hq, hl=hl, hs=hs, cfg=cfg)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(3):
                step()
        for seed in range(20):
            x.copy_(x_rows(M, H, 100 + seed))
            logits.copy_(torch.randn((M, E), device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)))
            if seed % 3 == 0:
                logits[2] = -math.inf
            graph.replay()
            got = [v.clone() for v in (ids, w, h, hq, hl, hs, y)]
            side.synchronize()
            want_ids, want_w, _ = route_ref(logits.cpu().numpy(), None, "softmax", 1, 1, 1, k, True, 1.0)
            assert np.array_equal(got[0].cpu().numpy(), want_ids)
            want, tol = glu_ref(gate, up, dict(xq=xq, xl=xl, xs=xs), mode, ids, E)
            there = (ids >= 0).flatten()
            assert bool(((got[2].double() - want).abs() <= tol)[there].all()), seed
            q = quantize(got[2], mode)
            assert torch.equal(got[3][there], q["xq"][there]) and torch.equal(got[4][there], q["xl"][there])
            want, tol = down_ref(down, dict(xq=hq, xl=hl, xs=hs), mode, ids, got[1], E)
            assert bool(((got[6].double() - want).abs() <= tol).all()), seed
    torch.cuda.current_stream().wait_stream(side)


@pytest.mark.parametrize("mode", ["int8act", "twopass"])
@pytest.mark.parametrize("M,E,k,F,K", CASES)
def test_kernels_agree(lk, mode, M, E, k, F, K):
    """The kernel for single rows and the tensor-core kernel give the same bits."""
    ex = lk.Experts(gate=experts(E, F, K, 1, DEV), up=experts(E, F, K, 2, DEV), down=experts(E, K, F, 3, DEV))
    m, n = lk.MODES[mode], M * k
    ids = make_ids(M, E, k, 4)
    acts, hs_ = quantize(x_rows(M, K, 3), m), as_h(quantize(x_rows(n, F, 5), m))
    w = torch.rand((M, k), device=DEV)
    got = []
    for path in (0, 2, 3):
        cfg = lk.launch_cfg(path=path)
        h, y = torch.zeros((n, F), device=DEV), torch.zeros((M, K), device=DEV)
        words = dict(hq=torch.zeros((n, F), dtype=torch.int8, device=DEV), hs=torch.zeros((n, F // 32), device=DEV),
                     hl=torch.zeros((n, F), dtype=torch.int8, device=DEV))
        cnt = torch.zeros((n * F // 32,), dtype=torch.int32, device=DEV)
        lk.lk_moe_glu_q8(ex, m, ids, h, cnt=cnt, cfg=cfg, **words, **acts)
        lk.lk_moe_down_q8(ex, m, ids, w, y, cfg=cfg, **hs_)
        assert not bool(cnt.any())
        got.append([bits(h), bits(y), bits(words["hs"]), words["hq"], words["hl"]])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    x = torch.zeros((M, K), device=DEV)
    for path in (1, 3):
        with pytest.raises(lk.LkError) as err:
            lk.lk_moe_glu_q8(ex, "dequant", ids, h, x=x, cfg=lk.launch_cfg(path=path))
        assert err.value.status == -3


@pytest.mark.parametrize("mode", ["dequant", "int8act", "twopass"])
@pytest.mark.parametrize("M,E,k,rows,K", [(40, 6, 8, 640, 384), (40, 6, 8, 640, 2048), (50, 4, 2, 1280, 1152),
                                          (7, 5, 3, 256, 4224), (7, 5, 3, 256, 4352), (1, 5, 3, 128, 4096)])
def test_single_rows_stages(lk, mode, M, E, k, rows, K):
    """The kernel for single rows with several groups of short rows in a stage (the last of a
    block with fewer), and with long rows in slices whose scales begin at 8 or 16 bytes."""
    mode, cfg = lk.MODES[mode], lk.launch_cfg(path=2)
    a, b = experts(E, rows, K, 1, DEV), experts(E, rows, K, 2, DEV)
    ids = make_ids(M, E, k, 3)
    there = ((ids >= 0) & (ids < E)).flatten()
    acts, h = acts_of(x_rows(M, K, 4), mode), torch.full((M * k, rows), 7.0, device=DEV)
    lk.lk_moe_glu_q8(lk.Experts(gate=a, up=b), mode, ids, h, cfg=cfg, **acts)
    want, tol = glu_ref(a, b, acts, mode, ids, E)
    assert bool(((h.double() - want).abs() <= tol)[there].all()) and bool((h[~there] == 7).all())
    hidden, w = acts_of(x_rows(M * k, K, 5), mode), torch.rand((M, k), device=DEV)
    y = torch.full((M, rows), math.nan, device=DEV)
    lk.lk_moe_down_q8(lk.Experts(down=a), mode, ids, w, y, cfg=cfg, **as_h(hidden))
    want, tol = down_ref(a, hidden, mode, ids, w, E)
    assert bool(((y.double() - want).abs() <= tol).all())


def test_two_streams_at_once(lk):
    """Calls on two streams, each with its own outputs and counters."""
    M, E, k, F, K, mode = 8, 12, 4, 256, 768, lk.LK_INT8ACT
    ex = lk.Experts(gate=experts(E, F, K, 1, DEV), up=experts(E, F, K, 2, DEV))
    n = M * k
    sets = []
    for s in range(2):
        acts = quantize(x_rows(M, K, 20 + s), mode)
        sets.append(dict(ids=make_ids(M, E, k, 30 + s, padding=False), h=torch.zeros((n, F), device=DEV),
                         hq=torch.zeros((n, F), dtype=torch.int8, device=DEV), hs=torch.zeros((n, F // 32), device=DEV),
                         cnt=torch.zeros((n * F // 32,), dtype=torch.int32, device=DEV), **acts))
    alone = []
    for s in sets:
        lk.lk_moe_glu_q8(ex, mode, **s)
        alone.append([s[v].clone() for v in ("h", "hq", "hs")])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for st, s in zip(streams, sets):
            lk.lk_moe_glu_q8(ex, mode, stream=st, **s)
    torch.cuda.synchronize()
    for s, want in zip(sets, alone):
        assert all(torch.equal(s[v], w) for v, w in zip(("h", "hq", "hs"), want))
        assert not bool(s["cnt"].any())


@pytest.mark.parametrize("mode", ["dequant", "int8act", "twopass"])
def test_no_experts_at_all(lk, mode):
    """Every pair absent: the products' rows stay, the sums are zeros."""
    M, E, k, F, K, m = 5, 4, 3, 128, 256, lk.MODES[mode]
    ex = lk.Experts(gate=experts(E, F, K, 1, DEV), up=experts(E, F, K, 2, DEV), down=experts(E, K, F, 3, DEV))
    ids = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31, 1023] * k, dtype=torch.int32, device=DEV).view(M, k)
    acts, hidden = acts_of(x_rows(M, K, 1), m), as_h(acts_of(x_rows(M * k, F, 2), m))
    for path in ((0, 2) if mode == "dequant" else (0, 2, 3)):
        h, y = torch.full((M * k, F), 7.0, device=DEV), torch.full((M, K), math.nan, device=DEV)
        cfg = lk.launch_cfg(path=path)
        lk.lk_moe_glu_q8(ex, m, ids, h, cfg=cfg, **acts)
        lk.lk_moe_down_q8(ex, m, ids, torch.ones((M, k), device=DEV), y, cfg=cfg, **hidden)
        assert bool((h == 7).all()) and bool((y == 0).all())


def test_stack_past_32_bits(lk):
    """Matrices that begin more than 2^32 bytes into their stacks."""
    E, F, K, k = 300, 4096, 4096, 2
    dev = torch.device(DEV)
    q = torch.zeros((E, F, K), dtype=torch.int8, device=dev)
    s = torch.zeros((E, F, K // 32), dtype=torch.float16, device=dev)
    for e in (3, E - 1):
        for t, r in zip((q, s), experts(1, F, K, e, DEV)):
            t[e] = r[0]
    assert (E - 1) * F * K > 2 ** 32
    ex = lk.Experts(gate=(q, s), up=(q, s), down=(q, s))
    for M, path in ((1, 2), (3, 3)):
        ids = torch.tensor([[E - 1, 3]] * M, dtype=torch.int32, device=DEV)
        acts, cfg = quantize(x_rows(M, K, 5), lk.LK_INT8ACT), lk.launch_cfg(path=path)
        h, y = torch.zeros((M * k, F), device=DEV), torch.zeros((M, F), device=DEV)
        lk.lk_moe_glu_q8(ex, "int8act", ids, h, cfg=cfg, **acts)
        want, tol = glu_ref((q, s), (q, s), acts, lk.LK_INT8ACT, ids, E)
        assert bool(((h.double() - want).abs() <= tol).all())
        hidden, w = quantize(x_rows(M * k, K, 6), lk.LK_INT8ACT), torch.ones((M, k), device=DEV)
        lk.lk_moe_down_q8(ex, "int8act", ids, w, y, cfg=cfg, **as_h(hidden))
        want, tol = down_ref((q, s), hidden, lk.LK_INT8ACT, ids, w, E)
        assert bool(((y.double() - want).abs() <= tol).all())


def test_limits(lk):
    """The largest activation that the header promises, and one past it."""
    e = lk.Experts(gate=experts(1, 128, 32768, 1, DEV), up=experts(1, 128, 32768, 2, DEV),
                   down=experts(1, 128, 128, 3, DEV))
    ids = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    x, h = x_rows(1, 32768, 1), torch.zeros((1, 128), device=DEV)
    lk.lk_moe_glu_q8(e, "dequant", ids, h, x=x)
    want, tol = glu_ref(e.gate, e.up, {"x": x}, lk.LK_DEQUANT, ids, 1)
    assert bool(((h.double() - want).abs() <= tol).all())
    big = lk.Experts(down=experts(1, 128, 51200, 3, DEV))
    with pytest.raises(lk.LkError) as err:
        lk.lk_moe_down_q8(big, "dequant", ids, torch.ones((1, 1), device=DEV), h, h=torch.zeros((1, 51200), device=DEV))
    assert err.value.status == -3
    empty = torch.zeros((0, 2), dtype=torch.int32, device=DEV)
    lk.lk_moe_glu_q8(e, "dequant", empty, torch.zeros((0, 128), device=DEV), x=torch.zeros((0, 32768), device=DEV))
