"""Append and attention as a program runs them, token after token in a captured
graph, on every path that the attention call takes: the streaming kernel and
the join, the tile kernel for the sequences, for the prefix behind a streaming
launch, for both, and clusters.  The append writes the queries that the
attention reads; lengths advance inside the graph; inputs and page-table
entries change between replays.  Two layers share the workspace.  Results are
held to the formula in 64 bits, and to the bits of the same calls with the
device idle before each."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gpuhelp import bits, host  # noqa: E402
from q8_quantized_gemv_gb300 import build, lk  # noqa: E402
from test_gpu_attn import (DEV, TYPES, check, gen, host_append, host_quant, make_cache, make_table, reference,  # noqa: E402
                           workspace)

pytestmark = pytest.mark.gpu

# path: n_q, n_kv, R, prefix, width of the table (pages of 16), lens, launches of f16 and bf16, of q8
PATHS = {
    "streaming": (8, 2, 1, 0, 700, [0, 31, -1, 300], 2, 2),
    "streaming prefix": (8, 2, 1, 700, 700, [0, 31, -1, 300], 2, 2),
    "own tiled": (8, 2, 12, 0, 600, [0, 120, 37], 2, 2),
    "prefix tiled": (8, 2, 1, 12000, 12, [40, 0, 7, -1, 64, 1, 90, 15, 16, 33, 5, 11], 3, 3),
    "both tiled": (8, 2, 12, 12000, 12, [0, 100, 37], 2, 2),
    "clusters": (8, 2, 1, 40, 12, [0, 15, 100], 1, 1),
}
STEPS = 6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    yield
    assert lk.lk_device_error(reset=True) == 0
    torch.cuda.empty_cache()


def dense(t, s):
    return t.double() if s is None else (t.double().view(*s.shape, 32) * s.double().unsqueeze(-1)).view(t.shape)


@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("pdl", [0, 1])
def test_token_by_token(path, type_, pdl):
    n_q, n_kv, R, prefix, width, first, most16, most8 = PATHS[path]
    B, D, page, layers, M = len(first), 128, 16, 2, len(first) * R
    g = gen(91)
    cfg = lk.launch_cfg(pdl=pdl)
    used = -(-(max(first) + R * (STEPS + 1)) // page)  # pages that sequences come to
    p_pages = -(-prefix // page)
    spare = 4
    n_pages = p_pages + B * used + spare
    caches = [make_cache(type_, n_pages, n_kv, page, D, g)[0] for _ in range(layers)]
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    ptable, others = order[:p_pages].contiguous(), order[p_pages + B * used:]
    table0 = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table0[:, :used] = order[p_pages:p_pages + B * used].view(B, used)
    table = table0.clone()
    assert lk.lk_attn_launches(caches[0], n_q, B, width, R, prefix) == (most8 if type_ == "q8" else most16)
    lens0 = torch.tensor(first, dtype=torch.int32, device=DEV)
    more = torch.where(lens0 >= 0, R, 0).to(torch.int32)
    lens = lens0.clone()
    ang = torch.rand((prefix + used * page, D // 2), generator=g, device=DEV) * 6
    cos, sin = ang.cos(), ang.sin()
    x = torch.zeros((layers, M, (n_q + 2 * n_kv) * D), device=DEV)
    xs = torch.randn((STEPS, *x.shape), generator=g, device=DEV)
    qr = torch.zeros((layers, M, n_q * D), device=DEV)
    out = torch.zeros_like(qr)
    ws = workspace(caches[0], n_q, B, R, prefix > 0)
    start = [[None if t is None else t.clone() for t in (c.k, c.v, c.ks, c.vs)] for c in caches]

    def step(cfg, idle=lambda: None):
        lens.add_(more)
        for l, c in enumerate(caches):
            q, k, v = x[l].split((n_q * D, n_kv * D, n_kv * D), 1)
            idle()
            lk.lk_kv_append(c, q, k, v, table, lens, cos, sin, qr[l], R=R, p0=prefix, cfg=cfg)
            idle()
            if prefix:
                lk.lk_attn_shared(c, qr[l], ptable, prefix, table, lens, ws, R=R, out=out[l], cfg=cfg)
            else:
                lk.lk_attn(c, qr[l], table, lens, ws, R=R, out=out[l], cfg=cfg)

    def restart():
        lens.copy_(lens0)
        table.copy_(table0)
        out.zero_()
        qr.zero_()
        for c, s in zip(caches, start):
            for t, b in zip((c.k, c.v, c.ks, c.vs), s):
                if t is not None:
                    t.copy_(b)

    def before(i):
        x.copy_(xs[i])
        if i % 2:  # sequence i's first page is another one from here on
            table[i % B, 0] = others[i % spare]

    restart()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cfg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(cfg)
    restart()
    got = []
    for i in range(STEPS):
        before(i)
        graph.replay()
        got.append((out.clone(), qr.clone(), lens.clone(), table.clone()))
        if i in (0, STEPS - 1):
            torch.cuda.synchronize()
            n = host(lens).tolist()
            assert n == [f + R * (i + 1) if f >= 0 else f for f in first]
            for l, c in enumerate(caches):
                want, tol = reference(dense(c.k, c.ks), dense(c.v, c.vs), qr[l], table, n, R, D ** -0.5,
                                      (ptable, prefix) if prefix else None, type_ == "bf16")
                check(out[l], want, tol)
    torch.cuda.synchronize()
    end = [[None if t is None else t.clone() for t in (c.k, c.v, c.ks, c.vs)] for c in caches]
    restart()
    for i in range(STEPS):
        before(i)
        step(None, torch.cuda.synchronize)
        torch.cuda.synchronize()
        for a, b in zip((out, qr, lens, table), got[i]):
            assert torch.equal(a, b), i
    for c, e in zip(caches, end):
        for t, b in zip((c.k, c.v, c.ks, c.vs), e):
            assert t is None or torch.equal(t, b)


@pytest.mark.parametrize("paired", [False, True])
def test_append_reads_tables_and_gains_of_the_launch_before(paired):
    """Rotation table and gains written by the launches just before a dependent
    append, new ones in every replay."""
    B, n_q, n_kv, D, page = 3, 8, 2, 128, 16
    g = gen(95)
    cache, _, _ = make_cache("q8", 8, n_kv, page, D, g)
    table = make_table(B, 2, 8, g)
    lens = torch.tensor([1, 17, 30], dtype=torch.int32, device=DEV)
    x = torch.randn((B, (n_q + 2 * n_kv) * D), generator=g, device=DEV)
    q, k, v = x.split((n_q * D, n_kv * D, n_kv * D), 1)
    new = torch.zeros((4, 30, D // 2), device=DEV)
    cos, sin = torch.zeros((30, D // 2), device=DEV), torch.zeros((30, D // 2), device=DEV)
    gains = torch.zeros((2, D), device=DEV)
    qr = torch.zeros((B, n_q * D), device=DEV)
    cfg = lk.launch_cfg(pdl=1)

    def step():
        cos.copy_(new[0])
        gains[0].copy_(new[2, :2].flatten())
        gains[1].copy_(new[3, :2].flatten())
        sin.copy_(new[1])
        for _ in range(2):  # the second one a dependent of a kernel that lets it start early
            lk.lk_kv_append(cache, q, k, v, table, lens, cos, sin, qr, paired=paired, q_gain=gains[0], k_gain=gains[1],
                            cfg=cfg)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    hx, ht = host(x).reshape(B, -1, D), host(table)
    for _ in range(4):
        new.copy_(torch.randn(new.shape, generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        n = host(new)
        for b, ln in enumerate(host(lens).tolist()):
            want = host_append(hx[b, :n_q], n[0], n[1], ln - 1, paired, n[2, :2].ravel())
            assert np.array_equal(bits(host(qr[b]).reshape(n_q, D)), bits(want))
            kw, ks = host_quant(host_append(hx[b, n_q:n_q + n_kv], n[0], n[1], ln - 1, paired, n[3, :2].ravel()))
            at = (int(ht[b, (ln - 1) // page]), slice(None), (ln - 1) % page)
            assert np.array_equal(host(cache.k)[at], kw) and np.array_equal(host(cache.ks)[at], ks)
