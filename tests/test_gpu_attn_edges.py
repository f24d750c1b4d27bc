"""Calls of the attention step that the documentation allows at its edges: every
form used for the first time inside a capture, after one call of another form;
neighbouring pairs over a part of the head; sequences without a table behind a
prefix; every page number absent."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from conftest import ROOT  # noqa: E402
from gpuhelp import bits, host  # noqa: E402
from q8_quantized_gemv_gb300 import build, lk  # noqa: E402
from test_gpu_attn import (DEV, TYPES, check, gen, host_append, make_cache, make_table, reference, roomy,  # noqa: E402
                           workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    yield
    assert lk.lk_device_error(reset=True) == 0


FIRST_USE = """
import sys, torch
sys.path.insert(0, "tests")
from test_gpu_attn import DEV, gen, make_cache, make_table, roomy, workspace
from q8_quantized_gemv_gb300 import lk
type_, D = sys.argv[1], int(sys.argv[2])
g = gen(3)
cfg = lk.launch_cfg(pdl=1)
small, _, _ = make_cache("f16" if type_ != "f16" else "bf16", 4, 1, 16, 64, g)
cache, _, _ = make_cache(type_, 800, 2, 16, D, g)
calls = []
for R, room, prefix, mode in ((1, 0, 0, 0), (1, 1, 0, 1), (12, 1, 0, 2), (12, 1, 11000, 0), (1, 1, 11000, 1)):
    B = 12 if R == 1 else 3
    table = make_table(B, 6, 800, g, 690)
    table = roomy(table, 16) if room else table
    lens = torch.full((B,), 80, dtype=torch.int32, device=DEV)
    q = torch.randn((B * R, 8 * D), generator=g, device=DEV)
    n = B * R
    out = torch.zeros_like(q)
    to = dict(hq=torch.zeros((n, 8 * D), dtype=torch.int8, device=DEV), hl=torch.zeros((n, 8 * D), dtype=torch.int8, device=DEV),
              hs=torch.zeros((n, D // 4), device=DEV)) if mode else {}
    calls.append((q, table, lens, workspace(cache, 8, B, R, prefix > 0), R, prefix, mode, out, to))
pt = torch.arange(688, dtype=torch.int32, device=DEV)
x = torch.randn((1, 12 * D), generator=g, device=DEV)
t1, l1 = torch.full((1, 6), 799, dtype=torch.int32, device=DEV), torch.ones((1,), dtype=torch.int32, device=DEV)
qr = torch.zeros((1, 8 * D), device=DEV)
# the one call before the capture: another type, head size and form
y = torch.zeros((1, 64), device=DEV)
z = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
lk.lk_attn(small, y, z, l1, workspace(small, 1, 1, 1), out=torch.zeros_like(y))
torch.cuda.synchronize()

def run():
    # (first: it writes a page that the others read, the same in every run)
    lk.lk_kv_append(cache, *x.split((8 * D, 2 * D, 2 * D), 1), t1, l1, None, None, qr, cfg=cfg)
    for q, table, lens, ws, R, prefix, mode, out, to in calls:
        if prefix:
            lk.lk_attn_shared(cache, q, pt, prefix, table, lens, ws, R=R, mode=mode, out=out, cfg=cfg, **to)
        else:
            lk.lk_attn(cache, q, table, lens, ws, R=R, mode=mode, out=out, cfg=cfg, **to)

side = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=side):
    run()
graph.replay()
torch.cuda.synchronize()
got = [c[7].clone() for c in calls]
for c in calls:
    c[7].zero_()
run()
torch.cuda.synchronize()
assert lk.lk_device_error(reset=True) == 0
for c, w in zip(calls, got):
    assert torch.equal(c[7], w) and torch.isfinite(w).all() and (w != 0).any()
print("fine")
"""


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
def test_first_use_inside_a_capture(type_, D):
    r = subprocess.run([sys.executable, "-c", FIRST_USE, type_, str(D)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300, env=dict(os.environ, PYTHONPATH=ROOT))
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]


@pytest.mark.parametrize("paired", [False, True])
def test_rotation_of_a_part_of_the_head(paired):
    g = gen(96)
    cache, _, _ = make_cache("bf16", 6, 3, 16, 128, g)
    table = make_table(2, 3, 6, g)
    lens = torch.tensor([48, 7], dtype=torch.int32, device=DEV)
    x = torch.randn((10, 12 * 128), generator=g, device=DEV)
    q, k, v = x.split((6 * 128, 3 * 128, 3 * 128), 1)
    ang = torch.rand((60, 32), generator=g, device=DEV) * 100
    cos, sin = ang.cos(), ang.sin()
    qg, kg = torch.rand((128,), generator=g, device=DEV), torch.rand((128,), generator=g, device=DEV)
    qr = torch.zeros((10, 6 * 128), device=DEV)
    lk.lk_kv_append(cache, q, k, v, table, lens, cos, sin, qr, R=5, p0=11, paired=paired, q_gain=qg, k_gain=kg)
    torch.cuda.synchronize()
    h, c, s = host(x).reshape(10, 12, 128), host(cos), host(sin)
    for m in range(10):
        p = [48, 7][m // 5] - 5 + m % 5
        assert np.array_equal(bits(host(qr[m]).reshape(6, 128)), bits(host_append(h[m, :6], c, s, 11 + p, paired, host(qg))))
        want = torch.from_numpy(host_append(h[m, 6:9], c, s, 11 + p, paired, host(kg))).to(torch.bfloat16)
        page = int(table[m // 5, p // 16])
        assert torch.equal(cache.k[page, :, p % 16].cpu(), want)
        assert torch.equal(cache.v[page, :, p % 16].cpu(), x[m].cpu().view(12, 128)[9:].to(torch.bfloat16))


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("R,prefix", [(1, 45), (1, 20000), (12, 45), (12, 12000)])
def test_prefix_and_no_table(type_, D, R, prefix):
    """No room for own tokens: rows see the prefix alone (padding nothing), however
    long the sequences say they are."""
    g = gen(97)
    pages = -(-prefix // 16)
    cache, kd, vd = make_cache(type_, pages + 1, 2, 16, D, g)
    pt = torch.randperm(pages + 1, generator=g, device=DEV)[:pages].to(torch.int32)
    lens = [0, 50, -1, 2 ** 31 - 1, 1]
    table = torch.empty((5, 0), dtype=torch.int32, device=DEV)
    q = torch.randn((5 * R, 8 * D), generator=g, device=DEV)
    out = torch.full((5 * R + 1, 8 * D), 3.0, device=DEV)
    lk.lk_attn_shared(cache, q, pt, prefix, table, torch.tensor(lens, dtype=torch.int32, device=DEV),
                      workspace(cache, 8, 5, R, True), R=R, out=out[:-1])
    torch.cuda.synchronize()
    check(out[:-1], *reference(kd, vd, q, table, lens, R, D ** -0.5, (pt, prefix), type_ == "bf16"))
    assert (out[-1] == 3.0).all() and (out[2 * R:3 * R] == 0).all()


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("R,prefix,room", [(1, 0, False), (1, 0, True), (12, 0, True), (1, 300, False), (12, 9000, True)])
def test_every_page_absent(type_, R, prefix, room):
    """Tables that list no page of the cache: nobody sees anything."""
    g = gen(98)
    cache, _, _ = make_cache(type_, 4, 2, 16, 128, g)
    for x in (cache.k, cache.v, cache.ks, cache.vs):
        if x is not None and x.dtype != torch.int8:
            x.fill_(float("nan"))
    table = torch.tensor([[-1, 4, 2 ** 31 - 1]] * 3, dtype=torch.int32, device=DEV)
    if room:
        table = roomy(table, 16)
    pt = torch.full((-(-prefix // 16),), 4, dtype=torch.int32, device=DEV)
    lens = torch.tensor([48, 0, 17], dtype=torch.int32, device=DEV)
    q = torch.randn((3 * R, 8 * 128), generator=g, device=DEV)
    out = torch.full_like(q, 3.0)
    ws = workspace(cache, 8, 3, R, prefix > 0)
    if prefix:
        lk.lk_attn_shared(cache, q, pt, prefix, table, lens, ws, R=R, out=out)
    else:
        lk.lk_attn(cache, q, table, lens, ws, R=R, out=out)
    torch.cuda.synchronize()
    assert (out == 0).all()
