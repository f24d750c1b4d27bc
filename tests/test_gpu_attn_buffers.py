"""Attention's buffers packed into one allocation without room between them, and
the result in place of the queries: the bits of separate buffers, nothing else
touched."""
import pytest

torch = pytest.importorskip("torch")

from gpuhelp import act_buffers  # noqa: E402
from q8_quantized_gemv_gb300 import build, lk  # noqa: E402
from test_gpu_attn import DEV, TYPES, gen, make_cache, make_table, roomy, workspace  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    yield
    assert lk.lk_device_error(reset=True) == 0


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("R,room,prefix", [(1, False, 0), (1, True, 0), (12, True, 0), (1, False, 5000), (1, True, 30000)])
def test_packed_buffers(type_, R, room, prefix):
    g = gen(64)
    n_q, n_kv, D, page, B = 16, 2, 128, 16, 3
    N, M, p_pages = n_q * D, B * R, -(-prefix // page)
    cache, _, _ = make_cache(type_, p_pages + 40, n_kv, page, D, g)
    table = make_table(B, 12, p_pages + 40, g, p_pages)
    if room:
        table = roomy(table, page)
    pt = torch.arange(p_pages, dtype=torch.int32, device=DEV)
    lens = torch.tensor([150, 0, 77], dtype=torch.int32, device=DEV)
    q0 = torch.randn((M, N), generator=g, device=DEV)

    def run(q, ws, **to):
        if prefix:
            lk.lk_attn_shared(cache, q, pt, prefix, table, lens, ws, R=R, mode=2, **to)
        else:
            lk.lk_attn(cache, q, table, lens, ws, R=R, mode=2, **to)

    hq, hl, hs = act_buffers(M, N, 2)
    want = torch.empty_like(q0)
    run(q0, workspace(cache, n_q, B, R, prefix > 0), out=want, hq=hq, hl=hl, hs=hs)
    nws = lk.lk_attn_workspace_bytes(n_q, n_kv, D, B, R, prefix > 0)
    sizes = [M * N * 4, M * N, nws, M * N // 8, M * N, M * N * 4]
    buf = torch.full((sum(sizes) + 64,), 0x55, dtype=torch.uint8, device=DEV)
    parts, at = [], 32
    for n in sizes:
        parts.append(buf[at:at + n])
        at += n
    q, hq2, ws, hs2, hl2, out = parts
    q, out, hs2 = q.view(torch.float32).view(M, N), out.view(torch.float32).view(M, N), hs2.view(torch.float32).view(M, N // 32)
    hq2, hl2 = hq2.view(torch.int8).view(M, N), hl2.view(torch.int8).view(M, N)
    q.copy_(q0)
    for place in (out, q):
        run(q, ws, out=place, hq=hq2, hl=hl2, hs=hs2)
        torch.cuda.synchronize()
        assert torch.equal(place, want) and torch.equal(hq2, hq) and torch.equal(hl2, hl) and torch.equal(hs2, hs)
        assert (buf[:32] == 0x55).all() and (buf[-32:] == 0x55).all()
        if place is out:
            assert torch.equal(q, q0)
    with pytest.raises(lk.LkError):
        run(q0, ws, out=out, hq=hq2, hl=hl2, hs=q0.view(-1)[:M * N // 32].view(M, N // 32))
