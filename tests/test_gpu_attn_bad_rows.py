"""Queries and cached values that are not finite: a head of a row that sees a
token comes out as NaN and not as the zeros of an empty one, a row that sees none as
zeros whatever its query holds, and every other result keeps its bits.  On each
path: clusters, the streaming kernel with the join, the tile kernel."""
import pytest

torch = pytest.importorskip("torch")

from q8_quantized_gemv_gb300 import build, lk  # noqa: E402
from test_gpu_attn import DEV, TYPES, gen, make_cache, make_table, roomy, workspace  # noqa: E402

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    yield
    assert lk.lk_device_error(reset=True) == 0


def attend(cache, q, prefix, table, lens, ws, R):
    out = torch.full_like(q, 5.0)
    if prefix is None:
        lk.lk_attn(cache, q, table, lens, ws, R=R, out=out)
    else:
        lk.lk_attn_shared(cache, q, prefix[0], prefix[1], table, lens, ws, R=R, out=out)
    return out


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("R,room", [(1, False), (1, True), (12, False), (12, True)])
@pytest.mark.parametrize("prefix", [0, 50, 9000])
def test_a_head_that_is_not_finite_shows(type_, D, R, room, prefix):
    g = gen(62)
    n_q, n_kv, page = 16, 2, 16
    lens = [150, 0, 77, 9, -1]
    B = len(lens)
    p_pages = -(-prefix // page)
    cache, _, _ = make_cache(type_, p_pages + 60, n_kv, page, D, g)
    table = make_table(B, 12, p_pages + 60, g, p_pages)
    if room:
        table = roomy(table, page)
    pre = (torch.arange(p_pages, dtype=torch.int32, device=DEV), prefix) if prefix else None
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = torch.randn((B * R, n_q * D), generator=g, device=DEV)
    ws = workspace(cache, n_q, B, R, bool(prefix))
    want = attend(cache, q, pre, table, lt, ws, R).view(B * R, n_q, D)
    bad = q.clone().view(B * R, n_q, D)
    spoilt = torch.zeros((B * R, n_q), dtype=torch.bool)

    def spoil(row, head, value, at=None):
        bad[row, head, slice(None) if at is None else at] = value
        spoilt[row, head] = True

    spoil(0, 0, INF), spoil(0, 1, NAN), spoil(0, 3, NAN, 5), spoil(0, 15, -INF, D - 1)
    spoil(R - 1, 7, INF, 33)
    for r in range(R):  # whole rows: of the empty sequence, the padding, and of 9 tokens those before the first
        for b in (1, 4):
            for h in range(n_q):
                spoil(b * R + r, h, NAN if r % 2 else INF)
        if 9 - R + 1 + r <= 0:
            for h in range(n_q):
                spoil(3 * R + r, h, NAN)
    spoil(2 * R + R // 2, 9, NAN, 0)
    got = attend(cache, bad.view(B * R, -1), pre, table, lt, ws, R).view(B * R, n_q, D)
    for m in range(B * R):
        b, r = divmod(m, R)
        sees = lens[b] >= 0 and (prefix > 0 or lens[b] - R + 1 + r > 0)
        for h in range(n_q):
            if not sees:
                assert (got[m, h] == 0).all(), (m, h)
            elif spoilt[m, h]:
                assert torch.isnan(got[m, h]).all(), (m, h)
            else:
                assert torch.equal(got[m, h], want[m, h]) and torch.isfinite(got[m, h]).all(), (m, h)


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("R", [1, 16])
def test_an_overflow_of_the_cache_shows(R, room):
    """Values past 65504 that an append rounds to infinity in an f16 cache."""
    g = gen(63)
    n_q, n_kv, D, page = 16, 2, 128, 16
    cache, _, _ = make_cache("f16", 30, n_kv, page, D, g)
    table = make_table(2, 12, 30, g)
    if room:
        table = roomy(table, page)
    lens = torch.tensor([100, 61], dtype=torch.int32, device=DEV)
    x = torch.randn((2 * R, (n_q + 2 * n_kv) * D), generator=g, device=DEV)
    qr = torch.empty((2 * R, n_q * D), device=DEV)
    ws = workspace(cache, n_q, 2, R)
    for part in (0, 1):  # the last token's first key head, its second value head
        y = x.clone()
        lo = (n_q + 2 * part + part) * D
        y[R - 1, lo:lo + D] = y[R - 1, lo:lo + D].sign() * 1e6
        lk.lk_kv_append(cache, *y.split((n_q * D, n_kv * D, n_kv * D), 1), table, lens, None, None, qr, R=R)
        out = attend(cache, qr, None, table, lens, ws, R).view(2 * R, n_kv, n_q // n_kv, D)
        assert not torch.isfinite(out[R - 1, part]).any()
        assert torch.isfinite(out[:R, 1 - part]).all() and torch.isfinite(out[R:]).all()
