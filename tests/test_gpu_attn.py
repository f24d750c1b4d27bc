"""The attention step on the GPU (include/lk_attn.h): the rotated append bit
for bit against the same operations on the host, the attention calls against
the formula in 64 bits.

Tolerance of the attention (derived, not fitted).  An f32 operand enters the
MMAs as 16-bit terms: the rest after two bf16 terms is at most 2^-8 * 2^-8 =
2^-16 of it (half a step each), after two f16 terms 2^-22.  A score is a sum of D <= 128 products in 8 chained MMA steps (each
at worst truncating at 2^-22 of the absolute sum) and a few f32 operations:
off by at most 2^-18 * A with A = scale * sum_i |q_i k_i|, in natural units, and
a weight by that relative to itself.  Weights enter numerator and denominator
(factor 2); the weights' own terms add 2^-16, the sums over keys (32 to an
accumulator, then f32 additions in a tree or over at most a few hundred units)
stay below 2^-16.  So |out - exact| <= (2^-15 + c * A) * W, W = sum p |v| / sum p,
with the row's largest A and c = 2 * 2^-18 (f16, Q8: at most 2^-22 from the
queries' terms) or, against bf16 keys, 2 * (2^-18 + 2^-16) <= 2^-14.

f16 terms also end at 2^-24, which counts where W is far below the largest
value (a winner whose own value is 0): weights are shifted to at least 2^10 at
the row's largest, so a weight's low term is off by at most 2^-25 / 2^10 of it;
Q8 multiplies that by a scale of at most 16, brought to 8 .. 16 at the largest,
and rounds the product's low term once more: (16 + 1) 2^-25 / (2^10 * 8) < 2^-33
of 127 times the largest scale, which is below 2 max|v|: 2^-32 max|v| a key.  A
scale below 2^-18 of the largest is off by 2^-25 / 8 of that: 2^-28 * 127 scales, below
2^-27 max|v| over all weights.  Together (2^-27 + N 2^-32) max|v| for N keys."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from gpuhelp import act_buffers, bits, host  # noqa: E402
from q8_quantized_gemv_gb300 import build, lk  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "q8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    yield
    assert lk.lk_device_error(reset=True) == 0
    torch.cuda.empty_cache()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def make_cache(type_, n_pages, n_kv, page, D, g, spread=1.0):
    """(KvCache, f64 keys, f64 values) with pages of random values."""
    shape = (n_pages, n_kv, page, D)
    parts = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device=DEV) * spread + 0.1
        if type_ != "q8":
            x = x.to(TYPES[type_])
            parts.append((x, None, x.double()))
            continue
        b = x.view(*shape[:3], D // 32, 32)
        s = (b.abs().amax(-1) / 127).half()
        q = torch.round(b / s.float().unsqueeze(-1)).nan_to_num().clamp(-127, 127).to(torch.int8)
        parts.append((q.view(shape), s, (q.double() * s.double().unsqueeze(-1)).view(shape)))
    (k, ks, kd), (v, vs, vd) = parts
    return lk.KvCache(k, v, ks, vs), kd, vd


def make_table(B, width, n_pages, g, first=0):
    return (torch.randperm(n_pages - first, generator=g, device=DEV)[:B * width] + first).to(torch.int32).view(B, width)


def roomy(table, page):
    """The table with room for 9000 tokens more (no pages there)."""
    return torch.cat([table, torch.full((table.shape[0], -(-9000 // page)), -1, device=DEV, dtype=torch.int32)], 1)


def poison(cache, table, lens, page):
    """Everything of the sequences' pages behind their tokens becomes NaN (the
    levels of a Q8 cache -128, its scales NaN)."""
    t = host(table)
    for b, n in enumerate(lens):
        for i, p in enumerate(t[b]):
            if not 0 <= p < cache.k.shape[0]:
                continue
            a = max(0, min(page, n - i * page))
            for x in (cache.k, cache.v, cache.ks, cache.vs):
                if x is not None:
                    x[int(p), :, a:] = -128 if x.dtype == torch.int8 else float("nan")


def reference(kd, vd, q, table, lens, R, scale, prefix=None, bf16=True):
    """out and its tolerance [M, n_q * D] in 64 bits, row by row.  prefix: (page
    list, length).  Pages outside the cache hold no tokens."""
    n_pages, n_kv, page, D = kd.shape
    M = q.shape[0]
    n_q = q.shape[1] // D
    G = n_q // n_kv
    q = q.double().view(M, n_kv, G, D)
    out = torch.zeros((M, n_kv, G, D), dtype=torch.float64, device=DEV)
    A, W = torch.zeros((M, n_kv, G, 1), dtype=torch.float64, device=DEV), torch.zeros_like(out)
    F = torch.zeros((M, n_kv, 1, 1), dtype=torch.float64, device=DEV)

    def tokens(pages, n):
        t = pages.long()
        at = torch.arange(n, device=DEV)
        pg = t[at // page]
        ok = (pg >= 0) & (pg < n_pages)
        at, pg = at[ok], pg[ok]
        return kd[pg, :, at % page], vd[pg, :, at % page]  # [tokens, n_kv, D]

    for m in range(M):
        b, r = divmod(m, R)
        n = max(0, min(int(lens[b]) - R + 1 + r, table.shape[1] * page))
        k, v = tokens(table[b], n) if n else (kd[:0, :, 0], vd[:0, :, 0])
        if prefix is not None and lens[b] >= 0:
            pk, pv = tokens(prefix[0], prefix[1])
            k, v = torch.cat((pk, k)), torch.cat((pv, v))
        if not k.shape[0]:
            continue
        s = torch.einsum("hgd,nhd->hgn", q[m], k) * scale
        p = torch.softmax(s, -1)
        out[m] = torch.einsum("hgn,nhd->hgd", p, v)
        W[m] = torch.einsum("hgn,nhd->hgd", p, v.abs())
        F[m] = (2.0 ** -27 + k.shape[0] * 2.0 ** -32) * v.abs().amax((0, 2))[:, None, None]
        A[m] = (torch.einsum("hgd,nhd->hgn", q[m].abs(), k.abs()) * abs(scale)).amax(-1, keepdim=True)
    c = 2.0 ** -14 if bf16 else 2.0 ** -17
    return out.view(M, -1), ((2.0 ** -15 + c * A) * W + F).reshape(M, -1)


def workspace(cache, n_q, B, R, shared=False):
    n = lk.lk_attn_workspace_bytes(n_q, cache.n_kv, cache.head_dim, B, R, shared)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN in every word


def check(out, want, tol):
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    bad = err > tol + 1e-30
    assert not bad.any(), (int(bad.sum()), float((err / (tol + 1e-30)).max()))


# ---- append --------------------------------------------------------------------------

def host_append(x, cos, sin, pos, paired, gain, eps=1e-6):
    """x f32 [heads, D] of one row (numpy), rounded as the header says."""
    x = x.astype(np.float32)
    if gain is not None:
        d = x.astype(np.float64)
        den = np.sqrt((d * d).sum(-1, keepdims=True) / x.shape[-1] + np.float64(np.float32(eps)))
        x = (d * gain.astype(np.float64) / den).astype(np.float32)
    if cos is None:
        return x
    rot = 2 * cos.shape[1]
    c, s = cos[pos], sin[pos]
    y = x.copy()
    ia = np.arange(0, rot, 2) if paired else np.arange(rot // 2)
    ib = ia + 1 if paired else ia + rot // 2
    a, b = x[:, ia], x[:, ib]
    y[:, ia] = a * c - b * s
    y[:, ib] = b * c + a * s
    return y


def host_quant(x):
    b = x.reshape(*x.shape[:-1], -1, 32)
    a = np.abs(b).max(-1)
    s = np.minimum(a / np.float32(127), np.float32(65504)).astype(np.float16)
    f = s.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(f > 0, np.clip(np.rint(b / f), -127, 127), 0)
    return z.astype(np.int8).reshape(x.shape), s


APPEND = [
    # type, D, n_q, n_kv, page, B, R, lens, rot, paired, norm, p0, fused
    ("f16", 128, 32, 8, 64, 1, 1, [1], 128, False, False, 0, True),
    ("f16", 64, 5, 5, 16, 3, 2, [2, 1, 40], 64, True, True, 7, False),
    ("bf16", 128, 10, 2, 32, 2, 17, [17, 65], 64, False, True, 0, True),
    ("bf16", 64, 4, 1, 128, 64, 1, None, 64, False, False, 100, True),
    ("bf16", 128, 7, 1, 16, 4, 1, [0, -5, 33, 16], 0, False, False, 0, False),
    ("q8", 128, 32, 8, 64, 5, 1, [1, 64, 65, 128, 0], 128, False, True, 0, True),
    ("q8", 64, 8, 4, 1024, 2, 3, [3, 1000], 64, True, False, 3, False),
    ("q8", 128, 4, 4, 16, 1, 64, [70], 128, True, True, 0, True),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c[:7]))
def test_append_bits(case):
    type_, D, n_q, n_kv, page, B, R, lens, rot, paired, norm, p0, fused = case
    g = gen(11 + D + B)
    if lens is None:
        lens = [1 + (37 * b) % 200 for b in range(B)]
    width = max(1, -(-max(lens) // page))
    n_pages = B * width + 2
    cache, _, _ = make_cache(type_, n_pages, n_kv, page, D, g)
    table = make_table(B, width, n_pages, g)
    M = B * R
    if fused:
        x = torch.randn((M, (n_q + 2 * n_kv) * D), generator=g, device=DEV)
        q, k, v = x.split((n_q * D, n_kv * D, n_kv * D), 1)
    else:
        pitch = max(n_q, n_kv) * D + 4
        x = torch.randn((3, M, pitch), generator=g, device=DEV)
        q, k, v = x[0, :, :n_q * D], x[1, :, :n_kv * D], x[2, :, :n_kv * D]
    if type_ == "q8":  # zero groups, tiny and huge ones
        v[0, :32] = 0
        k[-1, 32:64] = 1e-9
        v[-1, 32:64] *= 1e6
    n_pos = p0 + max(lens) + 1
    ang = torch.rand((n_pos, max(1, rot // 2)), generator=g, device=DEV) * 100
    cos, sin = (ang.cos(), ang.sin()) if rot else (None, None)
    qg = torch.rand((D,), generator=g, device=DEV) + 0.5 if norm else None
    kg = torch.rand((D,), generator=g, device=DEV) + 0.5 if norm else None
    qr = torch.full((M, n_q * D), 7.0, device=DEV)
    before = [None if t is None else host(t.float()).copy() for t in (cache.k, cache.v, cache.ks, cache.vs)]
    lk.lk_kv_append(cache, q, k, v, table, torch.tensor(lens, dtype=torch.int32, device=DEV), cos, sin, qr, R=R, p0=p0,
                    paired=paired, q_gain=qg, k_gain=kg)
    torch.cuda.synchronize()
    hq, hk, hv, t = host(q), host(k), host(v), host(table)
    hc, hs_ = (host(cos), host(sin)) if rot else (None, None)
    want_q = np.full((M, n_q * D), 7.0, np.float32)
    for m in range(M):
        b, r = divmod(m, R)
        p = lens[b] - R + r
        if p < 0:
            continue
        want_q[m] = host_append(hq[m].reshape(n_q, D), hc, hs_, p0 + p, paired, host(qg) if norm else None).ravel()
        nk = host_append(hk[m].reshape(n_kv, D), hc, hs_, p0 + p, paired, host(kg) if norm else None)
        nv = hv[m].reshape(n_kv, D)
        at = (int(t[b, p // page]), slice(None), p % page)
        if type_ == "q8":
            (before[0][at], before[2][at]), (before[1][at], before[3][at]) = host_quant(nk), host_quant(nv)
        else:
            for i, z in ((0, nk), (1, nv)):
                before[i][at] = torch.from_numpy(z.copy()).to(TYPES[type_]).float().numpy()
    assert np.array_equal(bits(host(qr)), bits(want_q))
    for t_, w in zip((cache.k, cache.v, cache.ks, cache.vs), before):
        if t_ is not None:
            assert np.array_equal(host(t_.float()), w)


def test_append_norm_bits():
    """The norm's quick form against its definition in 64 bits, over wide
    magnitudes (where it hands over to the f64 form) and signed zeros."""
    g = gen(6)
    cache, _, _ = make_cache("f16", 70, 1, 16, 128, g)
    table = torch.arange(64, dtype=torch.int32, device=DEV).view(64, 1)
    lens = torch.ones((64,), dtype=torch.int32, device=DEV)
    for spread, gain in ((1.0, 1.0), (1e-3, 1.0), (300.0, 1e-4), (1e-25, 1.0), (1e25, 1.0), (1e-6, 1e9)):
        x = torch.randn((64, 34 * 128), generator=g, device=DEV) * spread
        x[:, ::7] = 0.0
        x[:, 3::11] = -0.0
        qg = torch.randn((128,), generator=g, device=DEV) * gain
        qr = torch.empty((64, 32 * 128), device=DEV)
        lk.lk_kv_append(cache, *x.split((4096, 128, 128), 1), table, lens, None, None, qr, q_gain=qg, k_gain=qg)
        want = np.stack([host_append(r.reshape(32, 128), None, None, 0, False, host(qg)).ravel() for r in host(x[:, :4096])])
        assert np.array_equal(bits(host(qr)), bits(want)), (spread, gain)


def test_append_leaves_out_what_has_no_place():
    """Tokens past the table, in pages outside the cache or past the rotation
    table change nothing."""
    g = gen(5)
    cache, _, _ = make_cache("f16", 6, 2, 16, 64, g)
    k0, v0 = cache.k.clone(), cache.v.clone()
    table = torch.tensor([[0, 1], [-1, 99], [2, 3], [4, 6]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([33, 17, 31, 20], dtype=torch.int32, device=DEV)  # no room; bad page; past n_pos; page == n_pages
    x = torch.randn((4, 8 * 64), generator=g, device=DEV)
    cos = torch.ones((25, 32), device=DEV)
    qr = torch.full((4, 4 * 64), 3.0, device=DEV)
    lk.lk_kv_append(cache, *x.split((256, 128, 128), 1), table, lens, cos, cos, qr)
    lens.fill_(2 ** 31 - 1)
    lk.lk_kv_append(cache, *x.split((256, 128, 128), 1), table, lens, None, None, qr)
    lens.fill_(-2 ** 31)
    lk.lk_kv_append(cache, *x.split((256, 128, 128), 1), table, lens, None, None, qr)
    torch.cuda.synchronize()
    assert (qr == 3.0).all() and torch.equal(cache.k, k0) and torch.equal(cache.v, v0)


# ---- attention -----------------------------------------------------------------------

def run_attn(type_, D, n_q, n_kv, page, R, lens, seed=3, prefix=0, spread=1.0, scale=None, bad_pages=(), q_scale=2.0):
    g = gen(seed)
    B = len(lens)
    width = max(1, -(-max(max(lens), 1) // page))
    p_pages = -(-prefix // page) + (1 if prefix else 0)
    n_pages = p_pages + B * width + 1
    cache, kd, vd = make_cache(type_, n_pages, n_kv, page, D, g, spread)
    table = make_table(B, width, n_pages, g, p_pages)
    for b, i, p in bad_pages:
        table[b, i] = p
    poison(cache, table, lens, page)
    ptable = torch.arange(p_pages, device=DEV, dtype=torch.int32).flip(0).contiguous()
    if prefix:
        poison(cache, ptable[None], [prefix], page)
    q = q_scale * torch.randn((B * R, n_q * D), generator=g, device=DEV)
    out = torch.full((B * R + 1, n_q * D), 9.0, device=DEV)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    sc = D ** -0.5 if scale is None else scale
    ws = workspace(cache, n_q, B, R, bool(prefix))
    if prefix:
        lk.lk_attn_shared(cache, q, ptable, prefix, table, lt, ws, R=R, scale=scale, out=out[:-1])
    else:
        lk.lk_attn(cache, q, table, lt, ws, R=R, scale=scale, out=out[:-1])
    torch.cuda.synchronize()
    assert (out[-1] == 9.0).all()
    want, tol = reference(kd, vd, q, table, lens, R, sc, (ptable, prefix) if prefix else None, type_ == "bf16")
    check(out[:-1], want, tol)
    # with room for more, the keys are split in another way
    wide = roomy(table, page)
    if prefix:
        lk.lk_attn_shared(cache, q, ptable, prefix, wide, lt, ws, R=R, scale=scale, out=out[:-1])
    else:
        lk.lk_attn(cache, q, wide, lt, ws, R=R, scale=scale, out=out[:-1])
    torch.cuda.synchronize()
    assert (out[-1] == 9.0).all()
    check(out[:-1], want, tol)
    return out[:-1], want


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 255, 300]


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_attn_lengths(type_, D, page):
    run_attn(type_, D, 8, 2, page, 1, EDGES)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (8, 8), (10, 2), (7, 1), (16, 2), (40, 2), (71, 1)])
def test_attn_heads(type_, n_q, n_kv):
    run_attn(type_, 128, n_q, n_kv, 32, 1, [77, 1, 500])
    run_attn(type_, 64, n_q, n_kv, 16, 2, [33, 2])


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("R,lens", [(2, [2, 1, 0, 33, 64]), (5, [5, 3, 4, 100, 129, 31]), (64, [64]), (64, [700]),
                                    (21, [21, 400, 20]), (61, [33])])
def test_attn_several_new_tokens(type_, R, lens):
    """Row r of R sees the keys up to its own; rows before the first see none."""
    run_attn(type_, 128, 8, 2, 16, R, lens)
    run_attn(type_, 64, 3, 1, 64, R, lens)
    out, want = run_attn(type_, 128, 40, 8, 32, R, lens)
    if any(n >= R for n in lens):
        assert ((out.double() - want).norm() / want.norm()).item() < 2.0 ** -16


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_q", [32, 72])
def test_attn_many_pieces_to_a_block(type_, D, n_q):
    """Several new tokens of sequences from one tile to many, so that a block
    has the end of one, whole ones of a single tile and the start of another."""
    lens = [30, 700, 5, 64, 128, 2000, 129, 90, 65, 10, 300, 127]
    run_attn(type_, D, n_q, 8, 32, 5, lens)
    run_attn(type_, D, n_q, 8, 32, 5, lens, prefix=200)


@pytest.mark.parametrize("type_", list(TYPES))
def test_attn_long_ragged_batch(type_):
    """One long context among short ones and padding: split over the blocks."""
    out, want = run_attn(type_, 128, 32, 8, 64, 1, [20000, 1, 0, 300, 4097, 64, -3, 2000])
    assert ((out.double() - want).norm() / want.norm()).item() < 2.0 ** -16
    out, want = run_attn(type_, 64, 4, 1, 16, 1, [33333])
    assert ((out.double() - want).norm() / want.norm()).item() < 2.0 ** -16


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("spread", [1e-4, 30.0])
def test_attn_magnitudes(type_, spread):
    """Small and large cached values; scores from flat to a single winner."""
    run_attn(type_, 128, 8, 2, 32, 1, [300, 1000, 5], spread=spread)
    run_attn(type_, 128, 8, 2, 32, 1, [300, 1000, 5], spread=spread, scale=-0.02)
    run_attn(type_, 64, 8, 2, 32, 1, [300, 1000, 5], spread=spread, scale=0.0)
    run_attn(type_, 128, 8, 2, 32, 1, [300, 1000, 5], spread=spread, q_scale=1e-20)


def test_attn_pages_outside_the_cache_hold_no_tokens():
    for type_ in TYPES:
        run_attn(type_, 64, 4, 2, 16, 1, [100, 100, 16, 40],
                 bad_pages=[(0, 0, -1), (0, 3, 10 ** 6), (1, 6, -2 ** 31), (2, 0, 2 ** 31 - 1)])


def test_attn_lens_past_the_table():
    """A length past the table's room means the table's room."""
    g = gen(8)
    cache, kd, vd = make_cache("f16", 8, 2, 16, 64, g)
    table = make_table(2, 3, 8, g)
    q = torch.randn((2, 256), generator=g, device=DEV)
    out = torch.empty_like(q)
    lens = torch.tensor([2 ** 31 - 1, 49], dtype=torch.int32, device=DEV)
    lk.lk_attn(cache, q, table, lens, workspace(cache, 4, 2, 1), out=out)
    check(out, *reference(kd, vd, q, table, [48, 48], 1, 0.125, bf16=False))
    empty = torch.empty((2, 0), dtype=torch.int32, device=DEV)
    lk.lk_attn(cache, q, empty, lens, workspace(cache, 4, 2, 1), out=out)
    assert (out == 0).all()


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("B,R,n_q,n_kv,prefix", [(1, 1, 4, 4, 1), (3, 1, 8, 2, 31), (5, 2, 4, 1, 500),
                                                 (64, 1, 8, 2, 1029), (16, 4, 10, 2, 4000), (2, 1, 32, 8, 9000),
                                                 (5, 2, 8, 2, 14001), (7, 1, 28, 4, 22000), (64, 1, 8, 2, 4099)])
def test_shared_prefix(type_, B, R, n_q, n_kv, prefix):
    lens = [(R + 13 * b) % 70 for b in range(B)]
    run_attn(type_, 128, n_q, n_kv, 16, R, lens, prefix=prefix)
    out, want = run_attn(type_, 64, n_q, n_kv, 64, R, lens, prefix=prefix)
    # the terms' errors are independent: far below the worst case on the whole
    assert ((out.double() - want).norm() / want.norm()).item() < 2.0 ** -16


def test_shared_prefix_padding_and_empty():
    """lens 0: the prefix alone; lens < 0: zeros; prefix_len 0: lk_attn."""
    for type_ in TYPES:
        run_attn(type_, 128, 8, 2, 32, 1, [0, -1, 5, -2 ** 31, 0], prefix=77)
        run_attn(type_, 128, 16, 2, 32, 1, [0, -1, 5, -2 ** 31, 0], prefix=20000)
    g = gen(9)
    cache, _, _ = make_cache("bf16", 8, 2, 16, 64, g)
    table = make_table(2, 3, 8, g)
    q = torch.randn((2, 256), generator=g, device=DEV)
    lens = torch.tensor([40, 7], dtype=torch.int32, device=DEV)
    a, b = torch.empty_like(q), torch.empty_like(q)
    lk.lk_attn(cache, q, table, lens, workspace(cache, 4, 2, 1), out=a)
    lk.lk_attn_shared(cache, q, None, 0, table, lens, workspace(cache, 4, 2, 1), out=b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("room", [False, True])
def test_attn_quantized_output(mode, D, room):
    """The words are the quantizer's of the f32 rows, which they do not change."""
    g = gen(21)
    cache, _, _ = make_cache("q8", 40, 2, 32, D, g)
    table = make_table(4, 8, 40, g)
    if room:
        table = roomy(table, 32)
    lens = torch.tensor([200, 0, 1, 77], dtype=torch.int32, device=DEV)
    N = 8 * D
    q = torch.randn((4, N), generator=g, device=DEV)
    ws, plain, out = workspace(cache, 8, 4, 1), torch.empty_like(q), torch.empty_like(q)
    lk.lk_attn(cache, q, table, lens, ws, out=plain)
    hq, hl, hs = act_buffers(4, N, mode)
    lk.lk_attn(cache, q, table, lens, ws, mode=mode, out=out, hq=hq, hl=hl, hs=hs)
    torch.cuda.synchronize()
    assert torch.equal(out, plain)
    hi, lo, s = oracle.quantize(host(out), mode)
    assert np.array_equal(host(hq), hi) and np.array_equal(bits(host(hs)), bits(s))
    if mode == 2:
        assert np.array_equal(host(hl), lo)
    hq2, hl2, hs2 = act_buffers(4, N, mode)
    lk.lk_attn(cache, q, table, lens, ws, mode=mode, hq=hq2, hl=hl2, hs=hs2)  # no f32 rows
    assert torch.equal(hq, hq2) and torch.equal(hs, hs2)
    lk.lk_attn(cache, q, table, lens, ws, out=q)  # in place of the queries
    assert torch.equal(q, plain)


def test_offsets_past_32_bits():
    """Pages whose byte and element offsets pass 2^32."""
    for type_, n_pages in (("q8", 70000), ("f16", 40000)):
        page, n_kv, D = 64, 8, 128
        shape = (n_pages, n_kv, page, D)
        k = torch.empty(shape, dtype=TYPES[type_], device=DEV)
        v = torch.empty(shape, dtype=TYPES[type_], device=DEV)
        ks = vs = None
        if type_ == "q8":
            ks = torch.empty((*shape[:3], 4), dtype=torch.float16, device=DEV)
            vs = torch.empty_like(ks)
        cache = lk.KvCache(k, v, ks, vs)
        small, kd, vd = make_cache(type_, 4, n_kv, page, D, gen(31))
        at = [n_pages - 1, n_pages // 2 + 1, 0, n_pages - 7]
        for i, p in enumerate(at):
            for big, s in ((k, small.k), (v, small.v), (ks, small.ks), (vs, small.vs)):
                if big is not None:
                    big[p] = s[i]
        table = torch.tensor([at], dtype=torch.int32, device=DEV)
        lens = torch.tensor([250], dtype=torch.int32, device=DEV)
        q = torch.randn((1, 32 * D), generator=gen(32), device=DEV)
        out = torch.empty_like(q)
        lk.lk_attn(cache, q, table, lens, workspace(cache, 32, 1, 1), out=out)
        t4 = torch.arange(4, dtype=torch.int32, device=DEV)[None]
        check(out, *reference(kd, vd, q, t4, [250], 1, D ** -0.5, bf16=False))
        # an append there
        x = torch.randn((1, 48 * D), generator=gen(33), device=DEV)
        lens.fill_(251)
        lk.lk_kv_append(cache, *x.split((32 * D, 8 * D, 8 * D), 1), table, lens, None, None, out)
        lk.lk_kv_append(small, *x.split((32 * D, 8 * D, 8 * D), 1), t4, lens, None, None, out)
        assert torch.equal(k[at[3], :, 250 - 192], small.k[3, :, 250 - 192])
        assert torch.equal(v[at[3], :, 250 - 192], small.v[3, :, 250 - 192])
        del k, v, ks, vs, cache
        torch.cuda.empty_cache()


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("items", [1, 14, 15, 22, 23, 27, 28, 34, 35, 44, 45, 74, 75, 150, 151])
def test_attn_cluster_sizes(type_, items):
    """The numbers of key/value heads and sequences where the split changes."""
    n_kv, B = next((k, items // k) for k in (1, 2, 3, 5, 23, 37, 75, 151) if items % k == 0 and items // k <= 22)
    lens = [(97 * b + 700) % 901 for b in range(B)]
    run_attn(type_, 64, 3 * n_kv, n_kv, 32, 1, lens)
    run_attn(type_, 128, n_kv, n_kv, 64, 1, lens, prefix=45)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("R", [1, 12])
def test_attn_nothing_to_see(type_, R):
    """No sequence has a token."""
    out, _ = run_attn(type_, 128, 8, 2, 16, R, [0, -1, 0])
    assert (out == 0).all()
    run_attn(type_, 64, 8, 2, 1024, R, [0, 0], prefix=3)


@pytest.mark.parametrize("type_", list(TYPES))
def test_attn_many_rows_on_large_pages(type_):
    run_attn(type_, 128, 8, 2, 1024, 64, [1500])
    run_attn(type_, 64, 8, 2, 256, 16, [999, 20, 256])


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("R", [1, 16])
def test_attn_a_bad_row_changes_no_other(type_, R, room):
    """Padding rows may hold anything: NaN and infinity stay in their rows."""
    g = gen(61)
    cache, _, _ = make_cache(type_, 60, 2, 16, 128, g)
    table = make_table(3, 12, 60, g)
    if room:
        table = roomy(table, 16)
    lens = torch.tensor([150, 0, 77], dtype=torch.int32, device=DEV)
    q = torch.randn((3 * R, 16 * 128), generator=g, device=DEV)
    ws, want, out = workspace(cache, 16, 3, R), torch.empty_like(q), torch.empty_like(q)
    lk.lk_attn(cache, q, table, lens, ws, R=R, out=want)
    bad = q.clone()
    bad[R:2 * R] = float("nan")
    bad[0, :128], bad[0, 128:256] = float("inf"), float("nan")
    lk.lk_attn(cache, bad, table, lens, ws, R=R, out=out)
    assert (out[R:2 * R] == 0).all()
    assert torch.equal(out[0, 256:], want[0, 256:])
    assert torch.equal(out[1:R], want[1:R]) and torch.equal(out[2 * R:], want[2 * R:])


def test_one_workspace_for_calls_in_a_row():
    """Dependent launches of different calls on one stream share a workspace."""
    g = gen(71)
    cfg = lk.launch_cfg(pdl=1)
    cache, _, _ = make_cache("f16", 700, 4, 32, 128, g)
    ptable = torch.arange(600, 700, dtype=torch.int32, device=DEV)
    calls, n = [], 0
    for B, R, shared in ((4, 1, False), (2, 20, False), (8, 1, True), (64, 1, True), (1, 3, False), (9, 1, False)):
        table = torch.randint(0, 600, (B, 40), generator=g, device=DEV, dtype=torch.int32)
        lens = torch.randint(R, 1280, (B,), generator=g, device=DEV, dtype=torch.int32)
        q = torch.randn((B * R, 16 * 128), generator=g, device=DEV)
        n = max(n, lk.lk_attn_workspace_bytes(16, 4, 128, B, R, shared))
        calls.append((B, R, shared, table, lens, q, torch.empty_like(q), torch.empty_like(q)))
    ws = torch.empty((n,), dtype=torch.uint8, device=DEV)

    def run(c, out, cfg=None):
        B, R, shared, table, lens, q = c[:6]
        if shared:
            lk.lk_attn_shared(cache, q, ptable, 3190, table, lens, ws, R=R, out=out, cfg=cfg)
        else:
            lk.lk_attn(cache, q, table, lens, ws, R=R, out=out, cfg=cfg)

    for c in calls:
        run(c, c[6])
        torch.cuda.synchronize()
    for _ in range(10):
        for c in calls:
            run(c, c[7], cfg)
    torch.cuda.synchronize()
    for c in calls:
        assert torch.equal(c[6], c[7])


def test_shortest_wait_limit():
    """Under the shortest limit a call either keeps it and gives its result or
    raises the error word; the context and the next calls are as they were."""
    for type_ in TYPES:
        g = gen(81)
        cache, _, _ = make_cache(type_, 500, 2, 64, 128, g)
        lens = torch.tensor([12000, 9000], dtype=torch.int32, device=DEV)
        for R, width in ((1, 200), (24, 200), (1, 100)):
            table = make_table(2, width, 500, g)
            q = torch.randn((2 * R, 8 * 128), generator=g, device=DEV)
            ws, want, out = workspace(cache, 8, 2, R), torch.empty_like(q), torch.empty_like(q)
            lk.lk_attn(cache, q, table, lens, ws, R=R, out=want)
            torch.cuda.synchronize()
            assert lk.lk_device_error(reset=True) == 0
            lk.lk_set_option("wait_us", 1)
            try:
                lk.lk_attn(cache, q, table, lens, ws, R=R, out=out)
                torch.cuda.synchronize()
            finally:
                lk.lk_set_option("wait_us", 0)
            assert lk.lk_device_error(reset=True) != 0 or torch.equal(out, want)
            lk.lk_attn(cache, q, table, lens, ws, R=R, out=out)
            torch.cuda.synchronize()
            assert lk.lk_device_error(reset=True) == 0 and torch.equal(out, want)


# ---- a run of them together ------------------------------------------------------------

@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("pdl", [0, 1])
def test_append_and_attend_token_by_token(type_, pdl):
    """Tokens appended and attended one at a time, in a captured graph that is
    replayed with advancing lengths, against the formula on what the cache
    holds; the same steps as plain calls give the same bits."""
    B, n_q, n_kv, D, page, prefix = 3, 8, 2, 128, 16, 40
    g = gen(77)
    cfg = lk.launch_cfg(pdl=pdl)
    cache, _, _ = make_cache(type_, 24, n_kv, page, D, g)
    ptable = torch.tensor([20, 5, 23], dtype=torch.int32, device=DEV)
    free = torch.tensor([i for i in range(24) if i not in (20, 5, 23)], dtype=torch.int32, device=DEV)
    table = free[:18].view(3, 6)
    start = [k.clone() for k in (cache.k, cache.v)] + [k.clone() for k in (cache.ks, cache.vs) if k is not None]
    ang = torch.rand((200, D // 2), generator=g, device=DEV) * 6
    cos, sin = ang.cos(), ang.sin()
    x = torch.zeros((B, (n_q + 2 * n_kv) * D), device=DEV)
    lens = torch.tensor([0, 15, 30], dtype=torch.int32, device=DEV)
    qr, out = torch.zeros((B, n_q * D), device=DEV), torch.zeros((B, n_q * D), device=DEV)
    hq, _, hs = act_buffers(B, n_q * D, 1)
    ws = workspace(cache, n_q, B, 1, True)
    q, k, v = x.split((n_q * D, n_kv * D, n_kv * D), 1)

    def step():
        lens.add_(1)
        lk.lk_kv_append(cache, q, k, v, table, lens, cos, sin, qr, p0=prefix, cfg=cfg)
        lk.lk_attn_shared(cache, qr, ptable, prefix, table, lens, ws, mode=1, out=out, hq=hq, hs=hs, cfg=cfg)

    xs = torch.randn((9, *x.shape), generator=g, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()

    def restart():
        lens.copy_(torch.tensor([0, 15, 30], dtype=torch.int32))
        for t, s in zip([t for t in (cache.k, cache.v, cache.ks, cache.vs) if t is not None], start):
            t.copy_(s)

    def dense(t, s):
        return t.double() if s is None else (t.double().view(*s.shape, 32) * s.double().unsqueeze(-1)).view(t.shape)

    restart()
    got = []
    for i in range(9):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        got.append(out.clone())
        want, tol = reference(dense(cache.k, cache.ks), dense(cache.v, cache.vs), qr, table, host(lens).tolist(), 1,
                              D ** -0.5, (ptable, prefix), type_ == "bf16")
        check(out, want, tol)
        hi, _, s = oracle.quantize(host(out), 1)
        assert np.array_equal(host(hq), hi) and np.array_equal(bits(host(hs)), bits(s))
    restart()
    for i in range(9):
        x.copy_(xs[i])
        step()
        assert torch.equal(out, got[i])


@pytest.mark.parametrize("room", [False, True])
def test_two_streams_with_a_workspace_each(room):
    g = gen(41)
    cache, _, _ = make_cache("bf16", 300, 4, 32, 128, g)
    sets = []
    for i in range(2):
        table = make_table(4, 64, 300, g)
        if room:
            table = roomy(table, 32)
        lens = torch.tensor([2000, 100 + i, 33, 1500], dtype=torch.int32, device=DEV)
        q = torch.randn((4, 16 * 128), generator=g, device=DEV)
        sets.append((table, lens, q, workspace(cache, 16, 4, 1), torch.empty_like(q), torch.empty_like(q),
                     torch.cuda.Stream()))
    for table, lens, q, ws, want, _, _ in sets:
        lk.lk_attn(cache, q, table, lens, ws, out=want)
    torch.cuda.synchronize()
    for _ in range(20):
        for table, lens, q, ws, _, got, s in sets:
            lk.lk_attn(cache, q, table, lens, ws, out=got, stream=s)
    torch.cuda.synchronize()
    for _, _, _, _, want, got, _ in sets:
        assert torch.equal(want, got)


def test_binding_refusals():
    g = gen(51)
    cache, _, _ = make_cache("f16", 4, 2, 16, 64, g)
    table = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    lens = torch.ones((2,), dtype=torch.int32, device=DEV)
    q, ws = torch.zeros((2, 256), device=DEV), workspace(cache, 4, 2, 1)
    out = torch.zeros_like(q)
    for kw, err in ((dict(q=q[:1]), ValueError), (dict(q=q.double()), TypeError), (dict(q=q.cpu()), ValueError),
                    (dict(table=table[0]), ValueError), (dict(table=table.long()), TypeError),
                    (dict(lens=lens[:1]), ValueError), (dict(ws=ws[:-1]), lk.LkError), (dict(out=None), lk.LkError),
                    (dict(out=out[:1]), ValueError), (dict(R=2), ValueError), (dict(R=-1), ValueError),
                    (dict(scale=float("nan")), lk.LkError), (dict(q=q[:, ::2]), ValueError)):
        a = dict(q=q, table=table, lens=lens, ws=ws, out=out, R=1)
        a.update(kw)
        with pytest.raises(err):
            lk.lk_attn(cache, a.pop("q"), a.pop("table"), a.pop("lens"), a.pop("ws"), **a)
    k, q2, qr = (torch.zeros((2, 128), device=DEV) for _ in range(3))
    cos = torch.ones((9, 32), device=DEV)
    for kw, err in ((dict(k=k[:, :64]), ValueError), (dict(v=k[:1]), ValueError), (dict(q=q2.half()), TypeError),
                    (dict(k=torch.zeros((2, 256), device=DEV)[:, :128]), ValueError), (dict(sines=cos[:3]), ValueError),
                    (dict(cosines=None), ValueError), (dict(cosines=cos[:, :16].contiguous(), sines=None), lk.LkError),
                    (dict(qr=q2), lk.LkError), (dict(q_gain=cos), ValueError), (dict(qr=qr[:1]), ValueError)):
        a = dict(q=q2, k=k, v=k, table=table, lens=lens, cosines=cos, sines=cos, qr=qr)
        a.update(kw)
        with pytest.raises(err):
            lk.lk_kv_append(cache, *[a.pop(n) for n in ("q", "k", "v", "table", "lens", "cosines", "sines", "qr")], **a)
