"""Decode tokens with the attention step in place (DecodeStack(attn=...)): every
layer's append and attention against the formula in 64 bits on the layer's own
q, k and v, the o projection's quantized activation against the oracle's
quantizer, and the token as one captured graph of dependent launches with the
bits of the plain launches."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from gpuhelp import bits, host  # noqa: E402
from q8_quantized_gemv_gb300 import build, lk  # noqa: E402
from q8_quantized_gemv_gb300.decode import Attention, DecodeStack  # noqa: E402
from test_gpu_attn import check, host_append, host_quant, reference  # noqa: E402

pytestmark = pytest.mark.gpu

SMALL = dict(layers=2, hidden=1024, q_dim=1024, kv_dim=256, ffn=1536, vocab=3000, glu=True)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    yield
    assert lk.lk_device_error(reset=True) == 0


def dense(t, s):
    return t.double() if s is None else (t.double().view(*s.shape, 32) * s.double().unsqueeze(-1)).view(t.shape)


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("batch,tokens,prefix", [(1, 30, 0), (3, [0, 31, -1], 0), (8, 5, 50)])
def test_token_with_attention(kv, mode, batch, tokens, prefix):
    at = Attention(kv=kv, page=16, capacity=80, tokens=tokens, prefix=prefix)
    st = DecodeStack(**SMALL, batch=batch, mode=mode, attn=at)
    B, n_q, n_kv, D = batch, at.n_q, at.n_kv, at.D
    steps = []

    def hook(name, launch):
        if name == "attn":
            l = len(steps) % st.L
            torch.cuda.synchronize()
            before = [None if t is None else t.clone() for t in (at.caches[l].k, at.caches[l].v, at.caches[l].ks, at.caches[l].vs)]
            rec = dict(before=before, qkv=host(st.out_qkv).copy(), lens=host(at.lens).tolist())
            r = launch()
            torch.cuda.synchronize()
            rec.update(qr=at.qr.clone(), act={k: host(v).copy() for k, v in r.items()},
                       after=[None if t is None else t.clone() for t in (at.caches[l].k, at.caches[l].v, at.caches[l].ks, at.caches[l].vs)])
            steps.append(rec)
            return r
        return launch()

    st.run_token(hook=hook)
    st.run_token(hook=hook)
    torch.cuda.synchronize()
    assert len(steps) == 2 * st.L
    table, cos, sin = host(at.table), host(at.cos), host(at.sin)
    first = [tokens] * B if isinstance(tokens, int) else tokens
    for i, rec in enumerate(steps):
        l = i % st.L
        assert rec["lens"] == [t + 1 + i // st.L if t >= 0 else t for t in first]
        qg, kg = (host(g) for g in at.gains[l])
        want = [None if t is None else host(t.float()).copy() for t in rec["before"]]
        for b, n in enumerate(rec["lens"]):
            if n <= 0:
                continue
            x = rec["qkv"][b].reshape(-1, D)
            q = host_append(x[:n_q], cos, sin, prefix + n - 1, False, qg)
            assert np.array_equal(bits(host(rec["qr"][b]).reshape(n_q, D)), bits(q))
            k, v = host_append(x[n_q:n_q + n_kv], cos, sin, prefix + n - 1, False, kg), x[n_q + n_kv:]
            where = (int(table[b, (n - 1) // at.page]), slice(None), (n - 1) % at.page)
            if kv == "q8":
                (want[0][where], want[2][where]), (want[1][where], want[3][where]) = host_quant(k), host_quant(v)
            else:
                dt = rec["before"][0].dtype
                want[0][where], want[1][where] = (torch.from_numpy(z.copy()).to(dt).float().numpy() for z in (k, v))
        for t, w in zip(rec["after"], want):
            assert (t is None) == (w is None) and (t is None or np.array_equal(host(t.float()), w))
        out, tol = reference(dense(rec["after"][0], rec["after"][2]), dense(rec["after"][1], rec["after"][3]), rec["qr"],
                             at.table, rec["lens"], 1, D ** -0.5, (at.prefix_table, prefix) if prefix else None, kv == "bf16")
        if mode == 0:
            check(torch.from_numpy(rec["act"]["x"]).to(out.device), out, tol)
        else:
            # the words are the quantizer's of a row within the tolerance: at most one step from it
            a, s = rec["act"], np.repeat(rec["act"]["xs"].astype(np.float64), 32, 1)
            val = a["xq"] * s + (a["xl"] * s / 128 if mode == 2 else 0.0)
            step = s * (0.5 if mode == 1 else 0.5 / 128) * (1 + 2.0 ** -10)
            assert np.all(np.abs(val - host(out)) <= step + host(tol) + 1e-30)

    # one captured graph of dependent launches, from the same start
    plain = host(st.logits).copy(), host(st.idx).copy()
    st.pdl = True
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        st.run_token()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st.run_token()
    at.restart()
    for c, rec in zip(at.caches, steps):
        for t, b in zip((c.k, c.v, c.ks, c.vs), rec["before"]):
            if t is not None:
                t.copy_(b)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(host(st.logits)), bits(plain[0])) and np.array_equal(host(st.idx), plain[1])


def test_attention_needs_its_dataflow():
    with pytest.raises(ValueError):
        DecodeStack(**dict(SMALL, glu=False), attn=Attention(capacity=64))
    with pytest.raises(ValueError):
        DecodeStack(**SMALL, fused_qkv=False, attn=Attention(capacity=64))
    with pytest.raises(ValueError):
        DecodeStack(**dict(SMALL, kv_dim=192), attn=Attention(capacity=64))
    with pytest.raises(ValueError):
        DecodeStack(**SMALL, attn=Attention(capacity=64, tokens=64))
    with pytest.raises(ValueError):
        Attention(kv="f32")


def test_attention_belongs_to_one_stack():
    at = Attention(page=16, capacity=34, tokens=[30, -1])
    st = DecodeStack(**SMALL, batch=2, attn=at)
    with pytest.raises(ValueError):
        DecodeStack(**SMALL, batch=2, attn=at)
    for left in (4, 3, 2, 1):
        assert at.room() == left
        st.run_token()
    assert at.room() == 0
    # what a full sequence does not take changes nothing in the cache
    before = [t.clone() for c in at.caches for t in (c.k, c.v)]
    st.run_token()
    torch.cuda.synchronize()
    assert all(torch.equal(a, t) for a, t in zip(before, [t for c in at.caches for t in (c.k, c.v)]))
    at.restart()
    assert at.room() == 4
