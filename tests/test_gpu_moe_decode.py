"""Tokens of a small decoder stack whose layers have a mixture of experts and
whose tokens are drawn: every step against its definition in 64 bits on its own
inputs, and the same bits from a captured graph of dependent launches."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moehelp import act_value, down_ref, glu_ref, route_ref, sample_ref  # noqa: E402

pytestmark = pytest.mark.gpu
SIZE = dict(layers=2, hidden=512, q_dim=512, kv_dim=128, ffn=256, vocab=5003, glu=True)


@pytest.fixture(scope="module")
def lk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_gemv_gb300 import build, lk
    build.build()
    yield lk
    assert lk.lk_device_error(reset=True) == 0


def make(mode, batch, **kw):
    from q8_quantized_gemv_gb300.decode import Attention, DecodeStack, Mixture, Sampling
    moe = Mixture(experts=12, k=3, ffn=384, score="sigmoid", bias=True, n_group=4, top_group=2, group_sum=2, scale=1.5)
    how = Sampling(temperature=0.8, top_k=[50 + b for b in range(batch)], top_p=0.95, min_p=0.001)
    return DecodeStack(**SIZE, batch=batch, mode=mode, moe=moe, sample=how,
                       attn=Attention(head_dim=64, capacity=64, page=16, tokens=5), **kw)


@pytest.mark.parametrize("mode", ["dequant", "int8act", "twopass"])
@pytest.mark.parametrize("batch", [1, 5])
def test_tokens(lk, mode, batch):
    st = make(mode, batch)
    m, layers = st.moe, []

    def hook(name, fn):
        r = fn()
        if name == "moe":
            torch.cuda.synchronize()
            l = len(layers)
            act = {"x": st.xn} if st.mode == lk.LK_DEQUANT else st.acts[st.H]
            w, ws = m.routers[l]
            logits = act_value(act, st.mode) @ (w.double() * ws.view(torch.float16).double().repeat_interleave(32, -1)).T
            assert float((m.logits.double() - logits).abs().max()) <= 1e-4 * float(logits.abs().max())
            ids, weights, _ = route_ref(m.logits.cpu().numpy(), m.biases[l].cpu().numpy(), "sigmoid", 4, 2, 2, 3, True, 1.5)
            assert np.array_equal(m.ids.cpu().numpy(), ids)
            assert np.allclose(m.weights.cpu().numpy(), weights, rtol=2.0 ** -15, atol=0)
            ex = m.stacks[l]

            def half(pair):
                return pair[0], pair[1].view(torch.float16)
            h, tol = glu_ref(half(ex.gate), half(ex.up), act, st.mode, m.ids, m.E)
            assert bool(((m.h.double() - h).abs() <= tol).all())
            to = {{"hq": "xq", "hl": "xl", "hs": "xs"}[n]: t for n, t in m.words.items()} or {"x": m.h}
            y, tol = down_ref(half(ex.down), to, st.mode, m.ids, m.weights, m.E)
            assert bool(((st.out["down"].double() - y).abs() <= tol).all())
            layers.append(l)
        return r

    g = torch.Generator(device="cuda")
    g.manual_seed(batch)
    plain = []
    for _ in range(3):
        layers.clear()
        st.sample.u.copy_(torch.rand((batch,), generator=g, device="cuda"))
        idx = st.run_token(hook=hook)
        assert layers == list(range(st.L))
        torch.cuda.synchronize()
        logits, u = st.logits.cpu().numpy(), st.sample.u.cpu().numpy()
        for b in range(batch):
            i, p, margin = sample_ref(logits[b], np.float32(0.8), 50 + b, np.float32(0.95), np.float32(0.001), float(u[b]))
            assert margin < 2.0 ** -28 or (int(idx[b]) == i and abs(float(st.sample.prob[b]) / p - 1) < 2.0 ** -22)
        plain.append([t.clone() for t in (st.logits, idx, st.sample.prob, m.ids, m.h)])
    # the same tokens from one graph of dependent launches
    st.pdl = True
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        st.run_token()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            st.run_token()
        st.attn.restart()
        g.manual_seed(batch)
        for want in plain:
            st.sample.u.copy_(torch.rand((batch,), generator=g, device="cuda"))
            graph.replay()
            got = [t.clone() for t in (st.logits, st.idx, st.sample.prob, m.ids, m.h)]
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(lk):
    from q8_quantized_gemv_gb300.decode import DecodeStack, Mixture, Sampling
    small = {**SIZE, "glu": False}
    with pytest.raises(ValueError):
        DecodeStack(**small, moe=Mixture(experts=4, k=2, ffn=128))
    with pytest.raises(ValueError):
        DecodeStack(**small, sample=Sampling(top_k=3))
    moe = Mixture(experts=4, k=2, ffn=128)
    st = DecodeStack(**SIZE, moe=moe)
    with pytest.raises(ValueError):
        DecodeStack(**SIZE, moe=moe)
    assert st.launches_per_token() == 1 + 2 * (4 + 1 + 4) + 2
    draw = Sampling(top_k=3)
    DecodeStack(**SIZE, sample=draw)
    with pytest.raises(ValueError):
        DecodeStack(**SIZE, sample=draw)
