"""Decoder stacks with a mixture of experts under every GEMV kernel, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_gemv_gb300 import build, lk
    build.build()
    yield lk
    assert lk.lk_device_error(reset=True) == 0


@pytest.mark.parametrize("mode,batch,paths", [("int8act", 5, (1, 2, 3)), ("twopass", 5, (1, 2, 3)), ("int8act", 1, (1, 2)),
                                              ("int8act", 24, (3,)), ("dequant", 3, (1, 2))])
def test_every_gemv_kernel(lk, mode, batch, paths):
    """The same tokens whichever kernel the stack's GEMVs are given (under Dequant, where
    kernels round differently, the token is run)."""
    from q8_quantized_gemv_gb300.decode import DecodeStack, Mixture, Sampling
    size = dict(layers=2, hidden=512, q_dim=512, kv_dim=128, ffn=256, vocab=5003, glu=True, splitk=False, batch=batch, mode=mode)
    got = []
    for path in (0, *paths):
        st = DecodeStack(**size, path=path, moe=Mixture(experts=12, k=3, ffn=384), sample=Sampling(top_k=50))
        st.sample.u.fill_(0.4)
        idx = st.run_token()
        torch.cuda.synchronize()
        got.append([t.clone() for t in (st.moe.ids, st.moe.h, st.logits, idx)])
    for other in got[1:]:
        assert bool((other[-1] >= 0).all())
        if mode != "dequant":
            assert all(torch.equal(a, b) for a, b in zip(got[0], other))
