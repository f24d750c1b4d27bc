"""The bounded waits of the experts' products (include/lk_moe.h) on the GPU."""
import pytest

torch = pytest.importorskip("torch")

from moehelp import acts_of, as_h, experts  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
ERR_MOE_WAIT = 256


@pytest.fixture(scope="module")
def lk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_gemv_gb300 import build, lk
    build.build()
    yield lk
    assert lk.lk_device_error(reset=True) == 0


@pytest.mark.parametrize("mode,path", [("dequant", 2), ("int8act", 2), ("int8act", 3), ("twopass", 2), ("twopass", 3)])
@pytest.mark.parametrize("M", [1, 40])
def test_shortest_wait_limit(lk, mode, path, M):
    """Under the shortest limit a call keeps it and gives its result, or raises the
    bit of these waits in the error word (and no drain's); the context and,
    with the counters zeroed again, the next calls are as they were."""
    m, E, k, F, K = lk.MODES[mode], 48, 4, 1024, 4096
    ex = lk.Experts(gate=experts(E, F, K, 1, DEV), up=experts(E, F, K, 2, DEV), down=experts(E, K, F, 3, DEV))
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    ids = torch.rand((M, E), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
    n, cfg = M * k, lk.launch_cfg(path=path)
    acts = acts_of(torch.randn((M, K), generator=g, device=DEV), m)
    hidden = as_h(acts_of(torch.randn((n, F), generator=g, device=DEV), m))
    w, cnt = torch.rand((M, k), generator=g, device=DEV), torch.zeros((n * F // 32,), dtype=torch.int32, device=DEV)

    def buffers():
        out = [torch.zeros((n, F), device=DEV), torch.zeros((M, K), device=DEV)]
        return out + ([] if m == lk.LK_DEQUANT else [torch.zeros((n, F), dtype=torch.int8, device=DEV),
                                                     torch.zeros((n, F), dtype=torch.int8, device=DEV),
                                                     torch.zeros((n, F // 32), device=DEV)])

    def call(out):
        words = dict(zip(("hq", "hl", "hs"), out[2:]), cnt=cnt) if len(out) > 2 else {}
        lk.lk_moe_glu_q8(ex, m, ids, out[0], cfg=cfg, **words, **acts)
        lk.lk_moe_down_q8(ex, m, ids, w, out[1], cfg=cfg, **hidden)
        torch.cuda.synchronize()
        return lk.lk_device_error(reset=True)
    want = buffers()
    assert call(want) == 0
    for _ in range(3):
        out = buffers()
        lk.lk_set_option("wait_us", 1)
        try:
            err = call(out)
        finally:
            lk.lk_set_option("wait_us", 0)
        assert err in (0, ERR_MOE_WAIT)
        assert err or all(torch.equal(a, b) for a, b in zip(out, want))
        cnt.zero_()  # (as the header asks for after such a call)
        out = buffers()
        assert call(out) == 0 and not bool(cnt.any())
        assert all(torch.equal(a, b) for a, b in zip(out, want))
