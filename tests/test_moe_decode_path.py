"""The launch settings that a decoder stack's mixture of experts hands on, with
stand-ins for the calls.  No GPU."""
import pytest

torch = pytest.importorskip("torch")

from q8_quantized_gemv_gb300 import decode, lk  # noqa: E402


@pytest.mark.parametrize("path", [0, 1, 2, 3])
@pytest.mark.parametrize("mode", [lk.LK_DEQUANT, lk.LK_INT8ACT])
def test_the_stack_s_gemv_kernel_is_not_the_experts(monkeypatch, path, mode):
    """A stack's path names a GEMV kernel, for the router too; the experts' products, which
    have other kernels under these numbers (none under 1, one under Dequant), go by
    the library's choice.  The dependent launch is theirs as well."""
    calls = {}
    for name in ("lk_gemv_q8", "lk_moe_route", "lk_moe_glu_q8", "lk_moe_down_q8"):
        monkeypatch.setattr(lk, name, lambda *a, name=name, cfg=None, **k: calls.update({name: (cfg.path, cfg.pdl)}))
    m = decode.Mixture(experts=4, k=2, ffn=128)
    m.stacks, m.routers, m.biases = [None], [(None, None)], [None]
    m.logits = m.weights = m.h = m.cnt = None
    m.ids, m.words = torch.zeros((1, 2), dtype=torch.int32), {} if mode == lk.LK_DEQUANT else {"hq": None}
    cfg = lk.launch_cfg(path=path, pdl=1)
    m.step(0, {"x": None}, mode, None, cfg)
    assert calls["lk_gemv_q8"] == (path, 1) and calls["lk_moe_route"][1] == 1
    assert calls["lk_moe_glu_q8"] == calls["lk_moe_down_q8"] == (0, 1)
    assert cfg.path == path
