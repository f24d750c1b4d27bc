"""What a decoder stack refuses of its mixture of experts and its draw, before
anything is built.  No GPU."""
import pytest

pytest.importorskip("torch")

from q8_quantized_gemv_gb300.decode import DecodeStack, Mixture, Sampling  # noqa: E402

SIZE = dict(layers=1, hidden=256, q_dim=256, kv_dim=128, ffn=256, vocab=500, device="cpu")


class Part:
    """Stands for an Attention: counts how often it is built."""
    built = 0

    def build(self, *a):
        self.built += 1


@pytest.mark.parametrize("kw", [dict(glu=False), dict(glu=True, fused_qkv=False), dict(glu=True, fused=True), dict(glu=True, chain=True)])
@pytest.mark.parametrize("part", ["moe", "sample"])
def test_a_refused_stack_takes_none_of_its_parts(kw, part):
    at, moe, draw = Part(), Mixture(experts=4, k=2, ffn=128), Sampling(top_k=3)
    with pytest.raises(ValueError):
        DecodeStack(**SIZE, **kw, attn=at, **{part: moe if part == "moe" else draw})
    assert at.built == 0 and not hasattr(moe, "stacks") and not hasattr(draw, "set")


def test_parts_of_another_stack():
    """One that has the experts (the numbers) of another stack is refused, and the other
    parts are as free as they were."""
    at, moe, draw = Part(), Mixture(experts=4, k=2, ffn=128), Sampling(top_k=3)
    moe.stacks = []
    with pytest.raises(ValueError):
        DecodeStack(**SIZE, glu=True, attn=at, moe=moe, sample=draw)
    assert at.built == 0 and not hasattr(draw, "set")
    moe, draw.set = Mixture(experts=4, k=2, ffn=128), {}
    with pytest.raises(ValueError):
        DecodeStack(**SIZE, glu=True, attn=at, moe=moe, sample=draw)
    assert at.built == 0 and not hasattr(moe, "stacks")
