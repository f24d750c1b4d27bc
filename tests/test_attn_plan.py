"""Which kernels an attention call takes (lk_attn_launches: 1 in clusters, 2 with the
deal and the join), where the number of items decides: a cluster holds an item on
8 blocks however few items there are, the deal spreads them over the GPU.  No GPU."""
import pytest

torch = pytest.importorskip("torch")

from q8_quantized_gemv_gb300 import build, lk  # noqa: E402

F16, BF16, Q8 = 0, 1, 2


@pytest.fixture(scope="module")
def launches():
    build.build()
    f = lk._load().lk_attn_launches

    def of(type_, n_kv, D, B, tokens, prefix=0, G=4):
        return f(type_, n_kv * G, n_kv, D, B, 1, prefix, tokens)
    return of


@pytest.mark.parametrize("type_,n_kv,D,B,short,long", [
    # tokens where clusters were measured faster, and the deal
    (F16, 1, 128, 1, 4000, 8000), (F16, 2, 128, 1, 4000, 8000), (F16, 1, 128, 2, 4000, 8000), (F16, 4, 128, 1, 8000, 12700),
    (F16, 2, 128, 2, 6000, 12700), (F16, 6, 128, 1, 10000, 12700), (F16, 8, 128, 1, 12700, 14000),
    (BF16, 1, 128, 1, 2000, 6000), (BF16, 2, 128, 1, 2000, 6000), (BF16, 4, 128, 1, 4000, 8000), (BF16, 8, 128, 1, 8000, 10000),
    (Q8, 1, 128, 1, 4000, 8000), (Q8, 4, 128, 1, 8000, 10000), (Q8, 8, 128, 1, 10000, 12000),
    (F16, 1, 64, 1, 8000, 18000), (F16, 4, 64, 1, 18000, 25000), (F16, 8, 64, 1, 25000, 30000),
    (Q8, 1, 64, 1, 8000, 12000), (Q8, 8, 64, 1, 10000, 12000)])
def test_clusters_where_they_are_faster(launches, type_, n_kv, D, B, short, long):
    assert launches(type_, n_kv, D, B, short) == 1
    assert launches(type_, n_kv, D, B, long) == 2
    # a prefix counts as the room does
    assert launches(type_, n_kv, D, B, 500, prefix=short - 500) == 1
    assert launches(type_, n_kv, D, B, 500, prefix=long - 500) == 2


def test_more_items_never_take_fewer_tokens(launches):
    for type_ in (F16, BF16, Q8):
        for D in (64, 128):
            last = 0
            for n_kv in range(1, 9):
                most = max(t for t in range(1024, 30000, 64) if launches(type_, n_kv, D, 1, t) == 1)
                assert most >= last
                last = most
