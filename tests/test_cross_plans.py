"""Cross attention's plan at the sizes where its two forms meet, without a GPU."""
import pytest

kvq = pytest.importorskip("int4_quantized_paged_gb300.kvq",
                          reason="libkvq.so not built (run __graft_entry__.build())")


def _ctx(Hq=32, Hkv=8, D=128):
    return kvq.kvq_create(1, Hq, Hkv, D, 16, 4096, [3])


@pytest.mark.parametrize("batch, states", [(1, 60), (64, 1500), (8, 32768), (300, 100)])
def test_a_plan_of_one_query_serves_both_forms(batch, states):
    """Without query_start the call runs the decode, whose workspace a plan of 1 has to hold."""
    splits, need = kvq.kvq_cross_plan(_ctx(), 0, batch, 1, states)
    assert need >= kvq.kvq_decode_plan(_ctx(), 0, batch, states)[1]
    if splits > 1:
        assert need >= splits * batch * 32 * 129 * 4
    assert kvq.kvq_cross_plan(_ctx(), 0, 2, 1, 1000, 7)[0] == 7
