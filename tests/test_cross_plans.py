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


@pytest.mark.parametrize("Hq, Hkv, D", [(32, 8, 128), (512, 64, 128), (64, 64, 256), (2, 2, 256)])
@pytest.mark.parametrize("batch, most, states, splits", [
    (2 ** 31 - 1, 2 ** 31 - 1, 1 << 30, 0), (2 ** 31 - 1, 2 ** 31 - 1, 1 << 30, 1024),
    (1 << 30, 1 << 30, 1000, 0), (1 << 30, 1 << 30, 1000, 8), (2 ** 31 - 1, 1, 1 << 30, 0)])
def test_sizes_past_the_grid_are_refused(Hq, Hkv, D, batch, most, states, splits):
    """Their products pass 64 bits: a plan of them said (4, 0 bytes) for 2^60 queries."""
    with pytest.raises(kvq.KVQError, match="INVALID_ARG"):
        kvq.kvq_cross_plan(_ctx(Hq, Hkv, D), 0, batch, most, states, splits)


def test_the_largest_grids_are_planned():
    assert kvq.kvq_cross_plan(_ctx(), 0, 1 << 26, 2, 100) == (1, 0)
    # a loose bound of the queries needs no workspace
    assert kvq.kvq_cross_plan(_ctx(), 0, 4096, 1 << 20, 4096) == (1, 0)
    with pytest.raises(kvq.KVQError, match="INVALID_ARG"):
        kvq.kvq_cross_plan(_ctx(), 0, 4096, 1 << 20, 4096, 2)
