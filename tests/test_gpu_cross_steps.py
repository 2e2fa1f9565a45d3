"""One query a sequence, planned for either form."""
import pytest
import torch

from tests.gpu_harness import K
from tests.test_gpu_cross import Case

pytestmark = pytest.mark.gpu


def _decode(c):
    """kvq_decode_attention_bf16 under its own plan."""
    kvq = K()
    workers, need = kvq.kvq_decode_plan(c.ctx, 0, len(c.lens), max(c.lens))
    assert workers > 1
    out = torch.zeros_like(c.out[:len(c.lens)])
    y = c.layer
    kvq.kvq_decode_attention_bf16(
        c.ctx, 0, c.q, y["codes"][0], y["codes"][1], c.table, c.L, out, max_context=max(c.lens),
        k_scale=y["static"][0], v_scale=y["static"][1], k_cache_scale=y["scales"][0],
        v_cache_scale=y["scales"][1], num_workers=workers,
        workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))
    return out


@pytest.mark.parametrize("mode", [0, 2, 3, 4])
@pytest.mark.parametrize("batch, states", [(64, 700), (2, 9000)])
@pytest.mark.parametrize("most", [0, 1])
def test_the_decodes_own_plan_is_taken(mode, batch, states, most):
    """A plan of 1 counts splits of the keys (one, for 64 sequences); the call without query_start
    spreads over the SMs all the same: it gives the decode's bits and leaves partials behind."""
    lens = [states - 3 * b for b in range(batch)]
    c = Case(mode, 128, 16, 4, lens, [1] * batch, seed=batch)
    _, need = K().kvq_cross_plan(c.ctx, 0, batch, most, states)
    work = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    c.run(step=True, most=most, work=work)
    c.check()
    assert torch.equal(c.out[:batch], _decode(c))
    assert (work != 255).any()


def test_a_smaller_workspace_takes_the_count_that_it_was_planned_for():
    kvq = K()
    c = Case(3, 64, 8, 2, [900, 1, 333], [1] * 3, seed=4)
    workers, need = kvq.kvq_cross_plan(c.ctx, 0, 3, 0, 900, 3)
    assert workers == 3 and need < kvq.kvq_cross_plan(c.ctx, 0, 3, 1, 900)[1]
    y = c.layer
    kvq.kvq_cross_attention(
        c.ctx, 0, c.q, y["codes"][0], y["codes"][1], c.table, None, c.L, c.out, max_query_len=1,
        max_encoder_len=900, k_cache_scale=y["scales"][0], v_cache_scale=y["scales"][1],
        num_splits=workers, workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))
    c.check()
