"""A K scale of zero (a buffer's fill, a position that no write reached) is a key of zeros: its score
is 0 and its value counts, in whole key tiles and in partly used ones alike."""
import pytest
import torch

from tests import cross_model as cm
from tests.gpu_harness import K
from tests.test_gpu_cross import Case

pytestmark = pytest.mark.gpu


def _zero(c):
    """Keys 3, 64 to 79 and each sequence's last one get the scale 0."""
    for b, L in enumerate(c.lens):
        for p in {3, L - 1, *range(64, 80)}:
            if p < L:
                block = int(c.table[b, p // c.bs])
                c.layer["scales"][0][block, :, p % c.bs] = 0.0
                c.layer["values"][0][block, :, p % c.bs] = 0.0


@pytest.mark.parametrize("mode", [3, 4])
@pytest.mark.parametrize("D, lens, queries", [(128, [40, 100, 200, 64], [3, 1, 5, 2]), (64, [77, 500], [40, 130]),
                                              (256, [90, 30], [2, 9])])
def test_cross_attention(mode, D, lens, queries):
    c = Case(mode, D, 4, 2, lens, queries, seed=D)
    _zero(c)
    for splits in (0, 2):
        c.out.fill_(7.0)
        c.run(splits)
        c.check()


@pytest.mark.parametrize("mode", [3, 4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_and_decode(mode, D):
    """One new token a sequence sees every position, as in cross attention."""
    c = Case(mode, D, 4, 2, [40, 100, 200, 64], [1] * 4, seed=D + 1)
    _zero(c)
    c.run(step=True)
    c.check()
    y = c.layer
    out = torch.zeros(4, 4, D, device="cuda")
    K().kvq_prefill_attention(c.ctx, 0, c.q, y["codes"][0], y["codes"][1], c.table, c.qs, c.L, out,
                              max_query_len=1, k_cache_scale=y["scales"][0], v_cache_scale=y["scales"][1])
    assert K().kvq_get_device_error() == 0
    ref, tol = cm.attend(c.q, y, c.table, c.lens, c.starts, c.bs)
    assert ((out.double() - ref).abs() <= tol).all()
