"""The items of a call over whole prompts on the GPU: their order, their hand-over within a CTA, and
what starts that are wrong leave of them."""
import pytest
import torch

from tests import prompt_model as pm
from tests.gpu_harness import K
from tests.test_gpu_prompt import BAD, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D, Hq, Hkv", [(64, 4, 4), (128, 8, 1), (128, 16, 8), (256, 4, 1)])
@pytest.mark.parametrize("starts", [[0, 140, 10, 150], [0, 1000, 4, 1003, 8, 1000], [0, 700, 0, 700, 0, 700]])
def test_sequences_that_overlap(D, Hq, Hkv, starts):
    """Behind starts that descend a sequence may lie over another one. Their rows are undefined where
    they meet, and only there: more items than disjoint sequences of so many tokens have."""
    c = Case(D, Hq, Hkv, [max(starts)], seed=15)
    c.start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    c.run(max_seq_len=1000)
    spans = [(s, e) for s, e in zip(starts, starts[1:]) if s <= e]
    of = torch.zeros(c.T, dtype=torch.int32, device="cuda")
    for s, e in spans:
        of[s:e] += 1
    torch.cuda.synchronize()
    assert K().kvq_get_device_error() == BAD
    assert torch.all(c.out != 7.0)                           # every row was written
    for s, e in spans:
        ref, tol = pm.attend(c.q, c.k, c.v, [(s, e)])
        mine = of == 1
        mine[:s] = mine[e:] = False
        assert torch.all(((c.out.double() - ref).abs() <= tol)[mine])
