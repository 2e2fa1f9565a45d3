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


# KV heads enough for several hundred items: every CTA takes one behind another
TURNS = [(64, 16, 8), (64, 64, 8), (128, 8, 8), (128, 32, 8), (256, 8, 8), (256, 32, 8)]


def _ragged(seed, n, longest):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(1, longest + 1, (n,), generator=g)
    x[torch.randint(0, n, (n // 4,), generator=g)] = torch.randint(0, 40, (n // 4,), generator=g)
    x[n // 2] = longest
    return x.tolist()


@pytest.mark.parametrize("D, Hq, Hkv", TURNS)
@pytest.mark.parametrize("window", [0, 1, 100, 640])
def test_items_behind_one_another(D, Hq, Hkv, window):
    """Twelve sequences of up to 1,500 tokens: items of one to a dozen key tiles and of one query tile or
    two follow one another in a CTA."""
    c = Case(D, Hq, Hkv, _ragged(D + Hq + window, 12, 1500), seed=16, window=window, lead=5, tail=9, pad=8)
    c.run()
    c.check()


@pytest.mark.parametrize("D, Hq, Hkv", [(64, 8, 4), (128, 8, 4), (256, 8, 8)])
@pytest.mark.parametrize("window", [0, 33])
def test_levels_of_many_sequences(D, Hq, Hkv, window):
    """Seventy sequences: each level's items lie in several rounds of 32 sequences."""
    c = Case(D, Hq, Hkv, _ragged(D + window, 70, 700), seed=17, window=window)
    c.run()
    c.check()


@pytest.mark.parametrize("D, Hq, Hkv", [(64, 16, 8), (128, 16, 8), (256, 16, 8)])
def test_what_an_item_leaves_behind(D, Hq, Hkv):
    """Every third sequence is not finite, others have scores of a hundred: nothing of an item reaches the
    next one of its CTA."""
    lens = _ragged(D, 15, 900)
    c = Case(D, Hq, Hkv, lens, seed=18, scale=2.0)
    spans = []
    for i, (s, e) in enumerate(c.spans):
        if i % 3 == 1:
            for x in (c.q, c.k, c.v):
                x[s:e] = float("nan") if i % 2 else float("inf")
            continue
        spans.append((s, e))
        if i % 3 == 2:
            c.k[s:e] *= 0.05
    c.run()
    torch.cuda.synchronize()
    for i, (s, e) in enumerate(c.spans):
        if i % 3 == 1:
            c.out[s:e] = 7.0
    c.check(spans=spans)


@pytest.mark.parametrize("D, Hq, Hkv", [(64, 64, 8), (128, 32, 8), (256, 16, 8)])
def test_the_same_bits_again(D, Hq, Hkv):
    """Which CTA takes an item, and behind which other, changes from run to run; no bit does."""
    c = Case(D, Hq, Hkv, _ragged(D, 10, 1200), seed=19)
    c.run()
    want = c.out.clone()
    for _ in range(20):
        c.out.fill_(7.0)
        c.run()
        assert torch.equal(c.out, want)
    c.check()
