"""The order of the page calls: copies before the next call that changes the pool."""
import torch

import pytest

from tests.gpu_harness import K
from tests.page_model import SHORT
from tests.test_gpu_pages import Pair, _caches, _pointers

pytestmark = pytest.mark.gpu

MODES = [3, 0, 4]


def _contents(p, caches, lens):
    return [[None if t is None else [t[p.table[r, :p.m.used(n)].long()].transpose(1, 2).flatten(0, 1)[:n]
                                     for r, n in enumerate(lens)] for t in c] for c in caches]


def _equal(a, b):
    return all(x is None or all(torch.equal(u, v) for u, v in zip(x, y))
               for c, d in zip(a, b) for x, y in zip(c, d))


def test_every_holder_grows_again_and_again():
    """Beams of a shared prompt: all take a token, tails are copied, and the block that nobody holds
    any more is handed out by the next step. The prompt's positions keep their bytes."""
    p = Pair(40, 8, 6, 16, MODES)
    caches = _caches(p.ctx, MODES, 40)
    p.extend([0], [37])
    p.fork([0, 0, 0], [1, 2, 3])
    prompt = [37] * 4 + [0] * 4
    before = _contents(p, caches, prompt)
    shared = int(p.table[0, 2])
    c = p.extend([0, 1, 2, 3], [1] * 4)
    assert (c[:, 0] == shared).all() and int(p.ref[shared]) == 0
    K().kvq_copy_blocks(p.ctx, c, _pointers(caches))
    p.same()
    assert _equal(before, _contents(p, caches, prompt))
    c = p.extend([3, 1, 4], [11, 11, 5])               # past the tail: new blocks, the free one among them
    K().kvq_copy_blocks(p.ctx, c, _pointers(caches))
    p.same()
    assert shared in p.table.flatten().tolist()
    assert _equal(before, _contents(p, caches, prompt))
    moves, count = p.compact()
    K().kvq_copy_blocks(p.ctx, moves, _pointers(caches), num_pairs=count)
    p.same()
    assert _equal(before, _contents(p, caches, prompt))


@pytest.mark.parametrize("spare", [4, 3])
def test_a_pool_of_just_the_blocks_that_a_step_takes(spare):
    """Four holders of a tail take four blocks; with three free ones the last row waits."""
    p = Pair(3 + spare, 4, 6, 16)
    p.extend([0], [40])
    p.fork([0, 0, 0], [1, 2, 3])
    p.extend([0, 1, 2, 3], [1] * 4)
    assert p.m.errors == (set() if spare == 4 else {SHORT})
    p.same()
    assert p.lens.tolist() == [41, 41, 41, 41 if spare == 4 else 40]
    p.m.check()
