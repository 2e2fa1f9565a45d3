"""Page operators on the GPU against the list model, entry for entry."""
import random

import numpy as np
import pytest
import torch

from oracle import oracle as orc
from tests.gpu_harness import K
from tests.page_model import BAD, SHORT, Pool

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pair:
    """A pool on the device and its model; every call goes to both."""

    def __init__(self, num_blocks, rows, max_blocks, bs=16, modes=(orc.FP8_PER_TOKEN_HEAD,), Hkv=2, D=64):
        kvq = K()
        self.m = Pool(num_blocks, rows, max_blocks, bs)
        self.ctx = kvq.kvq_create(len(modes), Hkv, Hkv, D, bs, num_blocks, list(modes))
        self.ref = torch.zeros(num_blocks, dtype=torch.int32, device="cuda")
        self.table = torch.full((rows, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")

    def state(self):
        return self.ref, self.table, self.lens

    def same(self, word=True):
        assert self.ref.tolist() == self.m.ref
        assert self.table.tolist() == self.m.table
        assert self.lens.tolist() == self.m.lens
        if word:
            got = K().STATUS[K().kvq_get_device_error()]
            want = ("KVQ_ERR_" + (BAD if BAD in self.m.errors else SHORT)) if self.m.errors else "KVQ_OK"
            assert got == want
            self.m.errors.clear()

    def extend(self, rows, new, max_tokens=None):
        n = sum(max(x, 0) for x in new) if max_tokens is None else max_tokens
        qs = torch.full((len(rows) + 1,), 77, dtype=torch.int32, device="cuda")
        pos = torch.full((n,), 77, dtype=torch.int64, device="cuda")
        slots = torch.full((n,), 77, dtype=torch.int64, device="cuda")
        copies = torch.full((len(rows), 2), 77, dtype=torch.int32, device="cuda")
        K().kvq_extend_sequences(self.ctx, _i32(rows), _i32(new), *self.state(), qs, pos, slots, copies)
        want = self.m.extend(list(rows), list(new), n)
        assert qs.tolist() == want[0]
        assert pos.tolist() == want[1]
        assert slots.tolist() == want[2]
        assert [tuple(c) for c in copies.tolist()] == want[3]
        return copies

    def fork(self, parents, children):
        K().kvq_fork_sequences(self.ctx, _i32(parents), _i32(children), *self.state())
        self.m.fork(list(parents), list(children))

    def truncate(self, rows, keep=None):
        K().kvq_truncate_sequences(self.ctx, _i32(rows), None if keep is None else _i32(keep),
                                   *self.state())
        self.m.truncate(list(rows), keep)

    def compact(self):
        moves = torch.full((max(1, self.m.num_blocks // 2), 2), 77, dtype=torch.int32, device="cuda")
        count = _i32([77])
        K().kvq_compact_blocks(self.ctx, *self.state(), moves, count)
        want = self.m.compact()
        assert count.item() == len(want)
        assert [tuple(c) for c in moves[:len(want)].tolist()] == want
        assert torch.all(moves[len(want):] == 77)
        return moves, count


@pytest.mark.parametrize("bs, blocks, max_blocks", [(16, 1, 3), (16, 37, 5), (64, 1000, 9), (128, 300, 40)])
def test_one_row(bs, blocks, max_blocks):
    p = Pair(blocks, 3, max_blocks, bs)
    p.extend([1], [1])
    p.same()
    p.extend([1], [0])
    p.extend([1], [bs - 1])
    p.same()
    p.extend([1, 0], [bs + 1, 2 * bs])            # refused where blocks are too few
    p.same()
    p.truncate([1], [1])
    p.same()
    p.compact()
    p.truncate([1, 0])
    p.same()
    assert p.ref.sum().item() == 0


@pytest.mark.parametrize("seed", range(6))
def test_random_calls(seed):
    r = random.Random(seed)
    bs = r.choice([16, 32, 128])
    rows, max_blocks = r.choice([(8, 5), (40, 30), (130, 11)])
    p = Pair(r.choice([7, 60, 900, 20000]), rows, max_blocks, bs)
    for step in range(40):
        op = r.randrange(5)
        some = r.sample(range(rows), r.randint(1, rows))
        if op <= 1:
            new = [r.choice([0, 1, 1, 5, r.randrange(3 * bs)]) for _ in some]
            p.extend(some, new, sum(new) + r.choice([0, 3, -min(sum(new), 4)]))
        elif op == 2:
            empty = [x for x in range(rows) if p.m.lens[x] == 0]
            empty = r.sample(empty, r.randint(0, len(empty)))
            rest = [x for x in range(rows) if x not in empty]
            if empty and rest:
                p.fork([r.choice(rest) for _ in empty], empty)
        elif op == 3:
            p.truncate(some, None if r.random() < 0.3 else [r.randrange(1 + max_blocks * bs) for _ in some])
        else:
            p.compact()
        p.same()
        p.m.check()


def test_many_rows_and_a_large_pool():
    """Rows past one per thread, runs of blocks past one pass of a warp, a long table."""
    p = Pair(150001, 4096, 70, 16)
    p.extend(list(range(4096))[::-1], [(i * 37) % 900 for i in range(4096)])
    p.same()
    p.truncate(list(range(0, 4096, 3)), [(i * 11) % 700 for i in range(0, 4096, 3)])
    p.same()
    p.compact()
    p.same()
    p.extend(list(range(4096)), [1] * 4096, 5000)
    p.same()
    p.m.check()


def test_one_long_row():
    p = Pair(9000, 2, 8192, 16)
    p.extend([0], [8192 * 16 - 5])
    p.fork([0], [1])
    p.same()
    c = p.extend([0, 1], [5, 2])                  # a shared, partly filled tail: both get their own
    assert (c >= 0).all()
    p.same()
    p.truncate([0], [3])
    p.same()
    p.compact()
    p.same()
    p.truncate([1, 0])
    p.same()


def test_shared_tails():
    p = Pair(50, 6, 8, 16)
    p.extend([0], [40])
    p.fork([0, 0, 0], [1, 2, 3])
    p.same()
    c = p.extend([2, 0], [1, 0])                  # row 0 takes nothing: its tail stays shared
    assert c[0, 0] >= 0 and c[1, 0] == -1
    p.same()
    p.extend([3, 1, 0], [1, 30, 1])               # three holders left: each takes a block
    p.same()
    p.truncate([0, 1], [32, 20])                  # full and shared blocks at the cut
    p.fork([1], [4])
    p.same()
    p.extend([1], [1])                            # the cut left a shared block partly filled
    p.same()
    p.m.check()


def test_too_few_blocks_refuses_whole_rows():
    p = Pair(10, 5, 8, 16)
    p.extend([0, 1], [64, 60])                    # 8 blocks
    p.extend([2, 3, 1, 4], [16, 40, 4, 16])       # 1, 3 (refused), 0, 1 (after it: refused)
    p.same()
    assert p.lens.tolist() == [64, 64, 16, 0, 0]


def test_bad_rows():
    p = Pair(40, 4, 4, 16)
    p.extend([0, 1], [20, 64])
    p.same()
    p.extend([0, 9, -1, 0, 1, 2], [3, 4, 5, 6, 1, -2])       # no such row, twice, past its table, negative
    p.same()
    p.fork([0, 0, 1, 3, 7, 1], [2, 2, 0, 9, 3, 1])
    p.same()
    p.truncate([2, 2, 5, -3, 1], [1, 0, 0, 0, -1])
    p.same()
    p.lens[3] = 65                                # longer than its table row
    p.m.lens[3] = 65
    p.extend([3], [1])
    p.truncate([3], [0])
    p.fork([3], [2])
    assert K().kvq_get_device_error() == K().STATUS.index("KVQ_ERR_BAD_INDEX")
    p.lens[3] = p.m.lens[3] = 0
    p.m.errors.clear()
    p.same()


def test_bad_blocks_are_reported():
    kvq = K()
    bad = kvq.STATUS.index("KVQ_ERR_BAD_INDEX")
    for b in (-1, 40, 2 ** 31 - 1):
        p = Pair(40, 3, 4, 16)
        p.extend([0], [40])
        p.table[0, 1] = b
        p.fork([0], [1])
        assert kvq.kvq_get_device_error() == bad
        ref = p.ref.clone()
        p.compact_moves = torch.zeros(20, 2, dtype=torch.int32, device="cuda")
        kvq.kvq_compact_blocks(p.ctx, *p.state(), p.compact_moves, _i32([0]))
        assert kvq.kvq_get_device_error() == bad
        p.truncate([0])
        assert kvq.kvq_get_device_error() == bad
        assert p.ref.sum().item() == ref.sum().item() - 2 and p.ref.min().item() >= 0
        # a tail entry that is no block: the row is refused
        p.table[1, 2] = b
        q = torch.zeros(2, dtype=torch.int32, device="cuda")
        slots = torch.zeros(1, dtype=torch.int64, device="cuda")
        copies = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
        kvq.kvq_extend_sequences(p.ctx, _i32([1]), _i32([1]), *p.state(), q, slots.clone(), slots, copies)
        assert kvq.kvq_get_device_error() == bad
        assert slots.item() == -1 and p.lens[1].item() == 40
    # a block that nothing holds any more is not counted below zero
    p = Pair(40, 3, 4, 16)
    p.extend([0], [16])
    p.ref.zero_()
    p.truncate([0])
    assert kvq.kvq_get_device_error() == bad and p.ref.min().item() == 0


# ------------------------------------------------------------------- copy
def _caches(ctx, modes, nb, seed=0):
    kvq = K()
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for layer in range(len(modes)):
        kc, vc, ks, vs = kvq.alloc_layer_cache(ctx, layer)
        for t in (kc, vc):
            t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
        for t in (ks, vs):
            if t is not None:
                t.copy_(torch.rand(t.shape, generator=g, device="cuda"))
        out.append((kc, vc, ks, vs))
    return out


def _pointers(caches):
    return K().layer_pointers(*[[c[i] for c in caches] for i in range(4)])


@pytest.mark.parametrize("bs, Hkv, D", [(16, 1, 64), (16, 8, 128), (128, 3, 256), (32, 2, 64)])
@pytest.mark.parametrize("n", [1, 5, 90])
def test_copy_blocks(bs, Hkv, D, n):
    """Layers of every mode, one launch; every byte of every buffer is compared."""
    kvq = K()
    modes = [4, 0, 3, 1, 2, 3]
    nb = 2 * n + 7
    ctx = kvq.kvq_create(6, Hkv, Hkv, D, bs, nb, modes)
    caches = _caches(ctx, modes, nb, n)
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(n))
    pairs = torch.stack([perm[:n], perm[n:2 * n]], -1).to(torch.int32).cuda()
    pairs[n // 2, 0] = pairs[0, 0]                       # a source twice
    want = [[None if t is None else t.clone() for t in c] for c in caches]
    for c in want:
        for t in c:
            if t is not None:
                t[pairs[:, 1].long()] = t[pairs[:, 0].long()]
    kvq.kvq_copy_blocks(ctx, pairs, _pointers(caches))
    assert kvq.kvq_get_device_error() == 0
    for c, w in zip(caches, want):
        for t, u in zip(c, w):
            assert t is None or torch.equal(t, u)


def test_copy_skips_counts_and_reports():
    kvq = K()
    ctx = kvq.kvq_create(2, 2, 2, 64, 16, 20, [3, 0])
    caches = _caches(ctx, [3, 0], 20)
    before = [[None if t is None else t.clone() for t in c] for c in caches]
    layers = _pointers(caches)

    def unchanged(but=()):
        for c, w in zip(caches, before):
            for t, u in zip(c, w):
                if t is not None:
                    same = (t == u).flatten(1).all(1)
                    assert [i for i in range(20) if not same[i]] == sorted(but)
    pairs = _i32([[-1, -1], [-1, 3], [4, 5], [6, 7]])
    kvq.kvq_copy_blocks(ctx, pairs, layers, num_pairs=_i32([0]))
    kvq.kvq_copy_blocks(ctx, pairs, layers, num_pairs=_i32([-3]))
    unchanged()
    kvq.kvq_copy_blocks(ctx, pairs, layers, num_pairs=_i32([3]))
    unchanged([5])
    assert kvq.kvq_get_device_error() == 0
    kvq.kvq_copy_blocks(ctx, pairs, layers, num_pairs=_i32([1000]))       # at most max_pairs
    unchanged([5, 7])
    assert kvq.kvq_get_device_error() == 0
    for bad in ([20, 1], [1, 20], [1, -1]):
        kvq.kvq_copy_blocks(ctx, _i32([bad]), layers)
        assert kvq.kvq_get_device_error() == kvq.STATUS.index("KVQ_ERR_BAD_INDEX")
    unchanged([5, 7])
    # a part of the layers
    kvq.kvq_copy_blocks(ctx, _i32([[0, 9]]), _pointers(caches[1:]), first_layer=1)
    assert not torch.equal(caches[0][0][0], caches[0][0][9])
    assert torch.equal(caches[1][0][0], caches[1][0][9])


def test_copy_more_layers_than_one_launch_takes():
    kvq = K()
    modes = [3, 0] * 45
    ctx = kvq.kvq_create(90, 1, 1, 64, 16, 6, modes)
    caches = _caches(ctx, modes, 6)
    kvq.kvq_copy_blocks(ctx, _i32([[1, 4]]), _pointers(caches))
    for c in caches:
        for t in c:
            assert t is None or torch.equal(t[1], t[4])


def test_copy_past_four_gigabytes():
    """Byte offsets of a buffer of 4.5 GB."""
    kvq = K()
    nb = 140000
    ctx = kvq.kvq_create(1, 8, 8, 128, 16, nb, [0])
    kc, vc, _, _ = kvq.alloc_layer_cache(ctx, 0)
    kc[nb - 1] = 7
    vc[nb - 2] = 9
    kvq.kvq_copy_blocks(ctx, _i32([[nb - 1, 3], [nb - 2, nb - 3]]), kvq.layer_pointers([kc], [vc]))
    assert torch.all(kc[3] == 7) and torch.all(vc[nb - 3] == 9) and torch.all(vc[3] == 0)


def test_pages_keep_their_contents_through_compaction():
    kvq = K()
    modes = [3, 0, 4]
    p = Pair(120, 10, 12, 16, modes)
    caches = _caches(p.ctx, modes, 120)
    layers = _pointers(caches)
    p.extend(list(range(10)), [100 + 7 * i for i in range(10)])
    p.truncate([0, 3, 4, 8], [0, 17, 0, 40])

    def contents():
        return [[None if t is None else [t[p.table[r, :p.m.used(p.m.lens[r])].long()] for r in range(10)]
                 for t in c] for c in caches]
    before = contents()
    moves, count = p.compact()
    kvq.kvq_copy_blocks(p.ctx, moves, layers, num_pairs=count)
    p.same()
    for c, w in zip(contents(), before):
        for t, u in zip(c, w):
            assert t is None or all(torch.equal(x, y) for x, y in zip(t, u))


def test_calls_in_a_graph_on_another_stream():
    p = Pair(300, 6, 20, 16)
    p.extend([0, 1, 2], [100, 33, 64])
    p.same()
    book = [t.clone() for t in p.state()]
    out = [torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(6, dtype=torch.int64, device="cuda"),
           torch.zeros(6, dtype=torch.int64, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda")]
    rows, new, par, kid = _i32([1, 3, 0]), _i32([2, 2, 2]), _i32([0]), _i32([3])
    moves, count = torch.zeros(150, 2, dtype=torch.int32, device="cuda"), _i32([0])

    def calls():
        kvq = K()
        kvq.kvq_fork_sequences(p.ctx, par, kid, *p.state())
        kvq.kvq_extend_sequences(p.ctx, rows, new, *p.state(), *out)
        kvq.kvq_truncate_sequences(p.ctx, par, None, *p.state())
        kvq.kvq_compact_blocks(p.ctx, *p.state(), moves, count)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for t, b in zip(p.state(), book):
        assert torch.equal(t, b)                   # capturing runs nothing
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph.replay()
    side.synchronize()
    p.m.fork([0], [3])
    want = p.m.extend([1, 3, 0], [2, 2, 2], 6)
    p.m.truncate([0])
    p.m.compact()
    p.same()
    assert [t.tolist() for t in out[:3]] == [list(w) for w in want[:3]]
