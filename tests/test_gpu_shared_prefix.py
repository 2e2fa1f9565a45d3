"""Decode attention behind shared prefixes on the GPU against the 64-bit model (whose bound for one
rounded weight term covers the prefix's part, and the decode's own part lies within it)."""
import pytest
import torch

from tests import cross_model as cm
from tests.gpu_harness import K

pytestmark = pytest.mark.gpu
BAD = 6


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """groups: for each the shared length and its rows' own lengths (a row may be shorter than the
    prefix: then its own length is negative); lone: lengths of rows of no group, behind the others."""

    def __init__(self, mode, D, Hq, Hkv, groups, lone=(), bs=16, seed=0, scale=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.bs, self.mode, self.scale = bs, mode, scale or None
        self.start, self.shared, self.lens, first = [0], [], [], []
        for P, own in groups:
            first += [len(self.lens)] * len(own)
            self.lens += [P + o for o in own]
            self.shared.append(P)
            self.start.append(len(self.lens))
        for n in lone:
            first.append(len(self.lens))
            self.lens.append(n)
        B = len(self.lens)
        prefix = [P for P, own in groups for _ in own] + [0] * len(lone)
        used = [-(-n // bs) for n in self.lens]
        blocks = sum(used) + 3
        self.blocks = blocks
        self.ctx = K().kvq_create(1, Hq, Hkv, D, bs, blocks, [mode], [0], scale)
        ids = torch.randperm(blocks, generator=torch.Generator().manual_seed(seed)).tolist()
        self.layer = y = cm.layer(mode, blocks, Hkv, bs, D, g)
        live = torch.zeros(blocks, bs, dtype=torch.bool)
        width = max(max(used), 1)
        self.table = []
        for b in range(B):
            whole = min(prefix[b], self.lens[b]) // bs if first[b] != b else 0
            row = self.table[first[b]][:whole] if whole else []
            row = row + [ids.pop() for _ in range(used[b] - whole)]
            tail = min(prefix[b], self.lens[b]) % bs
            if first[b] != b and tail:                       # a copy of the prefix's last block
                s, d = self.table[first[b]][whole], row[whole]
                for parts in (y["codes"], y["values"], y["scales"]):
                    for x in parts:
                        if x is not None:
                            x[d, :, :tail] = x[s, :, :tail]
            for j, i in enumerate(row):
                live[i, :max(0, min(bs, self.lens[b] - j * bs))] = True
            self.table.append(row + [-1] * (width - used[b]))
        cm.poison(y, mode, live.cuda())
        self.q = torch.randn(B, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
        self.out = torch.full((B + 2, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.T, self.L = _i32(self.table), _i32(self.lens)
        self.gs, self.sl = _i32(self.start), _i32(self.shared)
        self.most = max([b - a for a, b in zip(self.start, self.start[1:])], default=0)
        self.max_own = max([n - p for n, p in zip(self.lens, prefix)] + [0])

    def run(self, splits=8, stream=None, out=None, work=None, groups=None, **kw):
        """splits 8: shared whether it gains or not; 0: the device's choice."""
        a = dict(max_group=self.most, max_shared=max(self.shared, default=0), max_own=self.max_own)
        a.update(kw)
        NG = len(self.shared) if groups is None else groups
        B = len(self.lens)
        ns, need = K().kvq_shared_prefix_plan(self.ctx, 0, B, NG, num_splits=splits, **a)
        if work is None:
            work = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        y = self.layer
        K().kvq_shared_prefix_attention(
            self.ctx, 0, self.q, y["codes"][0], y["codes"][1], self.T, self.L, self.gs, self.sl,
            self.out if out is None else out, num_groups=NG, k_scale=y["static"][0], v_scale=y["static"][1],
            k_cache_scale=y["scales"][0], v_cache_scale=y["scales"][1], num_splits=ns, workspace=work,
            stream=stream, **a)
        return ns

    def check(self, word=0):
        torch.cuda.synchronize()
        assert K().kvq_get_device_error() == word
        B = len(self.lens)
        ref, tol = cm.attend(self.q, self.layer, self.T, self.lens, list(range(B + 1)), self.bs, self.scale)
        err = (self.out[:B].double() - ref).abs()
        bad = ~(err <= tol)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(err[bad].max()),
                               float((err / tol.clamp_min(1e-30)).max()))
        assert torch.all(self.out[B:] == 7.0)


MODES = [0, 1, 2, 3, 4]
SHAPES = [(64, 2, 2), (64, 16, 2), (128, 8, 2), (128, 8, 8), (128, 16, 2), (256, 2, 2), (256, 4, 2)]
RAGGED = [(300, [5, 1, 40]), (64, [0, 200]), (17, [16, 15, 1, 2]), (15, [3, 4]), (90, [33]), (0, [9, 20])]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D, Hq, Hkv", SHAPES)
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_ragged(mode, D, Hq, Hkv, splits):
    c = Case(mode, D, Hq, Hkv, RAGGED, lone=[70, 0, 1], seed=D + Hq)
    c.run(splits)
    c.check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_block_sizes(mode, bs):
    c = Case(mode, 128, 8, 4, [(2 * bs, [5, 1, bs]), (3 * bs + 7, [1, 30, 9]), (bs - 1, [1, 2])], bs=bs, seed=bs)
    c.run()
    c.check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("rows", [2, 9, 33, 70])
def test_rows_of_a_group(mode, rows):
    """One query tile in its forms, and more than one pair of them."""
    c = Case(mode, 128, 16, 2, [(500, [1 + i % 20 for i in range(rows)])], seed=rows)
    for splits in (8, 0):
        c.out.fill_(7.0)
        c.run(splits)
        c.check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prefix(mode, D):
    c = Case(mode, D, 4, 2, [(20000, [3, 100, 1]), (12345, [2, 900])], seed=5)
    for splits in (0, 1, 40):
        c.out.fill_(7.0)
        c.run(splits)
        c.check()


def test_a_row_shorter_than_the_prefix():
    """The group shares what its shortest row has."""
    c = Case(3, 128, 8, 2, [(200, [5, -57, 30]), (100, [1, -100, 4])], seed=6)
    c.run()
    c.check()


def test_sizes_that_the_caller_underestimates():
    """max_shared and max_own size the plan only; a group past max_group is read row by row."""
    c = Case(2, 128, 8, 2, [(900, [5, 400]), (500, [1, 2, 3, 4])], seed=7)
    for splits in (3, 0):
        c.out.fill_(7.0)
        c.run(splits, max_shared=100, max_own=1)
        c.check()
    c.out.fill_(7.0)
    c.run(max_group=3)
    c.check()
    c.out.fill_(7.0)
    c.run(max_group=1)
    c.check()


def test_nothing_shared():
    c = Case(3, 64, 4, 2, [], lone=[100, 0, 33], seed=8)
    assert c.run(groups=0) == 0
    c.check()
    c = Case(3, 64, 4, 2, [(0, [10, 20]), (10, [3, 4])], seed=9)
    assert c.run() == 0
    c.check()


def test_bad_groups_share_nothing():
    for start, shared in (([0, 5, 3, 8], [50, 50, 50]), ([-1, 3, 5, 8], [50, 50, 50]), ([0, 3, 5, 9], [50, 50, 50]),
                          ([0, 3, 5, 8], [50, -1, 50])):
        c = Case(3, 128, 8, 2, [(50, [5, 1, 9]), (50, [2, 3]), (50, [4, 4, 4])], seed=10)
        c.gs, c.sl = _i32(start), _i32(shared)
        c.run()
        c.check(BAD)


def test_many_groups():
    """More groups than SMs, of all lengths; and one long prefix among short ones."""
    for c in (Case(3, 64, 4, 2, [(1 + (37 * i) % 300, [1 + i % 5, 2]) for i in range(170)], seed=20),
              Case(1, 128, 8, 2, [(40, [1, 2]), (9000, [3, 1, 1]), (70, [5, 5]), (1, [2, 2])], seed=21),
              Case(3, 128, 8, 2, [(20000, [5] * 40), (16, [1, 2]), (3000, [7, 2])], seed=22)):
        for splits in (0, 1, 5, 1024):
            c.out.fill_(7.0)
            c.run(splits)
            c.check()


def test_lengths_and_blocks_out_of_range():
    c = Case(1, 128, 8, 2, [(100, [5, 7, 9])], lone=[60], seed=11)
    c.T[3, 1] = c.blocks                          # that page's positions are left out
    c.lens[1] = -4
    c.L = _i32(c.lens)
    c.run()
    torch.cuda.synchronize()
    assert K().kvq_get_device_error() == BAD
    assert torch.all(c.out[1] == 0)
    assert torch.isfinite(c.out.float()).all()
    lens = c.lens
    c.lens = [lens[0], 0, lens[2], 16]            # and the other rows are what they are
    ref, tol = cm.attend(c.q, c.layer, c.T.clamp_max(c.blocks - 1), c.lens, [0, 1, 2, 3, 4], c.bs)
    assert torch.all(((c.out[:3].double() - ref[:3]).abs() <= tol[:3]))


def test_softmax_scale_and_large_scores():
    for mode in (0, 2, 3, 4):
        c = Case(mode, 128, 8, 2, [(600, [300, 20, 5])], seed=12, scale=4.0)
        c.run()
        c.check()


def test_streams_and_graphs():
    c = Case(3, 128, 8, 2, [(700, [9, 40, 1])], seed=13)
    d = Case(4, 64, 8, 2, [(300, [5, 2]), (100, [1, 1])], seed=14)
    c.run()
    d.run()
    torch.cuda.synchronize()
    want = c.out.clone(), d.out.clone()
    outs = torch.full_like(c.out, 7.0), torch.full_like(d.out, 7.0)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    works = [torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        c.run(out=outs[0], stream=s1, work=works[0])
        d.run(out=outs[1], stream=s2, work=works[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(work=works[0])
        d.run(work=works[0])                      # one workspace, one after the other
    c.q.copy_(torch.randn_like(c.q))
    for _ in range(3):
        c.out.fill_(7.0)
        d.out.fill_(7.0)
        graph.replay()
        c.check()
        d.check()
