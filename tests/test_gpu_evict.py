"""Eviction on the GPU, bit for bit against the list model."""
import pytest
import torch

from tests import evict_model as em
from tests.gpu_harness import K

pytestmark = pytest.mark.gpu
BAD = 6


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, lens, mode=3, D=128, Hkv=2, bs=16, seed=0, extra=5, refs=True, table_extra=0):
        g = torch.Generator().manual_seed(seed)
        self.gen, self.lens, self.bs, self.Hkv, self.mode = g, lens, bs, Hkv, mode
        used = [-(-n // bs) for n in lens]
        self.blocks = sum(used) + 3
        self.ctx = K().kvq_create(1, Hkv, Hkv, D, bs, self.blocks, [mode])
        perm = torch.randperm(self.blocks, generator=g).tolist()
        width = max(max(used), 1) + table_extra
        self.table = []
        for u in used:
            self.table.append([perm.pop() for _ in range(u)] + [-1] * (width - u))
        self.most = max(max(lens), 0)
        self.stride = self.most + extra
        self.ref = [0] * self.blocks
        for t in self.table:
            for b in t:
                if b >= 0:
                    self.ref[b] = 1
        self.with_refs = refs
        kc, vc, ks, vs = K().alloc_layer_cache(self.ctx, 0)
        self.bufs = [torch.randint(0, 256, kc.shape, generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
        if ks is not None:
            self.bufs += [torch.randn(ks.shape, generator=g).cuda() for _ in range(2)]
        self.weights = torch.exp(2 * torch.randn(len(lens), Hkv, self.stride, generator=g)).cuda()

    def run(self, rows, keeps, first, last, most=None, stream=None, device=None):
        """The call, checked against the model."""
        most = self.most if most is None else most
        before = [b.clone() for b in self.bufs]
        w = self.weights.cpu().tolist()
        want = em.Call(rows, keeps, self.table, self.lens, w, self.bs, self.blocks, self.Hkv, first, last, most,
                       self.ref if self.with_refs else None)
        new = torch.full((len(rows) + 2,), 77, dtype=torch.int32, device="cuda")
        self.call(_i32(rows), _i32(keeps), new, first, last, most, stream)
        torch.cuda.synchronize()
        assert K().kvq_get_device_error() == (BAD if want.bad else 0)
        assert new.tolist() == want.new_lens + [77, 77]
        if want.moves:
            src = torch.tensor([m[0] for m in want.moves], device="cuda").T
            dst = torch.tensor([m[1] for m in want.moves], device="cuda").T
            for b in before:
                b[tuple(dst)] = b[tuple(src)]
        for got, b in zip(self.bufs, before):
            assert torch.equal(got.view(torch.uint8), b.view(torch.uint8))
        ref = torch.tensor(w, dtype=torch.float32)
        got = self.weights.cpu()
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.nan_to_num(1.5), ref.nan_to_num(1.5))
        return want

    def call(self, rows, keeps, new, first, last, most, stream=None):
        b = self.bufs + [None, None]
        K().kvq_evict_cells(self.ctx, 0, rows, keeps, _i32(self.table), _i32(self.lens), self.weights, new, b[0],
                            b[1], b[2], b[3], first_kept=first, last_kept=last, max_context=most,
                            ref_count=_i32(self.ref) if self.with_refs else None, stream=stream)


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [16, 128])
def test_modes(mode, D, bs):
    c = Case([200, 33, 90, 300], mode, D, bs=bs, seed=mode + D)
    c.run([3, 0, 2], [100, 64, 90], 3, 17)


@pytest.mark.parametrize("first, last", [(0, 0), (4, 0), (0, 5), (1, 1), (20, 30), (50, 0), (0, 50), (49, 1)])
@pytest.mark.parametrize("over", [1, 2, 31, 50, 500])
def test_budgets(first, last, over):
    """One cell too many up to eleven times the budget; no middle at all; last cells that overlap
    their new places."""
    c = Case([50 + over, 50, 49], seed=first + last + over)
    c.run([0, 1, 2], [50, 50, 50], first, last)


@pytest.mark.parametrize("n", [1000, 2047, 5000, 9001])
@pytest.mark.parametrize("keep", [40, 900])
def test_clusters(n, keep):
    """Few rows of many cells: segments of several CTAs."""
    c = Case([n, n // 2], Hkv=1, seed=n)
    c.run([1, 0], [keep, keep], 7, 33)
    c = Case([n], Hkv=1, seed=n + 1)
    c.run([0], [n - 3], 2, 500)


def test_many_rows():
    lens = [100 + (37 * i) % 200 for i in range(90)]
    c = Case(lens, Hkv=4, D=64, seed=3)
    c.run(list(range(89, -1, -1)), [128] * 90, 4, 32)


@pytest.mark.parametrize("n, keep", [(70000, 20000), (393216, 200000)])
def test_long_row(n, keep):
    c = Case([n], mode=4, D=64, Hkv=1, seed=4, extra=0)
    c.run([0], [keep], 16, 1000)


@pytest.mark.parametrize("n", [300, 6000])
def test_ties(n):
    """Equal weights: the lowest positions stay, across the segments of a row."""
    for kind in range(4):
        c = Case([n], seed=kind, Hkv=1)
        if kind == 0:
            c.weights.fill_(0.25)
        elif kind == 1:
            c.weights.copy_(torch.randint(0, 3, c.weights.shape, generator=c.gen).float())
        elif kind == 2:
            c.weights.zero_()
            c.weights[..., ::7] = -0.0
        else:
            c.weights.copy_(torch.randint(0, 2, c.weights.shape, generator=c.gen).float() - 1.0)
        c.run([0], [n // 2 + 3], 5, 20)


def test_values_out_of_the_ordinary():
    c = Case([400, 400], seed=6)
    w = c.weights
    w[0, :, ::3] = float("nan")
    w[0, :, 1::5] = float("inf")
    w[0, :, 2::11] = float("-inf")
    w[1] = -w[1]
    w[1, :, ::4] *= 1e-42                       # subnormal
    c.run([0, 1], [200, 100], 4, 30)


def test_nothing_but_nan():
    c = Case([100], seed=7)
    c.weights.fill_(float("nan"))
    c.run([0], [50], 2, 3)


def test_bad_rows_are_left_alone():
    c = Case([100, 120, 0, 90], seed=8, table_extra=1)
    c.run([1, -1, 4, 1, 2, 0], [50, 50, 50, 40, 50, 60], 4, 8)
    c = Case([100, 120, 90], seed=9)
    c.run([0, 1, 2], [50, 11, -3], 4, 8)                     # keep below first + last
    c = Case([100, 120, 90], seed=10)
    c.run([0, 1, 2], [50, 50, 50], 4, 8, most=100)           # a row past the caller's bound
    c = Case([100, 120, 90], seed=11)
    c.lens = [100, -7, 5000]
    c.run([0, 1, 2], [50, 50, 50], 4, 8)


def test_shared_and_unknown_blocks():
    c = Case([100, 120, 90], seed=12)
    c.ref[c.table[1][6]] = 2
    c.table[2][0] = c.blocks
    c.run([0, 1, 2], [50, 50, 50], 4, 8)
    c = Case([100, 120], seed=13)
    c.table[0][5] = -1
    c.run([0, 1], [50, 50], 4, 8)
    c = Case([100, 120], seed=14, refs=False)                # no counts: the caller's word for it
    c.ref = [5] * c.blocks
    c.run([0, 1], [50, 50], 4, 8)
    c = Case([48, 120], seed=15)                             # a row that needs no eviction is not looked at
    c.ref[c.table[0][0]] = 2
    c.run([0, 1], [50, 50], 4, 8)


def test_again_and_again():
    """Cells evicted, others appended, evicted again: the last ones stay the last ones."""
    c = Case([300, 260], seed=16)
    for step in range(4):
        c.run([0, 1], [200, 200], 4, 64)
        c.lens = [200 + 25 * (step + 1), 200 + step]
        for r in range(2):
            c.weights[r, :, 200:c.lens[r]] = torch.rand(c.Hkv, c.lens[r] - 200, device="cuda") * 5


def test_stream_and_graph():
    c = Case([500, 400], seed=17)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.run([0, 1], [300, 300], 4, 100, stream=s)
    rows, keeps, new = _i32([0, 1]), _i32([150, 120]), _i32([0, 0])
    table, lens, ref = _i32(c.table), _i32(c.lens), _i32(c.ref)
    graph = torch.cuda.CUDAGraph()
    before = [b.clone() for b in c.bufs] + [c.weights.clone()]
    with torch.cuda.graph(graph):
        b = c.bufs
        K().kvq_evict_cells(c.ctx, 0, rows, keeps, table, lens, c.weights, new, b[0], b[1], b[2], b[3],
                            first_kept=4, last_kept=100, max_context=500, ref_count=ref)
    graph.replay()
    torch.cuda.synchronize()
    got = [b.clone() for b in c.bufs] + [c.weights.clone()]
    for x, y in zip(c.bufs + [c.weights], before):
        x.copy_(y)
    c.run([0, 1], [150, 120], 4, 100)
    for x, y in zip(c.bufs + [c.weights], got):
        assert torch.equal(x, y)
    assert new.tolist() == [150, 120]


def test_new_lengths_over_the_budgets():
    """keep_lens is new_lens: the same moves, rows that are refused among them."""
    lens = [3000, 100, 5000, 90, 120]
    rows, keeps = [0, 1, -1, 2, 3, 4], [2000, 50, 7, 3000, 100, 11]
    c, d = Case(lens, seed=18), Case(lens, seed=18)
    c.run(rows, keeps, 4, 8)
    over = _i32(keeps)
    d.call(_i32(rows), over, over, 4, 8, d.most, None)
    torch.cuda.synchronize()
    assert K().kvq_get_device_error() == BAD
    assert over.tolist() == [2000, 50, 0, 3000, 90, 120]
    for x, y in zip(c.bufs + [c.weights], d.bufs + [d.weights]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
