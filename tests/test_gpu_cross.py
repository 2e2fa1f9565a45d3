"""Cross attention on the GPU against the 64-bit model."""
import pytest
import torch

from tests import cross_model as cm
from tests.gpu_harness import K

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, mode, D, Hq, Hkv, lens, queries, bs=16, seed=0, window=0, softmax_scale=0.0):
        kvq = K()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.mode, self.bs, self.lens, self.n = mode, bs, lens, queries
        used = [-(-s // bs) for s in lens]
        blocks = sum(used) + 3
        self.ctx = kvq.kvq_create(1, Hq, Hkv, D, bs, blocks, [mode], [window], softmax_scale)
        self.scale = softmax_scale or None
        perm = torch.randperm(blocks, generator=torch.Generator().manual_seed(seed))
        self.table = torch.full((len(lens), max(max(used), 1)), -1, dtype=torch.int32)
        live = torch.zeros(blocks, bs, dtype=torch.bool)
        at = 0
        for b, u in enumerate(used):
            ids = perm[at:at + u]
            self.table[b, :u] = ids.to(torch.int32)
            for j, i in enumerate(ids.tolist()):
                live[i, :min(bs, lens[b] - j * bs)] = True
            at += u
        self.table = self.table.cuda()
        self.layer = cm.layer(mode, blocks, Hkv, bs, D, g)
        cm.poison(self.layer, mode, live.cuda())
        self.starts = [0]
        for n in queries:
            self.starts.append(self.starts[-1] + n)
        self.qs = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.L = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = torch.randn(self.starts[-1], Hq, D, generator=g, device="cuda").to(torch.bfloat16)
        self.out = torch.full((self.starts[-1] + 3, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")

    def run(self, splits=0, step=False, most=None, max_len=None, stream=None, out=None, work=None):
        kvq = K()
        most = (0 if step else max(self.n)) if most is None else most
        max_len = max(self.lens) if max_len is None else max_len
        ns, need = kvq.kvq_cross_plan(self.ctx, 0, len(self.lens), most, max_len, splits)
        if work is None:
            # a workspace's contents need no initialisation
            work = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
        y = self.layer
        kvq.kvq_cross_attention(
            self.ctx, 0, self.q, y["codes"][0], y["codes"][1], self.table, None if step else self.qs,
            self.L, self.out if out is None else out, max_query_len=most, max_encoder_len=max_len,
            k_scale=y["static"][0], v_scale=y["static"][1], k_cache_scale=y["scales"][0],
            v_cache_scale=y["scales"][1], num_splits=ns, workspace=work, stream=stream)
        return ns

    def check(self, word=0):
        torch.cuda.synchronize()
        assert K().kvq_get_device_error() == word
        ref, tol = cm.attend(self.q, self.layer, self.table, self.lens, self.starts, self.bs, self.scale)
        T = self.starts[-1]
        err = (self.out[:T].double() - ref).abs()
        bad = ~(err <= tol)
        assert not bad.any(), (int(bad.sum()), float(err[bad].max()), float((err / tol.clamp_min(1e-30)).max()))
        assert torch.all(self.out[T:] == 7.0)              # rows behind the last sequence


MODES = [0, 1, 2, 3, 4]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D, Hq, Hkv", [(64, 2, 2), (64, 16, 2), (128, 8, 2), (128, 8, 8), (128, 16, 2),
                                        (256, 2, 2), (256, 4, 2)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_ragged(mode, D, Hq, Hkv, splits):
    c = Case(mode, D, Hq, Hkv, [200, 1, 64, 0, 65, 500, 17], [3, 1, 0, 4, 33, 2, 70], seed=D + Hq)
    c.run(splits)
    c.check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_block_sizes(mode, bs):
    c = Case(mode, 128, 8, 4, [bs * 3 + 5, bs, 2 * bs - 1], [5, 40, 130], bs=bs, seed=bs)
    c.run()
    c.check()


@pytest.mark.parametrize("mode", MODES)
def test_many_queries(mode):
    """More than one query tile pair in a sequence, a partly filled last one."""
    c = Case(mode, 64, 8, 2, [700, 333], [301, 129], seed=3)
    c.run()
    c.check()
    c.run(4)
    c.check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_states(mode, D):
    c = Case(mode, D, 4, 2, [20000, 12345], [2, 1], seed=5)
    assert c.run() > 1
    c.check()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D, G", [(64, 1), (128, 8), (128, 4), (256, 2)])
def test_single_tokens(mode, D, G):
    """One query per sequence: with and without query_start."""
    c = Case(mode, D, 2 * G, 2, [1500, 1, 0, 333, 64], [1] * 5, seed=D + G)
    c.run(step=True)
    c.check()
    c.out.fill_(7.0)
    c.run()
    c.check()


def test_softmax_scale_and_large_scores():
    """Scores of several hundred: the reference max moves, O is rescaled."""
    for mode in (0, 2, 3, 4):
        c = Case(mode, 128, 8, 2, [900, 40], [9, 3], seed=8, softmax_scale=4.0)
        c.run(2)
        c.check()


def test_lengths_past_the_callers_bound():
    """max_encoder_len sizes the plan only: longer sequences are still read whole."""
    c = Case(3, 128, 8, 2, [900, 100], [4, 4], seed=9)
    c.run(3, max_len=200)
    c.check()
    c.out.fill_(7.0)
    c.run(max_len=0)
    c.check()


def test_queries_past_the_callers_bound():
    kvq = K()
    c = Case(1, 64, 4, 2, [100, 200], [3, 9], seed=10)
    for splits in (1, 2):
        c.out.fill_(7.0)
        c.run(splits, most=5)
        assert kvq.kvq_get_device_error() == kvq.STATUS.index("KVQ_ERR_BAD_INDEX")
        ref, tol = cm.attend(c.q, c.layer, c.table, c.lens, c.starts, c.bs)
        assert ((c.out[:8].double() - ref[:8]).abs() <= tol[:8]).all()
        assert torch.all(c.out[8:] == 7.0)


def test_bad_lengths_and_blocks():
    kvq = K()
    bad = kvq.STATUS.index("KVQ_ERR_BAD_INDEX")
    for splits in (1, 3):
        for L in (-1, 257):
            c = Case(3, 128, 4, 2, [256, 256], [2, 2], seed=11)
            c.L[0] = L
            c.run(splits)
            assert kvq.kvq_get_device_error() == bad
            assert torch.all(c.out[:2] == 7.0)
            ref, tol = cm.attend(c.q, c.layer, c.table, c.lens, c.starts, c.bs)
            assert ((c.out[2:4].double() - ref[2:4]).abs() <= tol[2:4]).all()
        for mode in MODES:
            c = Case(mode, 128, 4, 2, [256, 100], [2, 2], seed=12)
            for at, b in ((0, 10 ** 6), (5, -1), (15, c.table.numel() + 99)):
                c.table[0, at] = b
            c.run(splits)
            assert kvq.kvq_get_device_error() == bad
            # the other pages' positions are what is left
            keep = [j for j in range(16) if j not in (0, 5, 15)]
            left = torch.full_like(c.table, -1)
            left[0, :13] = c.table[0, keep]
            left[1] = c.table[1]
            ref, tol = cm.attend(c.q, c.layer, left, [13 * 16, 100], c.starts, c.bs)
            assert ((c.out[:4].double() - ref).abs() <= tol).all()
            # no page at all: zeros
            c.table[0].fill_(-5)
            c.run(splits)
            assert kvq.kvq_get_device_error() == bad
            assert torch.all(c.out[:2] == 0.0)


def test_shared_states_and_graph():
    """Beams share an encoder's pages; two captured calls with a workspace each, replayed."""
    kvq = K()
    c = Case(3, 64, 8, 2, [3000, 3000, 3000], [4, 4, 4], seed=13)
    c.table[1:] = c.table[0]
    ns, need = kvq.kvq_cross_plan(c.ctx, 0, 3, 4, 3000)
    assert ns > 1
    works = [torch.zeros(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.zeros_like(c.out) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for w, o in zip(works, outs):
            c.run(out=o, work=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    side.synchronize()
    assert torch.equal(outs[0][:12], outs[1][:12])
    c.out[:12] = outs[0][:12]
    c.check()


@pytest.mark.parametrize("splits", [2, 64, 1024])
def test_more_splits_than_key_tiles(splits):
    c = Case(4, 128, 8, 2, [500, 3, 130], [2, 7, 40], seed=15)
    c.run(splits)
    c.check()


@pytest.mark.parametrize("mode, D, Hkv", [(3, 64, 1), (0, 128, 1), (2, 256, 3)])
def test_many_sequences(mode, D, Hkv):
    lens = [(37 * b) % 211 for b in range(300)]
    c = Case(mode, D, 2 * Hkv, Hkv, lens, [(5 * b) % 4 for b in range(300)], bs=32, seed=16)
    c.run()
    c.check()
    c.out.fill_(7.0)
    c.run(2)
    c.check()


def test_rows_at_the_forms_borders():
    """Queries x heads of 32, 33, 64, 65, 128 and 129: copies of the rows, idle warps, two tiles."""
    for G, ns in ((8, (4, 8, 16, 17)), (1, (32, 33, 64, 65, 128, 129, 257))):
        for n in ns:
            c = Case(3, 64, G, 1, [700], [n], seed=n)
            c.run()
            c.check()


def test_two_streams_at_once():
    c = [Case(m, 128, 16, 2, [6000, 900], [3, 50], seed=17 + m) for m in (3, 0)]
    streams = [torch.cuda.Stream() for _ in c]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, s in zip(c, streams):
            with torch.cuda.stream(s):
                x.run()
    torch.cuda.synchronize()
    for x in c:
        x.check()


def test_repeats_are_bit_equal():
    for mode in MODES:
        c = Case(mode, 128, 16, 2, [5000, 77], [5, 60], seed=14)
        c.run()
        first = c.out.clone()
        for _ in range(3):
            c.out.fill_(7.0)
            c.run()
            assert torch.equal(first, c.out)
