"""Attention over whole prompts on the GPU against the 64-bit model."""
import pytest
import torch

from tests import prompt_model as pm
from tests.gpu_harness import K

pytestmark = pytest.mark.gpu
BAD = 6


class Case:
    """Packed sequences in one fused buffer; tokens of no sequence are NaN."""

    def __init__(self, D, Hq, Hkv, lens, seed=0, window=0, scale=0.0, lead=0, tail=0, pad=0, fused=True):
        kvq = K()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx = kvq.kvq_create(1, Hq, Hkv, D, 16, 0, [3], [window], scale)
        self.window, self.scale = window, scale or None
        self.lens = lens
        at, self.spans = lead, []
        for n in lens:
            self.spans.append((at, at + n))
            at += n
        self.T = T = at + tail
        self.start = torch.tensor([lead] + [e for _, e in self.spans], dtype=torch.int32, device="cuda")
        heads = Hq + 2 * Hkv
        live = torch.zeros(T, dtype=torch.bool, device="cuda")
        live[lead:at] = True
        self.live = live
        if fused:
            buf = torch.randn(T, heads * D + pad, generator=g, device="cuda").to(torch.bfloat16)
            buf[~live] = float("nan")
            buf[:, heads * D:] = float("nan")
            x = buf[:, :heads * D].unflatten(1, (heads, D))
            self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
            self.strides = dict(q_token_stride=heads * D + pad, kv_token_stride=heads * D + pad)
        else:
            self.q, self.k, self.v = [torch.randn(T, n, D, generator=g, device="cuda").to(torch.bfloat16)
                                      for n in (Hq, Hkv, Hkv)]
            for x in (self.q, self.k, self.v):
                x[~live] = float("nan")
            self.strides = {}
        self.out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")

    def run(self, out=None, **kw):
        a = dict(max_seq_len=max(self.lens, default=0), **self.strides)
        a.update(kw)
        K().kvq_prompt_attention(self.ctx, 0, self.q, self.k, self.v, self.start,
                                 self.out if out is None else out, **a)

    def check(self, word=0, spans=None):
        torch.cuda.synchronize()
        assert K().kvq_get_device_error() == word
        ref, tol = pm.attend(self.q, self.k, self.v, self.spans if spans is None else spans, self.window,
                             self.scale)
        live = self.live if spans is None else torch.zeros_like(self.live)
        for s, e in spans or []:
            live[s:e] = True
        err = (self.out.double() - ref).abs()[live]
        bad = ~(err <= tol[live])
        assert not bad.any(), (int(bad.sum()), float(err[bad].max()),
                               float((err / tol[live].clamp_min(1e-30)).max()), bad.nonzero()[:4].tolist())
        assert torch.all(self.out[~live] == 7.0)             # rows of no sequence


SHAPES = [(64, 2, 2), (64, 4, 2), (64, 16, 2), (128, 2, 2), (128, 8, 4), (128, 8, 2), (128, 8, 1), (256, 2, 2),
          (256, 4, 2), (256, 4, 1)]


@pytest.mark.parametrize("D, Hq, Hkv", SHAPES)
def test_one_token(D, Hq, Hkv):
    c = Case(D, Hq, Hkv, [1])
    c.run()
    c.check()


@pytest.mark.parametrize("D, Hq, Hkv", SHAPES)
def test_ragged(D, Hq, Hkv):
    c = Case(D, Hq, Hkv, [200, 1, 64, 0, 65, 129, 17, 128, 0, 333], seed=D + Hq, lead=3, tail=150)
    c.run()
    c.check()


@pytest.mark.parametrize("D, Hq, Hkv", SHAPES)
@pytest.mark.parametrize("window", [1, 2, 17, 64, 128, 130, 1000])
def test_windows(D, Hq, Hkv, window):
    c = Case(D, Hq, Hkv, [300, 5, 129, 520], seed=window, window=window, tail=1)
    c.run()
    c.check()


@pytest.mark.parametrize("D, Hq, Hkv", SHAPES)
def test_longer_than_the_ring(D, Hq, Hkv):
    c = Case(D, Hq, Hkv, [2100], seed=5)
    c.run()
    c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fused, pad", [(False, 0), (True, 8), (True, 104)])
def test_strides(D, fused, pad):
    c = Case(D, 8, 4, [77, 250], seed=pad, fused=fused, pad=pad)
    c.run()
    c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [15, 16, 31, 32, 33, 63, 127, 128, 255, 256, 257])
def test_ends(D, n):
    """Ends at and around the borders of 16 keys, of key tiles and of query tiles."""
    c = Case(D, 4, 1, [n, n, n], seed=n, tail=1)
    c.run()
    c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_scores(D):
    """Scores of a hundred: the reference maximum moves, O is rescaled."""
    c = Case(D, 4, 2, [700, 40], seed=8, scale=2.0)
    ramp = torch.linspace(0.05, 3.0, 700, device="cuda").to(torch.bfloat16)
    c.k[:700] *= ramp[:, None, None]
    c.run()
    c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_sequence_that_is_not_finite_stays_alone(D):
    c = Case(D, 4, 2, [100, 37, 260], seed=9)
    s, e = c.spans[1]
    for x in (c.q, c.k, c.v):
        x[s + 3:e] = float("nan")
    c.v[s + 5] = float("inf")
    c.run()
    torch.cuda.synchronize()
    c.out[s:e] = 7.0
    c.check(spans=[c.spans[0], c.spans[2]])


def test_lengths_past_the_callers_bound():
    c = Case(128, 8, 2, [300, 20], seed=10)
    c.run(max_seq_len=130)
    c.check(BAD, spans=[(0, 130), c.spans[1]])


def test_bad_starts_are_left_alone():
    c = Case(128, 4, 2, [100, 50], seed=11)
    good = c.start.clone()
    for bad in ([-5, 95, 150], [0, 200, 150], [0, 100, 151], [0, 100, 2 ** 31 - 1]):
        c.start = torch.tensor(bad, dtype=torch.int32, device="cuda")
        c.out.fill_(7.0)
        c.run(max_seq_len=150)
        spans = [(s, e) for s, e in zip(bad, bad[1:]) if 0 <= s <= e <= c.T]
        c.check(BAD, spans=spans)
    c.start = good
    c.out.fill_(7.0)
    c.run()
    c.check()


def test_nothing_to_do():
    c = Case(64, 2, 2, [0, 0], tail=5)
    c.run(max_seq_len=10)
    torch.cuda.synchronize()
    assert torch.all(c.out == 7.0) and K().kvq_get_device_error() == 0


def test_streams_and_graphs():
    """Two calls at once, and a captured one replayed on other inputs; the same bits each time."""
    c = Case(128, 8, 2, [513, 90], seed=12)
    d = Case(64, 8, 2, [300], seed=13)
    c.run()
    d.run()
    torch.cuda.synchronize()
    want = c.out.clone(), d.out.clone()
    outs = torch.zeros_like(c.out), torch.zeros_like(d.out)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        c.run(out=outs[0], stream=s1)
        d.run(out=outs[1], stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.q.copy_(torch.randn_like(c.q))
    for _ in range(2):
        c.out.fill_(7.0)
        graph.replay()
        c.check()


def test_many_sequences():
    lens = [1 + (7 * i) % 23 for i in range(300)]
    c = Case(64, 4, 2, lens, seed=14)
    c.run()
    c.check()
