"""Decode attention that accumulates its weights, output and weights against 64 bits."""
import math

import pytest
import torch

from tests import cross_model as cm
from tests.gpu_harness import K
from tests.test_gpu_cross import Case

pytestmark = pytest.mark.gpu
BAD = 6
U = 2.0 ** -24


class Weights(Case):
    """One query per row; weights rows longer than a context, with values behind it."""

    def __init__(self, mode, D, Hq, Hkv, lens, extra=5, **kw):
        super().__init__(mode, D, Hq, Hkv, lens, [1] * len(lens), **kw)
        self.Hkv, self.most = Hkv, max(lens)
        g = torch.Generator(device="cuda").manual_seed(1)
        self.w = torch.rand(len(lens), Hkv, self.most + extra, generator=g, device="cuda") * 2
        self.before = self.w.clone()

    def go(self, decay=1.0, workers=0, most=None, work=None, stream=None):
        most = self.most if most is None else most
        n, need = K().kvq_decode_weights_plan(self.ctx, 0, len(self.lens), most, workers)
        if work is None:
            work = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        y = self.layer
        K().kvq_decode_attention_weights(
            self.ctx, 0, self.q, y["codes"][0], y["codes"][1], self.table, self.L, self.w, self.out,
            max_context=most, decay=decay, k_scale=y["static"][0], v_scale=y["static"][1],
            k_cache_scale=y["scales"][0], v_cache_scale=y["scales"][1], num_workers=n, workspace=work,
            stream=stream)
        return n

    def verify(self, decay=1.0, lens=None):
        """The weights' bound, u = 2^-24, s the scores and e the log2 of their sum (log2 units),
        a_p = sum_d |q_d K_pd| scale log2 e: a score is off by 4 sqrt(D/16 + 3) u a_p (accumulation
        steps and roundings, four standard deviations) and two roundings of itself, e by the largest
        such error and two of its own, their difference by one: relative error ln 2 times the sum.
        The exponent and log2 add 2^-21, the fp32 sum of a row's weights 4 sqrt(n/16 + 2) u, the heads'
        sum and the update one rounding each."""
        torch.cuda.synchronize()
        lens = self.lens if lens is None else lens
        T, Hq, D = self.q.shape
        G = Hq // self.Hkv
        scale = (self.scale or 1.0 / math.sqrt(D)) * cm.LOG2E
        for b, L in enumerate(lens):
            assert torch.equal(self.w[b, :, L:], self.before[b, :, L:])
            if L <= 0:
                continue
            pages = self.table[b, :-(-L // self.bs)].long()
            for h in range(self.Hkv):
                k = self.layer["values"][0][pages, h].flatten(0, 1)[:L]
                q = self.q[b, h * G:(h + 1) * G].double()
                s = q @ k.T * scale
                a = q.abs() @ k.abs().T * scale
                top = s.amax(-1, keepdim=True)
                e = top + (s - top).exp2().sum(-1, keepdim=True).log2()
                p = (s - e).exp2()
                ds = 4 * math.sqrt(D / 16 + 3) * U * (a + a.amax(-1, keepdim=True))
                ds = ds + 2 * U * (s.abs() + s.abs().amax(-1, keepdim=True)) + 3 * U * e.abs() + U * (s - e).abs()
                t = (p * (math.log(2) * ds + 2.0 ** -21 + 4 * math.sqrt(L / 16 + 2) * U)).sum(0)
                want = decay * self.before[b, h, :L].double() + p.sum(0)
                t = t + (G + 1) * U * p.sum(0) + 2 * U * want
                err = (self.w[b, h, :L].double() - want).abs()
                assert torch.all(err <= t), (b, h, float((err / t).max()))


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("D, Hq, Hkv", [(64, 2, 2), (64, 4, 2), (64, 8, 2), (64, 16, 2), (128, 4, 2), (128, 8, 2),
                                        (128, 16, 2), (128, 2, 2), (256, 2, 2), (256, 4, 2)])
@pytest.mark.parametrize("workers", [0, 1, 5])
def test_ragged(mode, D, Hq, Hkv, workers):
    c = Weights(mode, D, Hq, Hkv, [200, 1, 64, 0, 65, 500, 17], seed=D + Hq)
    c.go(workers=workers)
    assert K().kvq_get_device_error() == 0
    c.check()
    c.verify()


@pytest.mark.parametrize("mode", [0, 2, 3, 4])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_block_sizes(mode, bs):
    c = Weights(mode, 128, 8, 4, [bs * 3 + 5, bs, 2 * bs - 1], bs=bs, seed=bs)
    c.go(decay=0.75)
    c.check()
    c.verify(decay=0.75)


@pytest.mark.parametrize("mode", [0, 3, 4])
def test_long_contexts(mode):
    c = Weights(mode, 64, 8, 2, [30000, 12345, 5000], seed=2, extra=0)
    assert c.go() > 1
    c.check()
    c.verify()


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
def test_decay(decay):
    c = Weights(3, 128, 8, 2, [300, 40], seed=3)
    c.go(decay=decay)
    c.verify(decay=decay)


def test_many_sequences():
    c = Weights(1, 64, 4, 2, [1 + (13 * i) % 90 for i in range(200)], seed=4)
    c.go()
    c.check()
    c.verify()


def test_large_scores():
    for mode in (0, 2, 3):
        c = Weights(mode, 128, 8, 2, [900, 40], seed=8, softmax_scale=4.0)
        c.go()
        c.check()
        c.verify()


def test_contexts_past_the_bound():
    """Only max_context positions are read and weighted."""
    c = Weights(3, 128, 8, 2, [300, 100], seed=5)
    c.go(most=123)
    torch.cuda.synchronize()
    assert K().kvq_get_device_error() == BAD
    c.lens = [123, 100]
    c.check()
    c.verify(lens=[123, 100])


def test_negative_lengths_and_bad_blocks():
    c = Weights(3, 128, 8, 2, [300, 100, 48], seed=6)
    c.L = torch.tensor([-3, 100, 48], dtype=torch.int32, device="cuda")
    c.table[1, 2] = -5
    c.table[2, :3] = 1 << 30
    c.go(decay=0.5)
    torch.cuda.synchronize()
    assert K().kvq_get_device_error() == BAD
    assert torch.equal(c.w[0], c.before[0])
    assert torch.all(c.out[0] == 0) and torch.isfinite(c.out.float()).all()
    # a page that was not read gets no weight, and nothing of a row without a page does
    assert torch.equal(c.w[1, :, 32:48], 0.5 * c.before[1, :, 32:48])
    assert torch.equal(c.w[2, :, :48], 0.5 * c.before[2, :, :48])
    got = (c.w[1, :, :100] - 0.5 * c.before[1, :, :100]).sum(-1)
    assert torch.all((got - 4.0).abs() < 1e-4)               # four heads, a weight of one each


def test_steps_streams_and_graphs():
    """Sums over steps; the same bits eagerly, on another stream and replayed."""
    c = Weights(3, 128, 8, 2, [700, 33, 400], seed=7)
    work = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        c.go(decay=0.5, work=work)
    torch.cuda.synchronize()
    want, out = c.w.clone(), c.out.clone()
    c.w.copy_(c.before)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        c.go(decay=0.5, work=work, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(c.w, want) and torch.equal(c.out, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.go(decay=0.5, work=work)
    c.w.copy_(c.before)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.w, want) and torch.equal(c.out, out)
