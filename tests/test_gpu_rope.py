"""Rotary positions on the GPU against the 64-bit model, and the fused write
against its parts."""
import numpy as np
import pytest
import torch

from oracle import oracle as orc
from tests import rope_model as rm
from tests.gpu_harness import K
from tests.helpers import bits

pytestmark = pytest.mark.gpu

FAR = [0, 1, 2, 7, 4095, 131071, 10 ** 6 + 3, 2 ** 31 - 1, 2 ** 40 + 12345, -1, -77777]


def _randn(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _positions(T, seed=0):
    return [FAR[(t + seed) % len(FAR)] if t % 3 == 0 else (t * 977 + seed) % 200000 for t in range(T)]


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("D, r", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256), (256, 64)])
@pytest.mark.parametrize("T, H", [(1, 1), (3, 5), (70, 8)])
def test_apply(D, r, layout, T, H):
    kvq = K()
    rope = kvq.kvq_rope_create(D, r, layout=layout, base=500000.0, magnitude=1.25)
    fs, m = kvq.kvq_rope_frequencies(rope)
    x = _randn((T, H, D), 11 * T + D)
    pos = _positions(T)
    p = torch.tensor(pos, dtype=torch.int64, device="cuda")
    for inverse in (False, True):
        out = torch.full_like(x, float("nan"))
        kvq.kvq_rope_apply(rope, x, p, out, inverse=inverse)
        xd = _np(x)
        rm.check_bf16(_np(out), rm.rotate(xd, pos, fs, layout, m, inverse),
                      rm.slack(xd, pos, fs, layout, m), f"inverse {inverse}")
        assert torch.equal(out[..., r:], x[..., r:])           # the rest of the head, bit for bit
    assert kvq.kvq_get_device_error() == 0


def test_apply_many_tokens_matches_few():
    """A warp per token and a token cut into slices give the same bits."""
    kvq = K()
    rope = kvq.kvq_rope_create(128)
    x = _randn((9000, 6, 128), 5)
    p = torch.arange(9000, device="cuda") * 13
    out = torch.empty_like(x)
    kvq.kvq_rope_apply(rope, x, p, out)
    for t in (0, 4099, 8999):
        one = torch.empty_like(x[t:t + 1])
        kvq.kvq_rope_apply(rope, x[t:t + 1], p[t:t + 1], one)
        assert torch.equal(one[0], out[t])


def test_apply_strides_and_in_place():
    kvq = K()
    rope = kvq.kvq_rope_create(64, layout=1)
    wide = _randn((33, 10, 64), 6)
    p = torch.arange(33, device="cuda")
    x = wide[:, 2:6]
    want = torch.empty(33, 4, 64, dtype=torch.bfloat16, device="cuda")
    kvq.kvq_rope_apply(rope, x.contiguous(), p, want)
    before = wide.clone()
    out = torch.zeros(33, 7, 64, dtype=torch.bfloat16, device="cuda")
    kvq.kvq_rope_apply(rope, x, p, out, x_token_stride=640, out_token_stride=448, num_heads=4)
    assert torch.equal(out[:, :4], want) and torch.all(out[:, 4:] == 0)
    kvq.kvq_rope_apply(rope, x, p, x, x_token_stride=640, out_token_stride=640, num_heads=4)
    assert torch.equal(wide[:, 2:6], want)
    assert torch.equal(wide[:, :2], before[:, :2]) and torch.equal(wide[:, 6:], before[:, 6:])


@pytest.mark.parametrize("layout", [0, 1])
def test_inverse_is_the_gradient(layout):
    """d <y, R x> / d x from differences of the 64-bit map (linear, so a step of 1 is exact up to
    rounding) against the inverse call."""
    kvq = K()
    rope = kvq.kvq_rope_create(64, 32, layout=layout, magnitude=1.5)
    fs, m = kvq.kvq_rope_frequencies(rope)
    pos = [3, 131072]
    y = _randn((2, 1, 64), 9)
    yd, x0 = _np(y), _np(_randn((2, 1, 64), 10))
    base = rm.rotate(x0, pos, fs, layout, m)
    grad = np.empty_like(x0)
    for t in range(2):
        for d in range(64):
            x1 = x0.copy()
            x1[t, 0, d] += 1.0
            grad[t, 0, d] = ((rm.rotate(x1, pos, fs, layout, m) - base) * yd).sum()
    out = torch.empty_like(y)
    kvq.kvq_rope_apply(rope, y, torch.tensor(pos, device="cuda"), out, inverse=True)
    # differences of sums of up to 64 doubles of size 10: 1e-12
    rm.check_bf16(_np(out), grad, rm.slack(yd, pos, fs, layout, m) + 1e-12)


# ------------------------------------------------------------------- fused write
MODES = [orc.BF16, orc.FP8_PER_TENSOR, orc.FP8_PER_HEAD, orc.FP8_PER_TOKEN_HEAD,
         orc.INT4_PER_TOKEN_HEAD]


def _e4m3(codes):
    return torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)


def _nibbles(codes):
    q = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.int64)
    return np.where(q > 7, q - 16, q).astype(np.float64)


class Write:
    """A fused projection's output and a paged layer for it."""

    def __init__(self, mode, D, Hq, Hkv, T, bs=16, r=None, layout=0, seed=1, scale=1.0, magnitude=1.0):
        kvq = K()
        self.mode, self.D, self.Hq, self.Hkv, self.T, self.bs, self.layout = mode, D, Hq, Hkv, T, bs, layout
        self.blocks = -(-T // bs) + 3
        self.ctx = kvq.kvq_create(1, Hq, Hkv, D, bs, self.blocks, [mode])
        self.rope = kvq.kvq_rope_create(D, r, layout=layout, magnitude=magnitude)
        self.qkv = _randn((T, Hq + 2 * Hkv, D), seed, scale)
        self.pos = _positions(T, seed)
        self.p = torch.tensor(self.pos, dtype=torch.int64, device="cuda")
        perm = torch.randperm(self.blocks * bs, generator=torch.Generator().manual_seed(seed))[:T]
        self.slots = perm.to(torch.int64).cuda()
        if T > 4:
            self.slots[2] = -1
            self.slots[T - 1] = -5
        self.ks = self.vs = None
        if mode == orc.FP8_PER_TENSOR:
            self.ks, self.vs = torch.tensor([0.01], device="cuda"), torch.tensor([0.02], device="cuda")
        if mode == orc.FP8_PER_HEAD:
            self.ks = torch.linspace(0.004, 0.03, Hkv, device="cuda")
            self.vs = torch.linspace(0.03, 0.002, Hkv, device="cuda")
        self.kc, self.vc, self.kcs, self.vcs = kvq.alloc_layer_cache(self.ctx, 0)
        self.q_out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")

    def run(self, q=True, stream=None):
        stride = (self.Hq + 2 * self.Hkv) * self.D
        K().kvq_rope_cache_write(
            self.ctx, self.rope, 0, self.qkv if q else None, self.q_out if q else None,
            self.qkv[:, self.Hq:], self.qkv[:, self.Hq + self.Hkv:], self.p, self.slots, self.kc,
            self.vc, self.kcs, self.vcs, self.ks, self.vs, q_token_stride=stride,
            kv_token_stride=stride, num_tokens=self.T, stream=stream)

    def check(self):
        kvq = K()
        Hq, Hkv, T, mode = self.Hq, self.Hkv, self.T, self.mode
        torch.cuda.synchronize()
        assert kvq.kvq_get_device_error() == 0
        # queries: the bits of the rotation alone, for every token
        alone = torch.empty_like(self.q_out)
        kvq.kvq_rope_apply(self.rope, self.qkv[:, :Hq].contiguous(), self.p, alone)
        assert torch.equal(alone, self.q_out)
        # values: the bits that kvq_cache_write stores, and the oracle's codes (either zero for
        # a zero: the library's quotient drops the sign of -0); unwritten cells stay zero
        pkc, pvc, pks, pvs = kvq.alloc_layer_cache(self.ctx, 0)
        kvq.kvq_cache_write(self.ctx, 0, self.qkv[:, Hq:], self.qkv[:, Hq + Hkv:], self.slots, pkc,
                            pvc, pks, pvs, self.ks, self.vs, (Hq + 2 * Hkv) * self.D, T)
        assert torch.equal(pvc, self.vc) and (pvs is None or torch.equal(pvs, self.vcs))
        okc, ovc, oks, ovs = orc.alloc_cache(mode, self.blocks, Hkv, self.bs, self.D)
        v = self.qkv[:, Hq + Hkv:].contiguous()
        orc.cache_write(mode, bits(v), bits(v), self.slots.cpu().numpy(), okc, ovc, oks, ovs,
                        block_size=self.bs, **({} if self.vs is None else dict(
                            k_scale=self.vs.cpu().numpy(), v_scale=self.vs.cpu().numpy())))
        zero = (lambda c: np.where(c == 128, 0, c)) if mode in MODES[1:4] else (lambda c: c)
        assert np.array_equal(zero(self.vc.cpu().numpy()), zero(ovc))
        if ovs is not None and self.vcs is not None:
            assert np.array_equal(self.vcs.cpu().numpy(), ovs)
        # keys
        fs, m = kvq.kvq_rope_frequencies(self.rope)
        x = _np(self.qkv[:, Hq:Hq + Hkv])
        want = rm.rotate(x, self.pos, fs, self.layout, m)
        slack = rm.slack(x, self.pos, fs, self.layout, m)
        live = (self.slots >= 0).cpu().numpy()
        slot = self.slots.cpu().numpy()[live]
        want, slack = want[live], slack[live]
        codes = self.kc.cpu().numpy()[slot // self.bs, :, slot % self.bs]
        if mode == orc.BF16:
            got = torch.from_numpy(codes).view(torch.bfloat16).float().numpy().astype(np.float64)
            rm.check_bf16(got, want, slack)
            rot = torch.empty(T, Hkv, self.D, dtype=torch.bfloat16, device="cuda")
            kvq.kvq_rope_apply(self.rope, self.qkv[:, Hq:Hq + Hkv].contiguous(), self.p, rot)
            assert np.array_equal(codes, rot.view(torch.uint8).cpu().numpy()[live])
        else:
            qmax = 7.0 if mode == orc.INT4_PER_TOKEN_HEAD else 448.0
            if self.kcs is not None:
                s = self.kcs.cpu().numpy().astype(np.float64)[slot // self.bs, :, slot % self.bs]
                ref = np.abs(want).max(-1) / qmax
                ref[ref == 0.0] = 1.0                   # a zero vector's scale
                # the amax is off by at most the slack, the division rounds once
                assert np.all(np.abs(s - ref) <= ref * 2.0 ** -24 + 2.0 ** -150 + slack.max(-1) / qmax)
            else:
                s = np.broadcast_to(self.ks.cpu().numpy().astype(np.float64), (len(slot), Hkv))
            s = s[..., None]
            if mode == orc.INT4_PER_TOKEN_HEAD:
                got = _nibbles(codes) * s
                tol = 0.5 * s * (1 + 2.0 ** -20) + slack
            else:
                got = _e4m3(codes) * s
                want = np.clip(want, -448 * s, 448 * s)
                # half a step of E4M3: 2^-4 relative, or half of 2^-9 below its normal numbers
                tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s) * (1 + 2.0 ** -20) + slack
            assert np.all(np.abs(got - want) <= tol)
        written = np.zeros((self.blocks, self.bs), dtype=bool)
        written[slot // self.bs, slot % self.bs] = True
        rest = self.kc.cpu().numpy().transpose(0, 2, 1, 3)[~written]
        assert not rest.any()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D, r, layout, Hq, Hkv", [(64, 64, 0, 4, 2), (64, 32, 1, 8, 8),
                                                   (128, 128, 0, 32, 8), (128, 32, 0, 3, 3),
                                                   (128, 128, 1, 16, 2), (256, 256, 0, 2, 1),
                                                   (256, 64, 1, 16, 8)])
@pytest.mark.parametrize("T, bs", [(1, 16), (37, 16), (301, 64)])
def test_write(mode, D, r, layout, Hq, Hkv, T, bs):
    w = Write(mode, D, Hq, Hkv, T, bs, r, layout, seed=T + D + r, magnitude=1.0 if r == D else 0.75)
    w.run()
    w.check()


@pytest.mark.parametrize("mode", MODES)
def test_write_many_tokens(mode):
    """More tokens than warps: several items per warp."""
    w = Write(mode, 64, 4, 2, 12000, seed=3)
    w.pos = [(7 * t) % 131072 for t in range(w.T)]
    w.p = torch.tensor(w.pos, device="cuda")
    w.run()
    kvq = K()
    torch.cuda.synchronize()
    assert kvq.kvq_get_device_error() == 0
    small = Write(mode, 64, 4, 2, 12000, seed=3)
    small.p = w.p
    for t0 in range(0, 12000, 1500):               # the same tokens in calls of 1500
        stride = 8 * 64
        kvq.kvq_rope_cache_write(
            small.ctx, small.rope, 0, small.qkv[t0:], small.q_out[t0:], small.qkv[t0:, 4:],
            small.qkv[t0:, 6:], small.p[t0:], small.slots[t0:], small.kc, small.vc, small.kcs,
            small.vcs, small.ks, small.vs, q_token_stride=stride, kv_token_stride=stride,
            num_tokens=1500)
    assert torch.equal(w.q_out, small.q_out)
    assert torch.equal(w.kc, small.kc) and torch.equal(w.vc, small.vc)
    if w.kcs is not None:
        assert torch.equal(w.kcs, small.kcs) and torch.equal(w.vcs, small.vcs)


@pytest.mark.parametrize("mode", [orc.FP8_PER_TOKEN_HEAD, orc.INT4_PER_TOKEN_HEAD])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -120, 2.0 ** 110])
def test_write_extreme_magnitudes(mode, scale):
    w = Write(mode, 64, 4, 2, 9, scale=scale)
    w.run()
    w.check()
    if scale == 0.0:
        live = w.slots[w.slots >= 0]
        assert torch.all(w.kcs[live // 16, :, live % 16] == 1.0)


def test_write_smallest_values():
    """The smallest bf16 subnormals: scales stay positive and codes finite."""
    for mode in (orc.FP8_PER_TOKEN_HEAD, orc.INT4_PER_TOKEN_HEAD):
        w = Write(mode, 64, 4, 2, 5, magnitude=0.0625)
        w.qkv.zero_()
        w.qkv.view(torch.int16)[..., ::3] = 1            # 2^-133
        w.run()
        torch.cuda.synchronize()
        live = w.slots[w.slots >= 0]
        s = w.kcs[live // 16, :, live % 16]
        assert torch.all(s > 0)
        codes = w.kc.cpu().numpy()
        assert np.isfinite(_nibbles(codes) if mode == orc.INT4_PER_TOKEN_HEAD else _e4m3(codes)).all()
        if mode == orc.INT4_PER_TOKEN_HEAD:
            assert np.abs(_nibbles(codes)).max() <= 7


def test_write_without_queries_and_bad_slots():
    kvq = K()
    w = Write(orc.FP8_PER_TOKEN_HEAD, 128, 8, 4, 40)
    w.run()
    kc, vc = w.kc.clone(), w.vc.clone()
    w.kc.zero_(), w.vc.zero_()
    w.run(q=False)
    assert torch.equal(w.kc, kc) and torch.equal(w.vc, vc)
    assert kvq.kvq_get_device_error() == 0
    t = 7
    old = w.slots[t].item()
    w.slots[t] = w.blocks * w.bs                        # one past the cache
    w.kc.zero_(), w.vc.zero_()
    w.q_out.fill_(float("nan"))
    w.run()
    assert kvq.kvq_get_device_error() == kvq.STATUS.index("KVQ_ERR_BAD_INDEX")
    kc[old // w.bs, :, old % w.bs] = 0
    assert torch.equal(w.kc, kc)
    assert torch.isfinite(w.q_out.float()).all()        # its queries are rotated all the same


def test_write_queries_in_place_in_the_fused_buffer():
    kvq = K()
    w = Write(orc.FP8_PER_HEAD, 64, 8, 2, 50, layout=1)
    w.run()
    stride = 12 * 64
    kc = w.kc.clone()
    w.kc.zero_()
    kvq.kvq_rope_cache_write(w.ctx, w.rope, 0, w.qkv, w.qkv, w.qkv[:, 8:], w.qkv[:, 10:], w.p, w.slots,
                             w.kc, w.vc, None, None, w.ks, w.vs, q_token_stride=stride,
                             q_out_token_stride=stride, kv_token_stride=stride, num_tokens=50)
    assert torch.equal(w.qkv[:, :8], w.q_out) and torch.equal(w.kc, kc)


def test_write_on_a_stream_and_in_a_graph():
    w = Write(orc.INT4_PER_TOKEN_HEAD, 128, 32, 8, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w.run(stream=side)
    side.synchronize()
    w.check()
    kc, q = w.kc.clone(), w.q_out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.run()
    w.kc.zero_(), w.q_out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w.kc, kc) and torch.equal(w.q_out, q)
    w.p += 5                                            # the graph reads the positions anew
    w.pos = [p + 5 for p in w.pos]
    graph.replay()
    w.check()
