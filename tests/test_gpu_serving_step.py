"""The operators together, as a server runs them: rows are extended, prompts and
single tokens rotated and written, attended to, forked, cut, closed up and cross
attended, over one pool of pages.

Every attention output of the pool is compared bit for bit with the same tokens
written into a fresh cache of their own (no page was ever shared, freed or moved
there), and the last ones with the 64-bit model."""
import numpy as np
import pytest
import torch

from oracle import oracle as orc
from tests import cross_model as cm
from tests import rope_model as rm
from tests.gpu_harness import K

pytestmark = pytest.mark.gpu

Hq, Hkv, D, BS = 8, 2, 64, 16


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, mode, blocks=96, rows=8, max_blocks=12, layers=2):
        kvq = K()
        self.mode, self.rows = mode, rows
        self.ctx = kvq.kvq_create(layers, Hq, Hkv, D, BS, blocks, [mode] * layers)
        self.rope = kvq.kvq_rope_create(D, 32, layout=1, scaling=kvq.ROPE_LINEAR, factor=2.0)
        self.caches = [kvq.alloc_layer_cache(self.ctx, i) for i in range(layers)]
        self.layers = kvq.layer_pointers(*[[c[i] for c in self.caches] for i in range(4)])
        self.ref = torch.zeros(blocks, dtype=torch.int32, device="cuda")
        self.table = torch.full((rows, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.static = torch.tensor([0.02, 0.03], device="cuda") if mode == orc.FP8_PER_HEAD else None
        self.history = [torch.zeros(0, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")] * rows
        self.gen = torch.Generator(device="cuda").manual_seed(mode + 1)

    def state(self):
        return self.ref, self.table, self.lens

    def scales(self, c):
        return dict(k_cache_scale=c[2], v_cache_scale=c[3], k_scale=self.static, v_scale=self.static)

    def step(self, rows, new):
        """Extends the rows, writes fresh tokens into every layer; (rotated q, query_start)."""
        kvq = K()
        T = sum(new)
        qs = torch.zeros(len(rows) + 1, dtype=torch.int32, device="cuda")
        pos = torch.zeros(T, dtype=torch.int64, device="cuda")
        slots = torch.zeros(T, dtype=torch.int64, device="cuda")
        copies = torch.zeros(len(rows), 2, dtype=torch.int32, device="cuda")
        kvq.kvq_extend_sequences(self.ctx, _i32(rows), _i32(new), *self.state(), qs, pos, slots, copies)
        kvq.kvq_copy_blocks(self.ctx, copies, self.layers)
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=self.gen, device="cuda").to(torch.bfloat16)
        q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        for i, c in enumerate(self.caches):
            self.write(self.ctx, c, i, qkv, q, pos, slots)
        at = 0
        for r, n in zip(rows, new):
            self.history[r] = torch.cat([self.history[r], qkv[at:at + n]])
            at += n
        return q, qs

    def write(self, ctx, c, layer, qkv, q, pos, slots):
        stride = (Hq + 2 * Hkv) * D
        K().kvq_rope_cache_write(ctx, self.rope, layer, qkv, q, qkv[:, Hq:], qkv[:, Hq + Hkv:], pos, slots,
                                 c[0], c[1], c[2], c[3], self.static, self.static, q_token_stride=stride,
                                 kv_token_stride=stride, num_tokens=qkv.shape[0])

    def prefill(self, ctx, c, table, lens, q, qs, layer):
        out = torch.empty(q.shape, device="cuda")
        K().kvq_prefill_attention(ctx, layer, q, c[0], c[1], table, qs, lens, out, max_query_len=q.shape[0],
                                  **self.scales(c))
        return out

    def fresh(self, rows):
        """The rows' whole histories in a cache of their own, page after page."""
        kvq = K()
        lens = [self.history[r].shape[0] for r in rows]
        used = [-(-n // BS) for n in lens]
        ctx = kvq.kvq_create(1, Hq, Hkv, D, BS, sum(used), [self.mode])
        c = kvq.alloc_layer_cache(ctx, 0)
        table = torch.full((len(rows), max(used)), -1, dtype=torch.int32)
        at = 0
        for i, u in enumerate(used):
            table[i, :u] = torch.arange(at, at + u)
            at += u
        qkv = torch.cat([self.history[r] for r in rows])
        pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
        tab = table.cuda()
        slots = torch.cat([tab[i, torch.arange(n, device="cuda") // BS].long() * BS +
                           torch.arange(n, device="cuda") % BS for i, n in enumerate(lens)])
        q = torch.empty(qkv.shape[0], Hq, D, dtype=torch.bfloat16, device="cuda")
        self.write(ctx, c, 0, qkv, q, pos, slots)
        return ctx, c, tab, _i32(lens), q

    def check(self, rows, q, qs):
        """Attention of the new queries over the pool, in every layer, against the fresh cache."""
        ctx, c, tab, lens, fq = self.fresh(rows)
        starts, total, want_q = qs.tolist(), lens.tolist(), []
        at = 0
        for i, n in enumerate(total):
            want_q.append(fq[at + n - (starts[i + 1] - starts[i]):at + n])
            at += n
        assert torch.equal(torch.cat(want_q), q)               # rotated alike whatever the batch
        want = self.prefill(ctx, c, tab, lens, q, qs, 0)
        r = torch.tensor(rows, device="cuda")
        assert torch.equal(self.lens[r], lens)
        for i, cache in enumerate(self.caches):
            got = self.prefill(self.ctx, cache, self.table[r].contiguous(), self.lens[r].contiguous(), q, qs, i)
            assert torch.equal(got, want)
        assert K().kvq_get_device_error() == 0
        return want

    def exact(self, row, n):
        """64-bit attention of the row's last n queries, from its history (no quantization)."""
        h = self.history[row].double().cpu().numpy()
        fs, m = K().kvq_rope_frequencies(self.rope)
        pos = list(range(h.shape[0]))
        rot = rm.rotate(h[:, :Hq + Hkv], pos, fs, 1, m)
        q, k, v = rot[:, :Hq], rot[:, Hq:], h[:, Hq + Hkv:]
        out = np.zeros((n, Hq, D))
        for i in range(n):
            L = h.shape[0] - n + i + 1
            for hq in range(Hq):
                s = k[:L, hq // (Hq // Hkv)] @ q[L - 1, hq] / np.sqrt(D)
                w = np.exp(s - s.max())
                out[i, hq] = (w / w.sum()) @ v[:L, hq // (Hq // Hkv)]
        return out


@pytest.mark.parametrize("mode", [orc.BF16, orc.FP8_PER_HEAD, orc.FP8_PER_TOKEN_HEAD,
                                  orc.INT4_PER_TOKEN_HEAD])
def test_serving(mode):
    kvq = K()
    s = Server(mode)
    # three prompts
    q, qs = s.step([0, 1, 2], [37, 64, 5])
    s.check([0, 1, 2], q, qs)
    # beams of request 1 (its last page is full) and of request 0 (partly filled)
    kvq.kvq_fork_sequences(s.ctx, _i32([1, 1, 0]), _i32([3, 4, 5]), *s.state())
    for p, c in ((1, 3), (1, 4), (0, 5)):
        s.history[c] = s.history[p]
    for _ in range(3):
        rows = [5, 0, 3, 1, 4, 2]
        q, qs = s.step(rows, [1] * 6)
        s.check(rows, q, qs)
    # one beam loses, a draft is taken back, another request ends
    kvq.kvq_truncate_sequences(s.ctx, _i32([4, 0, 2]), _i32([0, 35, 0]), *s.state())
    s.history[4] = s.history[4][:0]
    s.history[0] = s.history[0][:35]
    s.history[2] = s.history[2][:0]
    q, qs = s.step([0, 3, 1], [4, 1, 2])
    s.check([0, 3, 1], q, qs)
    # the pool closes up; a new request takes a freed row
    moves = torch.zeros(48, 2, dtype=torch.int32, device="cuda")
    count = _i32([0])
    kvq.kvq_compact_blocks(s.ctx, *s.state(), moves, count)
    kvq.kvq_copy_blocks(s.ctx, moves, s.layers, num_pairs=count)
    used = int((s.ref > 0).sum())
    assert (s.ref[:used] > 0).all() and count.item() > 0
    q, qs = s.step([2, 5, 3, 0], [20, 1, 1, 3])
    want = s.check([2, 5, 3, 0], q, qs)
    # the decode step of the pool agrees with its prefill of one token
    q, qs = s.step([2, 3], [1, 1])
    want = s.check([2, 3], q, qs)
    r = torch.tensor([2, 3], device="cuda")
    c = s.caches[1]
    out = torch.empty(2, Hq, D, device="cuda")
    kvq.kvq_decode_attention(s.ctx, 1, q, c[0], c[1], s.table[r].contiguous(), s.lens[r].contiguous(), out,
                             max_context=int(s.lens.max()), num_workers=1, **s.scales(c))
    assert torch.allclose(out, want, rtol=1e-4, atol=1e-4)
    # against the 64-bit model: the cache's own rounding is what is left.  A value is off by
    # half a code step (1/14 of the amax for INT4, 2^-4 for E4M3, 2^-8 for bf16), scores by
    # as much of about 8; outputs average some of it.  Static scales are coarse on purpose.
    exact = np.concatenate([s.exact(2, 1), s.exact(3, 1)])
    rel = np.linalg.norm(want.cpu().numpy() - exact) / np.linalg.norm(exact)
    assert rel < {orc.BF16: 2.0 ** -7, orc.FP8_PER_HEAD: 0.1, orc.FP8_PER_TOKEN_HEAD: 0.1,
                  orc.INT4_PER_TOKEN_HEAD: 0.35}[mode]
    # cross attention of the beams over an encoder's states shared by request 3's and 1's rows:
    # the pool's pages as they are now, all of them visible
    queries = torch.randn(5, Hq, D, generator=s.gen, device="cuda").to(torch.bfloat16)
    rows = torch.tensor([3, 1, 3], device="cuda")
    starts = _i32([0, 2, 2, 5])
    tab, lens = s.table[rows].contiguous(), s.lens[rows].contiguous()
    out = torch.zeros(5, Hq, D, dtype=torch.bfloat16, device="cuda")
    ns, need = kvq.kvq_cross_plan(s.ctx, 0, 3, 3, int(lens.max()))
    kvq.kvq_cross_attention(s.ctx, 0, queries, *s.caches[0][:2], tab, starts, lens, out, max_query_len=3,
                            max_encoder_len=int(lens.max()), num_splits=ns,
                            workspace=torch.empty(need, dtype=torch.uint8, device="cuda"),
                            **s.scales(s.caches[0]))
    assert kvq.kvq_get_device_error() == 0
    values = []
    for i in range(2):
        codes = s.caches[0][i]
        if mode == orc.BF16:
            v = codes.view(torch.bfloat16).double()
        elif mode == orc.INT4_PER_TOKEN_HEAD:
            n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int32)
            v = torch.where(n > 7, n - 16, n).double() * s.caches[0][2 + i][..., None].double()
        else:
            v = codes.view(torch.float8_e4m3fn).double()
            v = v * (s.static.double().view(1, -1, 1, 1) if s.static is not None
                     else s.caches[0][2 + i][..., None].double())
        values.append(v)
    ref, tol = cm.attend(queries, dict(values=values), tab, lens.tolist(), starts.tolist(), BS)
    assert ((out.double() - ref).abs() <= tol).all()
