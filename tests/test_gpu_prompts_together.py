"""The operators for long and shared prompts one after another, as a server uses them: prompts are
rotated, attended and cached, a prompt is forked, its rows decode behind it, caches are held to a
budget and go on decoding."""
import pytest
import torch

from tests import cross_model as cm
from tests import evict_model as em
from tests import prompt_model as pm
from tests.gpu_harness import K

pytestmark = pytest.mark.gpu
BAD = 6
Hq, BS = 8, 16


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, mode, D, Hkv, rows=6, blocks=120, max_blocks=24):
        kvq = K()
        self.mode, self.D, self.Hkv = mode, D, Hkv
        self.ctx = kvq.kvq_create(1, Hq, Hkv, D, BS, blocks, [mode])
        self.rope = kvq.kvq_rope_create(D, D)
        self.kc, self.vc, self.ks, self.vs = kvq.alloc_layer_cache(self.ctx, 0)
        self.layers = kvq.layer_pointers([self.kc], [self.vc], [self.ks], [self.vs])
        self.static = _f32([0.02] * Hkv) if mode == 2 else None
        self.ref = torch.zeros(blocks, dtype=torch.int32, device="cuda")
        self.table = torch.full((rows, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.tokens = [0] * rows                     # positions in the sequence, evicted ones too
        self.weights = torch.zeros(rows, Hkv, max_blocks * BS, device="cuda")
        self.gen = torch.Generator(device="cuda").manual_seed(mode + D)

    def scales(self):
        return dict(k_cache_scale=self.ks, v_cache_scale=self.vs, k_scale=self.static, v_scale=self.static)

    def grow(self, rows, new):
        """New tokens of the rows: rotated and written; (fused rows, their starts)."""
        kvq, D, Hkv = K(), self.D, self.Hkv
        T = sum(new)
        start, slots = _i32([0] * (len(rows) + 1)), torch.zeros(T, dtype=torch.int64, device="cuda")
        inside, copies = torch.zeros_like(slots), _i32([[0, 0]] * len(rows))
        kvq.kvq_extend_sequences(self.ctx, _i32(rows), _i32(new), self.ref, self.table, self.lens, start, inside,
                                 slots, copies)
        kvq.kvq_copy_blocks(self.ctx, copies, self.layers)
        position = torch.tensor([self.tokens[r] + i for r, n in zip(rows, new) for i in range(n)], device="cuda")
        for r, n in zip(rows, new):
            self.tokens[r] += n
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=self.gen, device="cuda").to(torch.bfloat16)
        stride = (Hq + 2 * Hkv) * D
        kvq.kvq_rope_apply(self.rope, x, position, x, x_token_stride=stride, out_token_stride=stride,
                           num_heads=Hq + Hkv)
        self.fused, self.start, self.slots, self.stride = x, start, slots, stride
        return x

    def cache(self):
        x, Hkv = self.fused, self.Hkv
        K().kvq_cache_write(self.ctx, 0, x[:, Hq:], x[:, Hq + Hkv:], self.slots, self.kc, self.vc, self.ks, self.vs,
                            self.static, self.static, kv_token_stride=self.stride, num_tokens=x.shape[0])

    def values(self):
        """The cache's vectors in 64 bits, as cross_model takes them."""
        out = []
        for c, s in ((self.kc, self.ks), (self.vc, self.vs)):
            if self.mode == 0:
                v = c.view(torch.bfloat16).double()
            elif self.mode == 4:
                n = torch.stack([c & 15, c >> 4], -1).flatten(-2).double()
                v = torch.where(n > 7, n - 16, n)
            else:
                v = c.view(torch.float8_e4m3fn).double()
            if s is not None:
                v = v * s.double()[..., None]
            if self.static is not None:
                v = v * self.static.double().view(1, -1, 1, 1)
            out.append(v.nan_to_num())
        return dict(values=out)

    def expect(self, q, rows):
        lens = self.lens[rows].tolist()
        return cm.attend(q, self.values(), self.table[rows], lens, list(range(len(rows) + 1)), BS)


def _f32(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


def _near(out, pair):
    torch.cuda.synchronize()
    ref, tol = pair
    assert torch.all((out.double() - ref).abs() <= tol)


@pytest.mark.parametrize("mode", [0, 2, 3, 4])
@pytest.mark.parametrize("D, Hkv", [(64, 2), (128, 2), (256, 4)])
def test_a_servers_day(mode, D, Hkv):
    kvq = K()
    s = Server(mode, D, Hkv)

    # two prompts in one pass, attended before they are cached
    new = [130, 77]
    x = s.grow([0, 1], new)
    out = torch.empty(sum(new), Hq, D, dtype=torch.bfloat16, device="cuda")
    kvq.kvq_prompt_attention(s.ctx, 0, x, x[:, Hq:], x[:, Hq + Hkv:], s.start, out, max_seq_len=130,
                             q_token_stride=s.stride, kv_token_stride=s.stride)
    s.cache()
    _near(out, pm.attend(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], [(0, 130), (130, 207)]))
    assert kvq.kvq_get_device_error() == 0

    # row 0 is forked twice; its rows decode behind it for some steps, row 1 by itself
    kvq.kvq_fork_sequences(s.ctx, _i32([0, 0]), _i32([2, 3]), s.ref, s.table, s.lens)
    s.tokens[2] = s.tokens[3] = 130
    batch = [0, 2, 3, 1]
    start, shared = _i32([0, 3]), _i32([130])
    sizes = dict(max_group=3, max_shared=130, max_own=160)
    splits, need = kvq.kvq_shared_prefix_plan(s.ctx, 0, 4, 1, num_splits=2, **sizes)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    for step in range(20):
        x = s.grow(batch, [1] * 4)
        s.cache()
        q = x[:, :Hq].contiguous()
        out = torch.empty(4, Hq, D, dtype=torch.bfloat16, device="cuda")
        kvq.kvq_shared_prefix_attention(s.ctx, 0, q, s.kc, s.vc, s.table[batch], s.lens[batch], start, shared, out,
                                        num_splits=splits, workspace=work, **sizes, **s.scales())
        if step % 6 == 0:
            _near(out, s.expect(q, batch))
    assert kvq.kvq_get_device_error() == 0

    # rows 1 and 3 go on with their weights accumulated
    n, need = kvq.kvq_decode_weights_plan(s.ctx, 0, 6, 24 * BS)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    lens = torch.zeros_like(s.lens)
    for step in range(12):
        x = s.grow([1, 3], [1, 1])
        s.cache()
        q = torch.zeros(6, Hq, D, dtype=torch.bfloat16, device="cuda")
        q[1], q[3] = x[0, :Hq], x[1, :Hq]
        lens.zero_()
        lens[[1, 3]] = s.lens[[1, 3]]                # the other rows rest
        out = torch.empty(6, Hq, D, dtype=torch.bfloat16, device="cuda")
        kvq.kvq_decode_attention_weights(s.ctx, 0, q, s.kc, s.vc, s.table, lens, s.weights, out,
                                         max_context=24 * BS, num_workers=n, workspace=work, **s.scales())
    _near(out[[1, 3]], s.expect(q[[1, 3]], [1, 3]))
    # twelve steps of a KV head's query heads gave one each in all; no one else got any
    assert torch.all((s.weights[[1, 3]].sum(-1) - 12 * Hq // Hkv).abs() < 1e-3)
    assert torch.all(s.weights[[0, 2, 4, 5]] == 0)

    # both are cut to 64 cells: row 3 still shares its prompt's blocks and is left as it is
    before, w = s.values()["values"], s.weights.cpu().tolist()
    L = s.lens.tolist()
    rows, keep, fresh = _i32([1, 3]), _i32([64, 64]), _i32([0, 0])
    kvq.kvq_evict_cells(s.ctx, 0, rows, keep, s.table, s.lens, s.weights, fresh, s.kc, s.vc, s.ks, s.vs,
                        first_kept=4, last_kept=16, max_context=24 * BS, ref_count=s.ref)
    torch.cuda.synchronize()
    assert kvq.kvq_get_device_error() == BAD
    assert fresh.tolist() == [64, L[3]]
    old = s.table[1].tolist()
    kvq.kvq_truncate_sequences(s.ctx, rows, fresh, s.ref, s.table, s.lens)
    assert s.lens.tolist() == L[:1] + [64] + L[2:]
    freed = old[4:-(-L[1] // BS)]
    assert len(freed) > 0 and all(int(s.ref[b]) == 0 for b in freed)

    # and decodes over what stayed, first by the list of its cells
    q = torch.randn(1, Hq, D, generator=s.gen, device="cuda").to(torch.bfloat16)
    kept = []
    for h in range(Hkv):
        cells = list(range(L[1]))
        for a, b in em.places(w[1][h], L[1], 64, 4, 16):
            cells[b] = a
        p = torch.tensor(sorted(cells[:64]), device="cuda")
        blk = torch.tensor(old, device="cuda")[p // BS]
        kept.append([v[blk, h, p % BS] for v in before])
    pages = dict(values=[torch.stack([k[i] for k in kept])[None] for i in range(2)])     # one block of 64
    want = cm.attend(q, pages, torch.zeros(1, 1, dtype=torch.int64, device="cuda"), [64], [0, 1], 64)
    out = torch.empty(1, Hq, D, dtype=torch.bfloat16, device="cuda")
    n, need = kvq.kvq_decode_plan(s.ctx, 0, 1, 64)
    kvq.kvq_decode_attention_bf16(s.ctx, 0, q, s.kc, s.vc, s.table[1:2], s.lens[1:2], out, max_context=64,
                                  num_workers=n, workspace=torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"),
                                  **s.scales())
    _near(out, want)

    # then with tokens appended, which start without weight
    for step in range(20):
        x = s.grow([1], [1])
        s.cache()
    q = x[:, :Hq].contiguous()
    out = torch.empty(1, Hq, D, dtype=torch.bfloat16, device="cuda")
    n, need = kvq.kvq_decode_weights_plan(s.ctx, 0, 1, 24 * BS)
    assert torch.all(s.weights[1, :, 64:] == 0)
    kvq.kvq_decode_attention_weights(s.ctx, 0, q, s.kc, s.vc, s.table[1:2], s.lens[1:2], s.weights[1:2], out,
                                     max_context=24 * BS, num_workers=n,
                                     workspace=torch.empty(need, dtype=torch.uint8, device="cuda"), **s.scales())
    _near(out, s.expect(q, [1]))
    assert torch.all(s.weights[1, :, 64:84] > 0) and torch.all(s.weights[1, :, 84:] == 0)
    assert kvq.kvq_get_device_error() == 0
