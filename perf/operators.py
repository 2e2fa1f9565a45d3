"""Measured cases of the operators around the paged cache: rotary positions
(alone and fused with the cache write), the page operators (extend, fork,
truncate, compact, copy) and cross attention to an encoder's cached states.

``run`` computes a case either in its plain form (``own`` false: elementary
torch operations in 32 bits, angles in 64) or through the library's entry
points (``own`` true).  ``exact`` computes it once more in 64 bits.
"""
import functools
import math

import torch

own = False

BF16, FP8_PER_TENSOR, FP8_PER_HEAD, FP8_PER_TOKEN_HEAD, INT4_PER_TOKEN_HEAD = range(5)
HALF, INTERLEAVED = 0, 1
PLAIN, LINEAR, BASE, PARTS = range(4)
DEV = "cuda"


# ------------------------------------------------------------------- cases
def _rope(kind, name, T, Hq, Hkv, D, r, layout, scaling, mode=FP8_PER_TOKEN_HEAD, seqs=1, start=0,
          factor=1.0, base=10000.0, inverse=False):
    return dict(name=name, op=kind, T=T, Hq=Hq, Hkv=Hkv, D=D, r=r, layout=layout, scaling=scaling,
                mode=mode, seqs=seqs, start=start, factor=factor, base=base, inverse=inverse, bs=16)


def _pages(kind, name, layers, Hkv, D, bs, mode, rows, blocks, lo, hi, forks, add, drop):
    return dict(name=name, op=kind, layers=layers, Hkv=Hkv, D=D, bs=bs, mode=mode, rows=rows,
                blocks=blocks, lo=lo, hi=hi, forks=forks, add=add, drop=drop)


def _cross(name, B, n_lo, n_hi, S_lo, S_hi, Hq, Hkv, D, bs, mode, step=False):
    return dict(name=name, op="cross", B=B, n_lo=n_lo, n_hi=n_hi, S_lo=S_lo, S_hi=S_hi, Hq=Hq,
                Hkv=Hkv, D=D, bs=bs, mode=mode, step=step)


def listed():
    return [
        # a decode step of 64 sequences: one token each, where latency counts
        _rope("rope_write", "rope_write_step", 64, 32, 8, 128, 128, HALF, PLAIN, seqs=64, start=4095),
        # a long prompt late in a 128K context, frequencies scaled by parts, static per-head scales
        _rope("rope_write", "rope_write_prompt", 32768, 64, 8, 128, 128, HALF, PARTS, FP8_PER_HEAD,
              start=98304, factor=8.0, base=500000.0),
        # an odd chunk of a wide-headed model that rotates a quarter of the head, INT4 pages
        _rope("rope_write", "rope_write_chunk_int4", 2053, 16, 8, 256, 64, INTERLEAVED, BASE,
              INT4_PER_TOKEN_HEAD, seqs=3, start=511, factor=4.0),
        # sixteen prompts of a narrow-headed model into a layer kept in BF16
        _rope("rope_write", "rope_write_bf16", 8192, 64, 8, 64, 64, HALF, LINEAR, BF16, seqs=16,
              factor=4.0, base=150000.0),
        # rotation alone of a chunk's queries
        _rope("rope_apply", "rope_apply_chunk", 16384, 32, 8, 128, 128, HALF, PLAIN),
        # its gradient for an odd number of tokens, half of the head rotated
        _rope("rope_apply", "rope_apply_inverse", 1021, 8, 8, 64, 32, INTERLEAVED, PLAIN,
              start=131072, inverse=True),
        # a step of beam search: every sequence forks, all take a token, shared tail pages are copied
        _pages("pages_beam", "pages_beam_step", 24, 8, 64, 16, FP8_PER_TOKEN_HEAD, 64, 12288, 200,
               2000, 3, 1, 0),
        # a small server's turnover: some sequences end, a prompt is shared, all grow, pages close up
        _pages("pages_turn", "pages_turnover", 2, 2, 64, 16, BF16, 24, 2048, 33, 900, 4, 37, 3),
        # half of the long sequences end and the pool is closed up
        _pages("pages_turn", "pages_compact", 4, 8, 128, 16, FP8_PER_TOKEN_HEAD, 32, 65536, 20000,
               32000, 0, 1, 2),
        # one token of each sequence to its encoder's states
        _cross("cross_step", 64, 1, 1, 1000, 1500, 32, 8, 128, 16, FP8_PER_TOKEN_HEAD, step=True),
        # a few tokens of each sequence to long encoder states, ragged, one of them empty
        _cross("cross_few", 8, 1, 5, 20000, 32768, 64, 8, 128, 16, FP8_PER_HEAD),
        # whole decoder prompts
        _cross("cross_prompt", 8, 900, 1024, 3000, 4096, 32, 8, 128, 16, FP8_PER_TOKEN_HEAD),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope_write", "rope_write", "rope_apply", "pages_beam", "pages_turn",
                       "cross", "cross", "cross"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    mode = rng.choice([BF16, FP8_PER_TENSOR, FP8_PER_HEAD, FP8_PER_TOKEN_HEAD, INT4_PER_TOKEN_HEAD])
    G = rng.choice([1, 2, 4, 8] if D < 256 else [1, 2])
    bs = rng.choice([16, 32, 64, 128])
    if kind.startswith("rope"):
        H = Hkv * G
        T = _log(rng, 1, 32768 if H * D <= 4096 else 8192)
        c = _rope(kind, "", T, H, Hkv, D, rng.choice([D, D, D // 2, D // 4]), rng.choice([0, 1]),
                  rng.choice([PLAIN, LINEAR, BASE, PARTS]), mode, seqs=rng.randint(1, min(T, 9)),
                  start=rng.choice([0, rng.randrange(1, 200000)]), factor=rng.choice([2.0, 8.0, 32.0]),
                  base=rng.choice([10000.0, 500000.0]), inverse=kind == "rope_apply" and rng.random() < 0.5)
        c["bs"] = bs
    elif kind.startswith("pages"):
        hi = _log(rng, 40, 4000)
        rows = _log(rng, 4, 64)
        forks = rng.randint(1, 3) if kind == "pages_beam" else rng.randint(0, rows // 4)
        per = -(-(hi + 80) // bs) + 1
        total = rows * (1 + (forks if kind == "pages_beam" else 0)) + forks
        mode = mode if mode != INT4_PER_TOKEN_HEAD else FP8_PER_TOKEN_HEAD
        c = _pages(kind, "", rng.randint(1, 6), Hkv, D, bs, mode, rows, total * per + rng.randrange(50),
                   max(1, hi // rng.randint(2, 20)), hi, forks, _log(rng, 1, 60), rng.randint(2, 5))
    else:
        step = rng.random() < 0.3
        S = _log(rng, 1, 16384)
        n = 1 if step else _log(rng, 1, 512)
        B = _log(rng, 1, max(1, min(64, 200000 // S, 4096 // n)))
        while 4 * B * n * S * Hkv * G * D > 4e11:
            n = n // 2
        c = _cross("", B, max(1, n // rng.randint(1, 4)), n, max(1, S // rng.randint(1, 8)), S, Hkv * G,
                   Hkv, D, bs, mode, step)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _row_bytes(mode, D):
    return 2 * D if mode == BF16 else D // 2 if mode == INT4_PER_TOKEN_HEAD else D


def _dynamic(mode):
    return mode in (FP8_PER_TOKEN_HEAD, INT4_PER_TOKEN_HEAD)


def _heads(n, g):
    """Per-head multipliers, log-uniform in [0.5, 32] as the workloads draw them."""
    return torch.exp(math.log(0.5) + torch.rand(n, generator=g, device=DEV) * math.log(64.0))


def prepare(case, seed):
    g = _gen(seed)
    if case["op"].startswith("rope"):
        return _prepare_rope(case, g)
    if case["op"].startswith("pages"):
        return _prepare_pages(case, g)
    return _prepare_cross(case, g)


def _prepare_rope(c, g):
    T, Hq, Hkv, D, bs, seqs = c["T"], c["Hq"], c["Hkv"], c["D"], c["bs"], c["seqs"]
    s = dict(c)
    each = -(-T // seqs)
    t = torch.arange(T, device=DEV)
    s["positions"] = c["start"] + t % each + 7 * (t // each)
    if c["op"] == "rope_apply":
        s["x"] = torch.randn(T, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["x"])
        return s
    # a fused projection's output: q, k and v rows side by side
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV)
    mult = _heads(Hkv, g)
    qkv[:, Hq:] *= torch.cat([mult, mult])[None, :, None]
    s["qkv"] = qkv.to(torch.bfloat16)
    s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    blocks = seqs * -(-each // bs) + 2
    cells = torch.randperm(blocks, generator=g, device=DEV)
    b, p = t // each, t % each
    s["slots"] = cells[b * -(-each // bs) + p // bs] * bs + p % bs
    if T > 40:
        s["slots"][T // 3] = -1                      # padding: nothing is stored for this token
    s["blocks"] = blocks
    s["cache"] = torch.zeros(2, blocks, Hkv, bs, _row_bytes(c["mode"], D), dtype=torch.uint8, device=DEV)
    s["scales"] = torch.zeros(2, blocks, Hkv, bs, device=DEV) if _dynamic(c["mode"]) else None
    s["static"] = None
    if c["mode"] == FP8_PER_TENSOR:
        s["static"] = torch.tensor([[0.25], [0.5]], device=DEV)
    if c["mode"] == FP8_PER_HEAD:
        s["static"] = torch.stack([mult, mult]) * (4.0 / 448.0)
    return s


def _prepare_pages(c, g):
    rows, bs, blocks = c["rows"], c["bs"], c["blocks"]
    s = dict(c)
    lens = torch.randint(c["lo"], c["hi"] + 1, (rows,), generator=g, device=DEV, dtype=torch.int32)
    extra = rows * c["forks"] if c["op"] == "pages_beam" else c["forks"]
    total = rows + extra
    max_blocks = -(-(c["hi"] + c["add"]) // bs) + 1
    used = -(-lens // bs)
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    at = used.cumsum(0) - used
    j = torch.arange(max_blocks, device=DEV)
    idx = (at[:, None] + j[None]).clamp_max(blocks - 1)
    table = torch.full((total, max_blocks), -1, dtype=torch.int32, device=DEV)
    table[:rows] = torch.where(j[None] < used[:, None], perm[idx], -1)
    ref = torch.zeros(blocks, dtype=torch.int32, device=DEV)
    ref[table[table >= 0].long()] = 1
    all_lens = torch.zeros(total, dtype=torch.int32, device=DEV)
    all_lens[:rows] = lens
    s["book"] = torch.cat([ref, table.reshape(-1), all_lens])
    s["total"], s["max_blocks"] = total, max_blocks
    i32 = dict(dtype=torch.int32, device=DEV)
    if c["op"] == "pages_beam":
        s["parents"] = torch.arange(rows, **i32).repeat_interleave(c["forks"])
        s["children"] = torch.arange(rows, total, **i32)
        s["grow"] = torch.arange(total, **i32)
        s["ended"] = torch.arange(rows, total, 2, **i32)         # beams that lose the step
        s["keep"] = None
    else:
        s["ended"] = torch.arange(0, rows, c["drop"], **i32) if c["drop"] else torch.zeros(0, **i32)
        s["keep"] = torch.where(s["ended"] % 3 == 1, all_lens[s["ended"].long()] // 2, 0).to(torch.int32)
        s["parents"] = torch.full((extra,), 1, **i32)            # a shared prompt
        s["children"] = torch.arange(rows, total, **i32)
        alive = torch.ones(total, dtype=torch.bool, device=DEV)
        alive[s["ended"].long()] = False
        s["grow"] = alive.nonzero().flatten().to(torch.int32)
    n = s["grow"].numel()
    s["added"] = torch.full((n,), c["add"], **i32)
    s["tokens"] = n * c["add"]
    rb = _row_bytes(c["mode"], c["D"])
    shape = (2, c["layers"], blocks, c["Hkv"], bs)
    dtype = torch.bfloat16 if c["mode"] == BF16 else torch.uint8
    s["cache"] = torch.randint(0, 0x7F, (*shape, rb), generator=g, device=DEV, dtype=torch.uint8).view(dtype)
    s["scales"] = torch.rand(*shape, generator=g, device=DEV) if _dynamic(c["mode"]) else None
    return s


def _prepare_cross(c, g):
    B, Hq, Hkv, D, bs, mode = c["B"], c["Hq"], c["Hkv"], c["D"], c["bs"], c["mode"]
    s = dict(c)
    S = torch.randint(c["S_lo"], c["S_hi"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    # the numbers of queries go by the case alone, so that every seed's outputs have one shape
    n = torch.randint(c["n_lo"], c["n_hi"] + 1, (B,), generator=_gen(7), device=DEV, dtype=torch.int32)
    S[0], n[B // 2] = c["S_hi"], c["n_hi"]
    if B > 2 and not c["step"]:
        S[1], n[2] = 0, 0                            # a sequence without states, one without queries
    used = -(-S // bs)
    max_blocks = -(-c["S_hi"] // bs)
    blocks = int(used.sum()) + 3
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    j = torch.arange(max_blocks, device=DEV)
    idx = ((used.cumsum(0) - used)[:, None] + j[None]).clamp_max(blocks - 1)
    s["table"] = torch.where(j[None] < used[:, None], perm[idx], -1).to(torch.int32).contiguous()
    s["lens"], s["blocks"] = S, blocks
    s["query_start"] = None if c["step"] else torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
    T = B if c["step"] else int(n.sum())
    s["q"] = torch.randn(T, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    mult = _heads(Hkv, g)
    s["static"] = s["scales"] = None
    if mode == FP8_PER_TENSOR:
        s["static"] = torch.tensor([[0.25], [0.5]], device=DEV)
    if mode == FP8_PER_HEAD:
        s["static"] = torch.stack([mult, mult]) * (4.0 / 448.0)
    parts = [_codes(torch.randn(blocks, Hkv, bs, D, generator=g, device=DEV) * mult[None, :, None, None],
                    mode, None if s["static"] is None else s["static"][i]) for i in range(2)]
    s["cache"] = torch.stack([p[0] for p in parts])
    if _dynamic(mode):
        s["scales"] = torch.stack([p[1] for p in parts])
    s["out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------- plain forms
def _codes(x, mode, static, head_axis=-3):
    """(code bytes, dynamic scales) of vectors x [..., D]; the KV head is the axis before the
    slot axis ([blocks, Hkv, bs, D]) or, with head_axis -2, the last axis but one."""
    if mode == BF16:
        return x.to(torch.bfloat16).view(torch.uint8), None
    if mode == INT4_PER_TOKEN_HEAD:
        m = x.abs().amax(-1)
        scale = torch.where(m > 0, m / torch.full_like(m, 7.0), torch.ones_like(m))
        q = torch.round(x / scale[..., None]).clamp(-7, 7).to(torch.int32) & 15
        return (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8), scale
    if mode == FP8_PER_TOKEN_HEAD:
        m = x.abs().amax(-1)
        scale = torch.where(m > 0, m / torch.full_like(m, 448.0), torch.ones_like(m))
        div = scale[..., None]
    else:
        scale = None
        shape = [1] * x.dim()
        shape[head_axis] = static.numel()
        div = static.view(shape)
    return (x / div).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _values(codes, mode):
    """fp32 values that code bytes [..., row] stand for, without their scales."""
    if mode == BF16:
        return codes.view(torch.bfloat16).float()
    if mode == INT4_PER_TOKEN_HEAD:
        c = codes.to(torch.int32)
        q = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        return (q - 16 * (q > 7)).float()
    return codes.view(torch.float8_e4m3fn).float()


@functools.lru_cache(maxsize=None)
def _nibbles():
    """For each byte its two INT4 values as a pair of halves in one 32-bit word."""
    b = torch.arange(256, dtype=torch.int32)
    q = torch.stack([b & 15, b >> 4], -1)
    return (q - 16 * (q > 7)).to(torch.float16).view(torch.int32).flatten().to(DEV)


def _shown(cache, mode):
    """A cache's codes as the values they stand for (a view, or one look-up for INT4)."""
    if mode == BF16:
        return cache.view(torch.bfloat16)
    if mode == INT4_PER_TOKEN_HEAD:
        return _nibbles()[cache.int()].view(torch.float16)
    return cache.view(torch.float8_e4m3fn)


def _frequencies(c):
    i = torch.arange(c["r"] // 2, dtype=torch.float64, device=DEV)
    base = c["base"]
    if c["scaling"] == BASE:
        base = base * c["factor"] ** (c["r"] / (c["r"] - 2.0))
    f = base ** (-2.0 * i / c["r"])
    if c["scaling"] == LINEAR:
        f = f / c["factor"]
    if c["scaling"] == PARTS:
        turns = 8192.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / c["factor"]
    return f


def _magnitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == PARTS else 1.0


def _rotated(c, x, positions, inverse=False):
    """x [T, H, D] in 32 bits, rotated."""
    angle = positions.double()[:, None] * _frequencies(c)[None]
    cos = (angle.cos() * _magnitude(c)).float()[:, None]
    sin = (angle.sin() * (-_magnitude(c) if inverse else _magnitude(c))).float()[:, None]
    r, y = c["r"], x.clone()
    if c["layout"] == HALF:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2] = a * cos - b * sin
        y[..., r // 2:r] = a * sin + b * cos
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2] = a * cos - b * sin
        y[..., 1:r:2] = a * sin + b * cos
    return y


def _plain_rope_write(s):
    Hq, Hkv, bs = s["Hq"], s["Hkv"], s["bs"]
    x = s["qkv"].float()
    turned = _rotated(s, x[:, :Hq + Hkv], s["positions"])
    k, v = turned[:, Hq:], x[:, Hq + Hkv:]
    live = s["slots"] >= 0
    blk, off = s["slots"][live] // bs, s["slots"][live] % bs
    static = s["static"]
    for_k = _codes(k[live], s["mode"], None if static is None else static[0], -2)
    for_v = _codes(v[live], s["mode"], None if static is None else static[1], -2)
    s["cache"][0][blk, :, off] = for_k[0]
    s["cache"][1][blk, :, off] = for_v[0]
    if s["scales"] is not None:
        s["scales"][0][blk, :, off] = for_k[1]
        s["scales"][1][blk, :, off] = for_v[1]
    return turned[:, :Hq].to(torch.bfloat16)


def _books(s):
    """The page tables as they stand before the pass: reference counts, block table, lengths."""
    book = s["book"].clone()
    nb, cells = s["blocks"], s["total"] * s["max_blocks"]
    return book[:nb], book[nb:nb + cells].view(s["total"], s["max_blocks"]), book[nb + cells:]


def _plain_truncate(s, ref, table, lens, rows, keep):
    r, bs = rows.long(), s["bs"]
    old = lens[r]
    new = torch.zeros_like(old) if keep is None else torch.minimum(old, keep)
    j = torch.arange(s["max_blocks"], device=DEV)[None]
    gone = (j >= -(-new // bs)[:, None]) & (j < -(-old // bs)[:, None])
    part = table[r]
    ref.index_add_(0, part[gone].long(), torch.full_like(part[gone], -1))
    table[r] = torch.where(gone, -1, part)
    lens[r] = new


def _plain_fork(s, ref, table, lens, parents, children):
    p, c = parents.long(), children.long()
    j = torch.arange(s["max_blocks"], device=DEV)[None]
    have = j < -(-lens[p] // s["bs"])[:, None]
    part = table[p]
    ref.index_add_(0, part[have].long(), torch.ones_like(part[have]))
    table[c] = torch.where(have, part, -1)
    lens[c] = lens[p]


def _plain_extend(s, ref, table, lens, rows, added, tokens):
    r, bs = rows.long(), s["bs"]
    old = lens[r]
    new = old + added
    have, want = -(-old // bs), -(-new // bs)
    tail = table[r, (have - 1).clamp_min(0).long()].clamp_min(0)
    shared = (old % bs != 0) & (added > 0) & (ref[tail.long()] > 1)
    need = want - have + shared
    upto = need.cumsum(0)
    free = (ref == 0).nonzero().flatten().to(torch.int32)
    ok = (need == 0) | (upto <= free.numel())
    need = torch.where(ok, need, 0)
    first = torch.where(shared, have - 1, have)
    at = torch.repeat_interleave(torch.arange(r.numel(), device=DEV), need)
    k = torch.arange(at.numel(), device=DEV)
    table[r[at], (first[at] + k - (upto - need)[at]).long()] = free[:at.numel()]
    ref[free[:at.numel()].long()] = 1
    copied = shared & ok
    fresh = table[r, (have - 1).clamp_min(0).long()]
    copies = torch.where(copied[:, None], torch.stack([tail, fresh], -1), -1)
    ref.index_add_(0, tail[copied].long(), torch.full_like(tail[copied], -1))
    lens[r] = torch.where(ok, new, old)
    start = torch.cat([added.new_zeros(1), added.cumsum(0)]).to(torch.int32)
    t = torch.arange(tokens, device=DEV)
    row = torch.repeat_interleave(torch.arange(r.numel(), device=DEV), added)
    position = old[row] + t - start[row]
    slot = table[r[row], (position // bs).long()].long() * bs + position % bs
    slot = torch.where(ok[row], slot, -1)
    return start, position.long(), slot, copies.to(torch.int32)


def _plain_compact(s, ref, table, lens):
    in_use = ref > 0
    n = int(in_use.sum())
    src = in_use[n:].nonzero().flatten() + n
    dst = (~in_use[:n]).nonzero().flatten()
    to = torch.arange(ref.numel(), dtype=torch.int32, device=DEV)
    to[src] = dst.to(torch.int32)
    ref[dst] = ref[src]
    ref[src] = 0
    j = torch.arange(s["max_blocks"], device=DEV)[None]
    have = j < -(-lens // s["bs"])[:, None]
    table.copy_(torch.where(have, to[table.clamp_min(0).long()], table))
    return torch.stack([src, dst], -1).to(torch.int32)


def _plain_copy(s, pairs):
    pairs = pairs[pairs[:, 0] >= 0].long()
    s["cache"][:, :, pairs[:, 1]] = s["cache"][:, :, pairs[:, 0]]
    if s["scales"] is not None:
        s["scales"][:, :, pairs[:, 1]] = s["scales"][:, :, pairs[:, 0]]


def _plain_pages(s):
    ref, table, lens = _books(s)
    if s["op"] == "pages_beam":
        _plain_fork(s, ref, table, lens, s["parents"], s["children"])
        grown = _plain_extend(s, ref, table, lens, s["grow"], s["added"], s["tokens"])
        _plain_copy(s, grown[3])
        _plain_truncate(s, ref, table, lens, s["ended"], s["keep"])
        moves = None
    else:
        _plain_truncate(s, ref, table, lens, s["ended"], s["keep"])
        _plain_fork(s, ref, table, lens, s["parents"], s["children"])
        grown = _plain_extend(s, ref, table, lens, s["grow"], s["added"], s["tokens"])
        _plain_copy(s, grown[3])
        moves = _plain_compact(s, ref, table, lens)
        _plain_copy(s, moves)
    return _pages_out(s, ref, table, lens, grown)


def _pages_out(s, ref, table, lens, grown):
    cache = s["cache"] if s["mode"] == BF16 else s["cache"].view(torch.float8_e4m3fn)
    return dict(ref=ref, table=table, lens=lens, start=grown[0], positions=grown[1], slots=grown[2],
                copies=grown[3], cache=cache, scales=s["scales"])


def _plain_cross(s):
    Hq, Hkv, D, B, mode = s["Hq"], s["Hkv"], s["D"], s["B"], s["mode"]
    S = s["lens"]
    blk = s["table"].clamp_min(0).long()
    # [B, Hkv, positions, D] keys and values
    kv = [_values(s["cache"][i][blk], mode).transpose(1, 2).flatten(2, 3) for i in range(2)]
    if s["scales"] is not None:
        kv = [x * s["scales"][i][blk].transpose(1, 2).flatten(2, 3)[..., None] for i, x in enumerate(kv)]
    if s["static"] is not None:
        kv = [x * s["static"][i].view(1, -1, 1, 1) for i, x in enumerate(kv)]
    if s["query_start"] is None:
        start, n, most = torch.arange(B, device=DEV), S.new_ones(B), 1
    else:
        start = s["query_start"][:-1].long()
        n, most = s["query_start"][1:] - s["query_start"][:-1], s["n_hi"]
    i = torch.arange(most, device=DEV)
    row = (start[:, None] + i[None]).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, most, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q.reshape(B, Hkv, -1, D), kv[0].transpose(-1, -2)) / math.sqrt(D)
    seen = torch.arange(kv[0].shape[2], device=DEV)[None] < S[:, None]
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    w = w / w.sum(-1, keepdim=True).clamp_min(1e-30)
    o = torch.matmul(w, kv[1]).view(B, Hkv, Hq // Hkv, most, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, most, Hq, D)
    live = i[None] < n[:, None]
    out = torch.zeros_like(s["q"])
    out[row[live]] = o[live].to(torch.bfloat16)
    return out


# -------------------------------------------------------- the library's own
@functools.lru_cache(maxsize=None)
def _context(layers, Hq, Hkv, D, bs, blocks, mode):
    from int4_quantized_paged_gb300 import kvq
    return kvq.kvq_create(layers, Hq, Hkv, D, bs, blocks, [mode] * layers)


@functools.lru_cache(maxsize=None)
def _rope_handle(D, r, layout, scaling, base, factor, magnitude):
    from int4_quantized_paged_gb300 import kvq
    return kvq.kvq_rope_create(D, r, layout=layout, base=base, scaling=scaling, factor=factor,
                               original_context=8192, low_rotations=1.0, high_rotations=32.0,
                               magnitude=magnitude)


def _own_rope(s):
    from int4_quantized_paged_gb300 import kvq
    rope = _rope_handle(s["D"], s["r"], s["layout"], s["scaling"], s["base"], s["factor"], _magnitude(s))
    if s["op"] == "rope_apply":
        kvq.kvq_rope_apply(rope, s["x"], s["positions"], s["out"], inverse=s["inverse"])
        return s["out"]
    Hq, Hkv, D, mode = s["Hq"], s["Hkv"], s["D"], s["mode"]
    ctx = _context(1, Hq, Hkv, D, s["bs"], s["blocks"], mode)
    stride = (Hq + 2 * Hkv) * D
    qkv, cache, scales, static = s["qkv"], s["cache"], s["scales"], s["static"]
    kvq.kvq_rope_cache_write(
        ctx, rope, 0, qkv, s["q_out"], qkv[:, Hq:], qkv[:, Hq + Hkv:], s["positions"], s["slots"],
        cache[0], cache[1], None if scales is None else scales[0], None if scales is None else scales[1],
        None if static is None else static[0], None if static is None else static[1],
        q_token_stride=stride, kv_token_stride=stride, num_tokens=s["T"])
    return s["q_out"]


def _own_pages(s):
    from int4_quantized_paged_gb300 import kvq
    ctx = _context(s["layers"], s["Hkv"], s["Hkv"], s["D"], s["bs"], s["blocks"], s["mode"])
    if "layers_of" not in s:                          # the pointers of every layer, kept by the program
        c, x = s["cache"], s["scales"]
        s["layers_of"] = kvq.layer_pointers(c[0].unbind(0), c[1].unbind(0),
                                            None if x is None else x[0].unbind(0),
                                            None if x is None else x[1].unbind(0))
    ref, table, lens = _books(s)
    n = s["grow"].numel()
    start = torch.empty(n + 1, dtype=torch.int32, device=DEV)
    positions = torch.empty(s["tokens"], dtype=torch.int64, device=DEV)
    slots = torch.empty(s["tokens"], dtype=torch.int64, device=DEV)
    copies = torch.empty(n, 2, dtype=torch.int32, device=DEV)
    beam = s["op"] == "pages_beam"
    if not beam:
        kvq.kvq_truncate_sequences(ctx, s["ended"], s["keep"], ref, table, lens)
    kvq.kvq_fork_sequences(ctx, s["parents"], s["children"], ref, table, lens)
    kvq.kvq_extend_sequences(ctx, s["grow"], s["added"], ref, table, lens, start, positions, slots, copies)
    kvq.kvq_copy_blocks(ctx, copies, s["layers_of"])
    if beam:
        kvq.kvq_truncate_sequences(ctx, s["ended"], s["keep"], ref, table, lens)
    else:
        moves = torch.empty(max(1, s["blocks"] // 2), 2, dtype=torch.int32, device=DEV)
        count = torch.empty(1, dtype=torch.int32, device=DEV)
        kvq.kvq_compact_blocks(ctx, ref, table, lens, moves, count)
        kvq.kvq_copy_blocks(ctx, moves, s["layers_of"], num_pairs=count)
    return _pages_out(s, ref, table, lens, (start, positions, slots, copies))


def _own_cross(s):
    from int4_quantized_paged_gb300 import kvq
    ctx = _context(1, s["Hq"], s["Hkv"], s["D"], s["bs"], s["blocks"], s["mode"])
    cache, scales, static = s["cache"], s["scales"], s["static"]
    most = 0 if s["query_start"] is None else s["n_hi"]      # 0: one query per sequence
    splits, need = kvq.kvq_cross_plan(ctx, 0, s["B"], most, s["S_hi"])
    work = torch.empty(need, dtype=torch.uint8, device=DEV)
    kvq.kvq_cross_attention(
        ctx, 0, s["q"], cache[0], cache[1], s["table"], s["query_start"], s["lens"], s["out"],
        max_query_len=most, max_encoder_len=s["S_hi"],
        k_cache_scale=None if scales is None else scales[0],
        v_cache_scale=None if scales is None else scales[1],
        k_scale=None if static is None else static[0], v_scale=None if static is None else static[1],
        num_splits=splits, workspace=work)
    return s["out"]


def run(s):
    if s["op"] == "rope_apply":
        return _own_rope(s) if own else _rotated(s, s["x"].float(), s["positions"], s["inverse"]).to(torch.bfloat16)
    if s["op"] == "rope_write":
        q = _own_rope(s) if own else _plain_rope_write(s)
        return dict(q=q, cache=_shown(s["cache"], s["mode"]), scales=s["scales"])
    if s["op"] == "cross":
        return _own_cross(s) if own else _plain_cross(s)
    return _own_pages(s) if own else _plain_pages(s)


# -------------------------------------------------------- what it cannot do without
def work(case):
    c = case
    if c["op"] == "rope_apply":
        n = c["T"] * c["Hq"] * c["D"]
        return dict(bytes=4 * n + 8 * c["T"], flops=3 * c["T"] * c["Hq"] * c["r"])
    if c["op"] == "rope_write":
        row = _row_bytes(c["mode"], c["D"]) + (4 if _dynamic(c["mode"]) else 0)
        per = 4 * c["Hq"] * c["D"] + 2 * c["Hkv"] * (2 * c["D"] + row) + 16
        return dict(bytes=per * c["T"], flops=c["T"] * (c["Hq"] + c["Hkv"]) * c["r"] * 3)
    mid = 0.5 * (c.get("lo", 0) + c.get("hi", 0))
    if c["op"].startswith("pages"):
        block = 2 * c["Hkv"] * c["bs"] * (_row_bytes(c["mode"], c["D"]) + (4 if _dynamic(c["mode"]) else 0))
        entries = c["rows"] * -(-mid // c["bs"])
        if c["op"] == "pages_beam":
            # nearly every sequence's tail page is shared: one copy for each beam
            pairs = c["rows"] * (1 + c["forks"]) * (1 - 1 / c["bs"])
            entries *= 1 + c["forks"]
        else:
            kept = entries * (1 - (1 / c["drop"] if c["drop"] else 0))
            moved = kept * max(0.0, 1 - kept / c["blocks"])
            pairs = moved + c["forks"]
        tokens = c["rows"] * c["add"]
        return dict(bytes=2 * block * pairs * c["layers"] + 4 * (c["blocks"] + 2 * entries) + 16 * tokens, flops=0)
    n = 0.5 * (c["n_lo"] + c["n_hi"])
    S = 0.5 * (c["S_lo"] + c["S_hi"])
    row = _row_bytes(c["mode"], c["D"]) + (4 if _dynamic(c["mode"]) else 0)
    return dict(bytes=c["B"] * (2 * S * c["Hkv"] * row + 4 * n * c["Hq"] * c["D"]),
                flops=4 * c["B"] * n * S * c["Hq"] * c["D"])


# ------------------------------------------------------------------ 64 bits
def _angles64(c, positions):
    """cos and sin of p f_i for every position, f_i formed one by one in 64 bits."""
    fs = []
    for i in range(c["r"] // 2):
        base = c["base"] * c["factor"] ** (c["r"] / (c["r"] - 2.0)) if c["scaling"] == BASE else c["base"]
        f = math.exp(-2.0 * i / c["r"] * math.log(base))
        if c["scaling"] == LINEAR:
            f /= c["factor"]
        if c["scaling"] == PARTS:
            t = (8192.0 * f / (2.0 * math.pi) - 1.0) / 31.0
            t = min(1.0, max(0.0, t))
            f = f * (t + (1.0 - t) / c["factor"])
        fs.append(f)
    a = positions.double()[:, None] * torch.tensor(fs, dtype=torch.float64, device=DEV)[None]
    m = 1.0 + 0.1 * math.log(c["factor"]) if c["scaling"] == PARTS else 1.0
    return m * torch.cos(a), m * torch.sin(a)


def _turn64(c, x, positions, inverse):
    """The rotation as a complex product."""
    cos, sin = _angles64(c, positions)
    turn = torch.complex(cos, -sin if inverse else sin)[:, None]
    r, out = c["r"], x.double().clone()
    first = slice(0, r // 2) if c["layout"] == HALF else slice(0, r, 2)
    second = slice(r // 2, r) if c["layout"] == HALF else slice(1, r, 2)
    z = torch.complex(out[..., first].contiguous(), out[..., second].contiguous()) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _quantum64(y, mode):
    if mode == INT4_PER_TOKEN_HEAD:
        return torch.round(y).clamp(-7, 7)
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -40))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_rope(s):
    if s["op"] == "rope_apply":
        return _turn64(s, s["x"], s["positions"], s["inverse"])
    Hq, Hkv, mode, bs = s["Hq"], s["Hkv"], s["mode"], s["bs"]
    x = s["qkv"].double()
    q = _turn64(s, x[:, :Hq], s["positions"], False)
    k = _turn64(s, x[:, Hq:Hq + Hkv], s["positions"], False)
    cache = torch.zeros(2, s["blocks"] * bs, Hkv, s["D"], dtype=torch.float64, device=DEV)
    scales = torch.zeros(2, s["blocks"] * bs, Hkv, dtype=torch.float64, device=DEV)
    keep = s["slots"] >= 0
    for i, v in enumerate((k, x[:, Hq + Hkv:])):
        v = v[keep]
        if mode == BF16:
            cache[i][s["slots"][keep]] = v
            continue
        if _dynamic(mode):
            top = v.abs().max(-1).values / (7.0 if mode == INT4_PER_TOKEN_HEAD else 448.0)
            # the codes' definition: the quotient by the scale as it is stored, rounded to 32 bits
            top = torch.where(top == 0, 1.0, top).float().double()
            scales[i][s["slots"][keep]] = top
        else:
            top = s["static"][i].double().expand(Hkv)[None]
        cache[i][s["slots"][keep]] = _quantum64((v / top[..., None]).float().double(), mode)
    paged = cache.view(2, s["blocks"], bs, Hkv, -1).transpose(2, 3).contiguous()
    shown = scales.view(2, s["blocks"], bs, Hkv).transpose(2, 3).contiguous()
    return dict(q=q, cache=paged, scales=shown if _dynamic(mode) else None)


def _exact_cross(s):
    """One sequence and KV head at a time."""
    Hq, Hkv, D, mode, bs = s["Hq"], s["Hkv"], s["D"], s["mode"], s["bs"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    starts = list(range(s["B"] + 1)) if s["query_start"] is None else s["query_start"].tolist()
    G = Hq // Hkv
    for b in range(s["B"]):
        S, rows = lens[b], slice(starts[b], starts[b + 1])
        if not S or rows.start == rows.stop:
            continue
        pages = s["table"][b][:-(-S // bs)].long()
        for h in range(Hkv):
            kv = []
            for i in range(2):
                x = s["cache"][i][pages, h].flatten(0, 1)[:S]
                if mode == INT4_PER_TOKEN_HEAD:
                    x = torch.stack([x % 16, x // 16], -1).flatten(-2).double()
                    x = torch.where(x >= 8, x - 16, x)
                else:
                    x = x.view(torch.bfloat16 if mode == BF16 else torch.float8_e4m3fn).double()
                if s["scales"] is not None:
                    x = x * s["scales"][i][pages, h].flatten(0, 1)[:S, None].double()
                if s["static"] is not None:
                    x = x * s["static"][i].double().expand(Hkv)[h]
                kv.append(x)
            q = s["q"][rows, h * G:(h + 1) * G].double()
            p = torch.softmax(q @ kv[0].T / math.sqrt(D), -1)
            out[rows, h * G:(h + 1) * G] = p @ kv[1]
    return out


def exact(case, seed):
    if case["op"].startswith("pages"):
        return None                                   # bytes and whole numbers: nothing is computed
    s = prepare(case, seed)
    return _exact_cross(s) if case["op"] == "cross" else _exact_rope(s)
