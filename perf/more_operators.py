"""Measured cases of the operators for long and shared prompts: attention over whole
prompts before they are cached, decode attention of a batch that shares a prefix,
decode attention that accumulates each cell's softmax weight, and the eviction of
the cells that gathered least.

``run`` computes a case either in its plain form (``own`` false: elementary torch
operations in 32 bits) or through the library's entry points (``own`` true).
``exact`` computes it once more in 64 bits.
"""
import functools
import math

import torch

own = False

BF16, FP8_PER_TENSOR, FP8_PER_HEAD, FP8_PER_TOKEN_HEAD, INT4_PER_TOKEN_HEAD = range(5)
DEV = "cuda"


# ------------------------------------------------------------------- cases
def _prompt(name, B, lo, hi, Hq, Hkv, D, window=0):
    return dict(name=name, op="prompt", B=B, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, D=D, window=window, bs=16,
                mode=BF16)


def _shared(name, groups, n_lo, n_hi, P_lo, P_hi, own_hi, Hq, Hkv, D, bs, mode):
    return dict(name=name, op="shared", groups=groups, n_lo=n_lo, n_hi=n_hi, P_lo=P_lo, P_hi=P_hi,
                own_hi=own_hi, Hq=Hq, Hkv=Hkv, D=D, bs=bs, mode=mode)


def _weights(name, B, lo, hi, Hq, Hkv, D, bs, mode, decay=1.0):
    return dict(name=name, op="weights", B=B, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, D=D, bs=bs, mode=mode,
                decay=decay)


def _evict(name, B, lo, hi, keep, first, last, Hkv, D, bs, mode):
    return dict(name=name, op="evict", B=B, lo=lo, hi=hi, keep=keep, first=first, last=last, Hq=Hkv,
                Hkv=Hkv, D=D, bs=bs, mode=mode)


def listed():
    return [
        # many short requests packed into one pass: latency and ragged ends
        _prompt("prompt_short", 48, 1, 120, 32, 8, 128),
        # a server's prefill batch, ragged
        _prompt("prompt_packed", 8, 500, 4096, 32, 8, 128),
        # one long document
        _prompt("prompt_long", 1, 16384, 16384, 32, 8, 128),
        # a window layer of a narrow-headed model
        _prompt("prompt_window", 4, 3000, 4096, 64, 8, 64, 128),
        # a wide-headed model
        _prompt("prompt_wide", 3, 1500, 4000, 16, 8, 256),
        # a few answers to one prompt, early on: latency
        _shared("shared_small", 1, 8, 8, 1500, 1500, 40, 32, 8, 128, 16, FP8_PER_TOKEN_HEAD),
        # a batch behind one long document, static scales
        _shared("shared_long", 1, 64, 64, 32000, 32768, 1000, 64, 8, 128, 16, FP8_PER_HEAD),
        # several prompts with beams of different numbers, INT4 pages
        _shared("shared_groups", 6, 1, 30, 100, 8000, 400, 32, 8, 128, 32, INT4_PER_TOKEN_HEAD),
        # a decode step of a batch whose caches are bounded
        _weights("weights_step", 64, 1500, 4200, 32, 8, 128, 16, FP8_PER_TOKEN_HEAD),
        # few long contexts, older weights fading
        _weights("weights_long", 4, 20000, 40000, 64, 8, 64, 16, BF16, 0.98),
        # caches a little over their budget, as every few dozen steps
        _evict("evict_some", 64, 1900, 2176, 2048, 4, 64, 8, 128, 16, FP8_PER_TOKEN_HEAD),
        # long prompts cut to an eighth before the decode begins
        _evict("evict_prompts", 4, 20000, 36000, 4096, 16, 200, 8, 128, 16, FP8_PER_HEAD),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "shared", "shared", "weights", "weights", "evict", "evict"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8] if D < 256 else [1, 2])
    mode = rng.choice([BF16, FP8_PER_TENSOR, FP8_PER_HEAD, FP8_PER_TOKEN_HEAD, INT4_PER_TOKEN_HEAD])
    bs = rng.choice([16, 32, 64, 128])
    if op == "prompt":
        hi = _log(rng, 1, 12000)
        B = _log(rng, 1, max(1, min(64, 40000 // hi)))
        c = _prompt("", B, max(1, hi // rng.randint(1, 20)), hi, Hkv * G, Hkv, D,
                    rng.choice([0, 0, rng.randint(1, 2000)]))
    elif op == "shared":
        P = _log(rng, 1, 32768)
        n = _log(rng, 1, 64)
        groups = _log(rng, 1, max(1, min(8, 65536 // P, 128 // n)))
        c = _shared("", groups, max(1, n // rng.randint(1, 4)), n, max(1, P // rng.randint(1, 6)), P,
                    _log(rng, 1, 1000), Hkv * G, Hkv, D, bs, mode)
    elif op == "weights":
        hi = _log(rng, 1, 40000)
        B = _log(rng, 1, max(1, min(64, 160000 // hi)))
        c = _weights("", B, max(1, hi // rng.randint(1, 8)), hi, Hkv * G, Hkv, D, bs, mode,
                     rng.choice([1.0, 1.0, 0.9, 0.995]))
    else:
        hi = _log(rng, 20, 36000)
        B = _log(rng, 1, max(1, min(64, 160000 // hi)))
        keep = rng.randint(max(1, hi // 8), hi)
        last = _log(rng, 1, max(1, keep // 2)) - 1
        first = min(rng.choice([0, 1, 4, 64]), keep - last)
        c = _evict("", B, max(1, hi // rng.randint(1, 3)), hi, keep, first, last, Hkv, D, bs, mode)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _row_bytes(mode, D):
    return 2 * D if mode == BF16 else D // 2 if mode == INT4_PER_TOKEN_HEAD else D


def _dynamic(mode):
    return mode in (FP8_PER_TOKEN_HEAD, INT4_PER_TOKEN_HEAD)


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def _lens(lo, hi, n, seed):
    """Lengths in [lo, hi], one of them hi. They go by the case alone, so that every seed's
    outputs have one shape."""
    x = torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(seed))
    x[n // 2] = hi
    return x.tolist()


def _running(x):
    out = [0]
    for v in x:
        out.append(out[-1] + v)
    return out


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c)
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "prompt":
        s["lens"] = _lens(c["lo"], c["hi"], c["B"], 11)
        s["start"] = _i32(_running(s["lens"]))
        s["T"] = sum(s["lens"])
        # a fused projection's output: q, k and v rows side by side
        s["qkv"] = torch.randn(s["T"], Hq + 2 * Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
        s["out"] = torch.empty(s["T"], Hq, D, dtype=torch.bfloat16, device=DEV)
        return s
    if c["op"] == "shared":
        n = _lens(c["n_lo"], c["n_hi"], c["groups"], 12)
        P = torch.randint(c["P_lo"], c["P_hi"] + 1, (c["groups"],), generator=g, device=DEV).tolist()
        P[0] = c["P_hi"]
        s["B"] = sum(n)
        s["group_start"], s["shared_lens"] = _i32(_running(n)), _i32(P)
        mine = torch.randint(1, c["own_hi"] + 1, (s["B"],), generator=g, device=DEV)
        mine[s["B"] // 2] = c["own_hi"]
        s["group_of"] = torch.arange(c["groups"], device=DEV).repeat_interleave(torch.tensor(n, device=DEV))
        s["lens"] = (s["shared_lens"][s["group_of"]] + mine).to(torch.int32)
        s["most"] = c["P_hi"] + c["own_hi"]
    else:
        s["lens"] = _i32(_lens(c["lo"], c["hi"], c["B"], 13))
        s["most"] = c["hi"]
    _paged(s, g)
    if c["op"] == "shared":
        _share(s)
    if c["op"] != "evict":
        s["q"] = torch.randn(s["B"], Hq, D, generator=g, device=DEV).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
    if c["op"] != "shared":
        # what earlier steps left: most cells little, a few much
        past = torch.exp(2.0 * torch.randn(s["B"], Hkv, c["hi"] + 7, generator=g, device=DEV) - 4.0)
        live = torch.arange(c["hi"] + 7, device=DEV) < s["lens"][:, None, None]
        s["weights"] = torch.where(live, past, 0.0)
    if c["op"] == "evict":
        s["rows"] = torch.randperm(s["B"], generator=g, device=DEV).to(torch.int32)
        s["keep_lens"] = torch.full((s["B"],), c["keep"], dtype=torch.int32, device=DEV)
        s["ref"] = torch.zeros(s["blocks"], dtype=torch.int32, device=DEV)
        s["ref"][s["table"][s["table"] >= 0].long()] = 1
        s["new_lens"] = torch.empty_like(s["keep_lens"])
    return s


def _paged(s, g):
    """Tables over a shuffled pool, and a layer's pages."""
    bs, Hkv, D, mode = s["bs"], s["Hkv"], s["D"], s["mode"]
    used = (s["lens"] + bs - 1) // bs
    max_blocks = -(-s["most"] // bs)
    blocks = int(used.sum()) + 3
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    j = torch.arange(max_blocks, device=DEV)
    idx = ((used.cumsum(0) - used)[:, None] + j[None]).clamp_max(blocks - 1)
    s["table"] = torch.where(j[None] < used[:, None], perm[idx], -1).to(torch.int32).contiguous()
    s["blocks"] = blocks
    s["static"] = s["scales"] = None
    shape = (2, blocks, Hkv, bs)
    if mode == BF16:
        x = torch.randn(*shape, D, generator=g, device=DEV)
        s["cache"] = x.to(torch.bfloat16).view(torch.uint8)
    elif mode == INT4_PER_TOKEN_HEAD:
        # two values in [-7, 7] a byte
        q = torch.randint(-7, 8, (*shape, D), generator=g, device=DEV, dtype=torch.int32) & 15
        s["cache"] = (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8)
    else:
        x = torch.randn(*shape, D, generator=g, device=DEV) * 100.0
        s["cache"] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    unit = 1.0 / 4.0 if mode == INT4_PER_TOKEN_HEAD else 1.0 / 100.0
    if _dynamic(mode):
        s["scales"] = (0.5 + torch.rand(*shape, generator=g, device=DEV)) * unit
    elif mode != BF16:
        s["static"] = (0.5 + torch.rand(2, 1 if mode == FP8_PER_TENSOR else Hkv, generator=g, device=DEV)) * unit


def _share(s):
    """Rows of a group read whole blocks of the prefix from the group's first row; a block that the
    prefix fills in part is each row's own copy, as a forked row gets it when it grows."""
    bs = s["bs"]
    first = s["group_start"][:-1].long()[s["group_of"]]
    P = s["shared_lens"][s["group_of"]]
    j = torch.arange(s["table"].shape[1], device=DEV)
    lead = s["table"][first]
    at = (P // bs).long().clamp_max(s["table"].shape[1] - 1)
    tail = P % bs
    part = (torch.arange(bs, device=DEV)[None] < tail[:, None])
    row = torch.arange(s["B"], device=DEV)
    src, dst = lead[row, at].clamp_min(0).long(), s["table"][row, at].clamp_min(0).long()
    b, o = part.nonzero(as_tuple=True)
    s["cache"][:, dst[b], :, o] = s["cache"][:, src[b], :, o]
    if s["scales"] is not None:
        s["scales"][:, dst[b], :, o] = s["scales"][:, src[b], :, o]
    s["table"] = torch.where(j[None] < (P // bs)[:, None], lead, s["table"]).contiguous()


# ------------------------------------------------------------- plain forms
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


def _cells(s, i, row, pos):
    """fp32 vectors [rows, Hkv, positions, D] of K (i 0) or V (1) at positions `pos` [rows, n] of
    table rows `row`."""
    bs = s["bs"]
    blk = s["table"][row[:, None], (pos // bs).clamp_max(s["table"].shape[1] - 1)].clamp_min(0).long()
    off = pos % bs
    x = _shown(s["cache"][i][blk, :, off], s["mode"]).float()          # [rows, n, Hkv, D]
    if s["scales"] is not None:
        x = x * s["scales"][i][blk, :, off][..., None]
    if s["static"] is not None:
        x = x * s["static"][i].view(1, 1, -1, 1)
    return x.transpose(1, 2)


def _softmax(score):
    """Weights of the last axis; rows with nothing to see get none."""
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    return w / w.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_prompt(s):
    Hq, Hkv, D, B, n, W = s["Hq"], s["Hkv"], s["D"], s["B"], s["hi"], s["window"]
    G = Hq // Hkv
    start = s["start"][:-1].long()
    length = (s["start"][1:] - s["start"][:-1]).long()
    t = torch.arange(n, device=DEV)
    row = (start[:, None] + t[None]).clamp_max(s["T"] - 1)
    x = s["qkv"][row].float()                                          # [B, n, heads, D]
    q = x[:, :, :Hq].reshape(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4)   # [B, Hkv, G, n, D]
    k = x[:, :, Hq:Hq + Hkv].permute(0, 2, 3, 1)                       # [B, Hkv, D, n]
    v = x[:, :, Hq + Hkv:].permute(0, 2, 1, 3)                         # [B, Hkv, n, D]
    o = torch.empty(B, n, Hq, D, device=DEV)
    # as many queries at a time as leave the scores within 4 GB
    step = max(1, min(n, (1 << 30) // (B * Hq * n)))
    for i0 in range(0, n, step):
        i1 = min(n, i0 + step)
        j0 = max(0, i0 + 1 - W) if W else 0
        score = torch.matmul(q[:, :, :, i0:i1].reshape(B, Hkv, -1, D), k[..., j0:i1]) / math.sqrt(D)
        score = score.view(B, Hkv, G, i1 - i0, i1 - j0)
        hidden = t[None, j0:i1] > t[i0:i1, None]
        if W:
            hidden |= t[None, j0:i1] <= t[i0:i1, None] - W
        w = _softmax(score.masked_fill(hidden, float("-inf")))
        part = torch.matmul(w.view(B, Hkv, -1, i1 - j0), v[:, :, j0:i1])
        o[:, i0:i1] = part.view(B, Hkv, G, i1 - i0, D).permute(0, 3, 1, 2, 4).reshape(B, i1 - i0, Hq, D)
    live = t[None] < length[:, None]
    out = torch.empty(s["T"], Hq, D, dtype=torch.bfloat16, device=DEV)
    out[row[live]] = o[live].to(torch.bfloat16)
    return out


def _plain_shared(s):
    """Scores to the group's prefix, once for all its rows, and to each row's own part."""
    Hq, Hkv, D, B, NG = s["Hq"], s["Hkv"], s["D"], s["B"], s["groups"]
    G = Hq // Hkv
    first, P = s["group_start"][:-1].long(), s["shared_lens"].long()
    grp = s["group_of"]
    place = torch.arange(B, device=DEV) - first[grp]
    n = s["n_hi"]
    pp = torch.arange(s["P_hi"], device=DEV)[None].expand(NG, -1)
    kp, vp = _cells(s, 0, first, pp), _cells(s, 1, first, pp)         # [NG, Hkv, P, D]
    op = P[grp][:, None] + torch.arange(s["own_hi"], device=DEV)[None]
    rows = torch.arange(B, device=DEV)
    ko, vo = _cells(s, 0, rows, op), _cells(s, 1, rows, op)           # [B, Hkv, own, D]
    q = s["q"].float().view(B, Hkv, G, D) / math.sqrt(D)
    member = (first[:, None] + torch.arange(n, device=DEV)[None]).clamp_max(B - 1)
    qg = q[member].permute(0, 2, 1, 3, 4).reshape(NG, Hkv, n * G, D)
    sp = torch.matmul(qg, kp.transpose(-1, -2)).masked_fill((pp >= P[:, None])[:, None, None], float("-inf"))
    sp = sp.view(NG, Hkv, n, G, -1)[grp, :, place]                    # [B, Hkv, G, P]
    so = torch.matmul(q, ko.transpose(-1, -2))
    so = so.masked_fill((op >= s["lens"][:, None])[:, None, None], float("-inf"))
    w = _softmax(torch.cat([sp, so], -1))
    wp = torch.zeros(NG, n, Hkv, G, s["P_hi"], device=DEV)
    wp[grp, place] = w[..., :s["P_hi"]]
    o = torch.matmul(wp.transpose(1, 2).reshape(NG, Hkv, n * G, -1), vp).view(NG, Hkv, n, G, D)[grp, :, place]
    o = o + torch.matmul(w[..., s["P_hi"]:], vo)
    return o.reshape(B, Hq, D).to(torch.bfloat16)


def _plain_weights(s):
    Hq, Hkv, D, B = s["Hq"], s["Hkv"], s["D"], s["B"]
    rows = torch.arange(B, device=DEV)
    pos = torch.arange(s["hi"], device=DEV)[None].expand(B, -1)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D) / math.sqrt(D)
    score = torch.matmul(q, _cells(s, 0, rows, pos).transpose(-1, -2))
    live = (pos < s["lens"][:, None])[:, None]
    w = _softmax(score.masked_fill(~live[:, :, None], float("-inf")))
    out = torch.matmul(w, _cells(s, 1, rows, pos)).view(B, Hq, D).to(torch.bfloat16)
    weights = s["weights"].clone()
    past = weights[..., :s["hi"]]
    weights[..., :s["hi"]] = torch.where(live, s["decay"] * past + w.sum(2), past)
    return dict(out=out, weights=weights)


def _plain_evict(s):
    first, last, bs = s["first"], s["last"], s["bs"]
    rows = s["rows"].long()
    weights = s["weights"].clone()
    L = s["lens"][rows].long()
    keep = torch.minimum(L, s["keep_lens"].long())
    cut = keep < L
    j = torch.arange(weights.shape[-1], device=DEV)
    w = weights[rows]                                                  # [n, Hkv, stride]
    middle = ((j >= first) & (j < (L - last)[:, None]) & cut[:, None])[:, None].expand_as(w)
    order = torch.where(middle, w, float("-inf")).argsort(dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order))
    stays = middle & (rank < (keep - first - last)[:, None, None])
    edge = (keep - last)[:, None, None]
    # cells that go into the places of evicted ones, in order: as many as there are places
    n, h, src = (stays & (j >= edge)).nonzero(as_tuple=True)
    dst = (middle & ~stays & (j < edge)).nonzero(as_tuple=True)[2]
    # and the last ones, which keep their order at the new end
    rn, rh, ri = torch.meshgrid(cut.nonzero().flatten(), torch.arange(w.shape[1], device=DEV),
                                torch.arange(last, device=DEV), indexing="ij")
    n, h = torch.cat([n, rn.flatten()]), torch.cat([h, rh.flatten()])
    src = torch.cat([src, (ri + (L - last)[rn]).flatten()])
    dst = torch.cat([dst, (ri + (keep - last)[rn]).flatten()])
    r = rows[n]
    weights[r, h, dst] = w[n, h, src]
    gone = (j >= keep[:, None]) & (j < L[:, None])
    weights[rows] = torch.where(gone[:, None], 0.0, weights[rows])
    sb, db = s["table"][r, src // bs].long(), s["table"][r, dst // bs].long()
    s["cache"][:, db, h, dst % bs] = s["cache"][:, sb, h, src % bs]
    if s["scales"] is not None:
        s["scales"][:, db, h, dst % bs] = s["scales"][:, sb, h, src % bs]
    return _evict_out(s, weights, keep.to(torch.int32))


def _evict_out(s, weights, new_lens):
    return dict(cache=_shown(s["cache"], s["mode"]), scales=s["scales"], weights=weights, new_lens=new_lens)


# -------------------------------------------------------- the library's own
@functools.lru_cache(maxsize=None)
def _context(Hq, Hkv, D, bs, blocks, mode, window):
    from int4_quantized_paged_gb300 import kvq
    return kvq.kvq_create(1, Hq, Hkv, D, bs, blocks, [mode], [window])


def _layer(s):
    """The layer's buffers as the calls take them."""
    c, x, t = s["cache"], s["scales"], s["static"]
    return (c[0], c[1]), dict(k_cache_scale=None if x is None else x[0], v_cache_scale=None if x is None else x[1],
                              k_scale=None if t is None else t[0], v_scale=None if t is None else t[1])


def _own(s):
    from int4_quantized_paged_gb300 import kvq
    Hq, Hkv, D, op = s["Hq"], s["Hkv"], s["D"], s["op"]
    ctx = _context(Hq, Hkv, D, s["bs"], s.get("blocks", 0), s["mode"], s.get("window", 0))
    if op == "prompt":
        qkv, stride = s["qkv"], (Hq + 2 * Hkv) * D
        kvq.kvq_prompt_attention(ctx, 0, qkv, qkv[:, Hq:], qkv[:, Hq + Hkv:], s["start"], s["out"],
                                 max_seq_len=s["hi"], q_token_stride=stride, kv_token_stride=stride)
        return s["out"]
    (kc, vc), scales = _layer(s)
    if op == "shared":
        sizes = dict(max_group=s["n_hi"], max_shared=s["P_hi"], max_own=s["own_hi"])
        splits, need = kvq.kvq_shared_prefix_plan(ctx, 0, s["B"], s["groups"], **sizes)
        work = torch.empty(need, dtype=torch.uint8, device=DEV)
        kvq.kvq_shared_prefix_attention(ctx, 0, s["q"], kc, vc, s["table"], s["lens"], s["group_start"],
                                        s["shared_lens"], s["out"], num_splits=splits, workspace=work,
                                        **sizes, **scales)
        return s["out"]
    weights = s["weights"].clone()
    if op == "weights":
        workers, need = kvq.kvq_decode_weights_plan(ctx, 0, s["B"], s["most"])
        work = torch.empty(need, dtype=torch.uint8, device=DEV)
        kvq.kvq_decode_attention_weights(ctx, 0, s["q"], kc, vc, s["table"], s["lens"], weights, s["out"],
                                         max_context=s["most"], decay=s["decay"], num_workers=workers,
                                         workspace=work, **scales)
        return dict(out=s["out"], weights=weights)
    x = s["scales"]
    kvq.kvq_evict_cells(ctx, 0, s["rows"], s["keep_lens"], s["table"], s["lens"], weights, s["new_lens"],
                        kc, vc, None if x is None else x[0], None if x is None else x[1],
                        first_kept=s["first"], last_kept=s["last"], max_context=s["most"], ref_count=s["ref"])
    return _evict_out(s, weights, s["new_lens"])


def run(s):
    if own:
        return _own(s)
    return dict(prompt=_plain_prompt, shared=_plain_shared, weights=_plain_weights, evict=_plain_evict)[s["op"]](s)


# -------------------------------------------------------- what it cannot do without
def work(case):
    c = case
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    cell = 2 * (_row_bytes(c["mode"], D) + (4 if _dynamic(c["mode"]) else 0))   # K and V of a position and head
    if c["op"] == "prompt":
        lens = _lens(c["lo"], c["hi"], c["B"], 11)
        W = c["window"] or c["hi"]
        pairs = sum(n * (n + 1) // 2 - max(0, n - W) * (max(0, n - W) + 1) // 2 for n in lens)
        return dict(bytes=sum(lens) * 2 * D * (2 * Hq + 2 * Hkv), flops=4 * D * Hq * pairs)
    if c["op"] == "shared":
        n = _lens(c["n_lo"], c["n_hi"], c["groups"], 12)
        P, mine = 0.5 * (c["P_lo"] + c["P_hi"]), 0.5 * (1 + c["own_hi"])
        B = sum(n)
        return dict(bytes=(c["groups"] * P + B * mine) * Hkv * cell + 4 * B * Hq * D,
                    flops=4 * D * Hq * B * (P + mine))
    lens = _lens(c["lo"], c["hi"], c["B"], 13)
    if c["op"] == "weights":
        return dict(bytes=sum(lens) * Hkv * (cell + 8) + 4 * c["B"] * Hq * D, flops=4 * D * Hq * sum(lens))
    # Of a row over its budget every cell's weight is read, and set to 0 behind the new end. The cells
    # that move are read and written: the last ones, and those that stay of the ones behind the new end.
    total, k = 16 * c["B"], c["keep"]
    for L in lens:
        if L > k:
            moved = c["last"] + (k - c["first"] - c["last"]) * (L - k) / (L - c["first"] - c["last"])
            total += Hkv * (4 * L + 4 * (L - k) + moved * (2 * cell + 4))
    return dict(bytes=total, flops=0)


# ------------------------------------------------------------------ 64 bits
def _vectors64(s, i, b, h, p0, p1):
    """K (i 0) or V (1) of positions [p0, p1) of row b and KV head h, page by page."""
    bs, mode = s["bs"], s["mode"]
    pages = s["table"][b, p0 // bs:-(-p1 // bs)].long()
    cut = slice(p0 % bs, p0 % bs + p1 - p0)
    x = s["cache"][i][pages, h].flatten(0, 1)[cut]
    if mode == INT4_PER_TOKEN_HEAD:
        x = torch.stack([x % 16, x // 16], -1).flatten(-2).double()
        x = torch.where(x >= 8, x - 16, x)
    else:
        x = x.view(torch.bfloat16 if mode == BF16 else torch.float8_e4m3fn).double()
    if s["scales"] is not None:
        x = x * s["scales"][i][pages, h].flatten(0, 1)[cut, None].double()
    if s["static"] is not None:
        x = x * s["static"][i].double().expand(s["Hkv"])[h]
    return x


def _exact_prompt(s):
    """One sequence and KV head at a time, a block of queries against the keys up to its end."""
    Hq, Hkv, D, W = s["Hq"], s["Hkv"], s["D"], s["window"]
    G = Hq // Hkv
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    at = s["start"].tolist()
    for b in range(s["B"]):
        x = s["qkv"][at[b]:at[b + 1]].double()
        n = at[b + 1] - at[b]
        for h in range(Hkv):
            q = x[:, h * G:(h + 1) * G]
            k, v = x[:, Hq + h], x[:, Hq + Hkv + h]
            for i in range(0, n, 2048):
                e = min(n, i + 2048)
                f = max(0, i - W + 1) if W else 0
                score = torch.einsum("qgd,kd->gqk", q[i:e], k[f:e]) / math.sqrt(D)
                away = torch.arange(i, e, device=DEV)[:, None] - torch.arange(f, e, device=DEV)[None]
                seen = (away >= 0) & (away < W) if W else away >= 0
                p = torch.softmax(torch.where(seen[None], score, -math.inf), -1)
                out[at[b] + i:at[b] + e, h * G:(h + 1) * G] = torch.einsum("gqk,kd->qgd", p, v[f:e])
    return out


def _exact_rows(s):
    """Every row against all of its own cells (a shared prefix read like any other)."""
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    G = Hq // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if "weights" in s else None
    for b, L in enumerate(s["lens"].tolist()):
        for h in range(Hkv):
            q = s["q"][b, h * G:(h + 1) * G].double()
            p = torch.softmax(q @ _vectors64(s, 0, b, h, 0, L).T / math.sqrt(D), -1)
            out[b, h * G:(h + 1) * G] = p @ _vectors64(s, 1, b, h, 0, L)
            if weights is not None:
                weights[b, h, :L] = weights[b, h, :L] * s["decay"] + p.sum(0)
    return out if weights is None else dict(out=out, weights=weights)


def _exact_evict(s):
    """One row and KV head at a time, in lists: who stays, then the places."""
    bs, first, last = s["bs"], s["first"], s["last"]
    weights = s["weights"].double()
    cache = _shown(s["cache"], s["mode"]).double()
    scales = None if s["scales"] is None else s["scales"].double()
    new = []
    for r, most in zip(s["rows"].tolist(), s["keep_lens"].tolist()):
        L = int(s["lens"][r])
        new.append(min(L, most))
        if L <= most:
            continue
        for h in range(s["Hkv"]):
            w = weights[r, h, :L].tolist()
            heavy = sorted(range(first, L - last), key=lambda p: (-w[p], p))[:most - first - last]
            stay = set(heavy)
            free = [p for p in range(first, most - last) if p not in stay]
            src = sorted(p for p in heavy if p >= most - last) + list(range(L - last, L))
            dst = free + list(range(most - last, most))
            a, b = (torch.tensor(x, dtype=torch.long, device=DEV) for x in (src, dst))
            weights[r, h, b] = weights[r, h, a]
            weights[r, h, most:L] = 0.0
            pages = s["table"][r].long()
            for x in [cache] if scales is None else [cache, scales]:
                x[:, pages[b // bs], h, b % bs] = x[:, pages[a // bs], h, a % bs]
    return dict(cache=cache, scales=scales, weights=weights, new_lens=torch.tensor(new, dtype=torch.int32))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s)
    return _exact_prompt(s) if case["op"] == "prompt" else _exact_rows(s)
