"""Cross attention in 64 bits over paged caches made of plain tensors, and the
bound that a bf16 output has to meet."""
import math

import torch

U32 = 2.0 ** -24
LOG2E = 1.4426950408889634


def layer(mode, blocks, Hkv, bs, D, gen, device="cuda"):
    """Codes, scales and the values they stand for, one entry per block (float64
    [blocks, Hkv, bs, D]); static scales for modes 1 and 2."""
    out = dict(static=[None, None], scales=[None, None], codes=[], values=[])
    for i in range(2):
        x = torch.randn(blocks, Hkv, bs, D, generator=gen, device=device)
        if mode == 0:
            c = x.to(torch.bfloat16)
            out["codes"].append(c.view(torch.uint8).clone())
            out["values"].append(c.double())
            continue
        if mode == 4:
            q = (x * 3).round().clamp(-7, 7).to(torch.int32)
            out["codes"].append(((q[..., 0::2] & 15) | ((q[..., 1::2] & 15) << 4)).to(torch.uint8))
            v = q.double()
        else:
            c = (x * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
            out["codes"].append(c.view(torch.uint8).clone())
            v = c.double()
        unit = 1 / 3 if mode == 4 else 1 / 64
        if mode in (3, 4):
            s = torch.exp(torch.randn(blocks, Hkv, bs, generator=gen, device=device)) * unit
            out["scales"][i] = s
            out["values"].append(v * s[..., None].double())
        else:
            s = (torch.rand(1 if mode == 1 else Hkv, generator=gen, device=device) + 0.5) * unit
            out["static"][i] = s
            out["values"].append(v * s.double().view(1, -1, 1, 1))
    return out


def poison(out, mode, used):
    """Everything that no position uses holds NaN (`used`: [blocks, bs] truth values)."""
    un = ~used
    for i in range(2):
        c = out["codes"][i]
        if mode == 0:
            c.view(torch.int16).transpose(1, 2)[un] = 0x7FC0
        elif mode != 4:
            c.transpose(1, 2)[un] = 0x7F
        if out["scales"][i] is not None:
            out["scales"][i].transpose(1, 2)[un] = float("nan")


def attend(q, out, table, lens, starts, bs, scale=None):
    """(reference, tolerance), float64 [T, Hq, D].

    The tolerance adds up, u = 2^-24, w the softmax weights, a_i = sum_d |q_d K_id| scale log2 e:
      * scores: D/16 accumulation steps and about three roundings, each u a_i, as a probabilistic
        bound of four standard deviations: 4 sqrt(D/16 + 3) u ln 2 sum w_i a_i |V_i - o|;
      * joining splits: log2 of a sum carried in fp32, 4 u max|s| ln 2 sum w_i |V_i - o|;
      * the weight in f16: half a step 2^-11 of w_i, and 2^-31 of the largest weight where P'
        leaves f16's normal numbers: 2^-11 sum w_i |V_i| + n 2^-31 max |V|;
      * exponent, scale products and the fp32 sums: (8 + 4 sqrt(n/16 + 2)) u sum w_i |V_i|;
      * the output's rounding to bf16, half a step 2^-8 of it."""
    T, Hq, D = q.shape
    Hkv = out["values"][0].shape[1]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    ref = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(ref)
    for b in range(len(lens)):
        S, rows = lens[b], slice(starts[b], starts[b + 1])
        if S <= 0 or rows.start >= rows.stop:
            continue
        pages = table[b, :-(-S // bs)].long()
        for h in range(Hkv):
            k, v = [x[pages, h].flatten(0, 1)[:S] for x in out["values"]]
            qq = q[rows, h * G:(h + 1) * G].double()
            s = qq @ k.T * scale
            w = torch.softmax(s, -1)
            o = w @ v
            ref[rows, h * G:(h + 1) * G] = o
            a = qq.abs() @ k.abs().T * (scale * LOG2E)
            mag = w @ v.abs()
            # sum w |V - o| <= sum w |V| + |o|
            aw = w * a
            spread = aw @ v.abs() + aw.sum(-1, keepdim=True) * o.abs()
            t = 4 * math.sqrt(D / 16 + 3) * U32 * math.log(2) * spread
            t = t + 4 * U32 * s.abs().amax(-1, keepdim=True) * (mag + o.abs())
            t = t + 2.0 ** -11 * mag + S * 2.0 ** -31 * v.abs().max()
            t = t + (8 + 4 * math.sqrt(S / 16 + 2)) * U32 * mag
            t = t + 2.0 ** -8 * (o.abs() + t)
            tol[rows, h * G:(h + 1) * G] = t
    return ref, tol
