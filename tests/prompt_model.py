"""Attention over packed prompts in 64 bits, and the bound that a bf16 output has to meet."""
import math

import torch

U32 = 2.0 ** -24
LOG2E = 1.4426950408889634


def attend(q, k, v, spans, window=0, scale=None):
    """(reference, tolerance), float64 [T, Hq, D]; spans: the sequences' (start, end).

    The tolerance adds up, u = 2^-24, w the softmax weights, a_i = sum_d |q_d k_id| scale log2 e:
      * scores: D/16 accumulation steps and about three roundings, each u a_i, as a probabilistic
        bound of four standard deviations: 4 sqrt(D/16 + 3) u ln 2 sum w_i a_i |v_i - o|, with
        sum w |v - o| <= sum w |v| + |o|;
      * the weight in bf16: half a step 2^-8 of w_i: 2^-8 sum w_i |v_i|;
      * exponent and the fp32 sums: (8 + 4 sqrt(n/16 + 2)) u sum w_i |v_i|;
      * the output's rounding to bf16, half a step 2^-8 of it."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    ref = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(ref)
    for s, e in spans:
        n = e - s
        if n <= 0:
            continue
        away = torch.arange(n, device=q.device)[:, None] - torch.arange(n, device=q.device)[None]
        seen = (away >= 0) & ((away < window) if window else True)
        for h in range(Hkv):
            kk, vv = k[s:e, h].double(), v[s:e, h].double()
            for hq in range(h * G, (h + 1) * G):
                x = q[s:e, hq].double()
                score = (x @ kk.T * scale).masked_fill(~seen, -math.inf)
                w = torch.softmax(score, -1)
                o = w @ vv
                ref[s:e, hq] = o
                a = x.abs() @ kk.abs().T * (scale * LOG2E)
                mag, aw = w @ vv.abs(), w * a
                spread = aw @ vv.abs() + aw.sum(-1, keepdim=True) * o.abs()
                t = 4 * math.sqrt(D / 16 + 3) * U32 * math.log(2) * spread
                t = t + (2.0 ** -8 + (8 + 4 * math.sqrt(n / 16 + 2)) * U32) * mag
                tol[s:e, hq] = t + 2.0 ** -8 * (o.abs() + t)
    return ref, tol
