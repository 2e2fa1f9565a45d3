"""V scales of one sequence that lie far apart: the weight times the V scale leaves f16's normal
numbers, and is off by 2^-31 of the largest V scale there, as the header says."""
import pytest
import torch

from tests import cross_model as cm
from tests.test_gpu_cross import Case

pytestmark = pytest.mark.gpu


def _bound(c):
    """cross_model's tolerance, with its term for small weights taken from the scales: n keys, each
    2^-31 of the largest V scale times a code."""
    ref, tol = cm.attend(c.q, c.layer, c.table, c.lens, c.starts, c.bs)
    Hkv = c.layer["values"][1].shape[1]
    G = c.q.shape[1] // Hkv
    for b, S in enumerate(c.lens):
        pages = c.table[b, :-(-S // c.bs)].long()
        rows = slice(c.starts[b], c.starts[b + 1])
        for h in range(Hkv):
            v = c.layer["values"][1][pages, h].flatten(0, 1)[:S]
            if c.mode == 0:
                # a V row's scale is 2^-14 of the power of two below its largest value
                scale = torch.exp2(torch.floor(torch.log2(v.abs().amax(-1).clamp_min(1e-300))) - 14)
            else:
                scale = c.layer["scales"][1][pages, h].flatten()[:S].double()
            code = (v.abs().amax(-1) / scale).max()
            tol[rows, h * G:(h + 1) * G] += S * 2.0 ** -31 * scale.max() * code * (1 + 2.0 ** -8)
    return ref, tol


@pytest.mark.parametrize("mode", [0, 3, 4])
@pytest.mark.parametrize("D, lens, queries", [(128, [700, 90, 1], [3, 40, 2]), (64, [1200, 333], [1, 130]),
                                              (256, [300], [5])])
@pytest.mark.parametrize("splits", [1, 3])
def test_scales_forty_powers_of_two_apart(mode, D, lens, queries, splits):
    c = Case(mode, D, 4, 2, lens, queries, seed=D + mode)
    y = c.layer
    g = torch.Generator(device="cuda").manual_seed(D)
    wide = torch.exp2(-torch.randint(0, 41, y["values"][1].shape[:3], generator=g, device="cuda").float())
    if mode == 0:
        v = y["codes"][1].view(torch.bfloat16) * wide[..., None].to(torch.bfloat16)
        y["codes"][1] = v.view(torch.uint8).contiguous()
    else:
        y["scales"][1] *= wide
    y["values"][1] *= wide[..., None].double()
    c.run(splits)
    torch.cuda.synchronize()
    ref, tol = _bound(c)
    err = (c.out[:c.starts[-1]].double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("mode", [3, 4])
def test_a_zero_value_among_small_ones(mode):
    """A vector of zeros is stored with the scale 1, 2^19 times that of its neighbours."""
    c = Case(mode, 128, 8, 2, [500, 64], [4, 20], seed=mode)
    y = c.layer
    for b, L in enumerate(c.lens):
        for p in range(L):
            block, at = int(c.table[b, p // 16]), p % 16
            if p == 5:
                y["codes"][1][block, :, at] = 0
                y["scales"][1][block, :, at] = 1.0
                y["values"][1][block, :, at] = 0.0
            else:
                y["scales"][1][block, :, at] *= 2.0 ** -13
                y["values"][1][block, :, at] *= 2.0 ** -13
    c.run()
    torch.cuda.synchronize()
    ref, tol = _bound(c)
    codes = 7.0 if mode == 4 else 448.0
    tol = tol + max(c.lens) * 2.0 ** -31 * codes         # the largest scale is the zero vector's 1
    err = (c.out[:c.starts[-1]].double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())
