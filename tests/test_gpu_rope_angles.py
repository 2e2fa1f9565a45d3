"""Angles near quarters of a turn, where a sine or a cosine is small and its error shows."""
import math

import numpy as np
import pytest
import torch

from tests import rope_model as rm
from tests.gpu_harness import K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("D", [64, 256])
def test_small_sines_and_cosines(D, layout):
    """Pair i turns by a quarter, a half, three quarters or a whole turn and a little more or less.

    The result may be off by half a step of bf16, 2^-8 of it; by the angle's fp32 value (2^-24 of
    what is left beyond the quarter), sine and cosine (2 ulp) and two products: under 2^-20 of it;
    and by the frequency's fraction of a turn, p f 2^-52 radians."""
    kvq = K()
    n = D // 2
    little = [(-1) ** i * 10.0 ** -(2 + 4.0 * i / (n - 1)) for i in range(n)]       # 1e-2 to 1e-6
    fs = [(i % 4 + 1) * math.pi / 2 + d for i, d in enumerate(little)]
    rope = kvq.kvq_rope_create(D, layout=layout, frequencies=fs)
    pos = [1, -1, 2, 3, 77, -1001]
    x = torch.zeros(len(pos), 2, D, dtype=torch.bfloat16, device="cuda")
    first = torch.arange(n) if layout == 0 else 2 * torch.arange(n)
    x[:, 0, first] = 1.0
    x[:, 1, first + (n if layout == 0 else 1)] = 1.0
    far = np.abs(np.array(pos, dtype=np.float64))[:, None] * np.array(fs)[None] * 2.0 ** -52
    unit = np.zeros((len(pos), 1, D))
    unit[:, 0, first] = far
    unit[:, 0, first + (n if layout == 0 else 1)] = far
    for inverse in (False, True):
        out = torch.empty_like(x)
        kvq.kvq_rope_apply(rope, x, torch.tensor(pos, device="cuda"), out, inverse=inverse)
        want = rm.rotate(x.float().cpu().numpy().astype(np.float64), pos, fs, layout, 1.0, inverse)
        got = out.float().cpu().numpy().astype(np.float64)
        err = np.abs(got - want)
        assert np.all(err <= np.abs(want) * (2.0 ** -8 + 2.0 ** -20) + unit), float((err / np.abs(want)).max())
    assert kvq.kvq_get_device_error() == 0


def test_whole_quarters_are_exact():
    """A quarter of a turn as the nearest double: its own error, 1e-16 radians, is all that is left."""
    kvq = K()
    rope = kvq.kvq_rope_create(64, frequencies=[math.pi / 2] * 32)
    x = torch.zeros(5, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[:, 0, :32] = 1.0
    out = torch.empty_like(x)
    kvq.kvq_rope_apply(rope, x, torch.arange(5, device="cuda"), out)
    for p, (c, s) in enumerate([(1, 0), (0, 1), (-1, 0), (0, -1), (1, 0)]):
        assert torch.all((out[p, 0, :32].float() - c).abs() <= 1e-15 * p)
        assert torch.all((out[p, 0, 32:].float() - s).abs() <= 1e-15 * p)
