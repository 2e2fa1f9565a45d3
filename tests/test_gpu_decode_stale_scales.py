"""Cells of a page behind the context may hold anything, NaN and infinite scales
among it: the decode reads none of it."""
import pytest
import torch

from int4_quantized_paged_gb300 import workloads as wl
from oracle import oracle as orc
from tests.gpu_harness import LayerRun

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [orc.FP8_PER_TOKEN_HEAD, orc.INT4_PER_TOKEN_HEAD])
@pytest.mark.parametrize("D, G", [(64, 4), (128, 8), (256, 2)])
@pytest.mark.parametrize("window", [0, 40])
def test_stale_scales(mode, D, G, window):
    w = wl.Workload("stale", Hq=2 * G, Hkv=2, D=D, block_size=16, context_lens=(37, 100, 1, 250),
                    windows=(window,), seed=D + G)
    r = LayerRun(w, mode)
    r.write()
    want = r.decode(num_workers=3).clone()
    live = torch.zeros(r.pg.num_blocks, 16, dtype=torch.bool)
    for b, L in enumerate(w.context_lens):
        for p in range(max(0, L - window) if window else 0, L):
            live[int(r.pg.block_table[b, p // 16]), p % 16] = True
    for bad in (float("nan"), float("inf")):
        for s in (r.ks, r.vs):
            s.transpose(1, 2)[~live.cuda()] = bad
        assert torch.equal(r.decode(num_workers=3), want)
