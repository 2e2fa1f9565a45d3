"""What the rotation does not touch keeps its bits, a NaN's payload and sign among them."""
import pytest
import torch

from tests.gpu_harness import K

pytestmark = pytest.mark.gpu

# quiet and signalling NaNs of both signs, infinities, subnormals, both zeros
ODD = [0x7FC1, 0x7F81, 0xFFA5, 0xFFFF, 0x7F80, 0xFF80, 0x0001, 0x8001, 0x0000, 0x8000, 0x3F80]


def _odd(*shape):
    n = torch.Size(shape).numel()
    v = torch.tensor([ODD[i % len(ODD)] for i in range(n)], dtype=torch.int32).to(torch.int16)
    return v.view(torch.bfloat16).view(shape).cuda()


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("D, r", [(64, 16), (128, 64), (256, 48)])
def test_the_rest_of_the_head(D, r, layout):
    kvq = K()
    x = _odd(37, 3, D)
    out = torch.zeros_like(x)
    kvq.kvq_rope_apply(kvq.kvq_rope_create(D, r, layout=layout), x, torch.arange(37, device="cuda"), out)
    assert torch.equal(out.view(torch.int16)[..., r:], x.view(torch.int16)[..., r:])


@pytest.mark.parametrize("D, r", [(64, 64), (128, 32)])
def test_values_and_keys_of_a_bf16_layer(D, r):
    kvq = K()
    T, Hkv = 40, 2
    k, v = _odd(T, Hkv, D), _odd(T, Hkv, D).flip(-1)
    pos = torch.arange(T, device="cuda")
    ctx = kvq.kvq_create(1, 4, Hkv, D, 16, 4, [kvq.BF16])
    caches = [kvq.alloc_layer_cache(ctx, 0)[:2] for _ in range(2)]
    kvq.kvq_rope_cache_write(ctx, kvq.kvq_rope_create(D, r), 0, None, None, k, v, pos, pos, *caches[0])
    kvq.kvq_cache_write(ctx, 0, k, v, pos, *caches[1])
    assert torch.equal(caches[0][1], caches[1][1])
    keys = [c[0].view(torch.int16)[..., r:] for c in caches]
    assert torch.equal(*keys)
