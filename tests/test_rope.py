"""Rotary handles and refusals, without a GPU."""
import math

import numpy as np
import pytest

from tests import rope_model as rm

kvq = pytest.importorskip("int4_quantized_paged_gb300.kvq",
                          reason="libkvq.so not built (run __graft_entry__.build())")
OK = 0x10000000                      # never dereferenced: validation fails first


@pytest.mark.parametrize("r", [16, 64, 128, 256])
@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
def test_frequencies(r, scaling):
    kw = dict(factor=8.0) if scaling else {}
    if scaling == 3:
        kw.update(original_context=8192.0, low_rotations=1.0, high_rotations=32.0)
    rope = kvq.kvq_rope_create(256, r, base=500000.0, scaling=scaling, magnitude=1.25, **kw)
    fs, m = kvq.kvq_rope_frequencies(rope)
    want = rm.frequencies(r, 500000.0, scaling, 8.0, 8192.0, 1.0, 32.0)
    # pow and exp(log) of a double, each a few ulp of an exponent of at most log(5e5 8^1.2) = 16
    assert np.allclose(fs, want, rtol=64 * 2.0 ** -53, atol=0)
    assert m == 1.25


def test_parts_keep_fast_pairs_and_divide_slow_ones():
    rope = kvq.kvq_rope_create(128, scaling=kvq.ROPE_PARTS, factor=4.0, original_context=4096.0,
                               low_rotations=1.0, high_rotations=4.0)
    fs, _ = kvq.kvq_rope_frequencies(rope)
    plain, _ = kvq.kvq_rope_frequencies(kvq.kvq_rope_create(128))
    assert fs[0] == plain[0] == 1.0
    assert fs[-1] == plain[-1] / 4.0
    ratio = [a / b for a, b in zip(fs, plain)]
    assert all(x >= y - 1e-15 for x, y in zip(ratio, ratio[1:]))


def test_given_frequencies_are_taken_as_they_are():
    given = [0.5 / (i + 1) for i in range(8)]
    rope = kvq.kvq_rope_create(64, 16, frequencies=given)
    assert kvq.kvq_rope_frequencies(rope)[0] == given
    with pytest.raises(ValueError):
        kvq.kvq_rope_create(64, 32, frequencies=given)


@pytest.mark.parametrize("match, kw", [
    ("UNSUPPORTED", dict(head_dim=96, rotary_dim=96)),
    ("UNSUPPORTED", dict(head_dim=128, rotary_dim=24)),
    ("INVALID_ARG", dict(head_dim=128, rotary_dim=0)),
    ("INVALID_ARG", dict(head_dim=64, rotary_dim=128)),
    ("INVALID_ARG", dict(head_dim=64, layout=2)),
    ("INVALID_ARG", dict(head_dim=64, scaling=4)),
    ("INVALID_ARG", dict(head_dim=64, base=0.0)),
    ("INVALID_ARG", dict(head_dim=64, base=math.inf)),
    ("INVALID_ARG", dict(head_dim=64, scaling=1, factor=0.0)),
    ("INVALID_ARG", dict(head_dim=64, scaling=1, factor=math.nan)),
    ("INVALID_ARG", dict(head_dim=64, scaling=3, factor=2.0)),
    ("INVALID_ARG", dict(head_dim=64, scaling=3, factor=2.0, original_context=4096.0,
                         low_rotations=4.0, high_rotations=4.0)),
    ("INVALID_ARG", dict(head_dim=64, magnitude=17.0)),
    ("INVALID_ARG", dict(head_dim=64, magnitude=-1.0)),
    ("INVALID_ARG", dict(head_dim=64, magnitude=math.nan)),
    ("INVALID_ARG", dict(head_dim=64, scaling=1, factor=2.0, frequencies=[1.0] * 32)),
    ("INVALID_ARG", dict(head_dim=64, frequencies=[math.inf] * 32)),
])
def test_create_refuses(match, kw):
    with pytest.raises(kvq.KVQError, match=match):
        kvq.kvq_rope_create(**kw)


def _apply(rope, **kw):
    a = dict(x=OK, xs=0, pos=OK, T=4, H=8, out=OK + 4096, os=0)
    a.update(kw)
    kvq.kvq_rope_apply(rope, a["x"], a["pos"], a["out"], x_token_stride=a["xs"],
                       out_token_stride=a["os"], num_tokens=a["T"], num_heads=a["H"], stream=0)


@pytest.mark.parametrize("match, kw", [
    ("INVALID_ARG", dict(x=None)), ("INVALID_ARG", dict(pos=None)), ("INVALID_ARG", dict(out=None)),
    ("INVALID_ARG", dict(T=-1)), ("INVALID_ARG", dict(H=0)), ("INVALID_ARG", dict(T=1 << 29)),
    ("INVALID_ARG", dict(xs=8 * 64 - 8)), ("INVALID_ARG", dict(os=8)),
    ("INVALID_ARG", dict(out=OK, os=8 * 64 + 8)),
    ("ALIGNMENT", dict(x=OK + 2)), ("ALIGNMENT", dict(out=OK + 8)), ("ALIGNMENT", dict(pos=OK + 4)),
    ("ALIGNMENT", dict(xs=8 * 64 + 4)), ("ALIGNMENT", dict(os=8 * 64 + 1)),
])
def test_apply_refuses(match, kw):
    with pytest.raises(kvq.KVQError, match=match):
        _apply(kvq.kvq_rope_create(64), **kw)


def test_no_tokens_is_nothing():
    _apply(kvq.kvq_rope_create(64), T=0, x=None, out=None, pos=None)


def _write(ctx, rope, layer=0, **kw):
    a = dict(q=OK, qo=OK + 4096, k=OK, v=OK, pos=OK, slots=OK, kc=OK, vc=OK, kcs=OK, vcs=OK, ks=OK,
             vs=OK, qs=0, qos=0, kvs=0, T=4)
    a.update(kw)
    kvq.kvq_rope_cache_write(ctx, rope, layer, a["q"], a["qo"], a["k"], a["v"], a["pos"], a["slots"],
                             a["kc"], a["vc"], a["kcs"], a["vcs"], a["ks"], a["vs"],
                             q_token_stride=a["qs"], q_out_token_stride=a["qos"],
                             kv_token_stride=a["kvs"], num_tokens=a["T"], stream=0)


@pytest.mark.parametrize("match, kw", [
    ("INVALID_ARG", dict(q=None)), ("INVALID_ARG", dict(qo=None)), ("INVALID_ARG", dict(k=None)),
    ("INVALID_ARG", dict(v=None)), ("INVALID_ARG", dict(pos=None)), ("INVALID_ARG", dict(slots=None)),
    ("INVALID_ARG", dict(kc=None)), ("INVALID_ARG", dict(vc=None)), ("INVALID_ARG", dict(kcs=None)),
    ("INVALID_ARG", dict(layer=1, vs=None)), ("INVALID_ARG", dict(layer=2)),
    ("INVALID_ARG", dict(T=-1)), ("INVALID_ARG", dict(T=1 << 28)), ("INVALID_ARG", dict(kvs=8)),
    ("INVALID_ARG", dict(qs=8)), ("INVALID_ARG", dict(qo=OK, qos=16 * 64 + 8)),
    ("ALIGNMENT", dict(q=OK + 8)), ("ALIGNMENT", dict(k=OK + 8)), ("ALIGNMENT", dict(vc=OK + 4)),
    ("ALIGNMENT", dict(kvs=8 * 64 + 4)), ("ALIGNMENT", dict(pos=OK + 4)),
    ("ALIGNMENT", dict(slots=OK + 4)), ("ALIGNMENT", dict(vcs=OK + 2)),
])
def test_write_refuses(match, kw):
    ctx = kvq.kvq_create(2, 16, 8, 64, 16, 64, [3, 2])
    with pytest.raises(kvq.KVQError, match=match):
        _write(ctx, kvq.kvq_rope_create(64), **kw)


def test_write_refuses_another_head_size():
    ctx = kvq.kvq_create(1, 16, 8, 64, 16, 64, [3])
    with pytest.raises(kvq.KVQError, match="INVALID_ARG"):
        _write(ctx, kvq.kvq_rope_create(128))
    _write(ctx, kvq.kvq_rope_create(64), T=0)
