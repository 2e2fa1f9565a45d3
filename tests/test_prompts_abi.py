"""Shared prefixes and accumulated weights without a GPU: the plans and the refusals."""
import pytest

kvq = pytest.importorskip("int4_quantized_paged_gb300.kvq",
                          reason="libkvq.so not built (run __graft_entry__.build())")
OK = 0x10000000                      # never dereferenced: validation fails first


def _ctx(modes=(3, 2), windows=None):
    return kvq.kvq_create(len(modes), 32, 8, 128, 16, 4096, list(modes), windows)


SIZES = dict(max_group=8, max_shared=2000, max_own=100)


def _plan(ctx=None, layer=0, batch=16, groups=2, splits=0, **kw):
    return kvq.kvq_shared_prefix_plan(ctx or _ctx(), layer, batch, groups, num_splits=splits, **{**SIZES, **kw})


def test_shared_plan():
    splits, need = _plan()
    assert splits == 0 and need % 16 == 0            # the device's choice stays that
    assert need < _plan(splits=1)[1]                 # too little to gain from: no room for partials
    assert _plan(max_shared=200000)[1] >= _plan(splits=1, max_shared=200000)[1]
    # two groups, a unit for each split: its entry, and a partial of 8 rows
    assert _plan(splits=7)[1] - _plan(splits=5)[1] == 2 * 2 * (16 + 8 * 32 * 129 * 4)
    assert _plan(splits=7)[0] == 7
    # nothing to share: no splits and no room for them
    for kw in (dict(groups=0), dict(max_group=1), dict(max_shared=15), dict(batch=1)):
        assert _plan(splits=3, **kw)[0] == 0
        assert _plan(splits=3, **kw)[1] < _plan(splits=1)[1]
    assert _plan(max_group=500)[1] == _plan(max_group=16)[1]         # no group has more rows than the batch


@pytest.mark.parametrize("match, kw", [
    ("INVALID_ARG", dict(layer=2)), ("INVALID_ARG", dict(batch=-1)), ("INVALID_ARG", dict(groups=-1)),
    ("INVALID_ARG", dict(max_group=-1)), ("INVALID_ARG", dict(max_shared=-1)), ("INVALID_ARG", dict(max_own=-1)),
    ("INVALID_ARG", dict(max_shared=(1 << 30) + 1)), ("INVALID_ARG", dict(max_own=(1 << 30) + 1)),
    ("INVALID_ARG", dict(max_shared=1 << 30, max_own=1 << 30)),
    ("INVALID_ARG", dict(splits=-1)), ("INVALID_ARG", dict(splits=1025)),
    ("INVALID_ARG", dict(groups=(1 << 31) - 1, batch=(1 << 31) - 1, max_group=(1 << 31) - 1)),
    ("INVALID_ARG", dict(groups=1 << 20, batch=1 << 20, max_group=1 << 20)),
    ("INVALID_ARG", dict(groups=1 << 26, batch=1 << 27, max_group=8, splits=1024)),
    ("UNSUPPORTED", dict(ctx=_ctx((3,), [128]))),
])
def test_shared_plan_refuses(match, kw):
    with pytest.raises(kvq.KVQError, match=match):
        _plan(**kw)


def _shared(ctx=None, **kw):
    a = dict(layer=0, q=OK, kc=OK, vc=OK, bt=OK, mb=256, lens=OK, B=16, gs=OK, sl=OK, NG=2, out=OK, splits=2, ws=OK,
             wsb=1 << 30, kcs=OK, vcs=OK, ks=OK, vs=OK, **SIZES)
    a.update(kw)
    kvq.kvq_shared_prefix_attention(
        ctx or _ctx(), a["layer"], a["q"], a["kc"], a["vc"], a["bt"], a["lens"], a["gs"], a["sl"], a["out"],
        max_group=a["max_group"], max_shared=a["max_shared"], max_own=a["max_own"], k_scale=a["ks"],
        v_scale=a["vs"], k_cache_scale=a["kcs"], v_cache_scale=a["vcs"], num_splits=a["splits"],
        workspace=a["ws"], workspace_bytes=a["wsb"], batch=a["B"], num_groups=a["NG"],
        max_blocks_per_seq=a["mb"], stream=0)


CACHE = [
    ("INVALID_ARG", dict(q=None)), ("INVALID_ARG", dict(kc=None)), ("INVALID_ARG", dict(vc=None)),
    ("INVALID_ARG", dict(bt=None)), ("INVALID_ARG", dict(lens=None)), ("INVALID_ARG", dict(out=None)),
    ("INVALID_ARG", dict(kcs=None)), ("INVALID_ARG", dict(layer=1, vs=None)), ("INVALID_ARG", dict(layer=2)),
    ("INVALID_ARG", dict(B=-1)), ("INVALID_ARG", dict(mb=-1)), ("WORKSPACE", dict(ws=None)),
    ("WORKSPACE", dict(wsb=100)), ("ALIGNMENT", dict(ws=OK + 8)), ("ALIGNMENT", dict(q=OK + 8)),
    ("ALIGNMENT", dict(out=OK + 2)), ("ALIGNMENT", dict(kc=OK + 4)), ("ALIGNMENT", dict(vc=OK + 8)),
    ("ALIGNMENT", dict(bt=OK + 2)), ("ALIGNMENT", dict(kcs=OK + 4)), ("ALIGNMENT", dict(vcs=OK + 8)),
    ("ALIGNMENT", dict(lens=OK + 3)),
]


@pytest.mark.parametrize("match, kw", CACHE + [
    ("INVALID_ARG", dict(gs=None)), ("INVALID_ARG", dict(sl=None)), ("INVALID_ARG", dict(NG=-1)),
    ("INVALID_ARG", dict(max_group=-1)), ("INVALID_ARG", dict(splits=-1)), ("INVALID_ARG", dict(splits=1025)),
    ("INVALID_ARG", dict(mb=1 << 27)), ("ALIGNMENT", dict(gs=OK + 2)), ("ALIGNMENT", dict(sl=OK + 1)),
])
def test_shared_refuses(match, kw):
    with pytest.raises(kvq.KVQError, match=match):
        _shared(**kw)


def test_shared_workspace_to_the_byte():
    need = _plan(splits=2)[1]
    with pytest.raises(kvq.KVQError, match="WORKSPACE"):
        _shared(wsb=need - 1)


def _weights(ctx=None, **kw):
    a = dict(layer=0, q=OK, kc=OK, vc=OK, bt=OK, mb=256, lens=OK, B=16, out=OK, w=OK, stride=4096, most=4096,
             decay=1.0, workers=4, ws=OK, wsb=1 << 30, kcs=OK, vcs=OK, ks=OK, vs=OK)
    a.update(kw)
    kvq.kvq_decode_attention_weights(
        ctx or _ctx(), a["layer"], a["q"], a["kc"], a["vc"], a["bt"], a["lens"], a["w"], a["out"],
        max_context=a["most"], decay=a["decay"], k_scale=a["ks"], v_scale=a["vs"], k_cache_scale=a["kcs"],
        v_cache_scale=a["vcs"], num_workers=a["workers"], workspace=a["ws"], workspace_bytes=a["wsb"],
        batch=a["B"], max_blocks_per_seq=a["mb"], weights_stride=a["stride"], stream=0)


@pytest.mark.parametrize("match, kw", CACHE + [
    ("INVALID_ARG", dict(w=None)), ("INVALID_ARG", dict(stride=4095)), ("INVALID_ARG", dict(most=-1)),
    ("INVALID_ARG", dict(most=4097, stride=5000)), ("INVALID_ARG", dict(decay=-0.1)),
    ("INVALID_ARG", dict(decay=1.5)), ("INVALID_ARG", dict(decay=float("nan"))),
    ("INVALID_ARG", dict(workers=-1)), ("INVALID_ARG", dict(B=65536)), ("ALIGNMENT", dict(w=OK + 2)),
])
def test_weights_refuse(match, kw):
    with pytest.raises(kvq.KVQError, match=match):
        _weights(**kw)


def test_weights_plan():
    n, need = kvq.kvq_decode_weights_plan(_ctx(), 0, 16, 4096, 4)
    decode = (16 * 8 + 4) * 4 * 130 * 4 + (16 * 8 + 1) * 8
    assert (n, need) == (4, -(-decode // 16) * 16 + 16 * 32 * 4 + 16 * 32 * 4096 * 4)
    with pytest.raises(kvq.KVQError, match="WORKSPACE"):
        _weights(wsb=need - 1)
    one = kvq.kvq_decode_weights_plan(_ctx(), 0, 16, 4096, 1)[1]      # the scores need it with one worker too
    assert one >= 16 * 32 * 4096 * 4
    for bad in (dict(layer=2), dict(batch=-1), dict(most=-1), dict(workers=-1),
                dict(batch=(1 << 31) - 1, most=(1 << 31) - 1)):
        a = dict(layer=0, batch=2, most=100, workers=0)
        a.update(bad)
        with pytest.raises(kvq.KVQError, match="INVALID_ARG"):
            kvq.kvq_decode_weights_plan(_ctx(), a["layer"], a["batch"], a["most"], a["workers"])


def test_windows_are_refused():
    ctx = _ctx((3,), [128])
    with pytest.raises(kvq.KVQError, match="UNSUPPORTED"):
        _weights(ctx)
    with pytest.raises(kvq.KVQError, match="UNSUPPORTED"):
        _shared(ctx)
    with pytest.raises(kvq.KVQError, match="UNSUPPORTED"):
        kvq.kvq_decode_weights_plan(ctx, 0, 2, 100)


def test_nothing_to_do():
    _shared(B=0)
    _weights(B=0)
