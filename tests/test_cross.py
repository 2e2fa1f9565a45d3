"""Cross attention without a GPU: the plan and the refusals."""
import pytest

kvq = pytest.importorskip("int4_quantized_paged_gb300.kvq",
                          reason="libkvq.so not built (run __graft_entry__.build())")
OK = 0x10000000                      # never dereferenced: validation fails first


def _ctx(modes=(3, 2), windows=None, D=128):
    return kvq.kvq_create(len(modes), 32, 8, D, 16, 4096, list(modes), windows)


def test_plan():
    ctx = _ctx()
    splits, need = kvq.kvq_cross_plan(ctx, 0, 1, 4, 32768)
    assert splits > 1
    assert need == splits * 4 * 32 * 129 * 4
    assert kvq.kvq_cross_plan(ctx, 0, 64, 1024, 4096) == (1, 0)       # the queries fill the SMs
    assert kvq.kvq_cross_plan(ctx, 0, 8, 4, 60)[0] == 1               # one key tile
    assert kvq.kvq_cross_plan(ctx, 0, 8, 4, 0)[0] == 1
    assert kvq.kvq_cross_plan(ctx, 0, 2, 5, 1000, 7) == (7, 7 * 10 * 32 * 129 * 4)
    assert kvq.kvq_cross_plan(ctx, 0, 8, 0, 1500) == kvq.kvq_decode_plan(ctx, 0, 8, 1500)


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(most=-1), dict(longest=-1), dict(longest=(1 << 30) + 1),
                                dict(splits=1025), dict(splits=-1), dict(layer=2),
                                dict(batch=1 << 30, most=1 << 10)])
def test_plan_refuses(kw):
    a = dict(layer=0, batch=2, most=4, longest=100, splits=0)
    a.update(kw)
    with pytest.raises(kvq.KVQError, match="INVALID_ARG"):
        kvq.kvq_cross_plan(_ctx(), a["layer"], a["batch"], a["most"], a["longest"], a["splits"])


def _call(ctx, **kw):
    a = dict(layer=0, q=OK, kc=OK, vc=OK, bt=OK, mb=256, qs=OK, lens=OK, B=2, most=4, longest=4096, out=OK,
             splits=2, ws=OK, wsb=1 << 30, kcs=OK, vcs=OK, ks=OK, vs=OK)
    a.update(kw)
    kvq.kvq_cross_attention(ctx, a["layer"], a["q"], a["kc"], a["vc"], a["bt"], a["qs"], a["lens"], a["out"],
                            max_query_len=a["most"], max_encoder_len=a["longest"], k_scale=a["ks"],
                            v_scale=a["vs"], k_cache_scale=a["kcs"], v_cache_scale=a["vcs"],
                            num_splits=a["splits"], workspace=a["ws"], workspace_bytes=a["wsb"],
                            batch=a["B"], max_blocks_per_seq=a["mb"], stream=0)


@pytest.mark.parametrize("match, kw", [
    ("INVALID_ARG", dict(q=None)), ("INVALID_ARG", dict(kc=None)), ("INVALID_ARG", dict(vc=None)),
    ("INVALID_ARG", dict(bt=None)), ("INVALID_ARG", dict(lens=None)), ("INVALID_ARG", dict(out=None)),
    ("INVALID_ARG", dict(kcs=None)), ("INVALID_ARG", dict(layer=1, vs=None)), ("INVALID_ARG", dict(layer=2)),
    ("INVALID_ARG", dict(B=-1)), ("INVALID_ARG", dict(most=-1)), ("INVALID_ARG", dict(longest=-1)),
    ("INVALID_ARG", dict(longest=4097)), ("INVALID_ARG", dict(splits=-1)), ("INVALID_ARG", dict(mb=-1)),
    ("INVALID_ARG", dict(qs=None, most=2)), ("INVALID_ARG", dict(qs=None, most=1, q=None)),
    ("INVALID_ARG", dict(splits=1025)),
    ("WORKSPACE", dict(ws=None)), ("WORKSPACE", dict(wsb=2 * 8 * 32 * 129 * 4 - 1)),
    ("ALIGNMENT", dict(ws=OK + 8)), ("ALIGNMENT", dict(q=OK + 8)), ("ALIGNMENT", dict(out=OK + 2)),
    ("ALIGNMENT", dict(kc=OK + 4)), ("ALIGNMENT", dict(bt=OK + 2)), ("ALIGNMENT", dict(qs=OK + 1)),
    ("ALIGNMENT", dict(kcs=OK + 4)), ("ALIGNMENT", dict(lens=OK + 3)),
])
def test_refuses(match, kw):
    with pytest.raises(kvq.KVQError, match=match):
        _call(_ctx(), **kw)


def test_refuses_windows():
    with pytest.raises(kvq.KVQError, match="UNSUPPORTED"):
        _call(_ctx((3,), [128]))


def test_nothing_to_do():
    _call(_ctx(), B=0)
    _call(_ctx(), most=0)
