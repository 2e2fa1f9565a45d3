"""Attention over whole prompts without a GPU: the refusals."""
import pytest

kvq = pytest.importorskip("int4_quantized_paged_gb300.kvq",
                          reason="libkvq.so not built (run __graft_entry__.build())")
OK = 0x10000000                      # never dereferenced: validation fails first


def _call(**kw):
    a = dict(layer=0, q=OK, k=OK, v=OK, start=OK, B=2, most=64, T=128, out=OK, qs=0, ks=0)
    a.update(kw)
    ctx = kvq.kvq_create(1, 32, 8, 128, 16, 0, [3])
    kvq.kvq_prompt_attention(ctx, a["layer"], a["q"], a["k"], a["v"], a["start"], a["out"], max_seq_len=a["most"],
                             q_token_stride=a["qs"], kv_token_stride=a["ks"], num_tokens=a["T"], batch=a["B"],
                             stream=0)


@pytest.mark.parametrize("match, kw", [
    ("INVALID_ARG", dict(layer=1)), ("INVALID_ARG", dict(layer=-1)), ("INVALID_ARG", dict(B=-1)),
    ("INVALID_ARG", dict(most=-1)), ("INVALID_ARG", dict(T=-1)), ("INVALID_ARG", dict(T=(1 << 31) - 256)),
    ("INVALID_ARG", dict(q=None)), ("INVALID_ARG", dict(k=None)), ("INVALID_ARG", dict(v=None)),
    ("INVALID_ARG", dict(start=None)), ("INVALID_ARG", dict(out=None)),
    ("INVALID_ARG", dict(qs=32 * 128 - 8)), ("INVALID_ARG", dict(ks=8 * 128 - 8)),
    ("INVALID_ARG", dict(qs=1 << 39)), ("INVALID_ARG", dict(ks=1 << 39)), ("INVALID_ARG", dict(qs=-8)),
    ("INVALID_ARG", dict(B=(1 << 31) - 1)), ("INVALID_ARG", dict(B=1 << 30, most=1 << 20, T=(1 << 31) - 300)),
    ("ALIGNMENT", dict(qs=32 * 128 + 4)), ("ALIGNMENT", dict(ks=8 * 128 + 4)), ("ALIGNMENT", dict(q=OK + 8)),
    ("ALIGNMENT", dict(k=OK + 2)), ("ALIGNMENT", dict(v=OK + 4)), ("ALIGNMENT", dict(out=OK + 8)),
    ("ALIGNMENT", dict(start=OK + 2)),
])
def test_refuses(match, kw):
    with pytest.raises(kvq.KVQError, match=match):
        _call(**kw)


def test_nothing_to_do():
    _call(B=0)
    _call(most=0)
    _call(T=0)
