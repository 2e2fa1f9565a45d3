"""Eviction without a GPU: the refusals, and the list model against a plain reading."""
import random

import pytest

from tests import evict_model as em

kvq = pytest.importorskip("int4_quantized_paged_gb300.kvq",
                          reason="libkvq.so not built (run __graft_entry__.build())")
OK = 0x10000000                      # never dereferenced: validation fails first


class Ints:
    """A tensor as far as the binding looks."""

    def __init__(self, ptr, *shape):
        self.ptr, self.shape = ptr, shape

    def data_ptr(self):
        return self.ptr

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n


def _call(windows=None, **kw):
    a = dict(layer=0, rows=OK, n=2, keep=OK, table=OK, blocks=256, lens=OK, w=OK, stride=4096, new=OK, kc=OK, vc=OK,
             ks=OK, vs=OK, first=4, last=64, most=4096, ref=OK)
    a.update(kw)
    ctx = kvq.kvq_create(2, 32, 8, 128, 16, 4096, [3, 2], windows)
    kvq.kvq_evict_cells(ctx, a["layer"], Ints(a["rows"], a["n"]), a["keep"], Ints(a["table"], 3, a["blocks"]),
                        a["lens"], a["w"], a["new"], a["kc"], a["vc"], a["ks"], a["vs"], first_kept=a["first"],
                        last_kept=a["last"], max_context=a["most"], ref_count=a["ref"], weights_stride=a["stride"],
                        stream=0)


@pytest.mark.parametrize("match, kw", [
    ("INVALID_ARG", dict(layer=2)), ("INVALID_ARG", dict(n=-1)), ("INVALID_ARG", dict(first=-1)),
    ("INVALID_ARG", dict(last=-1)), ("INVALID_ARG", dict(most=-1)), ("INVALID_ARG", dict(most=4097, stride=5000)),
    ("INVALID_ARG", dict(stride=4095)), ("INVALID_ARG", dict(blocks=1 << 27)), ("INVALID_ARG", dict(rows=None)),
    ("INVALID_ARG", dict(keep=None)), ("INVALID_ARG", dict(table=None)), ("INVALID_ARG", dict(lens=None)),
    ("INVALID_ARG", dict(w=None)), ("INVALID_ARG", dict(new=None)), ("INVALID_ARG", dict(kc=None)),
    ("INVALID_ARG", dict(vc=None)), ("INVALID_ARG", dict(ks=None)), ("INVALID_ARG", dict(vs=None)),
    ("INVALID_ARG", dict(n=1 << 29)),
    ("ALIGNMENT", dict(rows=OK + 2)), ("ALIGNMENT", dict(keep=OK + 1)), ("ALIGNMENT", dict(table=OK + 2)),
    ("ALIGNMENT", dict(lens=OK + 2)), ("ALIGNMENT", dict(w=OK + 2)), ("ALIGNMENT", dict(new=OK + 2)),
    ("ALIGNMENT", dict(kc=OK + 8)), ("ALIGNMENT", dict(vc=OK + 4)), ("ALIGNMENT", dict(ks=OK + 2)),
    ("ALIGNMENT", dict(ref=OK + 2)),
    ("UNSUPPORTED", dict(windows=[128, 0])),
    ("UNSUPPORTED", dict(most=393217, stride=400000, blocks=30000)),
])
def test_refuses(match, kw):
    with pytest.raises(kvq.KVQError, match=match):
        _call(**kw)


@pytest.mark.parametrize("kw", [
    dict(new=OK), dict(new=OK + 8), dict(new=OK - 4, n=2), dict(new=OK + 0x1000), dict(new=OK + 0x1004, n=2),
    dict(new=OK + 0xffc), dict(new=OK + 0x2004), dict(new=OK + 0x1ffc),
])
def test_lengths_are_not_written_over_what_the_call_reads(kw):
    """3 lengths at OK, 2 rows at OK + 0x1000, 2 budgets at OK + 0x2000."""
    with pytest.raises(kvq.KVQError, match="INVALID_ARG"):
        _call(rows=OK + 0x1000, keep=OK + 0x2000, table=OK + 0x3000, **kw)


def test_nothing_to_do():
    _call(n=0)


def test_the_model_keeps_what_it_should():
    rng = random.Random(0)
    for _ in range(300):
        L = rng.randint(2, 60)
        keep = rng.randint(0, L - 1)
        first = rng.randint(0, keep)
        last = rng.randint(0, keep - first)
        w = [rng.choice([0.0, 1.0, rng.random(), float("nan")]) for _ in range(L)]
        cells = list(range(L))
        for s, d in em.places(w, L, keep, first, last):
            cells[d] = s
        kept = cells[:keep]
        assert len(set(kept)) == keep and kept[:first] == list(range(first))
        assert kept[keep - last:] == list(range(L - last, L))
        value = [-1.0 if x != x else x for x in w]
        inside = sorted(kept[first:keep - last])
        out = sorted(set(range(first, L - last)) - set(inside))
        if inside and out:
            assert min((value[p], -p) for p in inside) > max((value[p], -p) for p in out)
