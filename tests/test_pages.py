"""Page operators without a GPU: the model keeps its invariant, and the entry
points refuse bad arguments before anything is launched."""
import random

import pytest

from tests.page_model import Pool

kvq = pytest.importorskip("int4_quantized_paged_gb300.kvq",
                          reason="libkvq.so not built (run __graft_entry__.build())")
OK = 0x10000000                      # never dereferenced: validation fails first


def test_model_keeps_the_counts():
    r = random.Random(3)
    p = Pool(200, 20, 12, 16)
    for _ in range(300):
        op = r.randrange(4)
        rows = r.sample(range(20), r.randint(1, 8))
        if op == 0:
            p.extend(rows, [r.randint(0, 40) for _ in rows], 1000)
        elif op == 1:
            empty = [x for x in range(20) if p.lens[x] == 0][:3]
            p.fork([r.choice([x for x in range(20) if x not in empty]) for _ in empty], empty)
        elif op == 2:
            p.truncate(rows, [r.randint(0, 150) for _ in rows] if r.random() < 0.5 else None)
        else:
            p.compact()
            assert all(p.ref[b] > 0 for b in range(sum(x > 0 for x in p.ref)))
        p.check()


class T(int):
    """A pointer with a shape, as the binding reads them."""
    def __new__(cls, at=OK, *shape):
        t = super().__new__(cls, at)
        t.shape = shape
        return t

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n


def _ctx(modes=(3,), nb=64):
    return kvq.kvq_create(len(modes), 8, 8, 64, 16, nb, list(modes))


def _extend(ctx, rows=T(OK, 4), new=OK, ref=OK, table=T(OK, 8, 16), lens=OK, qs=OK, pos=OK, slots=OK,
            copies=OK, max_tokens=64):
    kvq.kvq_extend_sequences(ctx, rows, new, ref, table, lens, qs, pos, slots, copies,
                             max_tokens=max_tokens, stream=0)


@pytest.mark.parametrize("match, kw", [
    ("INVALID_ARG", dict(new=None)), ("INVALID_ARG", dict(ref=None)), ("INVALID_ARG", dict(lens=None)),
    ("INVALID_ARG", dict(qs=None)), ("INVALID_ARG", dict(pos=None)), ("INVALID_ARG", dict(slots=None)),
    ("INVALID_ARG", dict(copies=None)), ("INVALID_ARG", dict(max_tokens=-1)),
    ("INVALID_ARG", dict(max_tokens=1 << 31)), ("INVALID_ARG", dict(max_tokens=(1 << 31) - 1)),
    ("INVALID_ARG", dict(table=T(OK, 8, 1 << 27))),
    ("UNSUPPORTED", dict(rows=T(OK, 4097))),
    ("ALIGNMENT", dict(rows=T(OK + 2, 4))), ("ALIGNMENT", dict(table=T(OK + 1, 8, 16))),
    ("ALIGNMENT", dict(pos=OK + 4)), ("ALIGNMENT", dict(slots=OK + 4)), ("ALIGNMENT", dict(copies=OK + 2)),
])
def test_extend_refuses(match, kw):
    with pytest.raises(kvq.KVQError, match=match):
        _extend(_ctx(), **kw)


def test_nothing_to_do():
    ctx = _ctx()
    empty = T(0, 0)
    _extend(ctx, rows=empty, new=None)
    kvq.kvq_fork_sequences(ctx, empty, None, OK, T(OK, 8, 16), OK, stream=0)
    kvq.kvq_truncate_sequences(ctx, empty, None, OK, T(OK, 8, 16), OK, stream=0)
    layers = kvq.layer_pointers([OK], [OK], [OK], [OK])
    kvq.kvq_copy_blocks(ctx, T(0, 0, 2), layers, stream=0)


@pytest.mark.parametrize("match, kw", [
    ("INVALID_ARG", dict(children=None)), ("INVALID_ARG", dict(ref=None)),
    ("INVALID_ARG", dict(lens=None)), ("ALIGNMENT", dict(parents=T(OK + 1, 2))),
    ("ALIGNMENT", dict(children=OK + 3)),
])
def test_fork_refuses(match, kw):
    a = dict(parents=T(OK, 2), children=OK, ref=OK, table=T(OK, 8, 16), lens=OK)
    a.update(kw)
    with pytest.raises(kvq.KVQError, match=match):
        kvq.kvq_fork_sequences(_ctx(), a["parents"], a["children"], a["ref"], a["table"], a["lens"],
                               stream=0)


@pytest.mark.parametrize("match, kw", [
    ("INVALID_ARG", dict(rows=T(0, 2))), ("INVALID_ARG", dict(ref=None)),
    ("ALIGNMENT", dict(keep=OK + 1)), ("ALIGNMENT", dict(lens=OK + 2)),
])
def test_truncate_refuses(match, kw):
    a = dict(rows=T(OK, 2), keep=None, ref=OK, table=T(OK, 8, 16), lens=OK)
    a.update(kw)
    with pytest.raises(kvq.KVQError, match=match):
        kvq.kvq_truncate_sequences(_ctx(), a["rows"] or None if a["rows"] else T(0, 2), a["keep"],
                                   a["ref"], a["table"], a["lens"], stream=0)


@pytest.mark.parametrize("match, kw", [
    ("INVALID_ARG", dict(ref=None)), ("INVALID_ARG", dict(moves=None)), ("INVALID_ARG", dict(count=None)),
    ("ALIGNMENT", dict(moves=OK + 2)), ("ALIGNMENT", dict(count=OK + 1)),
])
def test_compact_refuses(match, kw):
    a = dict(ref=OK, moves=OK, count=OK)
    a.update(kw)
    with pytest.raises(kvq.KVQError, match=match):
        kvq.kvq_compact_blocks(_ctx(), a["ref"], T(OK, 8, 16), OK, a["moves"], a["count"], stream=0)


@pytest.mark.parametrize("match, layers, kw", [
    ("INVALID_ARG", ([OK], [OK], None, None), dict(pairs=T(0, 4, 2))),
    ("INVALID_ARG", ([OK], [OK], None, None), {}),                        # dynamic layer, no scales
    ("INVALID_ARG", ([OK], [OK], [OK], [None]), {}),
    ("INVALID_ARG", ([OK], [None], [OK], [OK]), {}),
    ("INVALID_ARG", ([OK, OK, OK], [OK] * 3, [OK] * 3, [OK] * 3), {}),    # more layers than the context has
    ("INVALID_ARG", ([OK], [OK], [OK], [OK]), dict(first_layer=2)),
    ("INVALID_ARG", ([OK], [OK], [OK], [OK]), dict(first_layer=-1)),
    ("INVALID_ARG", ([OK], [OK], [OK], [OK]), dict(max_pairs=-1)),
    ("ALIGNMENT", ([OK + 8], [OK], [OK], [OK]), {}),
    ("ALIGNMENT", ([OK], [OK], [OK + 4], [OK]), {}),
    ("ALIGNMENT", ([OK], [OK], [OK], [OK]), dict(pairs=T(OK + 2, 4, 2))),
])
def test_copy_refuses(match, layers, kw):
    a = dict(pairs=T(OK, 4, 2))
    a.update(kw)
    with pytest.raises(kvq.KVQError, match=match):
        kvq.kvq_copy_blocks(_ctx((3, 0)), a.pop("pairs"), kvq.layer_pointers(*layers), stream=0, **a)


def test_layer_pointers_wants_every_layer():
    with pytest.raises(ValueError):
        kvq.layer_pointers([OK, OK], [OK])
