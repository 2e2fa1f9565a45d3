"""Eviction one cell at a time, on lists: the oracle of its tests. Follows the words of
include/kvq.h and nothing else."""
import math


def survivors(weights, L, keep, first, last):
    """Positions of the middle that stay, ascending."""
    def order(p):
        w = weights[p]
        return (1, 0.0, p) if math.isnan(w) else (0, -w, p)
    middle = sorted(range(first, L - last), key=order)
    return sorted(middle[:keep - first - last])


def places(weights, L, keep, first, last):
    """(source, destination) of every cell that moves, the middle's before the last ones."""
    stay = survivors(weights, L, keep, first, last)
    held = set(stay)
    free = [p for p in range(first, keep - last) if p not in held]
    late = [p for p in stay if p >= keep - last]
    assert len(free) == len(late)
    return list(zip(late, free)) + [(L - last + i, keep - last + i) for i in range(last)]


class Call:
    """What one call does to weights[row][head] (lists of floats) and to cells named
    (block, head, offset); `moves` collects (source, destination) cells, which happen at once."""

    def __init__(self, rows, keeps, table, lens, weights, bs, num_blocks, Hkv, first, last, most, ref=None):
        self.moves, self.bad, self.new_lens = [], False, []
        for i, (row, keep) in enumerate(zip(rows, keeps)):
            if row < 0 or row >= len(table) or row in rows[:i]:
                self.bad = True
                self.new_lens.append(0)
                continue
            L = lens[row]
            ok = 0 <= L <= most and L <= len(table[row]) * bs and keep >= first + last
            if ok and L > keep:
                used = table[row][:-(-L // bs)]
                ok = all(0 <= b < num_blocks and (ref is None or ref[b] == 1) for b in used)
            if not ok:
                self.bad = True
            if not ok or L <= keep:
                self.new_lens.append(L)
                continue
            self.new_lens.append(keep)
            for h in range(Hkv):
                w = weights[row][h]
                pairs = places(w, L, keep, first, last)
                old = list(w)
                for s, d in pairs:
                    w[d] = old[s]
                    self.moves.append(((table[row][s // bs], h, s % bs), (table[row][d // bs], h, d % bs)))
                w[keep:L] = [0.0] * (L - keep)
