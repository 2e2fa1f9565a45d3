"""The page operators one step at a time, on lists: the oracle of their tests.

Follows the words of include/kvq.h and nothing else; `errors` collects what the
device word would report."""

BAD, SHORT = "BAD_INDEX", "NO_BLOCKS"


class Pool:
    def __init__(self, num_blocks, rows, max_blocks, bs):
        self.bs, self.max_blocks, self.num_blocks = bs, max_blocks, num_blocks
        self.ref = [0] * num_blocks
        self.table = [[-1] * max_blocks for _ in range(rows)]
        self.lens = [0] * rows
        self.errors = set()

    def used(self, length):
        return -(-length // self.bs)

    def _row_ok(self, row):
        return 0 <= row < len(self.lens) and 0 <= self.lens[row] <= self.max_blocks * self.bs

    def extend(self, rows, new, max_tokens):
        bs = self.bs
        free = [b for b in range(self.num_blocks) if self.ref[b] == 0]
        old_ref = list(self.ref)
        start, positions, slots, copies = [0], [], [], []
        want = tokens = 0
        losers = []
        taken = 0
        for i, (row, n) in enumerate(zip(rows, new)):
            tokens += max(n, 0)
            start.append(tokens)
            ok = n >= 0 and self._row_ok(row) and row not in rows[:i]
            ok = ok and self.lens[row] + n <= self.max_blocks * bs
            copy = (-1, -1)
            if not ok:
                self.errors.add(BAD)
                positions += [0] * max(n, 0)
                slots += [-1] * max(n, 0)
                copies.append(copy)
                continue
            L = self.lens[row]
            have, need = self.used(L), self.used(L + n) - self.used(L)
            shared = n > 0 and L % bs != 0 and old_ref[self.table[row][have - 1]] > 1
            need += shared
            want += need
            granted = tokens <= max_tokens and (need == 0 or want <= len(free))
            if not granted:
                self.errors.add(BAD if tokens > max_tokens else SHORT)
            else:
                first = have - shared
                if shared:
                    losers.append(self.table[row][first])
                    copy = (self.table[row][first], free[taken])
                for k in range(need):
                    b = free[taken]
                    taken += 1
                    self.table[row][first + k] = b
                    self.ref[b] = 1
                self.lens[row] = L + n
            for p in range(L, L + n):
                positions.append(p)
                slots.append(self.table[row][p // bs] * bs + p % bs if granted else -1)
            copies.append(copy)
        for b in losers:
            self.ref[b] -= 1
        positions, slots = positions[:max_tokens], slots[:max_tokens]
        positions += [0] * (max_tokens - len(positions))
        slots += [-1] * (max_tokens - len(slots))
        return start, positions, slots, copies

    def fork(self, parents, children):
        for i, (p, c) in enumerate(zip(parents, children)):
            if c in children[:i] or p in children or not self._row_ok(p) or \
                    not 0 <= c < len(self.lens) or self.lens[c] != 0:
                self.errors.add(BAD)
                continue
            for j in range(self.used(self.lens[p])):
                self.table[c][j] = self.table[p][j]
                self.ref[self.table[p][j]] += 1
            self.lens[c] = self.lens[p]

    def truncate(self, rows, keep=None):
        for i, row in enumerate(rows):
            k = 0 if keep is None else keep[i]
            if row in rows[:i] or not self._row_ok(row) or k < 0:
                self.errors.add(BAD)
                continue
            left = min(self.lens[row], k)
            for j in range(self.used(left), self.used(self.lens[row])):
                self.ref[self.table[row][j]] -= 1
                self.table[row][j] = -1
            self.lens[row] = left

    def compact(self):
        n = sum(r > 0 for r in self.ref)
        moves = list(zip([b for b in range(n, self.num_blocks) if self.ref[b] > 0],
                         [b for b in range(n) if self.ref[b] == 0]))
        to = dict(moves)
        for s, d in moves:
            self.ref[d], self.ref[s] = self.ref[s], 0
        for row, length in enumerate(self.lens):
            for j in range(self.used(length)):
                b = self.table[row][j]
                self.table[row][j] = to.get(b, b)
        return moves

    def check(self):
        held = [0] * self.num_blocks
        for row, length in enumerate(self.lens):
            for j in range(self.used(length)):
                held[self.table[row][j]] += 1
            assert all(b == -1 for b in self.table[row][self.used(length):])
        assert held == self.ref
