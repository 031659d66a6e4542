"""Host model of the page operators, one page at a time (numpy), for the tests."""
import numpy as np

PAGE = 64


def pages_of(n):
    return (n + PAGE - 1) // PAGE


class PagesModel:
    """State: refs [num_pages], table [rows][stride], lens [rows], pool [num_pages][64][width]. Each
    operator returns the status code the library reports; a refused call changes nothing."""

    def __init__(self, refs, table, lens, pool=None):
        self.refs, self.table, self.lens, self.pool = refs, table, lens, pool
        self.cap = table.shape[1] * PAGE

    def _free_list(self):
        return [p for p in range(len(self.refs)) if self.refs[p] == 0]

    def _rows_ok(self, ids):
        return len(set(ids)) == len(ids) and all(0 <= i < len(self.lens) for i in ids)

    def reserve(self, ids, new_lens):
        if not self._rows_ok(ids) or any(not self.lens[i] <= n <= self.cap for i, n in zip(ids, new_lens)):
            return -7
        free = self._free_list()
        if sum(pages_of(n) - pages_of(self.lens[i]) for i, n in zip(ids, new_lens)) > len(free):
            return -10
        for i, n in zip(ids, new_lens):
            for c in range(pages_of(self.lens[i]), pages_of(n)):
                self.table[i, c] = free.pop(0)
                self.refs[self.table[i, c]] = 1
            self.lens[i] = n
        return 0

    def fork(self, src, dst):
        if not self._rows_ok(dst) or any(self.lens[d] for d in dst) or set(src) & set(dst):
            return -7
        if any(not 0 <= s < len(self.lens) for s in src):
            return -7
        free = self._free_list()
        if sum(self.lens[s] % PAGE != 0 for s in src) > len(free):
            return -10
        for s, d in zip(src, dst):
            n = self.lens[s]
            full, part = n // PAGE, n % PAGE
            self.table[d, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                self.refs[p] += 1
            if part:
                page = free.pop(0)
                self.table[d, full] = page
                self.refs[page] = 1
                if self.pool is not None:
                    self.pool[page, :part] = self.pool[self.table[s, full], :part]
            self.lens[d] = n
        return 0

    def free(self, ids):
        if not self._rows_ok(ids):
            return -7
        for i in ids:
            for p in self.table[i, :pages_of(self.lens[i])]:
                self.refs[p] -= 1
            self.lens[i] = 0
        return 0

    def compact(self):
        used = int((self.refs > 0).sum())
        holes = [p for p in range(used) if self.refs[p] == 0]
        high = [p for p in range(used, len(self.refs)) if self.refs[p] > 0]
        place = dict(zip(high, holes))
        for a, b in place.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            if self.pool is not None:
                self.pool[b] = self.pool[a]
        for r in range(len(self.lens)):
            for c in range(pages_of(self.lens[r])):
                self.table[r, c] = place.get(int(self.table[r, c]), self.table[r, c])
        return used

    def consistent(self):
        held = np.zeros_like(self.refs)
        for r in range(len(self.lens)):
            np.add.at(held, self.table[r, :pages_of(self.lens[r])], 1)
        return np.array_equal(held, self.refs)
