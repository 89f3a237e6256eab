"""Plain forms of the page management, for its tests: loops over requests and entries, on lists."""
import numpy as np


def up(n, m):
    return -(-n // m)


class Pool:
    """Tables, lengths, share counts and free list of a pool, as NumPy arrays."""

    def __init__(self, table, lens, shares, free, used, page):
        self.table, self.lens, self.shares, self.free = (np.array(x, dtype=np.int32) for x in
                                                         (table, lens, shares, free))
        self.used, self.page = int(used), page

    def copy(self):
        return Pool(self.table.copy(), self.lens.copy(), self.shares.copy(), self.free.copy(), self.used, self.page)

    def holders(self):
        """How many requests hold each page."""
        n = np.zeros(len(self.shares), dtype=int)
        for b, length in enumerate(self.lens):
            for j in range(up(int(length), self.page)):
                n[self.table[b, j]] += 1
        return n

    def check(self):
        """Every page is held as often as its count says, or free, once (or in no list at all)."""
        n, spare = self.holders(), self.free[self.used:].tolist()
        assert len(set(spare)) == len(spare) and not n[spare].any()
        assert np.array_equal(self.shares, np.maximum(n - 1, 0))
        assert (n > 0).sum() + len(spare) == len(self.free)

    def free_rows(self, rows, keep=None):
        back = []
        for i, row in enumerate(rows):
            if row < 0:
                continue
            kept = 0 if keep is None else int(keep[i])
            for j in range(up(kept, self.page), up(int(self.lens[row]), self.page)):
                p = self.table[row, j]
                if self.shares[p] == 0:
                    back.append(int(p))
                else:
                    self.shares[p] -= 1
            self.lens[row] = kept
        self.used -= len(back)
        self.free[self.used:self.used + len(back)] = sorted(back)

    def fork(self, parents, children, lens=None):
        copies = []
        for i, (parent, child) in enumerate(zip(parents, children)):
            copies.append((-1, -1, 0))
            if parent < 0:
                continue
            n = int(self.lens[parent]) if lens is None else int(lens[i])
            full, part = divmod(n, self.page)
            for j in range(full):
                self.table[child, j] = self.table[parent, j]
                self.shares[self.table[parent, j]] += 1
            if part:
                self.table[child, full] = self.free[self.used]
                copies[-1] = (int(self.table[parent, full]), int(self.free[self.used]), part)
                self.used += 1
            self.lens[child] = n
        return np.array(copies, dtype=np.int32).reshape(-1, 3)

    def compact(self, most):
        held = sorted(np.nonzero(self.holders())[0].tolist(), reverse=True)
        spare = sorted(self.free[self.used:].tolist())
        moves = []
        for high, low in zip(held, spare):
            if low > high or len(moves) == most:
                break
            moves.append((high, low, self.page))
        to = {a: b for a, b, _ in moves}
        for b, length in enumerate(self.lens):
            for j in range(up(int(length), self.page)):
                self.table[b, j] = to.get(int(self.table[b, j]), self.table[b, j])
        for a, b in to.items():
            self.shares[b], self.shares[a] = self.shares[a], 0
        self.free[self.used:] = sorted(set(spare) - set(to.values()) | set(to))
        return np.array(moves + [(-1, -1, 0)] * (most - len(moves)), dtype=np.int32).reshape(-1, 3)


def random_pool(rng, B, page, longest, spare=20, cols=2, fork=0.4, pinned=3):
    """A pool of B rows, some empty, some forks of others, its pages shuffled; `pinned` pages belong to
    no request and are not free either."""
    lens = rng.integers(1, longest + 1, B)
    lens[rng.random(B) < 0.3] = 0
    width = max(up(longest, page), 1) + cols
    need = int(sum(up(int(n), page) for n in lens)) + B
    n_pages = need + spare + pinned
    perm = rng.permutation(n_pages)
    pool = Pool(np.full((B, width), -9), lens, np.zeros(n_pages), perm[:n_pages - pinned], 0, page)
    for b in range(B):
        for j in range(up(int(lens[b]), page)):
            pool.table[b, j] = pool.free[pool.used]
            pool.used += 1
    living = np.nonzero(pool.lens)[0]
    empty = [b for b in np.nonzero(pool.lens == 0)[0] if rng.random() < fork]
    if len(living):
        parents = rng.choice(living, len(empty))
        pool.fork(parents, empty, [int(rng.integers(0, pool.lens[p] + 1)) for p in parents])
    return pool
