"""Row-by-row restatement of fork, extend and compact (include/pa.h) on Python
lists.  Nothing here shares code with the library."""
from __future__ import annotations

import random

import torch


def blocks(n, bs):
    return -(-n // bs)


class Book:
    """Tables, lengths and counts, as a program keeps them; `pools` [planes, blocks,
    ...] tensors on the CPU."""

    def __init__(self, tables, lens, refs, bs, pools=()):
        self.tables, self.lens, self.refs, self.bs = [list(r) for r in tables], list(lens), list(refs), bs
        self.pools = [p.clone() for p in pools]

    def used(self, r):
        return self.tables[r][:blocks(self.lens[r], self.bs)]

    def fork(self, parents, tables_out):
        tables, lens = [list(r) for r in tables_out], []
        for r in range(len(self.lens)):
            for b in self.used(r):
                self.refs[b] -= 1
        for s, parent in enumerate(parents):
            row = self.used(parent) if parent >= 0 else []
            lens.append(self.lens[parent] if parent >= 0 else 0)
            tables[s][:len(row)] = row
            for b in row:
                self.refs[b] += 1
        self.tables, self.lens = tables, lens

    def extend(self, new, num_slots, tables_out=None):
        """(slots, info).  Each row in turn takes the lowest free blocks."""
        bs, free = self.bs, [b for b, c in enumerate(self.refs) if c == 0]
        have, refs = len(free), list(self.refs)
        tables, slots, copies = [list(r) for r in (tables_out or self.tables)], [], []
        took = 0
        for r, n in enumerate(new):
            row = list(self.used(r))
            if n > 0 and self.lens[r] % bs and refs[row[-1]] > 1:
                refs[row[-1]] -= 1
                to = free[took] if took < have else -1
                copies.append((row[-1], to))
                row[-1] = to
                took += 1
            for _ in range(blocks(self.lens[r] + n, bs) - len(row)):
                row.append(free[took] if took < have else -1)
                took += 1
            tables[r][:len(row)] = row
            for p in range(self.lens[r], self.lens[r] + n):
                slots.append(row[p // bs] * bs + p % bs)
        info = [took, have - took]
        if took > have or len(slots) > num_slots:
            tables = [list(r) for r in (tables_out or self.tables)]
            for r in range(len(new)):
                tables[r][:len(self.used(r))] = self.used(r)
            self.tables = tables
            return [-1] * num_slots, info
        for b in free[:took]:
            refs[b] = 1
        for pool in self.pools:
            for src, dst in copies:
                pool[:, dst] = pool[:, src]
        self.refs, self.tables = refs, tables
        self.lens = [a + n for a, n in zip(self.lens, new)]
        return slots + [-1] * (num_slots - len(slots)), info

    def compact(self, tables_out=None):
        """(new_ids, info)"""
        n = sum(c > 0 for c in self.refs)
        src = [b for b, c in enumerate(self.refs) if c > 0 and b >= n]
        dst = [b for b, c in enumerate(self.refs) if c == 0 and b < n]
        ids = [b if c > 0 else -1 for b, c in enumerate(self.refs)]
        for a, b in zip(src, dst):
            ids[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
            for pool in self.pools:
                pool[:, b] = pool[:, a]
        tables = [list(r) for r in (tables_out or self.tables)]
        for r in range(len(self.lens)):
            for j, b in enumerate(self.used(r)):
                tables[r][j] = ids[b]
        self.tables = tables
        return ids, [n, len(src)]


def make_book(rows, max_blocks, bs, num_blocks, seed, share=0.5, shapes=((2, 16),)):
    """Random sequences of which some share blocks as after forks."""
    rng = random.Random(seed)
    free = list(range(num_blocks))
    rng.shuffle(free)
    tables, lens = [], []
    room = num_blocks * 3 // 4
    for r in range(rows):
        row, n = [], rng.choice([0, 1, bs, rng.randint(0, max_blocks * bs), rng.randint(0, max_blocks * bs)])
        if r and rng.random() < share:      # a fork of an earlier row, perhaps grown since
            of = rng.randrange(r)
            row = tables[of][:blocks(lens[of], bs)]
            n = lens[of]
            if rng.random() < 0.5 and len(row) < max_blocks:
                n = len(row) * bs + rng.randint(0, (max_blocks - len(row)) * bs)
        need = blocks(n, bs) - len(row)
        if need > room:
            n, need = len(row) * bs, 0
        room -= need
        row = row + [free.pop() for _ in range(need)]
        tables.append(row + [-7] * (max_blocks - len(row)))
        lens.append(n)
    refs = [0] * num_blocks
    for row, n in zip(tables, lens):
        for b in row[:blocks(n, bs)]:
            refs[b] += 1
    g = torch.Generator().manual_seed(seed)
    pools = [torch.randint(-100, 100, (s[0], num_blocks, *s[1:]), generator=g, dtype=torch.int8)
             for s in shapes]
    return Book(tables, lens, refs, bs, pools)
