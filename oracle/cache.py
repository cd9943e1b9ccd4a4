"""The paged cache's book-keeping, step by step on the host: pages given back, handed out lowest
number first, shared and copied; accepted tokens moved.  Arrays are changed in place."""
from __future__ import annotations

import numpy as np

PAGE = 16


def _pages(n):
    return -(-int(n) // PAGE)


def _copy(caches, src, dst):
    for c in caches:
        c[:, dst] = c[:, src]


def resize(caches, tables, lens, counts, new_lens) -> bool:
    """caches: arrays [layers, pages, 16, ...]; True if the free pages sufficed."""
    for b, new in enumerate(new_lens):
        for j in range(_pages(new), _pages(lens[b])):
            counts[tables[b, j]] -= 1
            tables[b, j] = -1
    places = []                                  # (row, table position, page to copy or None)
    for b, new in enumerate(new_lens):
        kept = min(int(lens[b]), int(new))
        last = _pages(kept) - 1
        if kept % PAGE and counts[tables[b, last]] > 1:
            places.append((b, last, int(tables[b, last])))
        places += [(b, j, None) for j in range(_pages(kept), _pages(new))]
    free = np.nonzero(counts == 0)[0]
    fits = len(places) <= len(free)
    if fits:
        for (b, j, old), page in zip(places, free):
            if old is not None:
                _copy(caches, old, page)
                counts[old] -= 1
            tables[b, j] = page
            counts[page] += 1
    for b, new in enumerate(new_lens):
        lens[b] = new if fits else min(int(lens[b]), int(new))
    return fits


def fork(caches, tables, lens, counts, src, dst) -> bool:
    free = np.nonzero(counts == 0)[0]
    at = [int(lens[s]) for s in src]
    if sum(1 for n in at if n % PAGE) > len(free):
        return False
    k = 0
    for s, d, n in zip(src, dst, at):
        for j in range(n // PAGE):
            tables[d, j] = tables[s, j]
            counts[tables[s, j]] += 1
        if n % PAGE:
            page = free[k]
            k += 1
            _copy(caches, tables[s, n // PAGE], page)
            tables[d, n // PAGE] = page
            counts[page] += 1
    for d, n in zip(dst, at):
        lens[d] = n
    return True


def compact(caches, tables, lens, nodes, index, count):
    """The new lengths; nodes: the tree's size in each row."""
    new = []
    for b, n in enumerate(nodes):
        start = int(lens[b]) - n
        for j in range(int(count[b]) + 1):
            a = start + int(index[b, j])
            for c in caches:
                c[:, tables[b, (start + j) // PAGE], (start + j) % PAGE] = \
                    c[:, tables[b, a // PAGE], a % PAGE]
        new.append(start + int(count[b]) + 1)
    return np.array(new, np.int32)
