"""Which pages of a paged KV cache are free, used, and shared: the host's side of forking,
compacting and freeing sequences.

A pool knows pages by index and keeps a count of the sequences that use each.  It moves no
bytes: where a call needs a page copied it returns the pairs (source, destination), and the
caller runs bi_kv_copy_pages on them, over the planes of every layer, before the next kernel
that reads or writes those pages.  The destinations of one call are free pages, so they are
distinct and none is a source.

Forking shares the full pages of a sequence (their keys and values are final: a later token
never changes them) and copies its open page, which both sequences go on to write.
"""
from __future__ import annotations

import heapq
from typing import Dict, List, Sequence, Tuple

from .inputs import PAGE_SIZE

Copies = List[Tuple[int, int]]


class PagePool:
    """Pages 0 .. num_pages-1, handed out lowest first."""

    def __init__(self, num_pages: int):
        if num_pages < 1:
            raise ValueError("a pool has at least one page")
        self.num_pages = num_pages
        self._count = [0] * num_pages      # sequences that use the page
        self._free = list(range(num_pages))  # a heap

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def uses(self, page: int) -> int:
        """How many sequences use a page (0: it is free)."""
        return self._count[page]

    def alloc(self, n: int) -> List[int]:
        """n free pages, each now used once; none is taken when there are too few."""
        if n < 0:
            raise ValueError("n must be >= 0")
        if n > len(self._free):
            raise MemoryError(f"{n} pages wanted, {len(self._free)} free")
        pages = [heapq.heappop(self._free) for _ in range(n)]
        for p in pages:
            self._count[p] = 1
        return pages

    def take(self, pages: Sequence[int]) -> None:
        """Takes particular free pages (a cache that is already laid out)."""
        if len(set(pages)) != len(pages) or any(
                not 0 <= p < self.num_pages or self._count[p] for p in pages):
            raise ValueError("pages must be free, in range and named once")
        for p in pages:
            self._count[p] = 1
        taken = set(pages)
        self._free = [p for p in self._free if p not in taken]
        heapq.heapify(self._free)

    def adopt(self, tables: Sequence[Sequence[int]]) -> None:
        """Takes the layout of given sequences, shared pages among them, into an unused pool."""
        if any(self._count):
            raise ValueError("the pool is in use")
        count = [0] * self.num_pages
        for t in tables:
            if len(set(t)) != len(t) or any(not 0 <= p < self.num_pages for p in t):
                raise ValueError("a sequence's pages must be in range and named once")
            for p in t:
                count[p] += 1
        self._count = count
        self._free = [p for p, c in enumerate(count) if not c]

    def release(self, pages: Sequence[int]) -> None:
        """A sequence gives its pages back; those that no other one uses are free again."""
        if len(set(pages)) != len(pages):
            raise ValueError("a sequence names a page once")
        for p in pages:
            if not 0 <= p < self.num_pages or self._count[p] < 1:
                raise ValueError(f"page {p} is not in use")
        for p in pages:
            self._count[p] -= 1
            if self._count[p] == 0:
                heapq.heappush(self._free, p)

    def fork(self, pages: Sequence[int], length: int) -> Tuple[List[int], Copies]:
        """The pages of a second sequence with the first `length` tokens of the one that has
        `pages`: the full ones shared, the open one (if the last page is not full) a copy."""
        need = -(-length // PAGE_SIZE)
        if length < 0 or need > len(pages):
            raise ValueError("length outside the sequence's pages")
        if any(not 0 <= p < self.num_pages or self._count[p] < 1 for p in pages[:need]):
            raise ValueError("a page of the sequence is not in use")
        full = length // PAGE_SIZE
        opened = self.alloc(need - full)
        for p in pages[:full]:
            self._count[p] += 1
        return list(pages[:full]) + opened, [(pages[full], d) for d in opened]

    def compact(self, tables: Sequence[List[int]]) -> Copies:
        """Moves the pages in use to the lowest indices, rewriting the given sequences' tables
        (all that use the pool, their lists changed in place).  Returns the copies to make; the
        pages from the number in use upwards are free afterwards."""
        used: Dict[int, int] = {}
        for t in tables:
            if len(set(t)) != len(t) or any(not 0 <= p < self.num_pages for p in t):
                raise ValueError("a sequence's pages must be in range and named once")
            for p in t:
                used[p] = used.get(p, 0) + 1
        if any(used.get(p, 0) != c for p, c in enumerate(self._count)):
            raise ValueError("the tables do not account for every page in use")
        n = len(used)
        holes = [p for p in range(n) if not self._count[p]]
        high = [p for p in range(n, self.num_pages) if self._count[p]]
        moves = dict(zip(high, holes))
        for t in tables:
            t[:] = [moves.get(p, p) for p in t]
        for s, d in moves.items():
            self._count[d], self._count[s] = self._count[s], 0
        self._free = list(range(n, self.num_pages))
        return list(moves.items())
