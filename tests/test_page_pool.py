"""The host's bookkeeping of cache pages: allocation, sharing, forks and compaction, against a
plain model of page contents (every page a list of the tokens written to it)."""
import random

import pytest

from invariant_bi_matmul_gb300.pages import PAGE_SIZE, PagePool


def test_alloc_release_and_refusals():
    pool = PagePool(5)
    a = pool.alloc(3)
    assert a == [0, 1, 2] and pool.free_pages == 2
    with pytest.raises(MemoryError):
        pool.alloc(3)
    assert pool.free_pages == 2            # nothing taken by the refused call
    pool.release([1])
    assert pool.alloc(1) == [1]
    for bad in ([4], [-1], [7], [0, 0]):
        with pytest.raises(ValueError):
            pool.release(bad)
    assert pool.uses(0) == 1
    with pytest.raises(ValueError):
        pool.alloc(-1)
    with pytest.raises(ValueError):
        pool.take([0, 3])
    assert pool.uses(3) == 0               # the refused call took nothing
    pool.take([4])
    assert pool.free_pages == 1
    with pytest.raises(ValueError):
        PagePool(0)
    with pytest.raises(ValueError):
        pool.adopt([[3]])


@pytest.mark.parametrize("length", [0, 1, PAGE_SIZE - 1, PAGE_SIZE, PAGE_SIZE + 1, 3 * PAGE_SIZE])
def test_fork_shares_full_pages_and_copies_the_open_one(length):
    pool = PagePool(10)
    pages = pool.alloc(4)
    forked, copies = pool.fork(pages, length)
    full = length // PAGE_SIZE
    assert forked[:full] == pages[:full] and all(pool.uses(p) == 2 for p in pages[:full])
    if length % PAGE_SIZE:
        assert copies == [(pages[full], forked[full])] and forked[full] not in pages
    else:
        assert copies == [] and len(forked) == full
    with pytest.raises(ValueError):
        pool.fork(pages, 4 * PAGE_SIZE + 1)
    with pytest.raises(ValueError):
        pool.fork([9], 1)


def test_fork_without_room_changes_nothing():
    pool = PagePool(2)
    pages = pool.alloc(2)
    with pytest.raises(MemoryError):
        pool.fork(pages, PAGE_SIZE + 1)
    assert [pool.uses(p) for p in pages] == [1, 1]


@pytest.mark.parametrize("seed", range(8))
def test_random_life_of_a_pool(seed):
    """Sequences grow, fork, end, and the pool is compacted; every sequence always reads back
    the tokens it was given."""
    rng = random.Random(seed)
    pool = PagePool(40)
    mem = [[None] * PAGE_SIZE for _ in range(40)]
    seqs = []  # (pages, tokens)

    def copy(copies):
        assert len({d for _, d in copies}) == len(copies)
        assert not {d for _, d in copies} & {s for s, _ in copies}
        before = [list(m) for m in mem]
        for s, d in copies:
            mem[d] = list(before[s])
    for step in range(400):
        what = rng.random()
        if what < 0.15 and pool.free_pages:
            seqs.append(([], []))
        elif what < 0.7 and seqs:
            pages, toks = rng.choice(seqs)
            for _ in range(rng.randint(1, 40)):
                if len(toks) % PAGE_SIZE == 0:
                    if not pool.free_pages:
                        break
                    pages += pool.alloc(1)
                mem[pages[-1]][len(toks) % PAGE_SIZE] = (step, len(toks))
                toks.append((step, len(toks)))
        elif what < 0.8 and seqs and pool.free_pages:
            pages, toks = rng.choice(seqs)
            n = rng.randint(0, len(toks))
            new, copies = pool.fork(pages, n)
            copy(copies)
            seqs.append((new, toks[:n]))
        elif what < 0.9 and seqs:
            pages, _ = seqs.pop(rng.randrange(len(seqs)))
            pool.release(pages)
        else:
            copies = pool.compact([p for p, _ in seqs])
            copy(copies)
            n = 40 - pool.free_pages
            assert all(p < n for pages, _ in seqs for p in pages)
        for pages, toks in seqs:
            assert [mem[pages[i // PAGE_SIZE]][i % PAGE_SIZE] for i in range(len(toks))] == toks
        assert pool.free_pages == 40 - len({p for pages, _ in seqs for p in pages})


def test_compact_needs_every_table():
    pool = PagePool(4)
    a, b = pool.alloc(1), pool.alloc(1)
    with pytest.raises(ValueError):
        pool.compact([a])
    pool.release(a)
    assert pool.compact([b]) == [(1, 0)] and b == [0]
