"""Compaction turns away tables that name pages outside the pool, or one page twice, and changes
nothing then."""
import pytest

from invariant_bi_matmul_gb300.pages import PagePool


@pytest.mark.parametrize("taken,table", [([0, 3], [0, 3, 7, 9]), ([0, 2], [0, 2, -1]),
                                         ([1], [1, 4]), ([1, 2], [1, -4, 2])])
def test_pages_outside_the_pool_are_refused(taken, table):
    pool = PagePool(4)
    pool.take(taken)
    tables = [list(table)]
    with pytest.raises(ValueError):
        pool.compact(tables)
    assert tables == [table] and pool.free_pages == 4 - len(taken)
    assert [pool.uses(p) for p in range(4)] == [int(p in taken) for p in range(4)]
    assert sorted(pool.alloc(4 - len(taken)) + taken) == [0, 1, 2, 3]     # no page is lost


def test_one_page_twice_in_a_table_is_refused():
    """A page that two sequences share, named twice by one of them and not by the other."""
    pool = PagePool(4)
    pool.take([1, 2])
    pool.fork([2], 64)
    tables = [[1], [2, 2]]
    with pytest.raises(ValueError):
        pool.compact(tables)
    assert tables == [[1], [2, 2]] and pool.uses(2) == 2 and pool.free_pages == 2
    tables = [[1, 2], [2]]
    assert pool.compact(tables) == [(2, 0)] and tables == [[1, 0], [0]]
