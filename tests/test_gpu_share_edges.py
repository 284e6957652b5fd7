"""Page sharing on the GPU where its lists are at odds with one another."""
import pytest

from tests.test_gpu_share import _ops, _ws, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
def test_compaction_tells_of_entries_on_the_free_list(in_place):
    """A table entry that is on the free list, below the limit (another request's page may be moved there) or at and above
    it; the free list is sound.  Nothing is told of tables that are."""
    ops = _ops()
    page, total = 4, 8
    ws = _ws(ops, ops.OP_COMPACT_PAGES, b=2, pages=total)
    src, dst, moves = (i32([-5] * 4) for _ in range(3))

    def compact(table, lens, limit=0):
        t = dict(counts=i32([0] * total), free=i32([1, 6, 3, 4]), n=i32([4]), table=i32(table))
        new = t if in_place else dict(counts=i32([-9] * total), free=i32([-9] * 4), n=i32([-9]), table=i32(table))
        ops.spec_compact_pages(len(lens), page, i32(list(range(len(lens)))), i32(lens), limit, t["counts"], t["free"], t["n"], t["table"], None, new["counts"], new["free"], new["n"],
                               new["table"], None, src, dst, moves, ws)
        return ws.last_error(), new["table"].tolist()

    # in use: 0, 2, 5, 7; free below the limit of four: 1 and 3
    assert compact([[0, 7, -1], [5, 2, -1]], [8, 8]) == (0, [[0, 3, -1], [1, 2, -1]])
    assert compact([[0, 7, 1], [5, 2, -1]], [8, 8]) == (0, [[0, 3, 1], [1, 2, -1]])  # (behind the request's tokens)
    error, table = compact([[0, 7, 1], [5, 2, -1]], [12, 8])  # 1 becomes another request's page
    assert error == ops.DEV_INVARIANT and table == [[0, 3, 1], [1, 2, -1]]
    error, table = compact([[0, 7, 6], [5, 2, -1]], [12, 8])
    assert error == ops.DEV_INVARIANT and table[0][:2] == [0, 3] and table[1] == [1, 2, -1]
    # a limit above every page: nothing is moved, and an entry on the list is told all the same
    assert compact([[0, 7, -1], [5, 2, -1]], [8, 8], limit=8) == (0, [[0, 7, -1], [5, 2, -1]])
    assert compact([[0, 4, -1], [5, 2, -1]], [8, 8], limit=8) == (ops.DEV_INVARIANT, [[0, 4, -1], [5, 2, -1]])
