"""Page sharing on the GPU where its lists are at odds with one another, and with as many requests as a call takes."""
import pytest

from tests import share_reference as R
from tests.test_gpu_share import Cache, _ops, _ws, i32

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


def test_the_most_requests_of_a_call():
    """16384 children of two prompts, grown by nothing, given back one half at a time; a compaction that lists them all."""
    ops = _ops()
    n, page = 16384, 8
    c = Cache(page, [20, 9], n + 2, 4, n + 3)
    ws = _ws(ops, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, ops.OP_COMPACT_PAGES, b=n, pages=c.total)
    r = c.rows
    lens = [(20, 17, 8)[i % 3] if i % 5 else 9 for i in range(n)]
    c.fork(ws, [r[0] if i % 5 else r[1] for i in range(n)], r[2:], lens)
    assert ws.last_error() == 0
    c.same()
    c.release(ws, r[2:n // 2], lens[:n // 2 - 2])
    assert ws.last_error() == 0
    c.same()
    rows, held = r[:2] + r[n // 2:], [20, 9] + lens[n // 2 - 2:]  # (fewer than a call takes)
    src, dst, moves = (i32([-5] * c.total) for _ in range(3))
    t = c.t
    ops.spec_compact_pages(len(rows), page, i32(rows), i32(held), 0, t["counts"], t["free"], t["n"], t["table"], None, t["counts"], t["free"], t["n"], t["table"], None, src, dst, moves, ws)
    assert ws.last_error() == 0
    want, c.n_free = R.compact(page, rows, held, 0, c.counts, c.free, c.n_free, c.table)
    c.same()
    assert moves.tolist()[0] == len(want) and list(zip(src.tolist(), dst.tolist()))[:len(want)] == want
    c.release(ws, rows, held)
    assert ws.last_error() == 0
    c.same()
    assert c.n_free == c.total
