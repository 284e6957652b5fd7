"""The release that goes over all SMs (table rows that may hold many pages): its counters, and calls at the same time."""
import pytest
import torch

from tests import share_reference as R
from tests.test_gpu_share import Cache, _ops, _ws, i32

pytestmark = pytest.mark.gpu

HEADER = 256  # bytes of a workspace before its counters


def _counters(ws):
    return ws.tensor[HEADER:HEADER + 1024].view(torch.int32)


def test_a_wait_that_runs_out():
    """A count that lies so far back that the meetings' wait (2 s) runs out: the call is told and changes nothing, and the
    next one on the workspace finds its counters as they should be, as does a fork."""
    ops = _ops()
    page, fan, L = 4, 60, 20001
    c = Cache(page, [L], fan + 1, 5002, fan + 4)
    ws = _ws(ops, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, b=fan + 1, pages=c.total)
    r = c.rows
    lens = [L - i for i in range(fan)]
    c.fork(ws, [r[0]] * fan, r[1:], lens)
    assert ws.last_error() == 0
    _counters(ws)[0] = -1000
    before = {k: c.t[k].clone() for k in ("counts", "free", "n", "table")}
    ops.spec_release_pages(fan, page, i32(r[1:]), i32(lens), None, c.t["counts"], c.t["free"], c.t["n"], c.t["table"], c.t["n"], ws)
    assert ws.last_error() == ops.DEV_TIMEOUT
    assert all(torch.equal(c.t[k], before[k]) for k in before)
    assert (_counters(ws) == 0).all()
    c.release(ws, r[1:], lens)
    assert ws.last_error() == 0
    c.same()
    assert (_counters(ws) == 0).all()
    c.fork(ws, [r[0]] * 2, r[1:3], [L, 7])
    assert ws.last_error() == 0
    c.same()


def test_wide_releases_on_two_streams():
    """Two graphs with a cache and a workspace each, replayed at once: each fork gives its pages back over all SMs.  Then the same
    from two streams without graphs."""
    ops = _ops()
    page, fan, lens = 4, 60, (20001, 16003)
    runs = []
    for L in lens:
        c = Cache(page, [L], fan + 1, 5002, fan + 4, seed=L)
        r, t = c.rows, c.t
        d = dict(c=c, ws=_ws(ops, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, b=fan, pages=c.total), before=(list(c.free), list(c.counts), c.n_free), parents=i32([r[0]] * fan), children=i32(r[1:]),
                 lens=i32([L - 7 * i for i in range(fan)]), src=i32([-5] * fan), dst=i32([-5] * fan), n=i32([-5]), left=i32([-5]), stream=torch.cuda.Stream(), graph=torch.cuda.CUDAGraph())

        def step(d=d, t=t):
            ops.spec_fork_pages(fan, page, d["parents"], d["children"], d["lens"], t["counts"], t["free"], t["n"], t["table"], None, d["src"], d["dst"], d["n"], d["left"], d["ws"])
            ops.spec_release_pages(fan, page, d["children"], d["lens"], None, t["counts"], t["free"], d["left"], t["table"], d["left"], d["ws"])

        d["step"] = step
        torch.cuda.synchronize()
        with torch.cuda.graph(d["graph"], stream=d["stream"]):
            step()
        runs.append(d)

    def check():
        torch.cuda.synchronize()
        for d in runs:
            assert d["ws"].last_error() == 0
            assert (d["c"].t["free"].tolist(), d["c"].t["counts"].tolist(), d["left"].tolist()[0]) == d["before"]
            assert (_counters(d["ws"]) == 0).all()

    for what in ("graph", "step"):
        for _ in range(20):
            for d in runs:
                with torch.cuda.stream(d["stream"]):
                    d["graph"].replay() if what == "graph" else d["step"]()
        check()


@pytest.mark.parametrize("b, width", [(256, 8192), (17, 8192), (16, 8192)])
def test_few_pages_in_wide_tables(b, width):
    """Rows of a table as wide as a model's longest request, that hold and give up a few pages; some requests nothing."""
    ops = _ops()
    page = 16
    lens = [(37 * i) % 900 for i in range(b)]
    keep = [x - x % 5 * (x // 5) for x in lens]
    c = Cache(page, lens, b + 1, width, 5)
    ws = _ws(ops, ops.OP_RELEASE_PAGES, b=b, pages=c.total)
    c.release(ws, c.rows[:b], lens, keep)
    assert ws.last_error() == 0
    c.same()
    c.release(ws, c.rows[:b], [-(-k // page) * page for k in keep])
    assert ws.last_error() == 0
    c.same()
    assert c.n_free == c.total and sorted(c.free) == list(range(c.total))


def test_one_page_held_by_many():
    """Every occurrence of a wide call is the same few pages: given up by all holders, by all but one, and once too often."""
    ops = _ops()
    page, b, width = 1, 40, 4096
    total = 9
    ws = _ws(ops, ops.OP_RELEASE_PAGES, b=b, pages=total)
    for more, error in ((0, 0), (1, 0), (-1, ops.DEV_INVARIANT)):
        table = [[(r + i) % 3 for i in range(width)] for r in range(b)]
        held = [sum(row.count(p) for row in table) for p in range(3)]
        counts, free = [h - 1 + more for h in held] + [0] * 6, [8, 7] + [-1] * 7
        t = dict(counts=i32(counts), free=i32(free), n=i32([2]), table=i32(table))
        n = R.release(page, range(b), [width] * b, [0] * b, counts, free, 2, table)
        ops.spec_release_pages(b, page, i32(list(range(b))), i32([width] * b), None, t["counts"], t["free"], t["n"], t["table"], t["n"], ws)
        assert ws.last_error() == error
        assert t["counts"].tolist() == counts and t["free"].tolist() == free and t["n"].tolist() == [n]
