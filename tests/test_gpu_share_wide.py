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
