"""Page sharing calls without a request (an idle batch), and what is called behind them."""
import pytest
import torch

from tests.test_gpu_share import _ops, _pools, _ws, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
def test_an_idle_call_leaves_nothing_to_copy(in_place):
    """Calls without a request, whose lists and counts a step before has filled: the copy behind them copies nothing."""
    ops = _ops()
    pools = _pools(2, 6, 16, 2, 64, False)
    keep = [[x.clone() for x in p] for p in pools[:2]]
    ws = _ws(ops, ops.OP_FORK_PAGES, ops.OP_COMPACT_PAGES, b=1, pages=6)
    none, table = i32([]), i32([[0, 1]])
    counts, free, n = i32([1, 0, 0, 0, 0, 0]), i32([3, 4]), i32([2])
    src, dst, count = i32([0, 1]), i32([2, 5]), i32([2])
    left = n if in_place else i32([-9])
    ops.spec_fork_pages(0, 16, none, none, none, counts, free, n, table, None, src, dst, count, left, ws)
    assert count.tolist() == [0] and left.tolist() == [2] and n.tolist() == [2]
    ops.spec_copy_pages(16, *pools, src, dst, count, ws)
    count.fill_(2)
    new = (counts, free) if in_place else (i32([-9] * 6), i32([-9] * 2))
    ops.spec_compact_pages(0, 16, none, none, 0, counts, free, n, table, None, *new, left, table, None, src, dst, count, ws)
    assert count.tolist() == [0] and left.tolist() == [2]
    assert new[0].tolist() == [1, 0, 0, 0, 0, 0] and new[1].tolist() == [3, 4]
    ops.spec_copy_pages(16, *pools, src, dst, count, ws)
    assert ws.last_error() == 0
    for p, q in zip(pools[:2], keep):
        for x, y in zip(p, q):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_an_idle_call_on_another_stream():
    ops = _ops()
    ws = _ws(ops, ops.OP_FORK_PAGES, b=1, pages=6)
    none, src, dst, count, n, left = i32([]), i32([0]), i32([1]), i32([1]), i32([2]), i32([-9])
    table, counts, free = i32([[0, 1]]), i32([0] * 6), i32([3, 4])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ops.spec_fork_pages(0, 16, none, none, none, counts, free, n, table, None, src, dst, count, left, ws)
    g.replay()
    torch.cuda.synchronize()
    assert count.tolist() == [0] and left.tolist() == [2]
    count.fill_(1)
    torch.cuda.synchronize()
    ops.spec_fork_pages(0, 16, none, none, none, counts, free, n, table, None, src, dst, count, left, ws, stream=s)
    s.synchronize()
    assert count.tolist() == [0]
