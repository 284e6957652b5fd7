"""Calls that let requests share pages, on the host: every refusal that needs no device, and the plain forms that the
GPU tests compare with, pinned on small examples (CPU only)."""
import ctypes

import pytest
import torch

from tests import share_reference as R

FAKE = 0x1000000  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    from accept_select_top_gb300 import ops
    return ops.LIB


def _fork(**change):
    a = dict(b=2, ps=16, parents=FAKE, children=FAKE, lens=FAKE, counts=FAKE, pages=10, free=FAKE, cap=8, n_free=FAKE, table=FAKE, rows=4, row_pages=8, slots=None, row_w=0,
             src=FAKE + 128, dst=FAKE + 192, copies=FAKE + 64, left=FAKE + 256, ws=FAKE, ws_bytes=4096, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change, code", [
    (dict(b=-1), -1), (dict(b=16385), -1), (dict(ps=0), -1), (dict(pages=0), -1), (dict(pages=1 << 28), -1), (dict(pages=(1 << 27)), -1), (dict(row_pages=1 << 27), -1),
    (dict(row_pages=0), -1), (dict(b=16384, row_pages=1 << 17), -1), (dict(b=16384, row_pages=(1 << 16) + 1), -1), 
    (dict(ps=(1 << 20) + 1), -1), (dict(ps=1, pages=(1 << 30) + 1), -1), (dict(cap=(1 << 30) + 1), -1), (dict(cap=-1), -1), (dict(slots=FAKE, row_w=0), -1), (dict(parents=None), -1), (dict(children=None), -1),
    (dict(lens=None), -1), (dict(counts=None), -1), (dict(free=None), -1), (dict(n_free=None), -1), (dict(table=None), -1), (dict(src=None), -1), (dict(dst=None), -1),
    (dict(copies=None), -1), (dict(left=None), -1), (dict(copies=FAKE), -1), (dict(ws=None), -2), (dict(ws=FAKE + 16), -2), (dict(ws_bytes=512), -2), (dict(b=0, parents=None), 0)])
def test_fork_refusals(lib, change, code):
    assert lib.spec_fork_pages(*_fork(**change)) == code


@pytest.mark.parametrize("change", [dict(src=FAKE + 4), dict(dst=FAKE + 28), dict(src=FAKE + 196), dict(copies=FAKE + 196), dict(left=FAKE + 64), dict(left=FAKE + 4), dict(copies=FAKE + 132)])
def test_fork_refuses_outputs_over_what_it_reads(lib, change):
    assert lib.spec_fork_pages(*_fork(**change)) == -1


def _release(**change):
    a = dict(b=2, ps=16, idx=FAKE, lens=FAKE, keep=None, counts=FAKE, pages=10, free=FAKE, cap=8, n_free=FAKE, table=FAKE, rows=4, row_pages=8, left=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change, code", [
    (dict(b=-1), -1), (dict(b=16385), -1), (dict(ps=-3), -1), (dict(ps=1 << 21), -1), (dict(cap=(1 << 30) + 1), -1), (dict(b=4096, row_pages=1 << 19, ps=1), -1), (dict(pages=0), -1), (dict(rows=0), -1), (dict(cap=-1), -1), (dict(idx=None), -1), (dict(lens=None), -1), (dict(counts=None), -1),
    (dict(free=None), -1), (dict(n_free=None), -1), (dict(table=None), -1), (dict(left=None), -1), (dict(ws=None), -2), (dict(pages=1 << 20), -2), (dict(b=0, lens=None), 0)])
def test_release_refusals(lib, change, code):
    assert lib.spec_release_pages(*_release(**change)) == code


def _compact(**change):
    a = dict(b=2, ps=16, idx=FAKE, lens=FAKE, limit=0, counts=FAKE, pages=10, free=FAKE, cap=8, n_free=FAKE, table=FAKE, rows=4, row_pages=8, slots=None, row_w=0, new_counts=FAKE,
             new_free=FAKE, left=FAKE, new_table=FAKE, new_slots=None, src=FAKE, dst=FAKE, moves=FAKE + 64, ws=FAKE, ws_bytes=1 << 20, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change, code", [
    (dict(b=-1), -1), (dict(limit=-1), -1), (dict(ps=0), -1), (dict(ps=1 << 21), -1), (dict(cap=(1 << 30) + 1), -1), (dict(ps=1, pages=(1 << 30) + 1), -1), (dict(cap=-1), -1), (dict(slots=FAKE, row_w=64), -1), (dict(counts=None), -1), (dict(free=None), -1), (dict(new_counts=None), -1),
    (dict(new_free=None), -1), (dict(new_table=None), -1), (dict(src=None), -1), (dict(dst=None), -1), (dict(moves=None), -1), (dict(moves=FAKE), -1), (dict(left=None), -1),
    (dict(ws=None), -2), (dict(pages=1 << 22), -2), (dict(b=0, idx=None), 0)])
def test_compact_refusals(lib, change, code):
    assert lib.spec_compact_pages(*_compact(**change)) == code


@pytest.mark.parametrize("change", [dict(src=FAKE + 4140), dict(dst=FAKE), dict(moves=FAKE + 4096), dict(left=FAKE + 4), dict(new_free=FAKE + 4), dict(new_counts=FAKE + 4), dict(src=FAKE + 8196),
                                    dict(dst=FAKE + 12292), dict(left=FAKE + 64)])
def test_compact_refuses_outputs_over_what_it_reads(lib, change):
    apart = dict(idx=FAKE, lens=FAKE, src=FAKE + 4096, dst=FAKE + 4160, moves=FAKE + 64, left=FAKE + 128, free=FAKE + 8192, new_free=FAKE + 8192, counts=FAKE + 12288, new_counts=FAKE + 12288)
    assert lib.spec_compact_pages(*_compact(**{**apart, **change})) == -1


@pytest.mark.parametrize("change", [dict(new_counts=FAKE + 12288 + 36), dict(new_free=FAKE + 8192 + 28), dict(new_table=FAKE + 16384 + 124), dict(new_table=FAKE + 16384 - 124),
                                    dict(new_slots=FAKE + 20480 + 512)])
def test_compact_refuses_outputs_shifted_over_their_inputs(lib, change):
    same = dict(idx=FAKE, lens=FAKE, src=FAKE + 4096, dst=FAKE + 4160, moves=FAKE + 64, left=FAKE + 128, free=FAKE + 8192, new_free=FAKE + 8192, counts=FAKE + 12288, new_counts=FAKE + 12288,
                table=FAKE + 16384, new_table=FAKE + 16384, slots=FAKE + 20480, new_slots=FAKE + 20480, row_w=64)
    assert lib.spec_compact_pages(*_compact(**{**same, **change})) == -1


def _copy(hole=None, **change):
    arr = (ctypes.c_void_p * 128)(*[FAKE] * 128)
    odd = (ctypes.c_void_p * 128)(*[FAKE + 8] * 128)
    none = (ctypes.c_void_p * 128)()
    A = ctypes.addressof
    a = dict(layers=2, page_bytes=4096, scale_bytes=0, k=A(arr), v=A(arr), ks=None, vs=None, pages=10, src=FAKE, dst=FAKE, most=4, copies=FAKE, ws=FAKE, ws_bytes=256, stream=None)
    a.update(change)
    for key, what in (hole or {}).items():
        a[key] = A(odd) if what == "odd" else A(none)
    return list(a.values()), (arr, odd, none)


@pytest.mark.parametrize("change, hole, code", [
    (dict(layers=0), None, -1), (dict(layers=129), None, -1), (dict(page_bytes=0), None, -1), (dict(page_bytes=4104), None, -1), (dict(scale_bytes=-1), None, -1), (dict(pages=0), None, -1),
    (dict(pages=1 << 31), None, -1), (dict(most=-1), None, -1), (dict(k=None), None, -1), (dict(scale_bytes=8), None, -1), (dict(src=None), None, -1), (dict(copies=None), None, -1),
    ({}, dict(k="odd"), -1), ({}, dict(v="none"), -1), (dict(scale_bytes=8, ks=FAKE), dict(ks="none", vs="none"), -1), (dict(ws_bytes=255), None, -2), (dict(ws=None), None, -2),
    (dict(most=0, k=None), None, 0)])
def test_copy_refusals(lib, change, hole, code):
    args, keep = _copy(hole=hole, **change)
    assert lib.spec_copy_pages(*args) == code


def test_workspace_sizes(lib):
    from accept_select_top_gb300 import ops
    base = ops.spec_workspace_size(ops.OP_FORK_PAGES, 8, 1, 1, 1)
    assert ops.spec_workspace_size(ops.OP_RELEASE_PAGES, 8, 1, 1, 1000) >= base + 8000
    assert ops.spec_workspace_size(ops.OP_COMPACT_PAGES, 8, 1, 1, 1000) >= base + 3 * 125
    assert ops.spec_workspace_size(ops.OP_COPY_PAGES, 8, 1, 1, 1000) == base


def test_binding_refuses_cpu_tensors():
    """(a machine without a GPU has no current device: whatever is raised, nothing is launched)"""
    from accept_select_top_gb300 import ops
    if torch.cuda.is_available():
        pytest.skip("CPU only")
    x = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(Exception):
        ops.spec_release_pages(1, 16, x, x, None, x, x, x, x.view(2, 2), x, None)


def test_plain_fork_then_release():
    """A request of 40 tokens (pages 7, 3, 5 of 16) forked twice: the whole pages are held three times, each child has a page of its own."""
    counts, free = [0] * 10, [1, 2, 4, 6, 8]
    table = [[7, 3, 5], [-1] * 3, [-1] * 3]
    slots = [[-1] * 48 for _ in range(3)]
    copies, left = R.fork(16, [0, 0], [1, 2], [40, 40], counts, free, 5, table, slots)
    assert copies == [(5, 8), (5, 6)] and left == 3
    assert table == [[7, 3, 5], [7, 3, 8], [7, 3, 6]]
    assert counts == [0, 0, 0, 2, 0, 0, 0, 2, 0, 0]
    assert slots[1][15:18] == [127, 48, 49] and slots[2][32] == 96 and slots[1][40] == -1
    assert R.release(16, [1, 2], [40, 40], [0, 0], counts, free, left, table) == 5
    assert free == [1, 2, 4, 6, 8] and counts == [0] * 10
    assert R.release(16, [0], [40], [17], counts, free, 4, table) == 5 and free == [1, 2, 4, 6, 5]


def test_plain_release_by_all_holders():
    counts = [2, 0, 0, 1]
    free = [0] * 6
    table = [[0, 1], [0, 3], [0, 3]]
    assert R.release(4, [0, 1, 2], [8, 8, 8], [0, 0, 0], counts, free, 0, table) == 3
    assert free[:3] == [3, 1, 0] and counts == [0, 0, 0, 0]


def test_plain_compact():
    """Pages 1, 4, 6 and 7 of eight in use: 6 and 7 move to 0 and 2 (4 is at the limit, and goes to 0 first)."""
    counts = [0, 0, 0, 0, 1, 0, 3, 0]
    free = [3, 0, 5, 2, -9]
    table = [[6, 1], [4, 7]]
    moves, left = R.compact(16, [0, 1], [20, 32], 0, counts, free, 4, table)
    assert moves == [(4, 0), (6, 2), (7, 3)] and left == 4
    assert table == [[2, 1], [0, 3]] and free == [7, 6, 5, 4, -9] and counts == [1, 0, 3, 0, 0, 0, 0, 0]
    moves, left = R.compact(16, [0], [20], 6, [0] * 8, f := [3, 0, 5, 2], 4, t := [[7, 1]])
    assert moves == [(6, 0), (7, 2)] and t == [[2, 1]] and f == [7, 6, 5, 3]
