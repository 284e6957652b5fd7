"""Page sharing and one-token attention, on the host: arrays that a call writes and that lie over what it reads or writes
besides are refused, whichever two they are (CPU only)."""
import pytest

BASE = 0x1000000  # an aligned address that no refused call reads
REFUSED, LAUNCH = -1, -3  # (without a GPU an accepted call ends where its kernel would start)


@pytest.fixture(scope="module")
def lib():
    from accept_select_top_gb300 import ops
    return ops.LIB


@pytest.fixture(autouse=True)
def _no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("CPU only: the accepted calls have no memory behind them")


def _compact(**change):
    """Two requests, 10 pages of 16, a list of 8, tables of 4 rows of 8 pages and 128 slots; in place."""
    a = dict(b=2, ps=16, idx=BASE, lens=BASE + 256, limit=0, counts=BASE + 512, pages=10, free=BASE + 768, cap=8, n_free=BASE + 1024, table=BASE + 2048, rows=4, row_pages=8, slots=BASE + 4096,
             row_w=128, new_counts=BASE + 512, new_free=BASE + 768, left=BASE + 1024, new_table=BASE + 2048, new_slots=BASE + 4096, src=BASE + 8192, dst=BASE + 8448, moves=BASE + 8704,
             ws=BASE + (1 << 20), ws_bytes=1 << 20, stream=None)
    a.update(change)
    return list(a.values())


APART = dict(new_counts=BASE + 16384, new_free=BASE + 16640, left=BASE + 16896, new_table=BASE + 20480, new_slots=BASE + 24576)
BYTES = dict(idx=8, lens=8, counts=40, free=32, n_free=4, table=128, slots=2048, new_counts=40, new_free=32, left=4, new_table=128, new_slots=2048, src=32, dst=32, moves=4)
OWN = dict(new_counts="counts", new_free="free", left="n_free", new_table="table", new_slots="slots")
WRITTEN = ["new_counts", "new_free", "left", "new_table", "new_slots", "src", "dst", "moves"]
PAIRS = [(w, o) for w in WRITTEN for o in BYTES if w != o and OWN.get(w) != o]


def test_compaction_in_place_and_apart_is_accepted(lib):
    assert lib.spec_compact_pages(*_compact()) == LAUNCH
    assert lib.spec_compact_pages(*_compact(**APART)) == LAUNCH
    for one in APART:
        assert lib.spec_compact_pages(*_compact(**{one: APART[one]})) == LAUNCH
    assert lib.spec_compact_pages(*_compact(slots=None, new_slots=None, row_w=0)) == LAUNCH
    # arrays side by side, without a byte between them
    assert lib.spec_compact_pages(*_compact(**{**APART, "new_counts": BASE + 8, "left": BASE + 48, "moves": BASE + 52, "new_free": BASE + 56})) == LAUNCH
    # pages of one token: the page table is the slot table
    one = dict(ps=1, slots=BASE + 2048, new_slots=BASE + 2048, row_w=8)
    assert lib.spec_compact_pages(*_compact(**one)) == LAUNCH
    assert lib.spec_compact_pages(*_compact(**{**one, "row_w": 16})) == REFUSED
    assert lib.spec_compact_pages(*_compact(**{**one, "ps": 2})) == REFUSED
    assert lib.spec_compact_pages(*_compact(**{**one, **APART, "new_slots": APART["new_table"]})) == LAUNCH
    assert lib.spec_compact_pages(*_compact(**{**one, **APART, "new_slots": BASE + 2048})) == REFUSED
    assert lib.spec_compact_pages(*_compact(cap=0, free=None, new_free=None, src=None, dst=None)) == LAUNCH


@pytest.mark.parametrize("written, other", PAIRS)
def test_compaction_refuses_overlaps(lib, written, other):
    where = {**dict(zip(["idx", "lens", "counts", "free", "n_free", "table", "slots", "src", "dst", "moves"],
                        [BASE, BASE + 256, BASE + 512, BASE + 768, BASE + 1024, BASE + 2048, BASE + 4096, BASE + 8192, BASE + 8448, BASE + 8704])), **APART}
    for at in (where[other], where[other] + BYTES[other] - 4, where[other] - BYTES[written] + 4):
        assert lib.spec_compact_pages(*_compact(**{**APART, written: at})) == REFUSED
