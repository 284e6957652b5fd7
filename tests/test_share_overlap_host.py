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


FORK = dict(parents=BASE, children=BASE + 256, lens=BASE + 512, counts=BASE + 1024, free=BASE + 2048, n_free=BASE + 2304, table=BASE + 4096, slots=BASE + 8192, src=BASE + 12288, dst=BASE + 12544,
            copies=BASE + 12800, left=BASE + 13056)
FORK_BYTES = dict(parents=8, children=8, lens=8, counts=40, free=32, n_free=4, table=128, slots=2048, src=8, dst=8, copies=4, left=4)
FORK_WRITTEN = ["counts", "table", "slots", "src", "dst", "copies", "left"]


def _fork(**change):
    """Two children, 10 pages of 16, a list of 8, tables of 4 rows of 8 pages and 128 slots."""
    a = dict(b=2, ps=16, parents=0, children=0, lens=0, counts=0, pages=10, free=0, cap=8, n_free=0, table=0, rows=4, row_pages=8, slots=0, row_w=128, src=0, dst=0, copies=0, left=0, ws=BASE + (1 << 20),
             ws_bytes=1 << 20, stream=None)
    a.update({**FORK, **change})
    return list(a.values())


def test_forks_are_accepted(lib):
    assert lib.spec_fork_pages(*_fork()) == LAUNCH
    assert lib.spec_fork_pages(*_fork(left=FORK["n_free"])) == LAUNCH
    assert lib.spec_fork_pages(*_fork(slots=None, row_w=0)) == LAUNCH
    assert lib.spec_fork_pages(*_fork(cap=0, free=None)) == LAUNCH
    assert lib.spec_fork_pages(*_fork(children=BASE, lens=BASE)) == LAUNCH  # (what is only read may be one array)
    assert lib.spec_fork_pages(*_fork(src=BASE + 8, dst=BASE + 16, copies=BASE + 24, left=BASE + 28)) == LAUNCH
    one = dict(ps=1, slots=FORK["table"], row_w=8)  # pages of one token: the page table is the slot table
    assert lib.spec_fork_pages(*_fork(**one)) == LAUNCH
    assert lib.spec_fork_pages(*_fork(**{**one, "row_w": 16})) == REFUSED
    assert lib.spec_fork_pages(*_fork(**{**one, "ps": 2})) == REFUSED


@pytest.mark.parametrize("written, other", [(w, o) for w in FORK_WRITTEN for o in FORK_BYTES if w != o])
def test_fork_refuses_overlaps(lib, written, other):
    for at in (FORK[other], FORK[other] + FORK_BYTES[other] - 4, FORK[other] - FORK_BYTES[written] + 4):
        want = LAUNCH if (written, other) == ("left", "n_free") else REFUSED
        assert lib.spec_fork_pages(*_fork(**{written: at})) == want


RELEASE = dict(idx=BASE, lens=BASE + 256, keep=BASE + 512, counts=BASE + 1024, free=BASE + 2048, n_free=BASE + 2304, table=BASE + 4096, left=BASE + 8192)
RELEASE_BYTES = dict(idx=8, lens=8, keep=8, counts=40, free=32, n_free=4, table=128, left=4)


def _release(**change):
    a = dict(b=2, ps=16, idx=0, lens=0, keep=0, counts=0, pages=10, free=0, cap=8, n_free=0, table=0, rows=4, row_pages=8, left=0, ws=BASE + (1 << 20), ws_bytes=1 << 20, stream=None)
    a.update({**RELEASE, **change})
    return list(a.values())


def test_releases_are_accepted(lib):
    assert lib.spec_release_pages(*_release()) == LAUNCH
    assert lib.spec_release_pages(*_release(left=RELEASE["n_free"])) == LAUNCH
    assert lib.spec_release_pages(*_release(keep=None)) == LAUNCH
    assert lib.spec_release_pages(*_release(keep=RELEASE["lens"])) == LAUNCH
    assert lib.spec_release_pages(*_release(cap=0, free=None)) == LAUNCH


@pytest.mark.parametrize("written, other", [(w, o) for w in ("counts", "free", "left") for o in RELEASE_BYTES if w != o])
def test_release_refuses_overlaps(lib, written, other):
    for at in (RELEASE[other], RELEASE[other] + RELEASE_BYTES[other] - 4, RELEASE[other] - RELEASE_BYTES[written] + 4):
        want = LAUNCH if (written, other) == ("left", "n_free") else REFUSED
        assert lib.spec_release_pages(*_release(**{written: at})) == want


DECODE = dict(q=BASE, table=BASE + 8192, idx=BASE + 16384, lens=BASE + 16640, start=BASE + 16896, shared=BASE + 17152, out=BASE + 20480, lse=BASE + 32768)
DECODE_BYTES = dict(q=2 * 2 * 1024, table=128, idx=8, lens=8, start=8, shared=4, out=2 * 8 * 128 * 2, lse=2 * 8 * 4)


def _decode(**change):
    a = dict(b=2, Hq=8, Hkv=2, D=128, ps=16, q=0, q_ld=1024, k=BASE + (1 << 20), v=BASE + (2 << 20), slots=160, table=0, rows=4, row_pages=8, idx=0, lens=0, most=100, groups=1, start=0, shared=0, scale=0.1,
             out=0, lse=0, ws=BASE + (16 << 20), ws_bytes=1 << 28, stream=None)
    a.update({**DECODE, **change})
    return list(a.values())


@pytest.mark.parametrize("written, other", [(w, o) for w in ("out", "lse") for o in DECODE_BYTES if w != o])
def test_decode_refuses_overlaps(lib, written, other):
    assert lib.spec_decode_attention(*_decode()) == LAUNCH
    step = 16 if written == "out" else 4  # (its alignment)
    for at in (DECODE[other], DECODE[other] - DECODE_BYTES[written] + step, DECODE[other] + (DECODE_BYTES[other] - 1) // step * step):
        assert lib.spec_decode_attention(*_decode(**{written: at})) == REFUSED
