"""The one-token attention over shared pages on the host: every refusal that needs no device (CPU only)."""
import pytest

FAKE = 0x1000000  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    from accept_select_top_gb300 import ops
    return ops.LIB


def _decode(**change):
    a = dict(b=2, Hq=8, Hkv=2, D=128, ps=16, q=FAKE, q_ld=1024, k=FAKE, v=FAKE, slots=160, table=FAKE, rows=4, row_pages=8, idx=FAKE, lens=FAKE, most=100, groups=1, start=FAKE, shared=FAKE, scale=0.1,
             out=FAKE << 4, lse=None, ws=FAKE, ws_bytes=1 << 10, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change, code", [
    (dict(b=-1), -1), (dict(b=2049), -1), (dict(Hkv=3), -1), (dict(Hq=0), -1), (dict(D=96), -4), (dict(ps=0), -4), (dict(ps=24), -4), (dict(ps=256), -4), (dict(q_ld=1000), -1), (dict(q_ld=1028), -1),
    (dict(slots=15), -1), (dict(slots=1 << 31), -1), (dict(rows=0), -1), (dict(row_pages=0), -1), (dict(row_pages=1 << 27), -1), (dict(most=-1), -1), (dict(b=1, Hq=1, Hkv=1, most=(1 << 30) + 1), -1), (dict(b=1, Hq=1, Hkv=1, groups=0, most=1 << 30), -2), (dict(groups=-1), -1), (dict(groups=3), -1),
    (dict(b=2048, Hq=64, Hkv=64, most=1 << 30, q_ld=8192), -1), (dict(q=None), -1), (dict(q=FAKE + 2), -1), (dict(k=None), -1), (dict(v=FAKE + 8), -1), (dict(table=None), -1), (dict(idx=None), -1),
    (dict(lens=None), -1), (dict(start=None), -1), (dict(shared=None), -1), (dict(out=None), -1), (dict(out=FAKE + 2048), -1), (dict(lse=FAKE + 4), -1), (dict(lse=(FAKE << 4) + 64), -1), (dict(q=FAKE << 5, out=FAKE - 4080), -1), (dict(out=(FAKE << 4) + 4), -1), (dict(ws=None), -2),
    ({}, -2), (dict(ws_bytes=1 << 16), -2), (dict(b=0, groups=0, q=None), 0)])
def test_decode_refusals(lib, change, code):
    assert lib.spec_decode_attention(*_decode(**change)) == code


def test_workspace_grows_with_the_rows(lib):
    from accept_select_top_gb300 import ops
    size = lambda b, Hq: ops.spec_workspace_size(ops.OP_DECODE_ATTENTION, b, 1, 1, 1, Hq, 1, 100)  # noqa: E731
    assert size(64, 32) - size(32, 32) >= 2 * 32 * 32 * (512 + 8)
    assert size(8, 0) == 0
