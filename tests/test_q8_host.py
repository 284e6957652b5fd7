"""The 8-bit cache and log-probability calls on the host: every refusal that
needs no device, the binding's checks, and the 64-bit forms the GPU tests
compare with, pinned against torch (CPU only)."""
import ctypes
import math

import pytest
import torch

from tests import q8_reference as R

FAKE = 0x1000000  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    from accept_select_top_gb300 import ops
    return ops.LIB


def _attention(**change):
    a = dict(b=2, n=4, Hq=8, Hkv=2, D=128, ps=16, q=FAKE, q_ld=1024, kn=FAKE, vn=FAKE, ld=256, kp=FAKE, vp=FAKE,
             ks=FAKE, vs=FAKE, pages=10, table=FAKE, rows=4, row_pages=8, idx=FAKE, lens=FAKE, most=100, mask=FAKE,
             scale=0.1, out=FAKE, lse=None, ws=FAKE, ws_bytes=0, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change, code", [
    (dict(b=-1), -1), (dict(b=2049), -1), (dict(n=0), -1), (dict(n=65), -1), (dict(Hkv=3), -1), (dict(D=96), -4),
    (dict(ps=1), -4), (dict(ps=48), -4), (dict(q_ld=1020), -1), (dict(q_ld=1000), -1), (dict(ld=128), -1),
    (dict(ld=257), -1), (dict(most=-1), -1), (dict(pages=0), -1), (dict(pages=1 << 30), -1), (dict(row_pages=0), -1),
    (dict(row_pages=1 << 27), -1), (dict(b=2048, most=1 << 30, row_pages=1 << 26), -1), (dict(q=None), -1),
    (dict(q=FAKE + 2), -1), (dict(kn=None), -1), (dict(vp=FAKE + 8), -1), (dict(out=FAKE + 4), -1), (dict(mask=None), -1),
    (dict(vs=None), -1), (dict(ws=None), -2), (dict(ws=FAKE + 16), -2), (dict(ws_bytes=1 << 20), -2), (dict(b=0, q=None), 0)])
def test_attention_refusals(lib, change, code):
    assert lib.spec_verify_attention_q8(*_attention(**change)) == code


def _commit(layers=1, hole=None, **change):
    arr = (ctypes.c_void_p * 128)(*[FAKE] * 128)
    odd = (ctypes.c_void_p * 128)(*[FAKE + 8] * 128)
    none = (ctypes.c_void_p * 128)()
    A = ctypes.addressof
    a = dict(b=2, Hkv=2, D=64, ps=32, layers=layers, kn=A(arr), vn=A(arr), num_rows=8, ld=128, kp=A(arr), vp=A(arr),
             ks=A(arr), vs=A(arr), pages=10, table=FAKE, rows=4, row_pages=8, idx=FAKE, lens=FAKE, index=FAKE, start=None,
             new=FAKE, width=4, after=FAKE, ws=FAKE, ws_bytes=256, stream=None)
    a.update(change)
    for key, what in (hole or {}).items():
        a[key] = A(odd) if what == "odd" else A(none)
    return list(a.values()), (arr, odd, none)


@pytest.mark.parametrize("change, hole, code", [
    (dict(b=-1), None, -1), (dict(Hkv=0), None, -1), (dict(D=32), None, -4), (dict(ps=24), None, -4),
    (dict(layers=0), None, -1), (dict(layers=129), None, -1), (dict(ld=120), None, -1), (dict(ld=132), None, -1),
    (dict(num_rows=0), None, -1), (dict(width=0), None, -1), (dict(index=None), None, -1), (dict(after=None), None, -1),
    (dict(b=1 << 30, width=1 << 20), None, -1), ({}, dict(kn="odd"), -1), ({}, dict(vp="odd"), -1),
    ({}, dict(ks="none"), -1), (dict(ws_bytes=255), None, -2), (dict(ws=None), None, -2), (dict(b=0), None, 0)])
def test_commit_refusals(lib, change, hole, code):
    args, keep = _commit(hole=hole, **change)
    assert lib.spec_commit_kv_q8(*args) == code


def _alloc(**change):
    a = dict(b=2, ps=16, idx=FAKE, lens=FAKE, new=FAKE, most=4, free=FAKE, cap=8, n_free=FAKE, pages=10, table=FAKE,
             rows=4, row_pages=8, slots=None, row_w=0, cu=FAKE, map=FAKE, pos=FAKE, slot_cap=8, left=FAKE, ws=FAKE,
             ws_bytes=4096, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change, code", [
    (dict(b=-1), -1), (dict(b=16385), -1), (dict(ps=0), -1), (dict(most=-1), -1), (dict(cap=-1), -1), (dict(slot_cap=-1), -1),
    (dict(pages=1 << 28), -1), (dict(row_pages=1 << 27), -1), (dict(slots=FAKE, row_w=0), -1), (dict(free=None), -1),
    (dict(map=None), -1), (dict(map=FAKE + 4), -1), (dict(pos=FAKE + 8), -1), (dict(left=None), -1), (dict(ws_bytes=512), -2),
    (dict(b=0), 0)])
def test_alloc_refusals(lib, change, code):
    assert lib.spec_alloc_slots(*_alloc(**change)) == code


def _logprobs(**change):
    a = dict(b=2, n=4, W=3, V=1000, dtype=0, logits=FAKE, index=FAKE, tokens=FAKE, temps=None, k=5, lp=FAKE, ent=None,
             ids=FAKE, top=FAKE, ws=FAKE, ws_bytes=0, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change, code", [
    (dict(b=-1), -1), (dict(n=65), -1), (dict(W=0), -1), (dict(W=66), -1), (dict(W=5, index=None), -1), (dict(k=-1), -1),
    (dict(k=33), -1), (dict(V=4, k=5), -1), (dict(dtype=2), -4), (dict(V=(1 << 22) + 1), -4), (dict(logits=None), -1),
    (dict(logits=FAKE + 2), -1), (dict(ids=None), -1), (dict(tokens=None), -1), (dict(ws=None), -2), (dict(ws_bytes=256), -2),
    (dict(b=0), 0)])
def test_logprobs_refusals(lib, change, code):
    assert lib.spec_token_logprobs(*_logprobs(**change)) == code


def test_workspace_sizes():
    from accept_select_top_gb300 import ops
    size = ops.spec_workspace_size
    assert size(ops.OP_ALLOC_SLOTS, 8, 1, 1, 1) >= 256 + 64
    assert size(ops.OP_COMMIT_KV_Q8, 8, 1, 1, 1) >= 256
    assert size(ops.OP_VERIFY_ATTENTION_Q8, 8, 4, 1, 1, 32, 8, 4096) > 1 << 20
    assert size(ops.OP_VERIFY_ATTENTION_Q8, 8, 4, 1, 1, 32, 5, 4096) == 0
    assert size(ops.OP_TOKEN_LOGPROBS, 8, 65, 32, 128256) > 0
    assert size(ops.OP_TOKEN_LOGPROBS, 8, 66, 32, 128256) == 0
    assert size(ops.OP_TOKEN_LOGPROBS, 8, 7, 33, 128256) == 0


def test_binding_refuses_wrong_tensors():
    """The checks come before any call into the library; CPU tensors are refused as such."""
    from accept_select_top_gb300 import ops
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ops.SpecError, match="expected torch.int32"):
        ops._in(i.long(), torch.int32, 4, 0, "x")
    with pytest.raises(ops.SpecError, match="CUDA"):
        ops._in(i, torch.int32, 4, 0, "x")
    with pytest.raises(ops.SpecError, match="elements"):
        ops._in(i, torch.int32, 5, -1, "x")
    with pytest.raises(ops.SpecError, match="contiguous"):
        ops._in(torch.zeros(8, dtype=torch.int32)[::2], torch.int32, 4, -1, "x")
    x = torch.zeros(6, 10, 64, dtype=torch.bfloat16)
    assert ops._rows_in(x[:, 2:4], 2, 64, 6, -1, "k") == (x.data_ptr() + 2 * 64 * 2, 640)
    for bad in (x[:, ::5], x[:, 2:4].float(), x[:, 2:5], x[:, 2:4, ::2], x[:3, 2:4]):
        with pytest.raises(ops.SpecError):
            ops._rows_in(bad, 2, 64, 6, -1, "k")
    p = torch.zeros(3, 2, 16, 64, dtype=torch.uint8)
    ops._pages_in(p, (2, 16, 64), -1, "pages")
    for bad in (p.float(), p[:, :, :8], p.transpose(1, 2)):
        with pytest.raises(ops.SpecError):
            ops._pages_in(bad, (2, 16, 64), -1, "pages")
    with pytest.raises(ops.SpecError):
        ops.LayerList([])
    with pytest.raises(ops.SpecError):
        ops.LayerList([p, p[:2]])


def test_reference_e4m3_is_torchs():
    byte = torch.arange(256, dtype=torch.uint8)
    want = byte.view(R.E4M3).double()
    got = R.e4m3_values(byte)
    assert torch.equal(got.nan_to_num(1e9), want.nan_to_num(1e9))
    x = torch.cat([torch.randn(4000, generator=torch.Generator().manual_seed(1)).double() * s for s in (1e-3, 0.05, 1, 60)])
    mid = (want[:126] + want[1:127]) / 2  # every tie
    x = torch.cat([x.clamp(-448, 448), mid, -mid, want[~want.isnan()]])
    assert torch.equal(R.e4m3_bytes(x), x.float().to(R.E4M3).view(torch.uint8))


def test_reference_scale():
    for a, e in ((448.0, 127), (449.0, 128), (224.0, 126), (1.75, 119), (1.0, 119), (1.7578125, 120), (0.0, 16), (1e-38, 16),
                 (float(torch.finfo(torch.bfloat16).max), 247)):
        assert R.need_exp(torch.tensor([a, -a / 2, math.inf, math.nan], dtype=torch.float64)) == e, a


def test_commit_refuses_rows_past_32_bits(lib):
    """A row number is kept in 32 bits: one past them would have been dropped without a word."""
    args, keep = _commit(num_rows=1 << 31)
    assert lib.spec_commit_kv_q8(*args) == -1


def test_logprobs_refuse_a_vocabulary_past_the_chunks(lib):
    assert lib.spec_token_logprobs(*_logprobs(V=(1 << 20) + 1)) == -4


@pytest.mark.parametrize("change, code", [
    (dict(after=FAKE, lens=FAKE), -1), (dict(after=FAKE + 4), -1), (dict(lens=FAKE + 8, after=FAKE + 12, idx=FAKE, new=FAKE), -1),
    (dict(after=FAKE + 0x1000, new=FAKE + 0x1000), -1), (dict(after=FAKE + 0x1000, idx=FAKE + 0x1000), -1),
    (dict(after=FAKE + 0x1000, index=None, start=FAKE + 0x1004), -1)])
def test_commit_refuses_lengths_in_place(lib, change, code):
    """Some of a request's CTAs would have read the new length for the old one."""
    args, keep = _commit(**change)
    assert lib.spec_commit_kv_q8(*args) == code


def test_workspaces_of_smaller_batches_keep_clear_of_the_counters():
    """The partial results of any batch size start behind the counters of every size that may share the workspace."""
    from accept_select_top_gb300 import ops
    # (an operation of no partial results: header and counters alone)
    sizes = [ops.spec_workspace_size(ops.OP_BUILD_TREE, b, 4, 1, 1000) for b in (1, 2, 600, 4096)]
    assert len(set(sizes)) == 1 and ops.spec_workspace_size(ops.OP_BUILD_TREE, 5000, 4, 1, 1000) > sizes[0]


def test_binding_refuses_a_workspace_of_another_device():
    from accept_select_top_gb300 import ops
    ws = ops.Workspace.__new__(ops.Workspace)
    ws.address, ws.device = FAKE, 1
    assert ops._workspace_in(ws, 1) == FAKE
    with pytest.raises(ops.SpecError, match="device 1"):
        ops._workspace_in(ws, 0)


@pytest.mark.parametrize("change", [
    dict(out=FAKE), dict(q=FAKE + 0x100000, kn=FAKE), dict(q=FAKE + 0x100000, kn=FAKE + 0x100000),
    # the last bytes of out and of strided rows
    dict(q=FAKE + 8 * 8 * 128 * 2 - 16, kn=FAKE + 0x100000, vn=FAKE + 0x100000),
    dict(q=FAKE + 0x100000, kn=FAKE + 0x100000, vn=FAKE - (7 * 2048 + 256) * 2 + 16, ld=2048)])
def test_attention_refuses_its_output_over_its_rows(lib, change):
    """out of 8 rows of 8 heads of 128: a warp writes it while others read the step's rows."""
    a = dict(ws_bytes=1 << 30)
    a.update(change)
    assert lib.spec_verify_attention_q8(*_attention(**a)) == -1


@pytest.mark.parametrize("change", [dict(cu=FAKE), dict(cu=FAKE - 8, lens=FAKE, new=FAKE + 0x100, idx=FAKE + 0x200),
                                    dict(cu=FAKE + 0x104, lens=FAKE, new=FAKE + 0x100, idx=FAKE + 0x200),
                                    dict(cu=FAKE + 0x204, lens=FAKE, new=FAKE + 0x100, idx=FAKE + 0x200)])
def test_alloc_refuses_offsets_over_its_lengths(lib, change):
    assert lib.spec_alloc_slots(*_alloc(ws_bytes=1 << 20, **change)) == -1
