"""The shared tokens of many query rows (the tcgen05 kernel) with scales of either sign, scores that rise, pages out of range and a
group for every request."""
import pytest
import torch

from tests.test_gpu_decode import DEV, Case, _ops, i32

pytestmark = pytest.mark.gpu

MANY = [([(640, [700 + r for r in range(20)])], [300]), ([(2048, [2048 + r for r in range(50)])], []), ([(20000, [20010 + r for r in range(12)])], [])]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("groups, alone", MANY)
@pytest.mark.parametrize("scale", [-0.1, 0.3, 2.0, 0.0])
def test_scales(groups, alone, scale, D):
    c = Case(groups, alone, D=D, seed=8)
    c.scale = scale
    c.check(*c.call())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("groups, alone", MANY)
@pytest.mark.parametrize("sign", [1, -1])
def test_rising_and_falling_scores(groups, alone, sign, D):
    c = Case(groups, alone, D=D, seed=9)
    at = c.slots_of(0)
    c.q[..., 0] = 4.0
    c.k[at, :, 0] = (torch.linspace(-60, 60, at.numel(), device=DEV) * sign)[:, None].bfloat16()
    c.check(*c.call())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("groups, alone", MANY)
def test_pages_out_of_range(groups, alone, D):
    """Shared pages that do not exist: told, and their keys do not count for any member."""
    ops = _ops()
    c = Case(groups, alone, D=D, seed=10)
    gone = [0, 3, 17, c.shared[0] // c.page - 1]
    table = c.table.clone()
    for r in range(c.starts[1]):
        for i, p in enumerate(gone):
            table[c.rows[r], p] = (-1, 1 << 30, c.slots // c.page, -(1 << 31))[i]
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_DECODE_ATTENTION, c.b, 1, 1, 1, c.Hq, c.Hkv, max(c.lens)))
    out, lse = torch.full((c.b, c.Hq, D), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((c.b, c.Hq), 7.0, device=DEV)
    ops.spec_decode_attention(c.b, c.Hq, c.Hkv, D, c.page, c.q, c.k, c.v, table, i32(c.rows), i32(c.lens), max(c.lens), i32(c.starts), i32(c.shared), c.scale, out, lse, ws)
    assert ws.last_error() == ops.DEV_INDEX

    def keys(r):
        at, page = c.slots_of(r), torch.arange(c.lens[r], device=DEV) // c.page
        return at[~torch.isin(page, torch.tensor(gone, device=DEV))] if r < c.starts[1] else at

    c.check(out, lse, keys=keys)


def test_a_group_for_every_request():
    """As many groups as a call takes, and requests: the lists that the kernels keep are at their longest."""
    c = Case([(16 * (r % 4), [16 * (r % 4) + r % 23]) for r in range(2048)], Hq=4, Hkv=2, D=64, seed=11)
    c.check(*c.call())


def test_large_groups_among_many_small_ones():
    """The batch's mean is below what the tcgen05 kernel takes (its launch is left out), or above it, the groups being the same."""
    small = [(32, [40, 50])] * 60
    for big in (1, 4):
        c = Case([(1024, [1030 + r for r in range(64)])] * big + small, Hq=8, Hkv=2, seed=12)
        c.check(*c.call())
