"""One-token attention over pools of more than 2^32 bytes, whose last pages the requests hold, in each of its kernels."""
import pytest
import torch

from tests.test_gpu_decode import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("groups, alone, most", [
    ([], [500], None), ([], [1500], 40000), ([], [3000] + [70] * 99, None), ([(640, [700, 650, 641])], [300], None), ([(640, [700 + r for r in range(20)])], [300], None),
    ([(1280, [1300 + r for r in range(50)])], [], None)])
def test_pages_behind_four_gigabytes(groups, alone, most, page, D):
    c = Case(groups, alone, page=page, Hq=32, Hkv=8, D=D, seed=page)
    more = ((4 << 30) + (1 << 20)) // (8 * D * 2 * page)  # pages ahead of the requests'
    for x in ("k", "v"):
        pool = torch.empty(more * page + c.slots, 8, D, dtype=torch.bfloat16, device="cuda")
        pool[more * page:] = getattr(c, x)
        setattr(c, x, pool)
    c.table = torch.where(c.table >= 0, c.table + more, c.table)
    c.check(*c.call(most=most))
