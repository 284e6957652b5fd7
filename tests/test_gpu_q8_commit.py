"""Commits into the 8-bit cache at the ends of what a page may hold."""
import math

import pytest
import torch

from tests.test_gpu_q8 import _gen, pools_of, run_commit, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held", [1, 2, 15, 16, 126, 127, 247, 248, 253, 254])
def test_pages_held_at_every_end_of_the_scales(held):
    """New rows of ordinary size, of the type's largest, infs and NaNs, behind rows of a page whose scale byte is `held`."""
    page, D, Hkv = 16, 64, 2
    big = torch.finfo(torch.bfloat16).max
    rows_t = torch.zeros(6, Hkv, D)
    for i, row in enumerate([[big, -big, 1.0], [1.0, -3.0, 448.0], [math.inf, -math.inf, 2.0], [math.nan, 5.0], [2.0 ** 120, 2.0 ** 119, 1e30], [0.0, 1e-30]]):
        rows_t[i, :, :len(row)] = torch.tensor(row)
    fresh = torch.stack([rows_t, -rows_t * 0.5], dim=1)[None].bfloat16()
    lens, src = [5, 1, 15, 9, 7, 3], [[i] for i in range(6)]
    table, rows, pages = tables([x + 1 for x in lens], page, _gen(1))
    pools = pools_of(1, pages, Hkv, page, D, _gen(2))
    pools[1][0].fill_(held), pools[3][0].fill_(held)
    run_commit(page, D, Hkv, 1, lens, src, 6, fresh, pools, table, rows)
