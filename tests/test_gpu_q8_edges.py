"""The 8-bit cache's attention at the ends of what the header allows: rows that see history alone, the largest batch,
shared tables, NaN in a page far below the others."""
import math

import pytest
import torch

from tests.test_gpu_q8 import DEV, Att, _ops, bounds, i32  # noqa: F401
from tests.test_gpu_q8_load import Load
from tests.test_gpu_q8_values import check

pytestmark = pytest.mark.gpu


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, Hq, D", [(1, 8, 128), (1, 2, 64), (5, 8, 128), (33, 8, 64), (64, 8, 128), (64, 2, 64)])
def test_rows_that_see_history_alone(n, Hq, D):
    """Every mask empty: out is the history's, a request without history gives 0 and -inf."""
    lens = [1, 16, 0, 17, 200, 0]
    check(Att(len(lens), n, Hq, 2, D, 16, lens, masks=[0] * (n * len(lens)), seed=n).device())


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, Hq, Hkv", [(1, 2, 1), (3, 4, 2), (64, 1, 1)])
def test_the_largest_batch(n, Hq, Hkv):
    x = Load(n, Hq, Hkv, 64, 16, [(7 * i) % 50 for i in range(2048)], seed=n, bound=50)
    x.launch()
    assert x.ws.last_error() == 0
    x.check(x.reference())


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n", [1, 4, 64])
def test_requests_that_share_a_table_row(n):
    """Several samples of one prompt read one history, at lengths of their own."""
    a = Att(4, n, 8, 2, 128, 32, [300, 300, 300, 300], seed=n)
    a.rows = [a.rows[0]] * 4
    a.lens = [300, 299, 33, 0]
    check(a.device())


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, D", [(1, 128), (4, 64), (33, 128), (64, 128), (64, 64)])
@pytest.mark.parametrize("page", [1, 6])
def test_nan_in_a_page_far_below_the_others(n, D, page):
    """A page of zeros but for one NaN, as a commit leaves such rows."""
    a = Att(40, n, 8, 2, D, 16, [150] * 40, seed=11)
    for r in (3, 17):
        p = int(a.table[a.rows[r], page])
        a.vp[p], a.vs[p] = 0, 16
        a.vp[p, 1, 3, 9] = 0x7f
    _ops().spec_verify_attention_q8(*a.device())
    assert a.ws.last_error() == 0
    bad = torch.isnan(a.out.float()).view(40, n, 2, 4, D)
    want = torch.zeros_like(bad)
    want[3, :, 1, :, 9] = want[17, :, 1, :, 9] = True
    assert torch.equal(bad, want)


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n", [2, 64])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_a_node_of_nothing_but_infs_or_nans(n, value):
    """A V row without a finite element: the rows that see it take it, the others keep their results to the bars."""
    masks = [1 << i | 1 for _ in range(3) for i in range(n)]
    a = Att(3, n, 8, 2, 128, 16, [60, 0, 200], masks=masks, seed=5)
    clean = a.reference()
    for r in range(3):
        a.v[r * n + 1] = value
    _ops().spec_verify_attention_q8(*a.device())
    assert a.ws.last_error() == 0
    out = a.out.double().cpu()
    at = [r * n + 1 for r in range(3)]
    assert not torch.isfinite(out[at]).any()
    assert value != value or (out[at] == value).all()
    out[at] = clean[0][at]
    a.check(out, a.lse, clean)
