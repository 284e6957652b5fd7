"""One-token attention over very many keys: values near the type's largest, whose sums fp32 holds only as long as the
weights are small enough."""
import math

import pytest
import torch

from tests.test_gpu_decode import _ops, i32

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_values_of_the_types_end_under_67_million_keys():
    """2^26 keys (two pages of 128, named over and over), every value 2^127.  Each CTA's first tile has scores of 0, all others
    scores 7.89 (as powers of two) above them, so that no CTA's reference moves and every weight is near the largest that a
    reference allows.

    P is rounded to bf16 (half a step 2^-8) and so is out (2^-8); a lane adds up 8 keys of each of its CTA's tiles in fp32, a
    matrix instruction 16: a rounding of 2^-24 each, in l and in O.  The scores: fp32 sums of 64 products, as d in test_gpu_decode."""
    ops = _ops()
    page, D, tiles = 128, 64, 1 << 19
    n = tiles * page
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 8.0
    k = torch.zeros(2 * page, 1, D, dtype=torch.bfloat16, device=DEV)
    k[page:, :, 0] = 5.46875
    v = torch.full((2 * page, 1, D), 2.0 ** 127, dtype=torch.bfloat16, device=DEV)
    ticks = 4 * tiles + 3  # four a tile, and the unit's end
    first = [(x * ticks // sms + 3) // 4 for x in range(sms)]
    table = torch.ones(1, tiles, dtype=torch.int32, device=DEV)
    table[0, first] = 0
    out, lse = torch.zeros(1, 1, D, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 1, device=DEV)
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_DECODE_ATTENTION, 1, 1, 1, 1, 1, 1, n))
    ops.spec_decode_attention(1, 1, 1, D, page, q, k, v, table, i32([0]), i32([n]), n, None, None, 0.125, out, lse, ws)
    assert ws.last_error() == 0
    high = 5.46875 * 8 * 0.125
    low_keys = len(set(first)) * page
    want = math.log(low_keys + (n - low_keys) * math.exp(high))
    adds = tiles / sms * 8
    d = 2.0 ** -19 + 2 * (D + 8) * 2.0 ** -24 * high + 2 * adds * 2.0 ** -24
    assert torch.isfinite(out).all()
    assert ((out.double() / 2.0 ** 127 - 1).abs() <= 2 * 2.0 ** -8 + d).all()
    assert abs(float(lse) - want) <= d + 2.0 ** -22 * want
