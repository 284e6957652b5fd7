"""NaN in what a request sees comes out of the one-token attention, whichever kernels, clusters and joins a call takes:
a query row of NaN, a key of NaN that is all that a part of a request's tokens has, a value of NaN under a weight that fp32
does not hold.  What does not see it is held to the bar of test_gpu_decode."""
import math

import pytest
import torch

from tests.test_gpu_decode import Case

pytestmark = pytest.mark.gpu

# (groups, requests alone, max_seq_len, the request with the NaN)
CALLS = {
    "cluster of eight": ([], [1001], None, 0),
    "cluster of eight, one tile": ([], [5], None, 0),
    "cluster of four": ([], [300] * 12, None, 5),
    "cluster of one": ([], [90 + r for r in range(60)], None, 33),
    "a unit of one CTA": ([], [40] * 200, None, 7),
    "units cut between CTAs": ([], [9000] + [40] * 99, None, 0),
    "one request over all SMs": ([], [20000], 40000, 0),
    "grouped": ([(640, [700, 650]), (64, [70] * 3)], [30], None, 1),
    "grouped, without a token of its own": ([(640, [640, 650])], [], None, 0),
    "grouped, many rows": ([(640, [700 + r for r in range(12)])], [300], None, 3),
    "grouped, more than 128 rows": ([(2048, [2100 + r for r in range(40)])], [], None, 37),
    "grouped, cut among many rows": ([(20000, [20100 + r for r in range(10)])], [], None, 0),
}


def _others(c, got, clean, hit):
    """The rows without NaN against the 64-bit form (`hit`: those with, taken from a run without)."""
    out, lse = (torch.where(hit[..., None] if x.dim() == 3 else hit, y, x) for x, y in zip(got, clean))
    c.check(out, lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", CALLS)
def test_a_query_of_nan(name, D):
    groups, alone, most, r = CALLS[name]
    c = Case(groups, alone, D=D, seed=3)
    clean = c.call(most=most)
    q = c.q.clone()
    c.q = q.clone()
    c.q[r, 5, 3] = math.nan
    got = c.call(most=most)
    hit = torch.zeros(c.b, c.Hq, dtype=torch.bool, device=q.device)
    hit[r, 5] = True
    assert got[0][hit].isnan().all() and got[1][hit].isnan().all()
    c.q = q
    _others(c, got, clean, hit)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", CALLS)
def test_a_last_key_of_nan(name, D):
    """The last token's key: where the tokens lie in parts, it may be the only one of its part."""
    groups, alone, most, r = CALLS[name]
    c = Case(groups, alone, D=D, seed=4)
    clean = c.call(most=most)
    at = c.slots_of(r)[-1]
    seen = torch.zeros(c.b, c.Hq, dtype=torch.bool, device=c.q.device)
    for x in range(c.b):
        seen[x, :c.Hq // c.Hkv] = bool((c.slots_of(x) == at).any())
    keep = c.k[at, 0].clone()
    c.k[at, 0, 1] = math.nan
    got = c.call(most=most)
    assert got[0][seen].isnan().all() and got[1][seen].isnan().all()
    c.k[at, 0] = keep
    _others(c, got, clean, seen)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("groups, alone", [
    ([(64, [65, 70])], []), ([(640, [641] + [700] * 11)], []), ([(2048, [2049] + [2100] * 39)], []), ([], [7 * 64 + 1]), ([], [7 * 128 + 1]), ([], [64 + 1] * 60)])
def test_one_key_of_its_own(groups, alone, D):
    """A member of a group with one token of its own, a CTA of a cluster with one: its key is all that the part has."""
    c = Case(groups, alone, D=D, seed=5)
    at = c.slots_of(0)[-1]
    c.k[at, 1] = math.nan
    out, lse = c.call()
    half = c.Hq // c.Hkv
    assert out[0, half:].isnan().all() and lse[0, half:].isnan().all()
    assert torch.isfinite(out[0, :half].float()).all() and torch.isfinite(lse[0, :half]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("groups, alone", [
    ([], [1001]), ([], [64, 9000] + [40] * 99), ([(64, [200, 90])], []), ([(640, [900] * 12)], []), ([], [7 * 64 + 1]), ([], [7 * 128 + 1]), ([(64, [65, 70])], []), ([(640, [641] + [700] * 11)], [])])
def test_a_value_of_nan_under_a_small_weight(groups, alone, D):
    """The last key's scores lie 300 below the others' (a weight of 2^-432), and it may be all that its part has: in 64 bits its value of NaN makes its column NaN."""
    c = Case(groups, alone, D=D, seed=6)
    r = 1 if len(alone) > 1 else 0
    at = c.slots_of(r)[-1]
    c.q[r, :, 0] = 8.0
    c.k[c.slots_of(r), :, 0] = 0.0
    c.k[at, :, 0] = -300.0 / 8 / c.scale
    clean = c.call()
    c.v[at, 0, 9] = math.nan
    out, lse = c.call()
    half = c.Hq // c.Hkv
    assert out[r, :half, 9].isnan().all()
    same = torch.ones(c.b, c.Hq, D, dtype=torch.bool, device=out.device)
    same[r, :half, 9] = False
    assert torch.equal(out[same], clean[0][same]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("groups, alone", [
    ([], [1001]), ([], [64, 9000] + [40] * 99), ([], [7 * 64 + 1]), ([], [7 * 128 + 1]), ([(64, [65, 70])], []), ([(640, [641] + [700] * 11)], []), ([(2048, [2049] + [2100] * 39)], [])])
def test_a_value_of_nan_under_no_weight(groups, alone, D):
    """The last key's scores are -inf: a weight of 0, and 0 times NaN is NaN, in 64 bits too.  A finite value there is without effect."""
    c = Case(groups, alone, D=D, seed=7)
    r = 1 if len(alone) > 1 else 0
    at = c.slots_of(r)[-1]
    c.q[r, :, 0] = 8.0
    c.k[at, :, 0] = -math.inf
    clean = c.call()
    c.check(*clean)
    c.v[at, 0, 9] = math.nan
    out, lse = c.call()
    half = c.Hq // c.Hkv
    assert out[r, :half, 9].isnan().all()
    same = torch.ones(c.b, c.Hq, D, dtype=torch.bool, device=out.device)
    same[r, :half, 9] = False
    assert torch.equal(out[same], clean[0][same]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("groups, alone", [([], [449]), ([], [64, 9000] + [40] * 99), ([(64, [65, 70])], []), ([(640, [641] + [700] * 11)], [])])
def test_scores_of_minus_infinity_only(groups, alone, D):
    """No key of one request has any weight: out 0 and lse -inf, as without a token."""
    c = Case(groups, alone, D=D, seed=7)
    r = 1 if len(alone) > 1 else 0
    c.q[r, :, 0] = -8.0
    others = c.call()
    keep = c.k.clone()
    c.k[c.slots_of(r), :, 0] = math.inf
    out, lse = c.call()
    assert (out[r] == 0).all() and (lse[r] == -math.inf).all()
    c.k = keep
    if not groups:
        rest = [x for x in range(c.b) if x != r]
        assert torch.equal(out[rest], others[0][rest]) and torch.equal(lse[rest], others[1][rest])
