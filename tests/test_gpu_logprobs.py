"""Token log probabilities, entropy and top alternatives on the GPU against the
64-bit form.

Bars.  Ids: equal (ties to the lowest index).  With y = (x - max) / T: every term
of the sum carries the rounding of c = log2(e) / T (two roundings, 2^-23), of
the FMA's result (2^-24 of y log2 e) and ex2.approx (2^-22), the sum itself at
most 2^-20 (per-thread sums of at most 512 terms, then trees), the logarithm
2^-22 of log2 s; so with R the largest |y| that still weighs in the sum (2^-30 of
it: R <= 21 + ln V, 33 here) ln s is off by at most R 2^-22 + 2^-20 < 1e-5, a log
probability by that and 2^-22 of itself, an entropy by twice that."""
import math

import pytest
import torch

from tests import q8_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAR = 1e-5


def _ops():
    from accept_select_top_gb300 import ops
    return ops


def run(n, W, logits, index, tokens, temps, k, entropy=True, ws=None, stream=None):
    ops = _ops()
    b = tokens.shape[0]
    V = logits.shape[1]
    dev = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    lp = torch.full((b, W), 7.0, device=DEV)
    ent = torch.full((b, W), 7.0, device=DEV) if entropy else None
    ids = torch.full((b, W, k), 7, dtype=torch.int32, device=DEV) if k else None
    top = torch.full((b, W, k), 7.0, device=DEV) if k else None
    ws = ws or ops.Workspace(ops.spec_workspace_size(ops.OP_TOKEN_LOGPROBS, b, W, max(1, k), V))
    ops.spec_token_logprobs(b, n, W, dev(logits), dev(index), dev(tokens), dev(temps), k, lp, ent, ids, top, ws, stream)
    return lp, ent, ids, top, ws


def check(n, W, logits, index, tokens, temps, k):
    lp, ent, ids, top, ws = run(n, W, logits, index, tokens, temps, k)
    assert ws.last_error() == 0
    wlp, went, wids, wtop = R.logprobs(n, W, logits, index, tokens, temps, k)
    if k:
        assert torch.equal(ids.cpu().long(), wids)
        near(top, wtop, 1)
    near(lp, wlp, 1)
    near(ent, went, 2)


def near(got, want, times):
    got = got.cpu().double()
    assert torch.equal(got == -math.inf, want == -math.inf) and torch.equal(got == math.inf, want == math.inf)
    fin = torch.isfinite(want)
    assert torch.isfinite(got[fin]).all()
    off = (got[fin] - want[fin]).abs() - 2.0 ** -22 * want[fin].abs()
    assert off.numel() == 0 or off.max() <= times * BAR, float(off.max())


def logits_of(rows, V, dtype, seed, std=2.0):
    return (torch.randn(rows, V, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def tokens_of(b, W, V, seed):
    return torch.randint(0, V, (b, W), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b, n, V, k", [
    (1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 31, 5), (1, 2, 33, 32), (3, 2, 255, 20), (2, 2, 1000, 8), (1, 1, 4099, 32), (2, 2, 32001, 5), (1, 4, 50257, 0), (5, 3, 8192, 1),
    (1, 1, 131072, 20), (1, 1, 200003, 10)])
def test_sizes(dtype, b, n, V, k):
    check(n, n, logits_of(b * n, V, dtype, V), None, tokens_of(b, n, V, 1), None, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_enough_for_a_cta_each(dtype):
    check(8, 8, logits_of(1200, 5003, dtype, 2), None, tokens_of(150, 8, 5003, 3), torch.rand(150, generator=torch.Generator().manual_seed(4)) + 0.3, 6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2000, 40000])
def test_accepted_rows_and_temperatures(dtype, V):
    b, n, W = 5, 6, 4
    index = torch.tensor([[0, 2, 5, -1], [6, -1, -1, -1], [12, 13, 14, 15], [23, 18, 18, 20], [-1, -1, -1, -1]], dtype=torch.int32)
    tokens = torch.where(index >= 0, tokens_of(b, W, V, 5), -1)
    tokens[2, 1] = -1  # a row without an asked token still has entropy and alternatives
    temps = torch.tensor([1.0, 0.0, -1.0, 0.05, 3.0])
    check(n, W, logits_of(b * n, V, dtype, 6, 0.5), index, tokens, temps, 3)


@pytest.mark.parametrize("V", [700, 9001, 70000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_and_tied_rows(V, dtype):
    """Masks down to fewer tokens than alternatives, everything masked, the type's lowest value, constant rows, ties across the cut, both zeros."""
    x = logits_of(12, V, dtype, 8)
    x[0, 3:] = -math.inf
    x[1] = -math.inf
    x[2] = -math.inf
    x[2, V - 1] = 2.0
    x[3] = 1.5
    x[4] = 0.0
    x[4, 1::2] = -0.0
    x[5, V // 2:] = torch.finfo(dtype).min
    x[6] = torch.finfo(dtype).min
    x[7] = torch.round(x[7].float()).to(dtype)
    x[8, :] = -math.inf
    x[8, V // 3:V // 3 + 40] = 4.0
    x[9, ::2] = math.nan
    x[10] = math.nan
    x[11, V - 30:] = 30.0
    tokens = torch.tensor([[0, 5, V - 1, 7], [1, 2, V - 1, 3], [V // 3, 0, 4, V - 1]], dtype=torch.int32)
    check(4, 4, x, None, tokens, None, 20)


def test_positive_infinity_gives_nan():
    x = logits_of(2, 3000, torch.float32, 9)
    x[0, 17] = math.inf
    lp, ent, ids, top, ws = run(2, 2, x, None, tokens_of(1, 2, 3000, 1), None, 4)
    assert torch.isnan(lp[0, 0]) and torch.isnan(ent[0, 0]) and torch.isnan(top[0, 0]).all() and ids[0, 0, 0] == 17
    assert torch.isfinite(lp[0, 1]) and torch.isfinite(ent[0, 1]) and torch.isfinite(top[0, 1]).all()


def test_confident_and_flat_rows():
    """Entropy near 0 (one token far ahead) and near ln V."""
    x = torch.zeros(4, 60000)
    x[0, 5] = 40.0
    x[1, 5] = 16.0
    x[2] = torch.linspace(0, 1e-3, 60000)
    x[3, :2] = 100.0
    check(4, 4, x, None, torch.tensor([[5, 6, 7, 1]], dtype=torch.int32), None, 3)


def test_offset_and_unaligned_logits():
    """Logits that start off a 16-byte boundary."""
    ops = _ops()
    base = torch.randn(1 + 3 * 5001, device=DEV)
    x = base[1:].view(3, 5001)
    tok = tokens_of(1, 3, 5001, 2)
    lp, ent, ids, top, ws = run(3, 3, x, None, tok, None, 5)
    assert ws.last_error() == 0
    wlp, went, wids, wtop = R.logprobs(3, 3, x.cpu(), None, tok, None, 5)
    assert torch.equal(ids.cpu().long(), wids)
    near(lp, wlp, 1)
    near(top, wtop, 1)


def test_bad_rows_and_tokens():
    ops = _ops()
    x = logits_of(4, 3000, torch.float32, 10)
    index = torch.tensor([[0, 4], [3, -2]], dtype=torch.int32)
    lp, ent, ids, top, ws = run(2, 2, x, index, torch.tensor([[1, 1], [3000, 1]], dtype=torch.int32), None, 2)
    assert ws.last_error() == ops.DEV_INDEX
    assert lp[0, 1] == 0 and ids[0, 1].tolist() == [-1, -1] and lp[1, 0] == 0 and lp[1, 1] == 0 and lp[0, 0] < 0 and ent[1, 0] > 0
    lp2, *_ , ws = run(2, 2, x, index, torch.tensor([[1, 1], [5, 1]], dtype=torch.int32), None, 0, entropy=False, ws=ws)
    assert ws.last_error() == ops.DEV_INDEX and lp2[0, 0] == lp[0, 0] and lp2[1, 0] < 0


def test_captured_and_repeated():
    ops = _ops()
    x, tok = logits_of(6, 70001, torch.bfloat16, 11).to(DEV), tokens_of(2, 3, 70001, 1)
    lp, ent, ids, top, ws = run(3, 3, x, None, tok, None, 9)
    got = [torch.empty_like(t) for t in (lp, ent, ids, top)]
    tok = tok.to(DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.spec_token_logprobs(2, 3, 3, x, None, tok, None, 9, *got, ws)
    for _ in range(3):
        for t in got:
            t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (lp, ent, ids, top)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run(3, 3, x, None, tok, None, 9, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again[:4], (lp, ent, ids, top)))


@pytest.mark.parametrize("V", [1 << 20, (1 << 20) - 5])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_largest_vocabulary(V, dtype):
    """A row in chunks of as many batches as a chunk may have."""
    gen = torch.Generator().manual_seed(V)
    logits = (4 * torch.randn(2, V, generator=gen)).to(dtype)
    tokens = torch.tensor([[V - 1, 17]], dtype=torch.int32)
    check(2, 2, logits, None, tokens, None, 32)


@pytest.mark.parametrize("b, V", [(1, 5000), (1, 9000), (3, 20000), (40, 70000), (120, 20000), (230, 9001)])
def test_rows_in_clusters_of_every_size(b, V):
    """Rows cut into 1, 2, 4 and 8 chunks; some rows left out, in the middle of others."""
    gen = torch.Generator().manual_seed(b)
    n, W = 3, 4
    logits = torch.randn(b * n, V, generator=gen).bfloat16()
    index = torch.randint(0, b * n, (b, W), generator=gen).to(torch.int32)
    index[torch.rand(b, W, generator=gen) < 0.3] = -1
    tokens = torch.randint(0, V, (b, W), generator=gen).to(torch.int32)
    check(n, W, logits, index, tokens, None, 7)


@pytest.mark.parametrize("V", [1000, 30000])
def test_temperatures_are_the_output_rows(V):
    """Rows of other requests: the temperature is that of the request that asks."""
    b, n, W = 4, 3, 4
    x = logits_of(b * n, V, torch.float32, 21)
    index = torch.tensor([[9, 0, 3, -1], [1, 4, 11, 6], [5, 5, -1, -1], [0, 2, 8, 10]], dtype=torch.int32)
    tokens = torch.where(index >= 0, tokens_of(b, W, V, 22), -1)
    temps = torch.tensor([0.5, 1.0, 0.0, 2.5])
    lp, ent, ids, top, ws = run(n, W, x, index, tokens, temps, 6)
    assert ws.last_error() == 0
    for r in range(b):
        # the request's rows gathered, as a batch of its own
        at = index[r][index[r] >= 0].long()
        m = at.numel()
        want = R.logprobs(m, m, x[at], None, tokens[r:r + 1, :m], temps[r:r + 1], 6)
        assert torch.equal(ids[r, :m].cpu().long(), want[2][0])
        near(lp[r, :m], want[0][0], 1)
        near(ent[r, :m], want[1][0], 2)
        near(top[r, :m], want[3][0], 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 1000, 20000])
def test_tokens_masked_by_the_lowest_value(V, dtype):
    """Fewer allowed tokens than alternatives, and asked tokens under the mask: their log probability is finite where
    fp32 holds it."""
    x = logits_of(4, V, dtype, 31)
    low = torch.finfo(dtype).min
    x[0, 3:] = low
    x[1, : V - 1] = low
    x[2, V // 2:] = low / 2
    x[3, 5:] = low
    x[3, 5:20] = -1e30
    tokens = torch.tensor([[5, 0, V - 1, V - 1]], dtype=torch.int32)
    for T in (1.0, 0.75, 2.0):
        lp, ent, ids, top, ws = run(4, 4, x, None, tokens, torch.tensor([T]), 20)
        assert ws.last_error() == 0
        wlp, went, wids, wtop = R.logprobs(4, 4, x, None, tokens, torch.tensor([T]), 20)
        past = lambda w: torch.where(w < -torch.finfo(torch.float32).max, -math.inf, w)  # noqa: E731
        assert torch.equal(ids.cpu().long(), wids)
        near(lp, past(wlp), 1)
        near(top, past(wtop), 1)
        near(ent, went, 2)


@pytest.mark.parametrize("V", [50, 3000, 30000])
@pytest.mark.parametrize("T", [1e-45, 1e-39, 4e-39, 1e-38, 1e-30, 1e-6, 1e30, 3e38, math.inf])
def test_temperatures_of_every_size(V, T):
    """Down to subnormal ones, whose inverse is past fp32's range (all the weight on the maximum), and up to inf (all equal)."""
    x = logits_of(3, V, torch.float32, 41)
    x[1, 7:9] = 20.0  # two maxima
    tokens = torch.tensor([[int(x[0].argmax()), 8, 0]], dtype=torch.int32)
    temps = torch.tensor([T], dtype=torch.float32)
    lp, ent, ids, top, ws = run(3, 3, x, None, tokens, temps, 5)
    assert ws.last_error() == 0
    wlp, went, wids, wtop = R.logprobs(3, 3, x, None, tokens, temps, 5)
    past = lambda w: torch.where(w < -torch.finfo(torch.float32).max, -math.inf, w)  # noqa: E731
    assert torch.equal(ids.cpu().long(), wids)
    near(lp, past(wlp), 1)
    near(top, past(wtop), 1)
    near(ent, went, 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_widest_rows_a_request(dtype):
    """65 output rows a request of 64 nodes, 32 alternatives, nodes asked for more than once."""
    b, n, W, V = 3, 64, 65, 5000
    gen = torch.Generator().manual_seed(51)
    index = torch.randint(0, n, (b, W), generator=gen).to(torch.int32) + torch.arange(b, dtype=torch.int32)[:, None] * n
    index[1, 40:] = -1
    check(n, W, logits_of(b * n, V, dtype, 52), index, tokens_of(b, W, V, 53), torch.tensor([1.0, 0.4, 0.0]), 32)
