"""The 8-bit paged cache on the GPU against its 64-bit forms: page allocation,
quantised commit, verify attention, and a run of them with the accept and the
log probabilities as a verify step uses them.

Bars.  Whole numbers, tables, scale bytes and e4m3 bytes: equal.  Attention, per
element, with P rounded to f16 (half a step, 2^-11), fp32 products and sums,
ex2.approx (2^-22) and out rounded to bf16 (2^-8 of the value):
    |out - ref| <= 2^-8 |ref| + (2^-11 + d) sum p |v|,   |lse - ref| <= d + 2^-22 |ref|,
    d = 2^-19 + 2 (D + 8) 2^-24 scale max_j sum |q| |k_j|
(d: how far fp32 sums of D products move an exponent, doubled for the
normalisation, plus the exponential's and the sum's own errors)."""
import math

import pytest
import torch

from tests import q8_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _ops():
    from accept_select_top_gb300 import ops
    return ops


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def tables(lens, page, gen, spare=2, width=None):
    """(table, rows, pages): scattered pages and table rows, unused entries -1."""
    need = [-(-x // page) for x in lens]
    total = sum(need) + spare
    width = width or max(need + [1]) + 1
    ids = torch.randperm(total, generator=gen).tolist()
    rows = torch.randperm(len(lens) + spare, generator=gen).tolist()[:len(lens)]
    table = torch.full((len(lens) + spare, width), -1, dtype=torch.int32)
    for r, k in zip(rows, need):
        for p in range(k):
            table[r, p] = ids.pop()
    return table, rows, total


def pool(pages, Hkv, page, D, gen, lo=110, hi=122):
    """Random e4m3 bytes (no NaN) and scale bytes."""
    x = torch.randint(0, 256, (pages, Hkv, page, D), generator=gen, dtype=torch.int64).to(torch.uint8)
    x = torch.where((x & 127) == 127, 64, x).to(torch.uint8)
    return x, torch.randint(lo, hi, (pages, Hkv), generator=gen).to(torch.uint8)


# ------------------------------------------------------------------ pages

def run_alloc(page, lens, new, free_more=0, slot_table=False, alias=False, seed=0, max_new=None):
    ops = _ops()
    gen = _gen(seed)
    b = len(lens)
    table, rows, used = tables(lens, page, gen, width=max(-(-(x + m) // page) for x, m in zip(lens, new)) + 2)
    need = sum(-(-(x + m) // page) - -(-x // page) for x, m in zip(lens, new))
    free = [used + int(i) for i in torch.randperm(need + free_more + 3, generator=gen)]
    n_free = need + free_more
    width = table.shape[1] * page
    slots = torch.full((table.shape[0], width), -7, dtype=torch.int32) if slot_table else None
    total = sum(new)
    dev = dict(table=table.to(DEV), slots=None if slots is None else slots.to(DEV), n_free=i32([n_free]),
               cu=i32([-5] * (b + 1)), map=i32([-5] * (total + 6)), pos=i32([-5] * (total + 6)), left=i32([-5]))
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_ALLOC_SLOTS, b, 1, 1, 1))
    ops.spec_alloc_slots(b, page, i32(rows), i32(lens), i32(new), max(new) if max_new is None else max_new, i32(free), dev["n_free"],
                         (used + need + free_more + 3) * page, dev["table"], dev["slots"], dev["cu"], dev["map"], dev["pos"],
                         dev["n_free"] if alias else dev["left"], ws)
    assert ws.last_error() == 0
    cu, got_slots, pos, left = R.alloc(page, rows, lens, new, free, n_free, table, slots)
    assert dev["cu"].tolist() == cu
    assert dev["map"].tolist() == got_slots + [-5] * 6
    assert dev["pos"].tolist() == pos + [-5] * 6
    assert torch.equal(dev["table"].cpu(), table)
    if slots is not None:
        assert torch.equal(dev["slots"].cpu(), slots)
    assert (dev["n_free"] if alias else dev["left"]).tolist() == [left]


@pytest.mark.parametrize("page", [1, 16, 32, 64, 7])
@pytest.mark.parametrize("lens, new", [
    ([0], [1]), ([5], [0]), ([16, 31, 0, 64], [1, 1, 0, 3]), ([15, 16, 17, 63, 64, 65, 0], [1, 2, 3, 1, 64, 130, 700]),
    ([0] * 300, [i % 5 for i in range(300)]), ([3] * 3 + [0] * 600 + [9], [0] * 603 + [5000])])
def test_alloc(page, lens, new):
    run_alloc(page, lens, new, free_more=2, slot_table=True)


def test_alloc_exactly_fitting_list_in_place():
    run_alloc(16, [10, 100], [30, 1], free_more=0, alias=True)


def test_alloc_many_tokens_and_requests():
    run_alloc(16, [i % 40 for i in range(1500)], [(i * 7) % 90 for i in range(1500)], alias=True, max_new=1 << 20)


@pytest.mark.parametrize("what", ["pages", "slots"])
def test_alloc_without_room_hands_out_nothing(what):
    ops = _ops()
    table = i32([[3, -1, -1], [4, -1, -1]])
    before = table.clone()
    free, n_free, left = i32([7, 8, 9]), i32([1 if what == "pages" else 3]), i32([-5])
    slots = torch.full((64 if what == "pages" else 20,), -5, dtype=torch.int32, device=DEV)
    cu, pos = i32([-5] * 3), slots.clone()
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_ALLOC_SLOTS, 2, 1, 1, 1))
    ops.spec_alloc_slots(2, 16, i32([0, 1]), i32([8, 16]), i32([16, 16]), 16, free, n_free, 160, table, None, cu, slots, pos, left, ws)
    assert ws.last_error() == ops.DEV_SPACE
    assert torch.equal(table, before) and cu.tolist() == [0, 0, 0] and left.tolist() == n_free.tolist()
    assert (slots == -5).all() and (pos == -5).all()
    if what == "pages":  # the workspace serves the next call, which fits
        ops.spec_alloc_slots(2, 16, i32([0, 1]), i32([8, 16]), i32([8, 3]), 16, free, n_free, 160, table, None, cu, slots, pos, left, ws)
        assert ws.last_error() == 0 and left.tolist() == [0] and table.tolist() == [[3, -1, -1], [4, 7, -1]]
        assert slots[:11].tolist() == [3 * 16 + i for i in range(8, 16)] + [7 * 16 + i for i in range(3)]


def test_alloc_bad_requests_get_nothing():
    ops = _ops()
    table = i32([[3, -1], [4, -1], [5, -1]])
    cu, left = i32([-5] * 5), i32([0])
    slots = torch.full((64,), -5, dtype=torch.int32, device=DEV)
    pos = slots.clone()
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_ALLOC_SLOTS, 4, 1, 1, 1))
    # a row past the table, a negative length, more tokens than the row holds, and a good request
    ops.spec_alloc_slots(4, 16, i32([3, 0, 1, 2]), i32([8, -1, 16, 16]), i32([4, 4, 17, 2]), 17, i32([7, 8, 9]), i32([3]), 160, table, None,
                         cu, slots, pos, left, ws)
    assert ws.last_error() == ops.DEV_LENGTH | ops.DEV_INDEX
    assert cu.tolist() == [0, 0, 0, 0, 2] and slots[:3].tolist() == [144, 145, -5] and left.tolist() == [2]
    # a free id past the pool: slot -1, and its table entry too
    ops.spec_alloc_slots(1, 16, i32([0]), i32([16]), i32([1]), 4, i32([10]), i32([1]), 160, table, None, cu, slots, pos, left, ws)
    assert ws.last_error() == ops.DEV_INDEX and slots[:1].tolist() == [-1] and table[0].tolist() == [3, -1]


# ----------------------------------------------------------------- commit

def run_commit(page, D, Hkv, layers, lens, src, rows_total, fresh, pools, table, rows, by_start=False, width=None):
    """fresh [layers, rows, 2, Hkv, D] bf16; pools: ([layers pools], [scales]) for K and V, CPU; both sides are changed."""
    ops = _ops()
    b = len(lens)
    width = width or max(len(s) for s in src)
    dev_new = fresh.to(DEV)
    kp, ks, vp, vs = ([x.to(DEV) for x in part] for part in pools)
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_COMMIT_KV_Q8, b, 1, 1, 1))
    after = i32([-5] * b)
    index = None if by_start else i32([s + [-1] * (width - len(s)) for s in src])
    start = i32([s[0] if s else 0 for s in src]) if by_start else None
    ops.spec_commit_kv_q8(b, Hkv, D, page, [dev_new[i, :, 0] for i in range(layers)], [dev_new[i, :, 1] for i in range(layers)], kp, vp, ks, vs,
                          table.to(DEV), i32(rows), i32(lens), index, start, i32([len(s) for s in src]), width, after, ws)
    assert ws.last_error() == 0
    assert after.tolist() == [x + len(s) for x, s in zip(lens, src)]
    for i in range(layers):
        for j, (got_p, got_s, pp, ss) in enumerate(((kp, ks, pools[0], pools[1]), (vp, vs, pools[2], pools[3]))):
            R.commit(page, table, rows, lens, src, fresh[i, :, j], pp[i], ss[i])
            assert torch.equal(got_s[i].cpu(), ss[i]), (i, j)
            g, w = got_p[i].cpu(), pp[i]
            nan = (w & 127) == 127
            assert torch.equal((g & 127) == 127, nan) and torch.equal(g[~nan], w[~nan]), (i, j)
    return kp, ks, vp, vs


def pools_of(layers, pages, Hkv, page, D, gen, **kw):
    got = [pool(pages, Hkv, page, D, gen, **kw) for _ in range(2 * layers)]
    return ([x[0] for x in got[:layers]], [x[1] for x in got[:layers]], [x[0] for x in got[layers:]], [x[1] for x in got[layers:]])


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("D, Hkv, layers", [(64, 1, 1), (128, 8, 2), (128, 3, 1), (64, 9, 3)])
def test_commit_accepted_rows(page, D, Hkv, layers):
    gen = _gen(page + D + Hkv)
    lens = [0, 1, 15, 16, 31, 63, 64, 100]
    n = 9
    src = [[b * n + j for j in path] for b, path in enumerate([[0], [0, 3, 4], [0, 1, 2, 5, 8], [0, 8], [0, 7], [0], [0, 1, 2, 3, 4, 5, 6], [0, 0, 3]])]
    table, rows, pages = tables([x + len(s) for x, s in zip(lens, src)], page, gen)
    fresh = torch.randn(layers, n * len(lens), 2, Hkv, D, generator=gen) * torch.exp2(torch.randint(-12, 12, (layers, n * len(lens), 2, Hkv, 1), generator=gen).float())
    run_commit(page, D, Hkv, layers, lens, src, n * len(lens), fresh.bfloat16(), pools_of(layers, pages, Hkv, page, D, gen), table, rows, width=8)


@pytest.mark.parametrize("page, D", [(16, 128), (64, 128), (32, 64), (64, 64)])
def test_commit_prompts(page, D):
    gen = _gen(page * D)
    lens, new = [0, 5, 64, 0, 77], [130, 64, 1, 0, 83]
    src, at = [], 0
    for m in new:
        src.append(list(range(at, at + m)))
        at += m
    table, rows, pages = tables([x + m for x, m in zip(lens, new)], page, gen)
    fresh = torch.randn(1, at, 2, 2, D, generator=gen).bfloat16()
    run_commit(page, D, 2, 1, lens, src, at, fresh, pools_of(1, pages, 2, page, D, gen), table, rows, by_start=True)


def test_commit_borders_of_scale_and_type():
    """Largest values at and next to 448 * 2^x, ties, zeros, values e4m3 flushes, inf, NaN, the type's extremes; a page whose
    scale is far above, far below, and equal to what the new rows need."""
    gen = _gen(3)
    page, D, Hkv = 16, 64, 2
    big = torch.finfo(torch.bfloat16).max
    specials = [[448.0, 1.0625, -1.1875, 0.0], [450.0, 1.0], [1.75, 0.0068359375, 0.001953125, 0.0009765625], [0.0] * 4, [1e-38, 9e-41],
                [math.inf, 1.0, -math.inf], [math.nan, 3.0], [big, -1.0, 1e30], [math.nan, math.inf, -math.inf, 0.0], [-0.0, 2.0 ** -120]]
    rows_t = torch.zeros(len(specials), Hkv, D)
    for i, s in enumerate(specials):
        rows_t[i, :, :len(s)] = torch.tensor(s)
    ties = torch.arange(64).float() * 0.0625 + 1.0  # halfway points between e4m3 values
    rows_t = torch.cat([rows_t, ties.view(1, 1, 64).expand(1, Hkv, 64)])
    fresh = torch.stack([rows_t, rows_t * 0.37], dim=1)[None].bfloat16()
    k = rows_t.shape[0]
    lens = [0] * k + [5] * (3 * k)
    src = [[i % k] for i in range(4 * k)]
    table, rows, pages = tables([x + 1 for x in lens], page, gen)
    pools = pools_of(1, pages, Hkv, page, D, gen)
    for b in range(k, 4 * k):
        for s in (pools[1][0], pools[3][0]):
            s[int(table[rows[b], 0])] = (16, 119, 247)[b // k - 1]
    run_commit(page, D, Hkv, 1, lens, src, k, fresh, pools, table, rows)


def test_commit_growth_keeps_held_values_and_repeats():
    """Committing the same rows again changes nothing (the scales have grown already); rows two requests name may be the same."""
    gen = _gen(4)
    page, D, Hkv = 32, 128, 2
    lens, src = [7, 40, 31], [[0, 1], [1, 2, 2], [0]]
    table, rows, pages = tables([x + len(s) for x, s in zip(lens, src)], page, gen)
    fresh = (torch.randn(1, 3, 2, Hkv, D, generator=gen) * 50).bfloat16()
    pools = pools_of(1, pages, Hkv, page, D, gen, lo=117, hi=121)
    first = run_commit(page, D, Hkv, 1, lens, src, 3, fresh, pools, table, rows)
    want = [x[0].cpu() for x in first]
    again = run_commit(page, D, Hkv, 1, lens, src, 3, fresh, tuple([x.clone()] for x in want), table, rows)
    assert all(torch.equal(x[0].cpu(), y) for x, y in zip(again, want))


def test_commit_bad_input_is_skipped():
    ops = _ops()
    gen = _gen(5)
    page, D, Hkv = 16, 64, 1
    fresh = torch.randn(4, Hkv, D, generator=gen).bfloat16().to(DEV)
    kp, ks = (x.to(DEV) for x in pool(4, Hkv, page, D, gen))
    vp, vs = kp.clone(), ks.clone()
    before, sb = kp.clone(), ks.clone()
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_COMMIT_KV_Q8, 1, 1, 1, 1))
    after = i32([-5])

    def call(row=0, L=0, index=(0,), m=1, table=((0, 1),)):
        ops.spec_commit_kv_q8(1, Hkv, D, page, [fresh], [fresh], [kp], [vp], [ks], [vs], i32([list(t) for t in table]), i32([row]), i32([L]), i32([list(index)]),
                              None, i32([m]), len(index), after, ws)
        return ws.last_error()

    assert call(row=1) == ops.DEV_INDEX and after.tolist() == [0]
    assert call(row=-1) == ops.DEV_INDEX
    assert call(L=-1) == ops.DEV_LENGTH
    assert call(L=32) == ops.DEV_LENGTH and after.tolist() == [32]
    assert call(m=2) == ops.DEV_LENGTH
    assert call(m=-1) == ops.DEV_LENGTH
    assert call(table=((4, 1),)) == ops.DEV_INDEX
    assert call(table=((-1, 1),)) == ops.DEV_INDEX
    assert call(m=0) == 0 and after.tolist() == [0]
    assert torch.equal(kp, before) and torch.equal(ks, sb) and torch.equal(vp, before)
    assert call(index=(4, 2), m=2) == ops.DEV_INDEX  # the bad row is left out, the good one written
    assert torch.equal(kp[0, 0, 0], before[0, 0, 0]) and not torch.equal(kp[0, 0, 1], before[0, 0, 1])
    assert torch.equal(kp[1:], before[1:])


# -------------------------------------------------------------- attention

@pytest.fixture(params=[0, 1 << 20], ids=["tight", "loose"])
def bounds(request, monkeypatch):
    monkeypatch.setattr(Att, "bound", request.param)


class Att:
    bound = 0  # of the lengths, at least: a loose one keeps a few short units from being taken by clusters

    def __init__(self, b, n, Hq, Hkv, D, page, lens, seed=0, masks=None, packed=False, scale=None, **kw):
        self.n, self.Hq, self.Hkv, self.D, self.page, self.lens = n, Hq, Hkv, D, page, lens
        gen = _gen(seed)
        self.table, self.rows, self.pages = tables(lens, page, gen)
        self.kp, self.ks = pool(self.pages, Hkv, page, D, gen, **kw)
        self.vp, self.vs = pool(self.pages, Hkv, page, D, gen, **kw)
        x = torch.randn(b * n, Hq + 2 * Hkv + 1, D, generator=gen).bfloat16()
        self.x, self.packed = x, packed
        self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv]
        if masks is None:
            masks = []
            for _ in range(b):
                m = [1]
                for i in range(1, n):
                    m.append(m[int(torch.randint(0, i, (1,), generator=gen))] | 1 << i)
                masks += m
        self.masks = masks
        self.scale = scale if scale is not None else 1 / math.sqrt(D)
        self.b = b

    def device(self):
        ops = _ops()
        if self.packed:
            x = self.x.to(DEV)
            q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:self.Hq + 2 * self.Hkv]
        else:
            q, k, v = (t.contiguous().to(DEV) for t in (self.q, self.k, self.v))
        most = max(self.lens + [self.bound])
        masks = torch.tensor([m - (1 << 64) if m >> 63 else m for m in self.masks], dtype=torch.int64, device=DEV)
        self.ws = ops.Workspace(ops.spec_workspace_size(ops.OP_VERIFY_ATTENTION_Q8, self.b, self.n, 1, 1, self.Hq, self.Hkv, most))
        self.out = torch.full((self.b * self.n, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.b * self.n, self.Hq), 7.0, device=DEV)
        self.args = (self.b, self.n, self.Hq, self.Hkv, self.D, self.page, q, k, v, self.kp.to(DEV), self.vp.to(DEV), self.ks.to(DEV), self.vs.to(DEV),
                     self.table.to(DEV), i32(self.rows), i32(self.lens), most, masks, self.scale, self.out, self.lse, self.ws)
        return self.args

    def reference(self):
        return R.attention(self.n, self.page, self.q, self.k, self.v, self.kp, self.vp, self.ks, self.vs, self.table, self.rows, self.lens, self.masks, self.scale)

    def check(self, got_out=None, got_lse=None, want=None):
        out, lse, size, dx = want or self.reference()
        d = 2.0 ** -19 + 2 * (self.D + 8) * 2.0 ** -24 * dx
        got = (self.out if got_out is None else got_out).double().cpu()
        gl = (self.lse if got_lse is None else got_lse).double().cpu()
        none = lse == -math.inf
        assert torch.equal(gl == -math.inf, none)
        assert (got[none] == 0).all()
        bar = 2.0 ** -8 * out.abs() + (2.0 ** -11 + d)[..., None] * size
        off = ((got - out).abs() / bar.clamp(min=1e-300))[~none]
        assert torch.isfinite(got[~none]).all() and (off.numel() == 0 or off.max() <= 1), float(off.max())
        dl = ((gl - lse).abs() / (d + 2.0 ** -22 * lse.abs()))[~none]
        assert dl.numel() == 0 or dl.max() <= 1, float(dl.max())

    def run(self):
        _ops().spec_verify_attention_q8(*self.device())
        assert self.ws.last_error() == 0
        self.check()
        return self


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("n, Hq, Hkv, D", [
    (1, 1, 1, 64), (1, 8, 8, 128), (1, 32, 4, 128), (2, 6, 2, 128), (3, 5, 1, 64), (4, 32, 8, 128), (7, 12, 4, 64), (16, 8, 2, 128), (17, 3, 3, 64),
    (33, 7, 1, 128), (63, 4, 1, 64), (64, 8, 2, 128), (64, 16, 2, 64), (64, 10, 2, 128)])
def test_attention_sizes(page, n, Hq, Hkv, D):
    Att(4, n, Hq, Hkv, D, page, [0, 1, 65, 130], seed=n * Hq + page, packed=n % 2 == 0).run()


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, Hq, Hkv", [(1, 4, 1), (4, 4, 1), (20, 4, 1), (64, 4, 1)])
@pytest.mark.parametrize("lens", [[1500], [2047, 3, 0, 17, 16, 15], [0, 0, 0], [31] * 40 + [900]])
def test_attention_ragged(n, Hq, Hkv, lens):
    """Units cut over warps and CTAs, many requests in one CTA's range, requests without history."""
    Att(len(lens), n, Hq, Hkv, 128, 16, lens, seed=len(lens) + n).run()


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, Hq, Hkv, D", [(1, 8, 1, 128), (4, 16, 4, 64), (64, 4, 1, 128)])
def test_attention_many_requests(n, Hq, Hkv, D):
    lens = [(37 * i) % 200 for i in range(90)]
    Att(90, n, Hq, Hkv, D, 32, lens, seed=1).run()


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n", [1, 5, 40, 64])
def test_attention_masks_that_leave_rows_empty(n):
    masks = [0, 0, 1, 0][:3] * 60 if n == 1 else None
    b = 3
    masks = [(0 if i % 2 else (1 << n) - 1) if r != 1 else 0 for r in range(b) for i in range(n)]
    Att(b, n, 8, 2, 128, 16, [0, 0, 20], masks=masks, seed=n).run()


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n", [1, 4, 33, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_scales_of_every_size(n, D):
    """Page scales spread over 2^40 and new rows of very different sizes: no over- or underflow inside."""
    a = Att(2, n, 4, 2, D, 16, [200, 77], seed=7, lo=90, hi=130, scale=2.0 ** -4)
    gen = _gen(8)
    a.ks.copy_(torch.randint(100, 118, a.ks.shape, generator=gen).to(torch.uint8))
    f = torch.exp2(torch.randint(-20, 20, (a.x.shape[0], 1, 1), generator=gen).float())
    a.v.copy_((a.v.float() * f).bfloat16())
    a.k.copy_((a.k.float() * torch.exp2(torch.randint(-8, 4, (a.x.shape[0], 1, 1), generator=gen).float())).bfloat16())
    a.run()


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n", [1, 4, 33, 64])
def test_attention_peaked_rows(n):
    """Large logits: most rows are one key; the running maximum moves often."""
    Att(2, n, 8, 2, 128, 16, [300, 5], seed=9, scale=1.0, lo=112, hi=114).run()


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n", [4, 20, 64])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_attention_nonfinite_values_in_masked_nodes(n, value):
    """A node whose K or V holds an inf or a NaN reaches the rows that see it and no other; bytes behind the last token of a
    page, and pages no request holds, may be NaN."""
    masks = [1 << i | 1 for _ in range(2) for i in range(n)]
    a = Att(2, n, 8, 2, 128, 32, [45, 64], masks=masks, seed=10)
    for x, lens in ((a.kp, a.lens), (a.vp, a.lens)):
        keep = torch.zeros(a.pages, a.page, dtype=torch.bool)
        for r, L in zip(a.rows, lens):
            for t in range(L):
                keep[int(a.table[r, t // a.page]), t % a.page] = True
        x[(~keep)[:, None, :].expand(-1, a.Hkv, -1)] = 0x7f
    clean = a.reference()
    a.k[2, 0, 3] = value
    a.v[2, 1, 5] = value
    a.v[n + 3, 0, 127] = value
    _ops().spec_verify_attention_q8(*a.device())
    assert a.ws.last_error() == 0
    G = a.Hq // a.Hkv
    out, lse = a.out.cpu().float(), a.lse.cpu()
    assert not torch.isfinite(out[2, G:, 5]).any()
    assert not torch.isfinite(out[n + 3, :G, 127]).any()
    if value != -math.inf or True:  # K row: scores of +-inf or NaN in heads 0..G-1 of row 2
        touched = torch.zeros(2 * n, a.Hq, a.D, dtype=torch.bool)
        touched[2, :G] = True
        touched[2, G:, 5] = True
        touched[n + 3, :G, 127] = True
    got = torch.where(touched, clean[0].float(), out)
    lse = torch.where(touched.all(-1), clean[1].float(), lse)
    a.check(got, lse, clean)


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n", [1, 4, 64])
def test_attention_nan_in_history(n):
    a = Att(2, n, 4, 1, 64, 16, [40, 40], seed=11)
    a.vp[int(a.table[a.rows[0], 1]), 0, 3, 9] = 0xff
    _ops().spec_verify_attention_q8(*a.device())
    bad = ~torch.isfinite(a.out.cpu().float())
    assert bad[:n, :, 9].all() and bad.sum() == n * 4


@pytest.mark.usefixtures("bounds")
def test_attention_bad_input():
    """Wrong lengths, rows and page ids are reported; nothing is read out of range and the other requests keep their results
    (within the bars: another total of keys splits the work elsewhere)."""
    ops = _ops()
    for n in (2, 64):
        a = Att(3, n, 4, 1, 128, 16, [40, 50, 30], seed=12)
        a.device()
        want = a.reference()

        def call(error, keep, **change):
            args = list(a.args)
            for at, v in change.items():
                args[int(at[1:])] = v
            ops.spec_verify_attention_q8(*args)
            assert a.ws.last_error() == error
            assert torch.isfinite(a.out.float()).all()
            mine = torch.zeros(3 * n, dtype=torch.bool)
            for r in keep:
                mine[r * n:(r + 1) * n] = True
            a.check(torch.where(mine[:, None, None], a.out.cpu().double(), want[0]), torch.where(mine[:, None], a.lse.cpu().double(), want[1]), want)

        call(0, (0, 1, 2))
        call(ops.DEV_INDEX, (1,), _14=i32([99, a.rows[1], -1]))
        table = a.table.clone()
        table[a.rows[0], 1] = a.pages
        table[a.rows[2], 0] = -3
        call(ops.DEV_INDEX, (1,), _13=table.to(DEV))
        call(ops.DEV_LENGTH, (0,), _15=i32([40, 50, -1]), _16=45)
        call(0, (0, 1, 2))


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, lens", [(1, [1000, 3]), (4, [700, 50, 0]), (64, [700, 50])])
def test_attention_captured_twice_and_on_another_stream(n, lens):
    """Two graphs that share one workspace, replayed in turn, and an eager call on a side stream: the same bits each time."""
    ops = _ops()
    a, c = Att(len(lens), n, 8, 2, 128, 16, lens, seed=13), Att(len(lens), n, 8, 2, 128, 16, lens[::-1], seed=14)
    a.device(), c.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.spec_verify_attention_q8(*a.args)
        ops.spec_verify_attention_q8(*c.args)
    side.synchronize()
    a.check()
    c.check()
    want = a.out.clone(), c.out.clone(), a.lse.clone(), c.lse.clone()
    graphs = []
    for x in (a, c):
        args = list(x.args)
        args[-1] = a.ws
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.spec_verify_attention_q8(*args)
        graphs.append(g)
    for _ in range(3):
        for x in (a, c):
            x.out.fill_(5.0)
            x.lse.fill_(5.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for got, w in zip((a.out, c.out, a.lse, c.lse), want):
            assert torch.equal(got, w)
    assert a.ws.last_error() == 0


@pytest.mark.usefixtures("bounds")
def test_attention_without_lse_and_idle_batch():
    ops = _ops()
    a = Att(2, 4, 8, 2, 64, 16, [20, 33], seed=15)
    args = list(a.device())
    args[20] = None
    ops.spec_verify_attention_q8(*args)
    want = a.reference()
    a.check(got_lse=want[1], want=want)
    a.out.fill_(3.0)
    args[0] = 0
    ops.spec_verify_attention_q8(*args)
    torch.cuda.synchronize()
    assert (a.out == 3.0).all()


def test_attention_history_past_32_bits():
    """Pages whose bytes lie past 4 GB in the pool."""
    ops = _ops()
    page, D, Hkv = 64, 128, 8
    pages = (5 << 30) // (page * D * Hkv)
    a = Att(1, 2, 8, Hkv, D, page, [150], seed=16)
    far = [pages - 1, pages - 3, pages // 2 + 7]
    a.device()
    args = list(a.args)
    table = a.table.clone()
    kp, vp = (torch.zeros(pages, Hkv, page, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((pages, Hkv), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    for i, p in enumerate(far):
        old = int(a.table[a.rows[0], i])
        table[a.rows[0], i] = p
        kp[p], vp[p], ks[p], vs[p] = a.kp[old].to(DEV), a.vp[old].to(DEV), a.ks[old].to(DEV), a.vs[old].to(DEV)
    args[9:14] = [kp, vp, ks, vs, table.to(DEV)]
    ops.spec_verify_attention_q8(*args)
    assert a.ws.last_error() == 0
    a.check()


# ------------------------------------------------------------ one verify step

def test_verify_steps_in_sequence():
    """Three steps as an engine runs them: attention over the cache, greedy accept, log probabilities of the accepted tokens,
    pages for them, commit -- with the 64-bit forms following alongside; the second step reads what the first committed."""
    import numpy as np

    import oracle
    ops = _ops()
    gen = _gen(20)
    b, n, S, Hq, Hkv, D, page, V = 3, 7, 3, 8, 2, 128, 16, 997
    lens = [30, 0, 15]
    table, rows, used = tables(lens, page, gen, width=8)
    pages = used + 12
    free = list(range(used, pages))
    kp, ks = pool(pages, Hkv, page, D, gen)
    vp, vs = pool(pages, Hkv, page, D, gen)
    parents = [-1, 0, 0, 1, 1, 2, 3]
    from tests.helpers import pointers_from_parents
    nt, ns = pointers_from_parents(parents)
    masks = []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
    dev = dict(table=table.to(DEV), kp=kp.to(DEV), vp=vp.to(DEV), ks=ks.to(DEV), vs=vs.to(DEV), lens=i32(lens), n_free=i32([len(free)]), free=i32(free),
               rows=i32(rows))
    tree = [i32(np.tile(x, b).tolist()) for x in (nt, ns)]
    size = max(ops.spec_workspace_size(ops.OP_VERIFY_ATTENTION_Q8, b, n, 1, V, Hq, Hkv, 100), ops.spec_workspace_size(ops.OP_TOKEN_LOGPROBS, b, S + 1, 4, V),
               ops.spec_workspace_size(ops.OP_VERIFY_GREEDY, b, n, 1, V))
    ws = ops.Workspace(size)
    for step in range(3):
        x = torch.randn(b * n, Hq + 2 * Hkv, D, generator=gen).bfloat16()
        drafts = torch.randint(0, V, (b * n,), generator=gen)
        logits = torch.randn(b * n, V, generator=gen)
        for i in range(b * n):  # most nodes' first child is the target's choice
            child = int(nt[i % n])
            if child >= 0 and int(torch.randint(0, 4, (1,), generator=gen)):
                logits[i, int(drafts[i // n * n + child])] = 9.0
        xd, ld = x.to(DEV), logits.to(DEV)
        out, lse = torch.empty(b * n, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(b * n, Hq, device=DEV)
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
        predict, acc, acc_lens, acc_tokens, root = z(b * n), z(b, S + 1), z(b), z(b, S + 1), z(b)
        cu, slots, pos, after = z(b + 1), z(b * (S + 1)), z(b * (S + 1)), z(b)
        lp, ent, ids, top = torch.zeros(b, S + 1, device=DEV), torch.zeros(b, S + 1, device=DEV), z(b, S + 1, 4), torch.zeros(b, S + 1, 4, device=DEV)
        ops.spec_verify_attention_q8(b, n, Hq, Hkv, D, page, xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], dev["kp"], dev["vp"], dev["ks"], dev["vs"], dev["table"],
                                     dev["rows"], dev["lens"], 100, i64(masks * b), D ** -0.5, out, lse, ws)
        ops.spec_verify_greedy(b, n, S, ld, drafts.int().to(DEV), i32(list(range(b * n))), tree[0], tree[1], predict, acc, acc_lens, acc_tokens, root, ws)
        ops.spec_token_logprobs(b, n, S + 1, ld, acc, acc_tokens, None, 4, lp, ent, ids, top, ws)
        ops.spec_alloc_slots(b, page, dev["rows"], dev["lens"], acc_lens, S + 1, dev["free"], dev["n_free"], pages * page, dev["table"], None, cu, slots, pos,
                             dev["n_free"], ws)
        ops.spec_commit_kv_q8(b, Hkv, D, page, [xd[:, Hq:Hq + Hkv]], [xd[:, Hq + Hkv:]], [dev["kp"]], [dev["vp"]], [dev["ks"]], [dev["vs"]], dev["table"], dev["rows"],
                              dev["lens"], acc, None, acc_lens, S + 1, after, ws)
        dev["lens"] = after
        assert ws.last_error() == 0

        a = Att.__new__(Att)
        a.D = D
        a.check(out, lse, R.attention(n, page, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kp, vp, ks, vs, table, rows, lens, masks * b, D ** -0.5))
        o = oracle.verify_greedy(b, n, S, logits.numpy(), drafts.int().numpy(), np.arange(b * n, dtype=np.int32), np.tile(nt, b), np.tile(ns, b))
        assert np.array_equal(acc.cpu().numpy(), o["accept_index"]) and np.array_equal(acc_tokens.cpu().numpy(), o["accepted_tokens"])
        wlp, went, wids, wtop = R.logprobs(n, S + 1, logits, acc.cpu(), acc_tokens.cpu(), None, 4)
        assert torch.equal(ids.cpu().long(), wids)
        for got, want in ((lp, wlp), (ent, went), (top, wtop)):
            assert (got.cpu().double() - want).abs().max() <= 1e-5
        new = [int(v) for v in o["accept_lens"]]
        wcu, wslots, wpos, left = R.alloc(page, rows, lens, new, free, len(free), table)
        assert slots[:len(wslots)].tolist() == wslots and dev["n_free"].tolist() == [left]
        src = [[int(v) for v in o["accept_index"][r][:m]] for r, m in enumerate(new)]
        R.commit(page, table, rows, lens, src, x[:, Hq:Hq + Hkv], kp, ks)
        R.commit(page, table, rows, lens, src, x[:, Hq + Hkv:], vp, vs)
        free, lens = free[:left], [x_ + m for x_, m in zip(lens, new)]
        assert after.tolist() == lens and torch.equal(dev["table"].cpu(), table)
        for got, want in ((dev["kp"], kp), (dev["vp"], vp), (dev["ks"], ks), (dev["vs"], vs)):
            assert torch.equal(got.cpu(), want)


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)
