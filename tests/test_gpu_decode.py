"""One-token attention over shared pages on the GPU against its 64-bit form, and runs of it with forks, copies,
appended tokens and compaction.

Bar, per element, with P rounded to bf16 (half a step, 2^-8), fp32 products and sums, ex2.approx (2^-22) and out
rounded to bf16 (2^-8 of the value):
    |out - ref| <= 2^-8 |ref| + (2^-8 + d) sum p |v|,   |lse - ref| <= d + 2^-22 |ref|,
    d = 2^-19 + 2 (D + 8) 2^-24 |scale| max_j sum |q| |k_j|
(d: how far fp32 sums of D products move an exponent, doubled for the normalisation, plus the exponential's and the
sum's own errors).  Values below 2^-94 of 1 may be lost (2^-90 absolute is allowed)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _ops():
    from accept_select_top_gb300 import ops
    return ops


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


class Case:
    """Requests over scattered pages: groups = [(shared tokens, [tokens of each member])], then requests of `alone`."""

    def __init__(self, groups, alone=(), page=16, Hq=8, Hkv=2, D=128, seed=0, spare=2, std=1.0):
        gen = _gen(seed)
        self.page, self.Hq, self.Hkv, self.D, self.scale = page, Hq, Hkv, D, 1 / math.sqrt(D)
        self.lens = [x for s, m in groups for x in m] + list(alone)
        self.starts = [0]
        for s, m in groups:
            self.starts.append(self.starts[-1] + len(m))
        self.shared = [s for s, m in groups]
        b = self.b = len(self.lens)
        need = sum(-(-x // page) for x in self.lens) + spare
        ids = torch.randperm(need, generator=gen).tolist()
        width = max([-(-x // page) for x in self.lens] + [1]) + 1
        self.rows = torch.randperm(b + 2, generator=gen).tolist()[:b]
        table = torch.full((b + 2, width), -1, dtype=torch.int32)
        r = 0
        for s, m in list(groups) + [(0, [x]) for x in alone]:
            common = [ids.pop() for _ in range(min(s, max(m, default=0)) // page)]
            for x in m:
                n = -(-x // page)
                mine = (common + [ids.pop() for _ in range(max(0, n - len(common)))])[:n]
                table[self.rows[r], :n] = torch.tensor(mine, dtype=torch.int32)
                r += 1
        self.table = table.to(DEV)
        self.slots = need * page
        g = torch.Generator(device=DEV).manual_seed(seed)
        draw = lambda *shape: (torch.randn(*shape, generator=g, device=DEV) * std).bfloat16()  # noqa: E731
        qkv = draw(b, Hq + 2 * Hkv, D)
        self.q = qkv[:, :Hq]
        self.k, self.v = draw(self.slots, Hkv, D), draw(self.slots, Hkv, D)
        # what is behind a request's last token, or in no request's pages, must not matter
        held = torch.zeros(self.slots, dtype=torch.bool, device=DEV)
        for r in range(b):
            held[self.slots_of(r)] = True
        self.k[~held] = math.nan
        self.v[~held] = math.inf

    def slots_of(self, r):
        pos = torch.arange(self.lens[r], device=DEV)
        return self.table[self.rows[r]].long()[pos // self.page] * self.page + pos % self.page

    def call(self, lse=True, groups=True, most=None, ws=None, out=None, lens=None, b=None):
        ops = _ops()
        b = self.b if b is None else b
        most = max(self.lens + [0]) if most is None else most
        ws = ws or ops.Workspace(ops.spec_workspace_size(ops.OP_DECODE_ATTENTION, b, 1, 1, 1, self.Hq, self.Hkv, most))
        out = torch.full((b, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
        ls = torch.full((b, self.Hq), 7.0, device=DEV) if lse else None
        share = groups and len(self.starts) > 1
        ops.spec_decode_attention(b, self.Hq, self.Hkv, self.D, self.page, self.q, self.k, self.v, self.table, i32(self.rows), i32(self.lens if lens is None else lens), most,
                                  i32(self.starts) if share else None, i32(self.shared) if share else None, self.scale, out, ls, ws)
        assert ws.last_error() == 0
        return out, ls

    def check(self, out, lse, keys=None):
        G = self.Hq // self.Hkv
        worst = torch.zeros(2, dtype=torch.float64, device=DEV)
        for r in range(self.b):
            at = self.slots_of(r) if keys is None else keys(r)
            q = self.q[r].double().view(self.Hkv, G, self.D)
            k, v = self.k[at].double().transpose(0, 1), self.v[at].double().transpose(0, 1)
            got = out[r].double().view(self.Hkv, G, self.D)
            if at.numel() == 0:
                assert (got == 0).all() and (lse is None or (lse[r] == -math.inf).all())
                continue
            x = q @ k.transpose(1, 2) * self.scale
            p = torch.softmax(x, dim=-1)
            ref, spread = p @ v, p @ v.abs()
            d = 2.0 ** -19 + 2 * (self.D + 8) * 2.0 ** -24 * abs(self.scale) * (q.abs() @ k.abs().transpose(1, 2)).amax(dim=-1, keepdim=True)
            bar = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + d) * spread + 2.0 ** -90
            far = (got - ref).abs() / bar
            worst[0] = torch.maximum(worst[0], torch.where(far.isnan(), math.inf, far).max())
            if lse is not None:
                want = torch.logsumexp(x, dim=-1)
                far = (lse[r].double().view(self.Hkv, G) - want).abs() / (d[..., 0] + 2.0 ** -22 * want.abs())
                worst[1] = torch.maximum(worst[1], torch.where(far.isnan(), math.inf, far).max())
        assert (worst <= 1).all(), worst.tolist()


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 2, 8, 16, 32, 64, 128])
def test_lengths_and_pages(D, page):
    c = Case([], LENS, page=page, D=D, seed=page)
    c.check(*c.call())


@pytest.mark.parametrize("Hq, Hkv", [(1, 1), (3, 3), (5, 1), (16, 1), (17, 1), (24, 2), (33, 1), (64, 2), (65, 1), (130, 1), (128, 1), (32, 8), (64, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(Hq, Hkv, D):
    c = Case([(32, [40, 32, 100])], [70, 5], Hq=Hq, Hkv=Hkv, D=D, seed=Hq)
    c.check(*c.call())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("groups, alone", [
    ([(64, [64, 65, 200])], []), ([(128, [130] * 4), (0, [3, 9]), (64, [64])], [5, 0]), ([(192, [192 + i for i in range(40)])], [100]),
    ([(64, [70, 90]), (128, []), (512, [600, 513, 512])], []), ([(1024, [1024 + 7 * i for i in range(9)]), (64, [300] * 33)], [1] * 5)])
def test_groups(D, page, groups, alone):
    c = Case(groups, alone, page=page, D=D, seed=len(groups))
    c.check(*c.call())
    c.check(*c.call(groups=False))


@pytest.mark.parametrize("fan", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 64, 100])
def test_members(fan):
    """Rows of the shared tokens from four to 400: every split of the warps, and several row tiles."""
    c = Case([(1600, [1600 + i % 50 for i in range(fan)])], seed=fan)
    c.check(*c.call())


def test_shared_lengths_inside_a_page():
    """A shared length that is no multiple of the page or the tile, where the tables name the same pages all the same."""
    c = Case([(96, [120, 111, 96, 400])], page=16)
    for shared in (1, 15, 63, 64, 65, 90, 96):
        c.shared = [shared]
        c.check(*c.call())


def test_members_shorter_than_the_shared_tokens():
    c = Case([(96, [120, 111, 96, 400])], page=16)
    c.lens[1], c.lens[2] = 50, 0
    c.check(*c.call())
    c.lens[0] = 10  # the first: nothing is shared
    c.check(*c.call())


@pytest.mark.parametrize("Hq, Hkv", [(8, 8), (40, 2), (64, 1), (96, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_few_requests(D, Hq, Hkv):
    """Units that clusters of every size take, some of them without a token, up to 64 rows."""
    for b in (1, 4, 9, 30):
        lens = [(i * 397) % 1500 for i in range(b)]
        c = Case([], lens, Hq=Hq, Hkv=Hkv, D=D, seed=b)
        c.check(*c.call())
    c = Case([], [0], Hq=Hq, Hkv=Hkv, D=D)
    c.check(*c.call(most=0))
    c.check(*c.call(most=9000))


@pytest.mark.parametrize("b, most", [(1, 1), (1, 40000), (3, 20000), (200, 900), (2048, 70)])
def test_batches(b, most):
    gen = _gen(b)
    lens = torch.randint(0, most + 1, (b,), generator=gen).tolist()
    lens[0] = most
    c = Case([], lens, Hq=4, Hkv=1, D=64, seed=b)
    c.check(*c.call())
    c.check(*c.call(most=2 * most + 1000, lse=False))


def test_many_groups():
    gen = _gen(5)
    groups = []
    for _ in range(300):
        s = int(torch.randint(0, 20, (1,), generator=gen)) * 16
        groups.append((s, [s + int(x) for x in torch.randint(0, 100, (int(torch.randint(1, 8, (1,), generator=gen)),), generator=gen)]))
    c = Case(groups, [33] * 7, Hq=4, Hkv=2, D=64)
    c.check(*c.call())


def test_every_member_of_a_full_batch():
    c = Case([(320, [320 + i % 3 for i in range(2048)])], Hq=2, Hkv=1, D=64)
    c.check(*c.call())


@pytest.mark.parametrize("scale", [0.0, 0.3, -0.1, 4.0])
def test_scales(scale):
    c = Case([(64, [100, 64])], [200])
    c.scale = scale
    c.check(*c.call())


def test_rising_and_falling_scores():
    """The reference of a row moves at every tile, or never."""
    c = Case([(1024, [1500, 1024])], [900], Hq=4, Hkv=1)
    for r in range(c.b):
        n = c.lens[r]
        for sign in (1, -1):
            ramp = torch.linspace(-30, 30, n, device=DEV) * sign
            c.k[c.slots_of(r), 0] = (c.q[0, 0].float()[None] * ramp[:, None] / c.D ** 0.5).bfloat16()
            c.check(*c.call())


def test_values_of_the_types_ends():
    """Values near the type's largest (sums of many would not fit 32 bits), and tiny ones."""
    c = Case([(128, [300, 290])], [5000, 64], Hq=4, Hkv=1)
    big = 2.0 ** 127
    c.v[torch.isfinite(c.v)] = big
    out, lse = c.call()
    c.check(out, lse)
    assert torch.isfinite(out).all()
    c.v[torch.isfinite(c.v)] = 2.0 ** -60
    c.check(*c.call())


@pytest.mark.parametrize("members", [2, 12])
@pytest.mark.parametrize("D", [64, 128])
def test_large_values_of_no_weight(D, members):
    """Keys whose scores lie hundreds below the others', seen first, with values near the type's largest.  Low and high
    keys take turns every 256, so that a CTA that has several tiles meets low ones before high ones wherever it begins."""
    c = Case([(4096, [4100 + 3 * r for r in range(members)])] * 4, [4096], Hq=32, Hkv=8, D=D)
    c.q[..., 0] = 8.0
    for r in range(0, c.b, members):  # what each group shares, and the request alone
        at = c.slots_of(r)
        low = at[(torch.arange(at.numel(), device=DEV) % 512) < 256]
        c.k[at, :, 0] = 0.0
        c.k[low, :, 0] = -400.0
        c.v[low] = 2.0 ** 127
    c.check(*c.call())


def test_infinities_and_nans_reach_who_sees_them():
    c = Case([(64, [100, 90])], [80, 70], Hq=4, Hkv=1)
    out, lse = c.call()
    c.v[c.slots_of(1)[70], 0, 5] = math.inf       # of request 1 alone
    c.v[c.slots_of(2)[3], 0, 6] = math.nan        # of request 2
    got, got_lse = c.call()
    assert torch.equal(got_lse, lse)
    same = torch.ones_like(out, dtype=torch.bool)
    same[1, :, 5] = same[2, :, 6] = False
    assert torch.equal(got[same], out[same])
    assert (got[1, :, 5] == math.inf).all() and got[2, :, 6].isnan().all()
    c.k[c.slots_of(0)[10], 0, 0] = math.nan       # shared by 0 and 1
    got, got_lse = c.call()
    assert got[:2].isnan().all() and got_lse[:2].isnan().all() and torch.equal(got_lse[3], lse[3])


def test_all_scores_minus_infinity():
    c = Case([], [20, 5], Hq=1, Hkv=1, D=64)
    c.q[0] = 0
    c.q[0, 0, 0] = 1
    c.k[c.slots_of(0), 0, 0] = -math.inf
    out, lse = c.call()
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    c.k[c.slots_of(0)[7], 0, 0] = 3.0
    out, lse = c.call()
    assert torch.equal(out[0, 0], c.v[c.slots_of(0)[7], 0]) and abs(float(lse[0, 0]) - 3 / 8) < 1e-6


def test_same_bits_again_and_on_a_workspace_used_by_others():
    ops = _ops()
    c = Case([(640, [700 + i for i in range(20)])], [3000, 100], Hq=8, Hkv=2)
    ws = ops.Workspace(max(ops.spec_workspace_size(ops.OP_DECODE_ATTENTION, 64, 1, 1, 1, 8, 2, 4096), ops.spec_workspace_size(ops.OP_VERIFY_ATTENTION, 64, 1, 1, 1, 8, 2, 4096)))
    first = c.call(ws=ws)
    other = Case([], [50, 60], Hq=8, Hkv=2, seed=9)
    other.check(*other.call(ws=ws))
    ws.tensor[ops.spec_workspace_size(ops.OP_BUILD_TREE, 64, 1, 1, 1):].fill_(255)  # (what other calls may leave behind the counters)
    again = c.call(ws=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    c.check(*again)


def test_idle_batch_and_short_batch():
    ops = _ops()
    c = Case([(64, [80, 90])], [33])
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_DECODE_ATTENTION, 3, 1, 1, 1, 8, 2, 100))
    out, lse = torch.full((3, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((3, 8), 7.0, device=DEV)
    ops.spec_decode_attention(0, 8, 2, 128, 16, c.q, c.k, c.v, c.table, i32(c.rows), i32(c.lens), 100, None, None, c.scale, out, lse, ws)
    assert ws.last_error() == 0 and (out == 7).all() and (lse == 7).all()
    # a call over the first two requests leaves the rows behind them as they were
    ops.spec_decode_attention(2, 8, 2, 128, 16, c.q, c.k, c.v, c.table, i32(c.rows), i32(c.lens), 100, i32(c.starts), i32(c.shared), c.scale, out, lse, ws)
    assert ws.last_error() == 0 and (out[2] == 7).all() and (lse[2] == 7).all()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: the request's pages lie at its end, and so does a page that is copied."""
    ops = _ops()
    Hkv, D, page = 8, 128, 64
    slots = (5 << 30) // (Hkv * D * 2) // page * page + 4 * page
    k = torch.empty(slots, Hkv, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    n = 3 * page
    k[-n:] = torch.randn(n, Hkv, D, device=DEV).bfloat16()
    v[-n:] = torch.randn(n, Hkv, D, device=DEV).bfloat16()
    pages = slots // page
    q = torch.randn(1, 16, D, device=DEV).bfloat16()
    out, lse = torch.empty_like(q), torch.empty(1, 16, device=DEV)
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_DECODE_ATTENTION, 1, 1, 1, 1, 16, Hkv, n))
    ops.spec_decode_attention(1, 16, Hkv, D, page, q, k, v, i32([[pages - 3, pages - 2, pages - 1]]), i32([0]), i32([n - 5]), n, None, None, 0.1, out, lse, ws)
    assert ws.last_error() == 0
    x = torch.einsum("hgd,khd->hgk", q[0].double().view(Hkv, 2, D), k[-n:-5].double()) * 0.1
    p = torch.softmax(x, dim=-1)
    ref, spread = (torch.einsum("hgk,khd->hgd", p, y).reshape(16, D) for y in (v[-n:-5].double(), v[-n:-5].double().abs()))
    assert ((out[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * spread).all()
    src, dst, count = i32([pages - 3]), i32([pages - 4]), i32([1])
    ops.spec_copy_pages(page, [k], [v], None, None, src, dst, count, ws)
    assert ws.last_error() == 0 and torch.equal(k[-4 * page:-3 * page], k[-3 * page:-2 * page]) and torch.equal(v[-4 * page:-3 * page], v[-3 * page:-2 * page])


# ------------------------------------------------------------- told on the device

def test_bad_lengths_rows_groups_and_pages():
    ops = _ops()
    c = Case([(64, [80, 90]), (32, [40])], [33])
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_DECODE_ATTENTION, 4, 1, 1, 1, 8, 2, 100))

    def call(rows=None, lens=None, starts=None, shared=None, most=90, table=None):
        out, lse = torch.full((4, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((4, 8), 7.0, device=DEV)
        ops.spec_decode_attention(4, 8, 2, 128, 16, c.q, c.k, c.v, c.table if table is None else table, i32(rows or c.rows), i32(lens or c.lens), most, i32(starts or c.starts),
                                  i32(shared or c.shared), c.scale, out, lse, ws)
        return out, lse, ws.last_error()

    for starts in ([0, 3, 2], [-1, 2, 3], [0, 2, 5], [1 << 30, 2, 3]):
        out, lse, err = call(starts=starts)
        assert err == ops.DEV_INDEX
        c.check(out, lse)
    for shared in ([-1, 32], [64, 91], [1 << 30, 32]):
        out, lse, err = call(shared=shared)
        assert err == ops.DEV_LENGTH
        c.check(out, lse)
    out, lse, err = call(lens=[80, 1000, 40, -5])
    assert err == ops.DEV_LENGTH and (out[3] == 0).all() and (lse[3] == -math.inf).all()
    c.lens[3] = 0
    c.check(out, lse)  # (1000 is clamped to 90)
    out, lse, err = call(rows=c.rows[:2] + [-1, 99], lens=[80, 90, 40, 33])
    assert err == ops.DEV_INDEX and (out[2:] == 0).all() and (lse[2:] == -math.inf).all()
    bad = c.table.clone()
    bad[c.rows[1], 5] = 1 << 20
    bad[c.rows[2], 0] = -1
    out, lse, err = call(table=bad, lens=[80, 90, 40, 0])
    assert err == ops.DEV_INDEX
    c.lens = [80, 80, 24, 0]  # keys of a bad page do not count
    c.check(out, lse, keys=lambda r: c.slots_of(r) if r != 2 else (c.table[c.rows[2]].long()[1 + torch.arange(24, device=DEV) // 16] * 16 + torch.arange(24, device=DEV) % 16))


def test_binding_refusals():
    ops = _ops()
    c = Case([(64, [80, 90])], [33])
    ws = ops.Workspace(ops.spec_workspace_size(ops.OP_DECODE_ATTENTION, 3, 1, 1, 1, 8, 2, 100))
    out, lse = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=DEV), torch.empty(3, 8, device=DEV)
    good = dict(b=3, Hq=8, Hkv=2, D=128, page=16, q=c.q, k=c.k, v=c.v, table=c.table, rows=i32(c.rows), lens=i32(c.lens), most=100, starts=i32(c.starts), shared=i32(c.shared), scale=0.1, out=out,
                lse=lse, ws=ws)
    ops.spec_decode_attention(*good.values())
    assert ws.last_error() == 0
    small = ops.Workspace(4096)
    for bad in (dict(q=c.q.float()), dict(q=c.q[:2]), dict(q=c.q.transpose(1, 2)), dict(k=c.k[:, :1]), dict(k=c.k.half()), dict(v=c.v[16:]), dict(table=c.table.long()), dict(rows=i32([0])),
                dict(lens=i32(c.lens).long()), dict(starts=None), dict(starts=i32([0])), dict(out=out[:2]), dict(lse=lse.double()), dict(page=48), dict(page=256), dict(Hq=7, q=c.q[:, :7]),
                dict(ws=small), dict(most=-1), dict(b=2049)):
        with pytest.raises(ops.SpecError):
            ops.spec_decode_attention(*{**good, **bad}.values())
    alias = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ops.SpecError):
        ops.spec_decode_attention(*{**good, "q": alias, "out": alias}.values())
    assert ws.last_error() == 0


# ------------------------------------------------------------------ runs

def test_captured_and_replayed_on_two_streams():
    """Two graphs with a workspace each, replayed at once; the lengths change between replays."""
    ops = _ops()
    cases = [Case([(256, [400 + i for i in range(6)])], [2000, 10], seed=1), Case([(64, [64] * 20)], [3000] * 3, seed=2, D=64)]
    graphs = []
    for c in cases:
        most = max(c.lens)
        s = torch.cuda.Stream()
        d = dict(ws=ops.Workspace(ops.spec_workspace_size(ops.OP_DECODE_ATTENTION, c.b, 1, 1, 1, c.Hq, c.Hkv, most)), lens=i32(c.lens), rows=i32(c.rows), starts=i32(c.starts), shared=i32(c.shared),
                 out=torch.empty(c.b, c.Hq, c.D, dtype=torch.bfloat16, device=DEV), lse=torch.empty(c.b, c.Hq, device=DEV), s=s, g=torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(d["g"], stream=s):
            ops.spec_decode_attention(c.b, c.Hq, c.Hkv, c.D, c.page, c.q, c.k, c.v, c.table, d["rows"], d["lens"], most, d["starts"], d["shared"], c.scale, d["out"], d["lse"], d["ws"])
        graphs.append(d)
    for step in range(3):
        for c, d in zip(cases, graphs):
            c.lens = [max(0, x - step) for x in c.lens]
            d["lens"].copy_(i32(c.lens))
        torch.cuda.synchronize()
        for _ in range(5):
            for d in graphs:
                with torch.cuda.stream(d["s"]):
                    d["g"].replay()
        torch.cuda.synchronize()
        for c, d in zip(cases, graphs):
            assert d["ws"].last_error() == 0
            c.check(d["out"], d["lse"])


def test_samples_of_a_prompt():
    """A prompt's pages forked, the children grown token by token with the attention after each, some ended, the
    cache compacted, and the attention again: always what the 64-bit form gives over the tokens each request has."""
    ops = _ops()
    page, Hq, Hkv, D, rows, width, total = 16, 8, 2, 64, 12, 16, 90
    gen = _gen(11)
    draw = lambda *s: torch.randn(*s, generator=gen).bfloat16().to(DEV)  # noqa: E731
    k, v = torch.full((total * page, Hkv, D), math.nan, dtype=torch.bfloat16, device=DEV), torch.full((total * page, Hkv, D), math.nan, dtype=torch.bfloat16, device=DEV)
    t = dict(counts=i32([0] * total), free=i32(list(range(total))), n=i32([total]), table=i32([[-1] * width] * rows))
    ws = ops.Workspace(max(ops.spec_workspace_size(op, rows, 1, 1, total, Hq, Hkv, 256) for op in
                           (ops.OP_ALLOC_SLOTS, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, ops.OP_COMPACT_PAGES, ops.OP_DECODE_ATTENTION)))
    held = {}

    def grow(reqs, m):
        b = len(reqs)
        cu, slots, pos = i32([0] * (b + 1)), i32([-1] * (b * m)), i32([-1] * (b * m))
        ops.spec_alloc_slots(b, page, i32(reqs), i32([len(held.get(r, ([], []))[0]) for r in reqs]), i32([m] * b), m, t["free"], t["n"], total * page, t["table"], None, cu, slots, pos, t["n"], ws)
        kk, vv = draw(b * m, Hkv, D), draw(b * m, Hkv, D)
        k[slots.long()], v[slots.long()] = kk, vv
        for i, r in enumerate(reqs):
            had = held.get(r, (kk[:0], vv[:0]))
            held[r] = (torch.cat([had[0], kk[i * m:(i + 1) * m]]), torch.cat([had[1], vv[i * m:(i + 1) * m]]))

    def attend(groups, alone):
        reqs = [r for _, m in groups for r in m] + alone
        starts = [0]
        for _, m in groups:
            starts.append(starts[-1] + len(m))
        q = draw(len(reqs), Hq, D)
        out, lse = torch.empty_like(q), torch.empty(len(reqs), Hq, device=DEV)
        ops.spec_decode_attention(len(reqs), Hq, Hkv, D, page, q, k, v, t["table"], i32(reqs), i32([len(held[r][0]) for r in reqs]), 256, i32(starts), i32([s for s, _ in groups]), D ** -0.5,
                                  out, lse, ws)
        assert ws.last_error() == 0
        for i, r in enumerate(reqs):
            kk, vv = (x.double().transpose(0, 1) for x in held[r])
            x = q[i].double().view(Hkv, Hq // Hkv, D) @ kk.transpose(1, 2) * D ** -0.5
            p = torch.softmax(x, dim=-1)
            ref, spread = p @ vv, p @ vv.abs()
            got = out[i].double().view(Hkv, Hq // Hkv, D)
            assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * spread).all(), r

    def fork(parent, children, lens):
        n = len(children)
        src, dst, count = i32([0] * n), i32([0] * n), i32([0])
        ops.spec_fork_pages(n, page, i32([parent] * n), i32(children), i32(lens), t["counts"], t["free"], t["n"], t["table"], None, src, dst, count, t["n"], ws)
        ops.spec_copy_pages(page, [k], [v], None, None, src, dst, count, ws)
        for c, x in zip(children, lens):
            held[c] = (held[parent][0][:x], held[parent][1][:x])

    grow([4], 150)
    grow([7], 37)
    fork(4, [0, 1, 2, 3], [150, 150, 150, 131])
    attend([(144, [4, 0, 1, 2]), (128, [3])], [7])
    for _ in range(3):
        grow([0, 1, 2, 3, 4, 7], 5)
        attend([(128, [4, 0, 1, 2, 3])], [7])
    ended = [4, 1]
    ops.spec_release_pages(2, page, i32(ended), i32([len(held[r][0]) for r in ended]), None, t["counts"], t["free"], t["n"], t["table"], t["n"], ws)
    for r in ended:
        del held[r]
    attend([(128, [0, 2, 3])], [7])
    reqs = list(held)
    src, dst, count = i32([0] * total), i32([0] * total), i32([0])
    ops.spec_compact_pages(len(reqs), page, i32(reqs), i32([len(held[r][0]) for r in reqs]), 0, t["counts"], t["free"], t["n"], t["table"], None, t["counts"], t["free"], t["n"], t["table"], None,
                           src, dst, count, ws)
    ops.spec_copy_pages(page, [k], [v], None, None, src, dst, count, ws)
    k[int(total - t["n"]) * page:] = math.nan
    attend([(128, [0, 2, 3])], [7])
    fork(7, [5, 6], [52, 16])
    grow([0, 2, 3, 5, 6], 17)
    attend([(128, [0, 2, 3]), (16, [7, 5, 6])], [])
