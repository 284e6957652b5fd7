"""Verify attention over the 8-bit cache under load: many units a CTA, units of one tile beside
long ones, both ways the tcgen05 kernel gives rows to its two groups, calls on two streams.
The reference is float64 torch on the GPU; repeats of a call have to give the same bits."""
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


class Load:
    def __init__(self, n, Hq, Hkv, D, page, lens, seed, scale=None, lo=110, hi=122, bound=None):
        ops = _ops()
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.b, self.n, self.Hq, self.Hkv, self.D, self.page, self.lens = len(lens), n, Hq, Hkv, D, page, lens
        need = [-(-x // page) for x in lens]
        pages = sum(need) + 1
        ids = torch.randperm(pages, generator=gen, device=DEV).tolist()
        table = torch.full((self.b, max(need + [1])), -1, dtype=torch.int32)
        for r, k in enumerate(need):
            table[r, :k] = torch.tensor(ids[:k], dtype=torch.int32)
            ids = ids[k:]
        self.table = table.to(DEV)

        def pool():
            x = torch.randint(0, 256, (pages, Hkv, page, D), generator=gen, device=DEV, dtype=torch.uint8)
            return torch.where((x & 127) == 127, x ^ 64, x), torch.randint(lo, hi, (pages, Hkv), generator=gen, device=DEV).to(torch.uint8)
        (self.kp, self.ks), (self.vp, self.vs) = pool(), pool()
        x = torch.randn(self.b * n, Hq + 2 * Hkv, D, generator=gen, device=DEV).bfloat16()
        self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        # a tree: every node sees itself and the nodes its parent sees
        see = torch.zeros(self.b, n, n, dtype=torch.bool, device=DEV)
        rows = torch.arange(self.b, device=DEV)
        for i in range(n):
            if i > 0:
                see[:, i] = see[rows, torch.randint(0, i, (self.b,), generator=gen, device=DEV)]
            see[:, i, i] = True
        self.see = see
        bits = (see.long() << torch.arange(n, device=DEV)).sum(-1)
        self.scale = 1 / math.sqrt(D) if scale is None else scale
        most = max(lens) if bound is None else bound
        self.ws = ops.Workspace(ops.spec_workspace_size(ops.OP_VERIFY_ATTENTION_Q8, self.b, n, 1, 1, Hq, Hkv, most))
        self.out = torch.empty(self.b * n, Hq, D, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.empty(self.b * n, Hq, device=DEV)
        self.args = (self.b, n, Hq, Hkv, D, page, self.q, self.k, self.v, self.kp, self.vp, self.ks, self.vs, self.table, i32(list(range(self.b))),
                     i32(lens), most, bits.reshape(-1), self.scale, self.out, self.lse, self.ws)

    def launch(self):
        _ops().spec_verify_attention_q8(*self.args)

    def reference(self):
        n, D, G = self.n, self.D, self.Hq // self.Hkv
        values = R.e4m3_values(torch.arange(256)).to(DEV)
        out = torch.empty(self.b * n, self.Hq, D, dtype=torch.float64, device=DEV)
        size, lse = torch.empty_like(out), torch.empty(self.b * n, self.Hq, dtype=torch.float64, device=DEV)
        dx = torch.empty_like(lse)
        for r, L in enumerate(self.lens):
            ids = self.table[r, :-(-L // self.page)].long()
            own = slice(r * n, (r + 1) * n)

            def keys(pages, scales, fresh):  # [Hkv, L + n, D]
                held = values[pages[ids].long()] * torch.exp2(scales[ids].double() - R.BIAS)[..., None, None]
                return torch.cat([held.transpose(0, 1).reshape(self.Hkv, -1, D)[:, :L], fresh[own].double().transpose(0, 1)], 1)
            k, v = keys(self.kp, self.ks, self.k), keys(self.vp, self.vs, self.v)
            q = self.q[own].double().reshape(n, self.Hkv, G, D).permute(1, 0, 2, 3).reshape(self.Hkv, n * G, D)
            hide = torch.cat([torch.zeros(n, L, dtype=torch.bool, device=DEV), ~self.see[r]], 1).repeat_interleave(G, 0)
            x = (self.scale * (q @ k.transpose(1, 2))).masked_fill(hide, -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - z[..., None])
            most = (abs(self.scale) * (q.abs() @ k.abs().transpose(1, 2))).masked_fill(hide, 0.0).amax(-1)

            def rows(t):
                return t.reshape(self.Hkv, n, G, *t.shape[2:]).transpose(0, 1).reshape(n, self.Hq, *t.shape[2:])
            out[own], size[own], lse[own], dx[own] = rows(p @ v), rows(p @ v.abs()), rows(z), rows(most)
        return out, lse, size, dx

    def check(self, want):
        out, lse, size, dx = want
        # fp32 products and sums of D terms move x by 2 (D + 8) 2^-24 dx; P is rounded to 2^-11, the output to 2^-8
        d = 2.0 ** -19 + 2 * (self.D + 8) * 2.0 ** -24 * dx
        off = (self.out.double() - out).abs() / (2.0 ** -8 * out.abs() + (2.0 ** -11 + d)[..., None] * size)
        assert torch.isfinite(self.out).all() and off.max() <= 1, float(off.max())
        dl = (self.lse.double() - lse).abs() / (d + 2.0 ** -22 * lse.abs())
        assert dl.max() <= 1, float(dl.max())


def mixed(b, short, long, seed):
    """Histories of 0, of a few keys and of up to `long`, in no order."""
    gen = torch.Generator().manual_seed(seed)
    kind = torch.randint(0, 4, (b,), generator=gen).tolist()
    few, many = torch.randint(0, short, (b,), generator=gen).tolist(), torch.randint(0, long, (b,), generator=gen).tolist()
    return [0 if k < 2 else few[i] if k == 2 else many[i] for i, k in enumerate(kind)]


@pytest.mark.parametrize("n, Hq, Hkv, D, page, lens", [
    (64, 32, 8, 128, 16, [2048] * 24),             # two groups of 128 rows, a tree tile every seventeenth
    (64, 32, 8, 128, 64, mixed(40, 300, 4000, 1)),
    (64, 16, 4, 64, 32, mixed(60, 300, 2000, 2)),
    (64, 16, 8, 128, 32, mixed(150, 200, 1500, 3)),  # 128 rows: the groups alternate tiles
    (48, 8, 8, 64, 16, mixed(300, 140, 1500, 4)),    # 48 rows, mostly units of one tile
    (64, 8, 8, 128, 64, [0] * 200 + [700]),
    (64, 20, 4, 128, 16, mixed(40, 200, 2500, 5)),   # 320 rows: a block of each kind
    (4, 32, 8, 128, 16, mixed(250, 300, 3000, 6)),
    (7, 32, 8, 64, 64, mixed(200, 300, 3000, 7)),
    (1, 16, 2, 128, 32, [30000, 5, 0, 17000]),
])
def test_attention_under_load(n, Hq, Hkv, D, page, lens):
    x = Load(n, Hq, Hkv, D, page, lens, seed=n + len(lens))
    x.launch()
    assert x.ws.last_error() == 0
    x.check(x.reference())
    first, z = x.out.clone(), x.lse.clone()
    for _ in range(20):
        x.out.fill_(3.0)
        x.launch()
        assert torch.equal(first, x.out) and torch.equal(z, x.lse)
    assert x.ws.last_error() == 0


@pytest.mark.parametrize("bound", [None, 1 << 20])
@pytest.mark.parametrize("n, Hq, Hkv, D, page, lens", [
    (1, 1, 1, 64, 16, [0, 1, 65, 130]), (1, 8, 8, 128, 32, [40, 0, 700]), (2, 6, 2, 128, 64, [0, 1, 65, 130]), (3, 5, 1, 64, 16, [2000]),
    (4, 32, 8, 128, 16, [1000]), (7, 16, 4, 64, 32, [1, 900, 16, 15]), (16, 8, 4, 128, 64, [300, 0, 17]), (32, 4, 4, 64, 16, [129, 1500]),
    (1, 16, 2, 128, 32, [30000, 5, 0, 17000]), (5, 12, 2, 128, 64, [12000]), (1, 8, 1, 64, 16, [0] * 15 + [4000]), (4, 8, 2, 128, 16, [333] * 36),
    (4, 8, 2, 64, 32, [100, 0, 3] * 25), (33, 7, 1, 128, 16, [200, 0, 1000]), (63, 4, 1, 64, 64, [65, 1]), (64, 10, 2, 128, 32, [0, 300]),
    (48, 8, 8, 64, 16, [129]), (64, 16, 2, 64, 16, [1500])])
def test_attention_by_clusters_and_by_the_whole_gpu(n, Hq, Hkv, D, page, lens, bound):
    """Few units: a cluster of CTAs takes each (of 8, 4, 2, 1), unless the bound of the lengths allows long ones; then
    the GPU's warps share the work, and long contexts are joined by CTA first."""
    x = Load(n, Hq, Hkv, D, page, lens, seed=3 * n + len(lens), bound=bound)
    x.launch()
    assert x.ws.last_error() == 0
    x.check(x.reference())
    first, z = x.out.clone(), x.lse.clone()
    for _ in range(5):
        x.out.fill_(3.0)
        x.launch()
        assert torch.equal(first, x.out) and torch.equal(z, x.lse)


@pytest.mark.parametrize("scale", [-0.11, 0.0])
@pytest.mark.parametrize("n, Hq, Hkv", [(4, 32, 8), (64, 16, 8), (64, 32, 8)])
def test_attention_scale_below_or_at_zero_under_load(n, Hq, Hkv, scale):
    x = Load(n, Hq, Hkv, 128, 32, mixed(30, 200, 1500, 9), seed=8, scale=scale)
    x.launch()
    assert x.ws.last_error() == 0
    x.check(x.reference())


def test_attention_on_two_streams_at_once():
    """Two calls with a workspace each, of both kernels, in flight together."""
    both = [Load(64, 16, 8, 128, 16, mixed(60, 300, 1500, 10), seed=1), Load(4, 32, 8, 128, 16, mixed(120, 300, 1500, 11), seed=2)]
    want = [x.reference() for x in both]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s in zip(both, streams):
            with torch.cuda.stream(s):
                x.launch()
    torch.cuda.synchronize()
    for x, w in zip(both, want):
        assert x.ws.last_error() == 0
        x.check(w)


def test_commit_of_more_pages_than_get_a_cta_for_each_layer():
    """A CTA takes K and V of several layers in turn: bytes and scales of whole prompts, against torch's own e4m3."""
    ops = _ops()
    b, page, Hkv, D, layers = 120, 16, 8, 64, 3
    gen = torch.Generator().manual_seed(12)
    lens = torch.randint(1, 700, (b,), generator=gen).tolist()
    lens[3], lens[50] = 0, 699
    start = [sum(lens[:r]) for r in range(b)]
    need = [-(-x // page) for x in lens]
    ids = torch.randperm(sum(need), generator=gen).tolist()
    table = torch.full((b, max(need)), -1, dtype=torch.int32)
    owner = []  # (page id, first row, rows) of every page
    for r in range(b):
        for p in range(need[r]):
            table[r, p] = ids.pop()
            owner.append((int(table[r, p]), start[r] + p * page, min(page, lens[r] - p * page)))
    on = torch.Generator(device=DEV).manual_seed(13)
    x = [[(torch.randn(sum(lens), Hkv, D, generator=on, device=DEV) * torch.exp2(torch.randint(-9, 10, (sum(lens), 1, 1), generator=on, device=DEV))).bfloat16()
          for _ in range(layers)] for _ in "kv"]
    pools = [[torch.full((sum(need), Hkv, page, D), 0x55, dtype=torch.uint8, device=DEV) for _ in range(layers)] for _ in "kv"]
    scales = [[torch.zeros(sum(need), Hkv, dtype=torch.uint8, device=DEV) for _ in range(layers)] for _ in "kv"]
    after, ws = torch.empty(b, dtype=torch.int32, device=DEV), ops.Workspace(ops.spec_workspace_size(ops.OP_COMMIT_KV_Q8, b, 1, 1, 1))
    ops.spec_commit_kv_q8(b, Hkv, D, page, x[0], x[1], pools[0], pools[1], scales[0], scales[1], table.to(DEV), i32(list(range(b))), i32([0] * b),
                          None, i32(start), i32(lens), 699, after, ws)
    assert ws.last_error() == 0 and after.tolist() == lens
    pid = torch.tensor([o[0] for o in owner], device=DEV)
    rows = torch.tensor([o[1] for o in owner], device=DEV)[:, None] + torch.arange(page, device=DEV)
    held = torch.arange(page, device=DEV) < torch.tensor([o[2] for o in owner], device=DEV)[:, None]
    for kv in range(2):
        for layer in range(layers):
            y = x[kv][layer].float()[torch.where(held, rows, 0)].transpose(1, 2)  # [pages, Hkv, page, D]
            there = held[:, None, :, None].expand_as(y)
            most = torch.where(there, y, 0.0).abs().amax((2, 3)).double()
            e = torch.full_like(most, 16.0)
            for k in range(100, 150):
                e = torch.where(most > 448 * 2.0 ** (k - 127), k + 1.0, e)
            assert torch.equal(scales[kv][layer][pid].double(), e)
            want = (y * torch.exp2(127 - e)[..., None, None].float()).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(pools[kv][layer][pid], torch.where(there, want, 0x55))
