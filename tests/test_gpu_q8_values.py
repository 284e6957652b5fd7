"""Verify attention over the 8-bit cache where values lie far apart: rows and pages of zeros,
tiny beside large ones, the type's largest.  A key counts in the softmax by its score alone,
whatever its value's size.

Bars.  Those of test_gpu_q8, and what P may lose below f16's range.  P_j = kappa p_j 2^e_j with e_j
the exponent that v_j is divided by, and its largest in a row is at least 2^5 (the reference
puts it into (2^5, 2^6] and only rises); so kappa >= 2^5 / M, M = max_j p_j 2^e_j.  Below 2^-14 an
f16 is off by at most 2^-25: out moves by at most
    2^-25 sum_j |v_j| 2^-e_j / kappa <= 2^-30 M sum_j |v_j| 2^-e_j.
A value whose exponent counts as the base's less 64 (M is taken with those: the base is at most the
largest exponent) is off by at most 2^-25 in v_j 2^-e_j: out moves by at most 2^-25 M for each of
the K keys (P_j / kappa <= M).  A subnormal bf16 is off by at most 2^-134."""
import math

import pytest
import torch

from tests import q8_reference as R
from tests.test_gpu_q8 import DEV, Att, _gen, _ops, bounds  # noqa: F401
from tests.test_gpu_q8_load import Load, mixed

pytestmark = pytest.mark.gpu

EXP_ONE = 118  # 448 * 2^(118 - 127) is just below 1


def reference(n, q, k_new, v_new, kp, vp, ks, vs, table, rows, lens, see, scale):
    """float64 (out, lse, bar of out, bar of lse) for [b*n] rows; see [b, n, n]."""
    Hq, D = q.shape[1:]
    Hkv = k_new.shape[1]
    G, page = Hq // Hkv, kp.shape[2]
    dev = q.device
    values = R.e4m3_values(torch.arange(256)).to(dev)
    got = [[] for _ in range(4)]
    for r, L in enumerate(lens):
        own = slice(r * n, (r + 1) * n)
        ids = table[rows[r], :-(-L // page)].long()

        def keys(pages, scales, fresh):  # [Hkv, L + n, D], and the exponents [Hkv, L + n]
            e = scales[ids].double() - R.BIAS
            held = (values[pages[ids].long()] * torch.exp2(e)[..., None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :L]
            x = fresh[own].double().transpose(0, 1)
            most = x.abs().amax(-1)
            ex = torch.where(most > 0, torch.floor(torch.log2(most.clamp(min=1e-300))) - 14, -200.0)
            return torch.cat([held, x], 1), torch.cat([e.repeat_interleave(page, 0).T[:, :L], ex], 1)
        (k, _), (v, e) = keys(kp, ks, k_new), keys(vp, vs, v_new)
        qq = q[own].double().reshape(n, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, n * G, D)
        hide = torch.cat([torch.zeros(n, L, dtype=torch.bool, device=dev), ~see[r]], 1).repeat_interleave(G, 0)
        x = (scale * (qq @ k.transpose(1, 2))).masked_fill(hide, -math.inf)
        z = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[..., None])
        dx = (abs(scale) * (qq.abs() @ k.abs().transpose(1, 2))).masked_fill(hide, 0.0).amax(-1)
        d = 2.0 ** -19 + 2 * (D + 8) * 2.0 ** -24 * dx
        out = p @ v
        M = (p * torch.exp2(torch.maximum(e, e.amax(-1, keepdim=True) - 64))[:, None]).amax(-1, keepdim=True)
        seen = (~hide).double()[None]
        lost = 2.0 ** -30 * M * (seen @ (v.abs() * torch.exp2(-e)[..., None])) + 2.0 ** -25 * M * seen.sum(-1, keepdim=True)
        bar = 2.0 ** -8 * out.abs() + (2.0 ** -11 + d)[..., None] * (p @ v.abs()) + lost + 2.0 ** -134

        def back(t):
            return t.reshape(Hkv, n, G, *t.shape[2:]).transpose(0, 1).reshape(n, Hq, *t.shape[2:])
        for to, t in zip(got, (out, z, bar, d + 2.0 ** -22 * torch.where(z == -math.inf, 0.0, z).abs())):
            to.append(back(t))
    return [torch.cat(t) for t in got]


def check(args):
    """Runs the call and compares; args as the entry point has them."""
    b, n, q, k, v, kp, vp, ks, vs, table, rows, lens, mask, scale, out, lse, ws = (args[i] for i in (0, 1, *range(6, 16), 17, 18, 19, 20, 21))
    out.fill_(7.0), lse.fill_(7.0)
    _ops().spec_verify_attention_q8(*args)
    assert ws.last_error() == 0
    see = ((mask.view(b, n, 1) >> torch.arange(n, device=DEV)) & 1).bool()
    want, z, bar, dz = reference(n, q, k, v, kp, vp, ks, vs, table, rows.tolist(), lens.tolist(), see, scale)
    none = z == -math.inf
    assert torch.equal(lse == -math.inf, none) and (out[none] == 0).all()
    assert torch.isfinite(out).all()
    off = ((out.double() - want).abs() / bar.clamp(min=1e-300))[~none]
    dl = ((lse.double() - z).abs() / dz)[~none]
    assert dl.max() <= 1 and off.max() <= 1, (float(off.max()), float(dl.max()))


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("cached", [0, 7, 10, 20])  # log2 of the cached values
@pytest.mark.parametrize("nodes", ["root", "leaf", "all", "all but one"])
@pytest.mark.parametrize("n", [1, 4, 33, 64])
def test_nodes_of_zeros(n, nodes, cached):
    """Weights of the zero rows from 1 down to 2^-12 and less beside cached values of every size."""
    a = Att(4, n, 8, 2, 128, 16, [0, 1, 20, 200], seed=n + cached, lo=EXP_ONE + cached, hi=EXP_ONE + cached + 2, scale=1.5 / math.sqrt(128))
    a.ks.copy_(torch.randint(116, 119, a.ks.shape, generator=_gen(1)).to(torch.uint8))
    v = a.v.view(4, n, 2, 128)
    if nodes == "root":
        v[:, 0] = 0
    elif nodes == "leaf":
        v[:, n - 1] = 0
    else:
        kept = v[:, n // 2].clone()
        v[:] = 0
        if nodes == "all but one":
            v[:, n // 2] = kept
    check(a.device())


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("cached", [0, 20])
@pytest.mark.parametrize("where", ["first", "last", "some", "all but one", "all"])
@pytest.mark.parametrize("n, D, page", [(1, 128, 16), (4, 64, 32), (33, 64, 16), (64, 128, 64), (64, 128, 16)])
def test_pages_of_zeros(n, D, page, where, cached):
    a = Att(3, n, 8, 2, D, page, [40, 333, 64], seed=n + cached, lo=EXP_ONE + cached, hi=EXP_ONE + cached + 2, scale=1.5 / math.sqrt(D))
    a.ks.copy_(torch.randint(116, 119, a.ks.shape, generator=_gen(2)).to(torch.uint8))
    for r, L in zip(a.rows, a.lens):
        ids = [int(a.table[r, p]) for p in range(-(-L // page))]
        for p in {"first": ids[:1], "last": ids[-1:], "some": ids[1::2], "all but one": ids[:len(ids) // 2] + ids[len(ids) // 2 + 1:], "all": ids}[where]:
            a.vp[p], a.vs[p] = 0, 16  # (as the commit leaves rows of zeros)
    check(a.device())


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("cached", [1, 8, 15])
@pytest.mark.parametrize("n, Hq", [(1, 2), (4, 8), (33, 4), (64, 4)])
def test_a_zero_node_of_every_weight(n, Hq, cached):
    """One cached key of weight 1 and one visible node of zeros, of weight 1 down to 2^-12."""
    b, D = 13, 64
    a = Att(b, n, Hq, 1, D, 16, [1] * b, seed=3, masks=[1] * (b * n), scale=1.0)
    a.q[:] = 0
    a.q[:, :, 0] = 1
    a.kp[:] = 0
    a.vp[:] = 0x7e  # 448
    a.vs[:] = 119 + cached
    a.k[:] = 0
    a.v[:] = 0
    for r in range(b):
        a.k[r * n, 0, 0] = -r * math.log(2.0)
    check(a.device())


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, D", [(1, 128), (4, 64), (20, 128), (33, 128), (64, 64), (64, 128)])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_value_scales_in_every_order(n, D, order):
    """Cached values from 2^-37 to 2^23 and nodes from 2^-30 to 2^30: larger ones after smaller, smaller after larger."""
    page = 16
    a = Att(3, n, 8, 2, D, page, [350, 77, 0], seed=4, lo=116, hi=119, scale=1.5 / math.sqrt(D))
    gen = _gen(5)
    for r, L in zip(a.rows, a.lens):
        count = -(-L // page)
        e = torch.randint(90, 151, (count, 2), generator=gen)
        if order != "mixed":
            e = e.sort(dim=0, descending=order == "falling").values
        for p in range(count):
            a.vs[int(a.table[r, p])] = e[p].to(torch.uint8)
    f = torch.randint(-30, 31, (a.x.shape[0],), generator=gen).double()
    a.v.copy_((a.v.double() * torch.exp2(f)[:, None, None]).bfloat16())
    check(a.device())


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, D", [(1, 128), (4, 64), (33, 128), (64, 64), (64, 128)])
@pytest.mark.parametrize("low", [-100, -60])
def test_all_values_tiny(n, D, low):
    """Tiny values with nothing larger beside them keep their bits, in the cache and in the tree."""
    a = Att(3, n, 8, 2, D, 16, [200, 3, 0], seed=12, lo=EXP_ONE + low, hi=EXP_ONE + low + 2, scale=1.5 / math.sqrt(D))
    a.ks.copy_(torch.randint(116, 119, a.ks.shape, generator=_gen(2)).to(torch.uint8))
    a.v.copy_((a.v.float() * 2.0 ** low).bfloat16())
    check(a.device())


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, Hq, D", [(1, 4, 128), (4, 8, 64), (16, 4, 128), (33, 4, 128), (64, 4, 64)])
@pytest.mark.parametrize("ahead", [20, 60, 100, 140])  # log2 of the weight of the small values' keys
@pytest.mark.parametrize("low", [16, 60, 95])
def test_small_values_of_great_weight_before_large_ones(n, Hq, D, ahead, low):
    """The base rises by up to 103 while the sum of weights is all the small values': of keys whose weights differ
    from one another by 2^12."""
    b, page = 40, 16
    a = Att(b, n, Hq, 1, D, page, [120] * b, seed=3, lo=119, hi=120, masks=[1 << i for _ in range(b) for i in range(n)], scale=ahead * math.log(2.0) / 16)
    a.q[:] = 0
    a.q[:, :, 0] = 4
    a.kp[:] = 0
    a.ks[:] = 127
    a.k[:] = 0
    a.v.copy_((a.v.float() * 8).bfloat16())
    for r in a.rows[:b]:
        p = int(a.table[r, 0])
        a.kp[p, 0, :, 0] = torch.tensor([0x48, 0x47, 0x46, 0x45, 0x44, 0x43, 0x42, 0x41] * 2)  # 4, 3.75 .. 2.25
        a.vs[p] = low
    check(a.device())


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, D", [(1, 128), (4, 64), (33, 128), (64, 64), (64, 128)])
@pytest.mark.parametrize("lens", [[2000, 3, 0], [200] * 40])
def test_values_near_the_types_largest(n, D, lens):
    """Values up to 2^122: sums of many stay an average."""
    a = Att(len(lens), n, 4, 1, D, 16, lens, seed=13, lo=EXP_ONE + 119, hi=EXP_ONE + 121, scale=0.1 / math.sqrt(D))
    a.ks.fill_(114)
    a.v.copy_((a.v.float() * 2.0 ** 119).bfloat16())
    check(a.device())


@pytest.mark.usefixtures("bounds")
@pytest.mark.parametrize("n, Hq", [(4, 8), (33, 4), (64, 8)])
def test_a_dominant_key_of_zeros(n, Hq):
    """Nearly all the weight on a zero row: what is left of the others is small, not lost, and lse is that row's."""
    a = Att(2, n, Hq, 1, 128, 16, [50, 300], seed=6, lo=130, hi=133, scale=1.0 / math.sqrt(128))
    a.ks.fill_(114)
    a.v[:] = 0
    a.k.view(2, n, 1, 128)[:, 0] = a.q.view(2, n, Hq, 128)[:, 0, :1] * 2
    check(a.device())


@pytest.mark.parametrize("bound", [None, 1 << 20])
@pytest.mark.parametrize("what", ["nodes", "pages", "far"])
@pytest.mark.parametrize("n, Hq, Hkv, D, page", [(64, 8, 2, 128, 16), (64, 4, 2, 64, 32), (33, 8, 2, 128, 64), (48, 8, 8, 64, 16), (4, 32, 8, 128, 16), (1, 8, 8, 64, 32)])
def test_zeros_and_far_values_under_load(n, Hq, Hkv, D, page, what, bound):
    """Pieces of several units a CTA: history and tree in one, in both ways the rows are shared out."""
    x = Load(n, Hq, Hkv, D, page, mixed(150, 300, 1500, n), seed=n, scale=1.5 / math.sqrt(D), lo=125, hi=129, bound=bound)
    x.ks.fill_(115)
    gen = torch.Generator(device=DEV).manual_seed(n)
    pages, rows = x.vs.shape[0], x.v.shape[0]
    if what == "nodes":
        x.v[torch.rand(rows, generator=gen, device=DEV) < 0.4] = 0
    elif what == "pages":
        empty = torch.rand(pages, generator=gen, device=DEV) < 0.4
        x.vp[empty], x.vs[empty] = 0, 16
    else:
        x.vs.copy_(torch.randint(95, 146, x.vs.shape, generator=gen, device=DEV))
        f = torch.randint(-25, 26, (rows, 1, 1), generator=gen, device=DEV)
        x.v.copy_((x.v.double() * torch.exp2(f.double())).bfloat16())
    check(x.args)


@pytest.mark.parametrize("bound", [None, 1 << 20])
@pytest.mark.parametrize("n, Hq, Hkv, D", [(2, 10, 2, 128), (4, 12, 4, 128), (8, 6, 2, 64), (16, 2, 2, 128), (64, 4, 2, 64)])
def test_short_histories_beside_zero_nodes_of_great_weight(n, Hq, Hkv, D, bound):
    """A zero node with nearly all the weight must not take the others' P below f16's range."""
    x = Load(n, Hq, Hkv, D, 16, [i % 7 for i in range(300)], seed=n, scale=4 / math.sqrt(D), lo=125, hi=126, bound=bound)
    x.ks.fill_(113)
    gen = torch.Generator(device=DEV).manual_seed(n)
    x.v.copy_((x.v.float() * 2.0 ** 4).bfloat16())
    x.v[torch.rand(x.v.shape[0], generator=gen, device=DEV) < 0.4] = 0
    check(x.args)
