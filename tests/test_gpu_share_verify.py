"""Forked requests through a verify step: pages for the tree's nodes, attention of the tree over the fork's slot tables, the
accepted rows' commit, the pages of the rest given back, and the one-token attention over what remains."""
import pytest
import torch

from tests.test_gpu_share import _gen, _ops, i32

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("page", [1, 16])
def test_verify_steps_of_samples(page):
    ops = _ops()
    Hq, Hkv, D, n, W, rows, width, total = 8, 2, 64, 21, 5, 6, -(-320 // page), -(-1100 // page)
    scale, gen = D ** -0.5, _gen(page)
    draw = lambda *s: torch.randn(*s, generator=gen).bfloat16().to(DEV)  # noqa: E731
    k, v = torch.zeros(total * page, Hkv, D, dtype=torch.bfloat16, device=DEV), torch.zeros(total * page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    t = dict(counts=i32([0] * total), free=i32(list(range(total))), n=i32([total]), table=i32([[-1] * width] * rows), slots=i32([[-1] * (width * page)] * rows))
    ws = ops.Workspace(max(ops.spec_workspace_size(op, rows, n if op in (ops.OP_VERIFY_ATTENTION, ops.OP_COMMIT_KV) else 1, 1, total, Hq, Hkv, 320) for op in
                           (ops.OP_ALLOC_SLOTS, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, ops.OP_DECODE_ATTENTION, ops.OP_VERIFY_ATTENTION, ops.OP_COMMIT_KV)))
    held = {}  # row -> its tokens' K and V

    def put(reqs, m):
        """m more slots a request, with K and V in them; the requests' tokens are not changed."""
        b = len(reqs)
        cu, slots, pos = i32([0] * (b + 1)), i32([-1] * (b * m)), i32([-1] * (b * m))
        lens = [held[r][0].shape[0] if r in held else 0 for r in reqs]
        ops.spec_alloc_slots(b, page, i32(reqs), i32(lens), i32([m] * b), m, t["free"], t["n"], total * page, t["table"], t["slots"], cu, slots, pos, t["n"], ws)
        kk, vv = draw(b * m, Hkv, D), draw(b * m, Hkv, D)
        k[slots.long()], v[slots.long()] = kk, vv
        return lens, slots, kk, vv

    def attention(q, kk, vv):
        x = q.double().view(Hkv, Hq // Hkv, D) @ kk.double().permute(1, 2, 0) * scale
        p = torch.softmax(x, dim=-1)
        return (p @ vv.double().transpose(0, 1)).view(Hq, D), (p @ vv.double().abs().transpose(0, 1)).view(Hq, D)

    def near(got, want, spread):  # (P and out rounded to bf16; scores of 64 products)
        assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * spread).all()

    def verify(reqs):
        b = len(reqs)
        lens, loc, kk, vv = put(reqs, n)
        parents = [-1] + [int(torch.randint(0, i, (1,), generator=gen)) for i in range(1, n)]
        paths = [[0]]
        for i in range(1, n):
            paths.append(paths[parents[i]] + [i])
        mask = torch.tensor([sum(1 << j for j in path) for path in paths] * b, dtype=torch.int64, device=DEV)
        q = draw(b * n, Hq, D)
        out, lse = torch.empty_like(q), torch.empty(b * n, Hq, device=DEV)
        ops.spec_verify_attention(b, n, Hq, Hkv, D, page, q, k, v, t["slots"], i32(reqs), i32(lens), 320, loc, mask, scale, out, lse, ws)
        accept, paths_of = [], []
        for i, r in enumerate(reqs):
            for node in range(0, n, 3):
                at = torch.tensor(paths[node], device=DEV) + i * n
                near(out[i * n + node], *attention(q[i * n + node], torch.cat([held[r][0], kk[at]]), torch.cat([held[r][1], vv[at]])))
            path = paths[int(torch.randint(0, n, (1,), generator=gen))][:W]
            paths_of.append(path)
            accept.append([i * n + x for x in path] + [-1] * (W - len(path)))
        new, freed, n_freed = i32([-1] * b), i32([-1] * (b * n)), i32([-1])
        ops.spec_commit_kv(b, n, W, Hkv, D, page, [k], [v], t["slots"], i32(reqs), i32(lens), loc, i32(accept), i32([len(p) for p in paths_of]), new, freed, n_freed, ws)
        assert new.tolist() == [x + len(p) for x, p in zip(lens, paths_of)]
        before = t["n"].tolist()[0]
        ops.spec_release_pages(b, page, i32(reqs), i32([x + n for x in lens]), new, t["counts"], t["free"], t["n"], t["table"], t["n"], ws)
        # the pages that go back are those of the commit's own free list
        assert sorted(t["free"][before:t["n"].tolist()[0]].tolist()) == sorted(freed[:n_freed.tolist()[0]].tolist())
        for i, (r, path) in enumerate(zip(reqs, paths_of)):
            at = torch.tensor(path, device=DEV) + i * n
            held[r] = (torch.cat([held[r][0], kk[at]]), torch.cat([held[r][1], vv[at]]))

    def check(groups):
        assert ws.last_error() == 0
        reqs = [r for _, m in groups for r in m]
        for r in reqs:
            at = t["slots"][r, :held[r][0].shape[0]].long()
            assert torch.equal(k[at], held[r][0]) and torch.equal(v[at], held[r][1])
        pages = {int(x) for r in reqs for x in t["table"][r, :-(-held[r][0].shape[0] // page)]}
        free = t["free"][:t["n"].tolist()[0]].tolist()
        assert sorted(list(pages) + free) == list(range(total))
        starts = [0]
        for _, m in groups:
            starts.append(starts[-1] + len(m))
        q = draw(len(reqs), Hq, D)
        out = torch.empty_like(q)
        ops.spec_decode_attention(len(reqs), Hq, Hkv, D, page, q, k, v, t["table"], i32(reqs), i32([held[r][0].shape[0] for r in reqs]), 320, i32(starts), i32([s for s, _ in groups]), scale, out,
                                  None, ws)
        for i, r in enumerate(reqs):
            near(out[i], *attention(q[i], *held[r]))
        assert ws.last_error() == 0

    def end(reqs):
        ops.spec_release_pages(len(reqs), page, i32(reqs), i32([held[r][0].shape[0] for r in reqs]), None, t["counts"], t["free"], t["n"], t["table"], t["n"], ws)
        for r in reqs:
            del held[r]

    for r, m in ((4, 150), (5, 33)):
        _, _, kk, vv = put([r], m)
        held[r] = (kk, vv)
    src, dst, count = i32([0] * 3), i32([0] * 3), i32([0])
    ops.spec_fork_pages(3, page, i32([4] * 3), i32([0, 1, 2]), i32([150, 150, 131]), t["counts"], t["free"], t["n"], t["table"], t["slots"], src, dst, count, t["n"], ws)
    ops.spec_copy_pages(page, [k], [v], None, None, src, dst, count, ws)
    for c, x in ((0, 150), (1, 150), (2, 131)):
        held[c] = (held[4][0][:x], held[4][1][:x])
    check([(128, [4, 0, 1, 2]), (0, [5])])
    for _ in range(3):
        verify([4, 0, 5, 1, 2])
        check([(144, [4, 0, 1]), (128, [2]), (0, [5])])
    end([4])
    for _ in range(2):
        verify([2, 1, 0, 5])
        check([(128, [0, 1, 2]), (0, [5])])
    end([0, 1, 2, 5])
    assert ws.last_error() == 0 and t["n"].tolist() == [total] and not t["counts"].any()
