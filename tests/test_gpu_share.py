"""Forks, copies, releases and compaction of pages on the GPU, equal to their plain forms, and runs of them with page
allocation as an engine that samples a prompt several times makes them."""
import pytest
import torch

from tests import share_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _ops():
    from accept_select_top_gb300 import ops
    return ops


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _ws(ops, *ops_of, b, pages):
    return ops.Workspace(max(ops.spec_workspace_size(op, b, 1, 1, pages) for op in ops_of))


class Cache:
    """Tables of `rows` requests over a pool, on both sides: `t` on the GPU, lists on the host."""

    def __init__(self, page, lens, rows, width, spare, seed=0, slots=False, slot_width=None):
        gen = _gen(seed)
        need = [-(-x // page) for x in lens]
        self.page, self.total = page, sum(need) + spare
        ids = torch.randperm(self.total, generator=gen).tolist()
        self.rows = torch.randperm(rows, generator=gen).tolist()
        self.table = [[-1] * width for _ in range(rows)]
        self.slots = [[-7] * (slot_width or width * page) for _ in range(rows)] if slots else None
        for r, k in zip(self.rows, need):
            for i in range(k):
                self.table[r][i] = ids.pop()
        self.free, self.n_free = ids + [-3] * (self.total - len(ids)), len(ids)
        self.counts = [0] * self.total
        self.t = {k: i32(v) for k, v in (("table", self.table), ("free", self.free), ("n", [self.n_free]), ("counts", self.counts))}
        self.t["slots"] = i32(self.slots) if slots else None

    def same(self):
        assert self.t["table"].tolist() == self.table
        assert self.t["counts"].tolist() == self.counts
        assert self.t["n"].tolist() == [self.n_free]
        assert self.t["free"].tolist() == self.free
        if self.slots is not None:
            assert self.t["slots"].tolist() == self.slots

    def fork(self, ws, parents, children, lens):
        ops = _ops()
        n = len(parents)
        src, dst, count = i32([-5] * n), i32([-5] * n), i32([-5])
        ops.spec_fork_pages(n, self.page, i32(parents), i32(children), i32(lens), self.t["counts"], self.t["free"], self.t["n"], self.t["table"], self.t["slots"], src, dst, count,
                            self.t["n"], ws)
        copies, self.n_free = R.fork(self.page, parents, children, lens, self.counts, self.free, self.n_free, self.table, self.slots)
        pad = n - len(copies)
        assert src.tolist() == [c[0] for c in copies] + [-5] * pad and dst.tolist() == [c[1] for c in copies] + [-5] * pad
        assert count.tolist() == [len(copies)]
        return src, dst, count

    def release(self, ws, rows, lens, keep=None):
        ops = _ops()
        ops.spec_release_pages(len(rows), self.page, i32(rows), i32(lens), None if keep is None else i32(keep), self.t["counts"], self.t["free"], self.t["n"], self.t["table"], self.t["n"], ws)
        self.n_free = R.release(self.page, rows, lens, keep or [0] * len(rows), self.counts, self.free, self.n_free, self.table)


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("lens, fan", [([0], 2), ([1], 1), ([16, 33, 64], 3), ([5, 64, 130, 0, 1000], 4), ([40] * 200, 2), ([9000], 40)])
def test_fork_and_release(page, lens, fan):
    ops = _ops()
    n = len(lens)
    c = Cache(page, lens, n * (fan + 1) + 1, -(-max(lens) // page) + 2, n * fan + 3, slots=True)
    before = (list(c.free), c.n_free)
    parents = [c.rows[i] for i in range(n) for _ in range(fan)]
    children = [c.rows[n + i] for i in range(n * fan)]
    at = [max(0, x - (i % 3)) for x in lens for i in range(fan)]  # (some from a little earlier)
    ws = _ws(ops, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, b=n * fan, pages=c.total)
    c.fork(ws, parents, children, at)
    assert ws.last_error() == 0
    c.same()
    c.release(ws, children, at)
    assert ws.last_error() == 0
    c.same()
    assert (c.free, c.n_free) == before  # what one call took goes back to where it was
    c.release(ws, c.rows[:n], lens)
    assert ws.last_error() == 0
    c.same()
    assert c.n_free == c.total and sorted(c.free) == list(range(c.total))


@pytest.mark.parametrize("slot_width", [130, 128, 161])
def test_fork_into_slot_tables_of_any_width(slot_width):
    ops = _ops()
    c = Cache(16, [100, 117], 5, 9, 9, slots=True, slot_width=slot_width)
    ws = _ws(ops, ops.OP_FORK_PAGES, b=3, pages=c.total)
    c.fork(ws, [c.rows[0], c.rows[1], c.rows[1]], c.rows[2:5], [100, 117, 48])
    assert ws.last_error() == 0
    c.same()


def test_forks_of_forks():
    """Children forked again, parents ending first: a page goes back with its last holder."""
    ops = _ops()
    c = Cache(16, [77], 8, 8, 20)
    ws = _ws(ops, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, b=4, pages=c.total)
    r = c.rows
    c.fork(ws, [r[0], r[0]], [r[1], r[2]], [77, 70])
    c.fork(ws, [r[1], r[1], r[2]], [r[3], r[4], r[5]], [77, 40, 64])
    c.release(ws, [r[0]], [77])
    c.same()
    c.release(ws, [r[4], r[1]], [40, 77])
    c.same()
    c.release(ws, [r[5], r[2], r[3]], [64, 70, 77])
    c.same()
    assert ws.last_error() == 0 and c.n_free == c.total and c.counts == [0] * c.total


@pytest.mark.parametrize("b, most", [(1, 10), (300, 600), (40, 20000)])
def test_release_cut_back(b, most):
    ops = _ops()
    gen = _gen(b)
    lens = torch.randint(0, most, (b,), generator=gen).tolist()
    keep = [int(torch.randint(0, x + 1, (1,), generator=gen)) for x in lens]
    c = Cache(16, lens, b + 1, -(-most // 16) + 1, 4)
    ws = _ws(ops, ops.OP_RELEASE_PAGES, b=b, pages=c.total)
    c.release(ws, c.rows[:b], lens, keep)
    assert ws.last_error() == 0
    c.same()


@pytest.mark.parametrize("b, width, total", [(50, 40, 500), (40, 4500, 5000), (40, 4500, 2000000), (80, 40000, 60000)])
def test_release_of_pages_held_in_one_call_and_outside(b, width, total):
    """Pages shared among the call's requests and one outside of it, in a random pattern; the same row twice is an error of the caller that is told."""
    ops = _ops()
    gen = _gen(3)
    table = torch.randint(0, total, (b, width), generator=gen).tolist()
    lens = torch.randint(0, width * 4 + 1, (b,), generator=gen).tolist()
    held = {}
    for r in range(b):
        for i in range(-(-lens[r] // 4)):
            held[table[r][i]] = held.get(table[r][i], 0) + 1
    counts = [max(0, held.get(p, 0) - 1 + (p % 3 == 0)) for p in range(total)]
    free, n_free = [-1] * total, 0
    t = dict(counts=i32(counts), free=i32(free), n=i32([0]), table=i32(table))
    ws = _ws(ops, ops.OP_RELEASE_PAGES, b=b, pages=total)
    n_free = R.release(4, range(b), lens, [0] * b, counts, free, n_free, table)
    ops.spec_release_pages(b, 4, i32(list(range(b))), i32(lens), None, t["counts"], t["free"], t["n"], t["table"], t["n"], ws)
    assert ws.last_error() == 0
    assert t["counts"].tolist() == counts and t["free"].tolist() == free and t["n"].tolist() == [n_free]
    two = dict(counts=i32([0, 0]), free=i32([9, 9]), n=i32([0]))
    ops.spec_release_pages(2, 4, i32([0, 0]), i32([8, 8]), None, two["counts"], two["free"], two["n"], i32([[0, 1]]), two["n"], ws)
    assert ws.last_error() == ops.DEV_INVARIANT
    assert two["free"].tolist() == [1, 0] and two["n"].tolist() == [2] and two["counts"].tolist() == [0, 0]


@pytest.mark.parametrize("total, b, fill", [(1, 1, 1.0), (5, 2, 0.5), (64, 3, 0.0), (31, 2, 0.9), (1000, 30, 0.5), (33000, 40, 0.7), (70000, 300, 0.2)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("extra", [0, 7])
def test_compact(total, b, fill, in_place, extra):
    ops = _ops()
    gen = _gen(total + b)
    live = int(total * fill)
    ids = torch.randperm(total, generator=gen).tolist()
    used, free = ids[:live], ids[live:]
    n_free = len(free)
    free = free + [-2] * 3
    page, width = 4, live // b + 2
    rows = torch.randperm(b + 1, generator=gen).tolist()[:b]
    table, lens = [[-1] * width for _ in range(b + 1)], []
    for i, r in enumerate(rows):
        mine = used[i * live // b:(i + 1) * live // b]
        table[r][:len(mine)] = mine
        lens.append(max(0, len(mine) * page - i % page))
    slots = [[-7] * (width * page) for _ in range(b + 1)]
    counts = [0] * total
    for p in used:
        counts[p] = p % 5
    limit = live + extra if extra else 0
    t = dict(counts=i32(counts), free=i32(free), n=i32([n_free]), table=i32(table), slots=i32(slots))
    new = t if in_place else dict(counts=i32([-9] * total), free=i32([-2] * len(free)), n=i32([-9]), table=i32(table), slots=i32(slots))
    kept = {k: v.clone() for k, v in t.items()}
    src, dst, moved = i32([-5] * len(free)), i32([-5] * len(free)), i32([-5])
    ws = _ws(ops, ops.OP_COMPACT_PAGES, b=b, pages=total)
    ops.spec_compact_pages(b, page, i32(rows), i32(lens), limit, t["counts"], t["free"], t["n"], t["table"], t["slots"], new["counts"], new["free"], new["n"], new["table"], new["slots"],
                           src, dst, moved, ws)
    assert ws.last_error() == 0
    if not in_place:
        assert all(torch.equal(t[k], kept[k]) for k in t)
    moves, left = R.compact(page, rows, lens, limit, counts, free, n_free, table, slots)
    assert moved.tolist() == [len(moves)] and new["n"].tolist() == [left]
    assert src.tolist()[:len(moves)] == [m[0] for m in moves] and dst.tolist()[:len(moves)] == [m[1] for m in moves]
    assert src.tolist()[len(moves):] == [-5] * (len(free) - len(moves))
    assert new["counts"].tolist() == counts and new["free"].tolist() == free
    assert new["table"].tolist() == table and new["slots"].tolist() == slots


def _bits(x):
    return x.view(torch.uint8)  # (random bits: NaNs among them)


def _pools(layers, pages, page, heads, dim, quantised, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *shape: torch.randint(0, 256, shape, generator=gen, device=DEV, dtype=torch.uint8)  # noqa: E731
    if quantised:
        return [[rand(pages, heads, page, dim) for _ in range(layers)] for _ in range(2)] + [[rand(pages, heads) for _ in range(layers)] for _ in range(2)]
    return [[rand(pages * page, heads, dim * 2).view(torch.bfloat16) for _ in range(layers)] for _ in range(2)] + [None, None]


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("layers, pages, page, heads, dim, n", [(1, 4, 16, 1, 64, 1), (3, 40, 16, 8, 128, 17), (2, 30, 64, 3, 128, 0), (128, 12, 1, 1, 64, 5), (2, 300, 32, 5, 64, 140)])
def test_copy(quantised, layers, pages, page, heads, dim, n):
    ops = _ops()
    pools = _pools(layers, pages, page, heads, dim, quantised)
    ids = torch.randperm(pages, generator=_gen(n)).tolist()
    src, dst = ids[:n], ids[n:2 * n]
    want = []
    for p in pools:
        for x in p or []:
            y = x.view(torch.uint8).reshape(pages, -1).clone()
            y[dst] = y[src]
            want.append(y)
    ws = _ws(ops, ops.OP_COPY_PAGES, b=1, pages=pages)
    more = 2
    ops.spec_copy_pages(page, *pools, i32(src + [0] * more), i32(dst + [1] * more), i32([n]), ws)
    assert ws.last_error() == 0
    got = [x.view(torch.uint8).reshape(pages, -1) for p in pools for x in p or []]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_copy_leaves_out_bad_pairs_and_counts():
    ops = _ops()
    pools = _pools(2, 6, 16, 2, 64, False)
    before = [[x.clone() for x in p] for p in pools[:2]]
    ws = _ws(ops, ops.OP_COPY_PAGES, b=1, pages=6)
    ops.spec_copy_pages(16, *pools, i32([-1, 6, 2, 0]), i32([1, 1, 7, 3]), i32([4]), ws)
    assert ws.last_error() == ops.DEV_INDEX
    for p, q in zip(pools[:2], before):
        for x, y in zip(p, q):
            y[3 * 16:4 * 16] = y[:16]
            assert torch.equal(_bits(x), _bits(y))
    ops.spec_copy_pages(16, *pools, i32([0]), i32([1]), i32([2]), ws)  # more than there are
    assert ws.last_error() == ops.DEV_LENGTH
    ops.spec_copy_pages(16, *pools, i32([0]), i32([2]), i32([-1]), ws)
    assert ws.last_error() == ops.DEV_LENGTH
    got, was = _bits(pools[0][0]), _bits(before[0][0])
    assert torch.equal(got[16:32], was[:16]) and torch.equal(got[32:48], was[32:48])


def test_refused_on_the_device():
    """Lists that are too short, lengths and rows out of range: told, and nothing (of that request) is changed."""
    ops = _ops()
    c = Cache(16, [100, 40], 5, 8, 3)
    ws = _ws(ops, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, ops.OP_COMPACT_PAGES, b=4, pages=c.total)
    r, t = c.rows, c.t
    src, dst, n = i32([-5] * 4), i32([-5] * 4), i32([-5])

    def fork(parents, children, lens):
        ops.spec_fork_pages(len(lens), 16, i32(parents), i32(children), i32(lens), t["counts"], t["free"], t["n"], t["table"], None, src, dst, n, t["n"], ws)

    fork([r[0]] * 4, r[1:5], [100] * 4)  # four pages are needed, three are there
    assert ws.last_error() == ops.DEV_SPACE and n.tolist() == [0]
    c.same()
    fork([r[0], -1, r[0], r[1]], [r[2], r[3], 5, r[1]], [-1, 10, 10, 10])
    assert ws.last_error() == ops.DEV_INDEX | ops.DEV_LENGTH and n.tolist() == [0]
    c.same()
    fork([r[0]], [r[2]], [16 * 8 + 1])
    assert ws.last_error() == ops.DEV_LENGTH
    c.same()
    fork([r[0], r[0]], [r[2], r[3]], [1000, 99])  # one bad, one good
    assert ws.last_error() == ops.DEV_LENGTH
    R.fork(16, [r[0]], [r[3]], [99], c.counts, c.free, c.n_free, c.table)
    c.n_free -= 1
    c.same()

    def release(rows, lens, keep=None, cap=None):
        free = t["free"] if cap is None else t["free"][:cap]
        ops.spec_release_pages(len(rows), 16, i32(rows), i32(lens), None if keep is None else i32(keep), t["counts"], free, t["n"], t["table"], t["n"], ws)

    release([r[0], 5, -1], [16 * 9, 10, 10])
    assert ws.last_error() == ops.DEV_INDEX | ops.DEV_LENGTH
    c.same()
    release([r[0]], [100], [101])
    assert ws.last_error() == ops.DEV_LENGTH
    c.same()
    release([r[1]], [40], cap=c.n_free + 2)  # three pages, room for two
    assert ws.last_error() == ops.DEV_SPACE
    c.same()
    t["n"].fill_(-1)
    release([r[1]], [40])
    assert ws.last_error() == ops.DEV_SPACE and t["n"].tolist() == [-1]
    moves = i32([-5])
    ops.spec_compact_pages(1, 16, i32([r[1]]), i32([40]), 0, t["counts"], t["free"], t["n"], t["table"], None, t["counts"], t["free"], t["n"], t["table"], None, src.repeat(9), dst.repeat(9), moves, ws)
    assert ws.last_error() == ops.DEV_SPACE and moves.tolist() == [0]
    t["n"].fill_(c.n_free)
    c.same()


def test_bad_page_ids_are_told_and_passed_over():
    ops = _ops()
    ws = _ws(ops, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, ops.OP_COMPACT_PAGES, b=4, pages=8)
    counts, free, n = i32([0] * 8), i32([5, 99, 6]), i32([3])
    table, slots = i32([[0, -1, 2], [7, 7, 7], [7, 7, 7]]), i32([[-7] * 48] * 3)
    src, dst, copies, left = i32([-5, -5]), i32([-5, -5]), i32([-5]), i32([-5])
    ops.spec_fork_pages(2, 16, i32([0, 0]), i32([1, 2]), i32([40, 40]), counts, free, n, table, slots, src, dst, copies, left, ws)
    assert ws.last_error() == ops.DEV_INDEX
    assert table.tolist() == [[0, -1, 2], [0, -1, 6], [0, -1, -1]] and counts.tolist() == [2, 0, 0, 0, 0, 0, 0, 0]
    assert src.tolist() == [2, 2] and dst.tolist() == [6, 99] and left.tolist() == [1]
    assert slots[1].tolist() == list(range(16)) + [-1] * 16 + list(range(96, 104)) + [-7] * 8 and slots[2][32:40].tolist() == [-1] * 8
    ops.spec_release_pages(2, 16, i32([1, 2]), i32([40, 40]), None, counts, free, left, table, left, ws)
    assert ws.last_error() == ops.DEV_INDEX
    assert left.tolist() == [2] and free.tolist() == [5, 6, 6] and counts.tolist() == [0] * 8
    # a free list with a bad id and one twice; a table entry that is on it
    free, n, table = i32([5, 8, 1, 5, 0]), i32([5]), i32([[7, 6, 1, -4]])
    src, dst = i32([-5] * 5), i32([-5] * 5)
    ops.spec_compact_pages(1, 16, i32([0]), i32([64]), 0, counts, free, n, table, None, counts, free, n, table, None, src, dst, copies, ws)
    assert ws.last_error() == ops.DEV_INDEX | ops.DEV_INVARIANT
    # in use: 2, 3, 4, 6, 7; five pages are the limit: 6 and 7 move to 0 and 1
    assert n.tolist() == [3] and copies.tolist() == [2] and src.tolist()[:2] == [6, 7] and dst.tolist()[:2] == [0, 1]
    assert table.tolist() == [[1, 0, 1, -1]] and free.tolist()[:3] == [7, 6, 5]


def test_binding_refusals():
    ops = _ops()
    ws = _ws(ops, ops.OP_FORK_PAGES, b=2, pages=8)
    x, table, pools = i32([0, 1]), i32([[0, 1], [2, 3]]), _pools(2, 4, 16, 2, 64, False)
    q8 = _pools(2, 4, 16, 2, 64, True)
    good = dict(parents=x, children=x, lens=x, counts=i32([0] * 8), free=x, n=x, table=table, slots=None, src=i32([0] * 2), dst=i32([0] * 2), copies=i32([0]), left=i32([0]))
    for bad in (dict(parents=x.long()), dict(children=x[:1]), dict(lens=x.cpu()), dict(src=i32([0] * 4)[::2]), dict(slots=i32([[0] * 8])), dict(dst=i32([0]))):
        with pytest.raises(ops.SpecError):
            ops.spec_fork_pages(2, 16, *{**good, **bad}.values(), ws)
    one = i32([0])
    for args in ((16, pools[0], pools[1][:1], None, None), (16, pools[0], pools[1], q8[2], q8[3]), (16, q8[0], q8[1], None, None), (32, q8[0], q8[1], q8[2], q8[3]),
                 (16, q8[0], pools[1], None, None), (16, [p.float() for p in pools[0]], pools[1], None, None), (128, pools[0], pools[1], None, None),
                 (16, q8[0], q8[1], [s[:2].contiguous() for s in q8[2]], q8[3])):
        with pytest.raises(ops.SpecError):
            ops.spec_copy_pages(*args, one, one, one, ws)
    with pytest.raises(ops.SpecError):
        ops.spec_compact_pages(1, 16, x, x, 0, x, x, x, table, None, x, x[:1], x, table, None, x, x, x, ws)
    with pytest.raises(ops.SpecError):
        ops.spec_compact_pages(1, 16, x, x, 0, x, x, x, table, None, x, x, x, table[:1], None, x, x, x, ws)


def test_captured_and_replayed():
    """A step's fork, copy and release in one graph, replayed, on a stream of its own."""
    ops = _ops()
    c = Cache(16, [50, 20], 6, 8, 8)
    pools = _pools(2, c.total, 16, 2, 64, False)
    keep = [[x.clone() for x in p] for p in pools[:2]]
    ws = _ws(ops, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, b=4, pages=c.total)
    layers = [ops.LayerList(p) for p in pools[:2]]
    r, t = c.rows, c.t
    parents, children, lens = i32([r[0], r[0], r[1], r[1]]), i32(r[2:6]), i32([50, 48, 20, 7])
    src, dst, n, left = i32([-5] * 4), i32([-5] * 4), i32([-5]), i32([-5])

    def step():
        ops.spec_fork_pages(4, 16, parents, children, lens, t["counts"], t["free"], t["n"], t["table"], None, src, dst, n, left, ws)
        ops.spec_copy_pages(16, *layers, None, None, src, dst, n, ws)
        ops.spec_release_pages(4, 16, children, lens, None, t["counts"], t["free"], left, t["table"], left, ws)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert ws.last_error() == 0
    copies, _ = R.fork(16, [r[0], r[0], r[1], r[1]], r[2:6], [50, 48, 20, 7], c.counts, c.free, c.n_free, c.table)
    R.release(16, r[2:6], [50, 48, 20, 7], [0] * 4, c.counts, c.free, c.n_free - len(copies), c.table)
    c.same()
    for p, q in zip(pools[:2], keep):
        for x, y in zip(p, q):
            for a, b in copies:
                y[b * 16:b * 16 + 16] = y[a * 16:a * 16 + 16]
            assert torch.equal(_bits(x), _bits(y))


def test_wide_release_captured_and_replayed():
    """Many rows: the release is one launch over many SMs.  Forks of a long prompt given back in one graph, three
    times; then every holder's pages in one call."""
    ops = _ops()
    page, fan, L = 4, 60, 20001
    c = Cache(page, [L], fan + 1, 5002, fan + 4)
    ws = _ws(ops, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, b=fan + 1, pages=c.total)
    r, t = c.rows, c.t
    before = (list(c.free), c.n_free, list(c.counts))
    parents, children, lens = i32([r[0]] * fan), i32(r[1:]), i32([L - i for i in range(fan)])
    src, dst, n, left = i32([-5] * fan), i32([-5] * fan), i32([-5]), i32([-5])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.spec_fork_pages(fan, page, parents, children, lens, t["counts"], t["free"], t["n"], t["table"], None, src, dst, n, left, ws)
        ops.spec_release_pages(fan, page, children, lens, None, t["counts"], t["free"], left, t["table"], left, ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert ws.last_error() == 0
    assert (t["free"].tolist(), left.tolist()[0], t["counts"].tolist()) == before
    c.fork(ws, [r[0]] * fan, r[1:], [L - i for i in range(fan)])
    c.release(ws, r, [L] + [L - i for i in range(fan)])
    assert ws.last_error() == 0
    c.same()
    assert c.n_free == c.total


def test_engine_run():
    """Prompts admitted, sampled several times, grown, ended in another order, the cache compacted, and what every
    request holds read back after each step: the values written into each token's slot follow the request."""
    ops = _ops()
    page, heads, dim, rows, width = 16, 2, 64, 12, 12
    total = 70
    k = torch.zeros(total * page, heads, dim, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    t = dict(counts=i32([0] * total), free=i32(list(range(total))[::-1]), n=i32([total]), table=i32([[-1] * width] * rows), slots=i32([[-1] * (width * page)] * rows))
    ws = _ws(ops, ops.OP_ALLOC_SLOTS, ops.OP_FORK_PAGES, ops.OP_RELEASE_PAGES, ops.OP_COMPACT_PAGES, b=rows, pages=total)
    tokens = {}  # row -> its tokens' values
    stamp = [0]

    def grow(more):
        reqs = list(more)
        b, lens = len(reqs), [len(tokens.get(r, [])) for r in reqs]
        new = [more[r] for r in reqs]
        cu, slots, pos = i32([0] * (b + 1)), i32([-1] * sum(new)), i32([-1] * sum(new))
        ops.spec_alloc_slots(b, page, i32(reqs), i32(lens), i32(new), max(new), t["free"], t["n"], total * page, t["table"], t["slots"], cu, slots, pos, t["n"], ws)
        values = torch.arange(stamp[0], stamp[0] + sum(new)) % 251
        stamp[0] += sum(new)
        k[slots.long()] = values.to(DEV).bfloat16()[:, None, None]
        v[slots.long()] = -values.to(DEV).bfloat16()[:, None, None]
        at = 0
        for r, m in zip(reqs, new):
            tokens.setdefault(r, []).extend(values[at:at + m].tolist())
            at += m

    def fork(parent, children, lens):
        n = len(children)
        src, dst, count = i32([0] * n), i32([0] * n), i32([0])
        ops.spec_fork_pages(n, page, i32([parent] * n), i32(children), i32(lens), t["counts"], t["free"], t["n"], t["table"], t["slots"], src, dst, count, t["n"], ws)
        ops.spec_copy_pages(page, [k], [v], None, None, src, dst, count, ws)
        for c, x in zip(children, lens):
            tokens[c] = tokens[parent][:x]

    def end(reqs):
        ops.spec_release_pages(len(reqs), page, i32(reqs), i32([len(tokens[r]) for r in reqs]), None, t["counts"], t["free"], t["n"], t["table"], t["n"], ws)
        for r in reqs:
            del tokens[r]

    def compact():
        reqs = list(tokens)
        src, dst, count = i32([0] * total), i32([0] * total), i32([0])
        ops.spec_compact_pages(len(reqs), page, i32(reqs), i32([len(tokens[r]) for r in reqs]), 0, t["counts"], t["free"], t["n"], t["table"], t["slots"], t["counts"], t["free"], t["n"],
                               t["table"], t["slots"], src, dst, count, ws)
        ops.spec_copy_pages(page, [k], [v], None, None, src, dst, count, ws)
        held = {int(t["table"][r, i]) for r in tokens for i in range(-(-len(tokens[r]) // page))}
        assert held == set(range(len(held)))

    def check():
        assert ws.last_error() == 0
        held = set()
        for r, x in tokens.items():
            slots = t["slots"][r, :len(x)].long()
            ids = t["table"][r, torch.arange(len(x), device=DEV) // page].long()
            assert torch.equal(slots, ids * page + torch.arange(len(x), device=DEV) % page)
            want = torch.tensor(x, device=DEV).bfloat16()[:, None, None].expand(-1, heads, dim)
            assert torch.equal(k[slots], want) and torch.equal(v[slots], -want)
            held |= set(ids.tolist())
        n = int(t["n"])
        assert sorted(held | set(t["free"][:n].tolist())) == list(range(total)) and len(held) + n == total

    grow({3: 100, 7: 33, 0: 16})
    check()
    fork(3, [1, 2, 4], [100, 100, 90])
    fork(7, [5], [32])
    check()
    grow({3: 5, 1: 9, 2: 1, 4: 40, 5: 3, 7: 1})
    check()
    end([3, 0])
    check()
    compact()
    check()
    fork(1, [6, 8], [109, 64])
    grow({1: 20, 6: 1, 8: 30})
    check()
    end([1, 7, 4])
    compact()
    check()
    end([2, 5, 6, 8])
    check()
    assert int(t["n"]) == total and t["counts"].sum() == 0
