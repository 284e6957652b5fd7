"""Measured cases of the operators that let requests share pages of a cache, and of
the attention of one new token that reads them:

  fork      children of a request share its whole pages (a count of further holders a
            page), get a page of their own for the part of one behind them, and copy it;
            then the children end and their pages are given back
  release   pages given back to the free list: those of a step's new tokens, or of
            whole requests, right after they were taken from it
  compact   the pages in use moved to the lowest ids: tables, counts, free list, and
            the pages of every layer
  decode    attention of one new token a request over the paged bf16 cache; requests
            of a group share the pages of their first tokens

``run`` computes them in elementary torch operations where ``own`` is false, and
through ``accept_select_top_gb300.ops`` where it is true.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    return [
        # eight samples of one prompt, every layer of a GQA model, with the slot table: latency and the tails
        dict(name="fork samples", kind="fork", b=1, fan=8, page=16, lo=1001, hi=1001, layers=32, heads=8, dim=128, q8=False, slots=True),
        # beams of a batch of ragged contexts over the 8-bit cache
        dict(name="fork beams", kind="fork", b=64, fan=4, page=64, lo=256, hi=4096, layers=8, heads=8, dim=128, q8=True, slots=False),
        # many samples of two long documents: tables and slot tables of a few million entries
        dict(name="fork long", kind="fork", b=2, fan=32, page=16, lo=32759, hi=131061, layers=2, heads=8, dim=128, q8=False, slots=True),
        # a verify step's slots of a large batch taken, and taken back
        dict(name="release step", kind="release", b=256, page=16, lo=256, hi=4096, new_lo=1, new_hi=64),
        # a batch of long requests ends
        dict(name="release batch", kind="release", b=256, page=16, lo=0, hi=0, new_lo=256, new_hi=16384),
        # a small cache after some requests have ended
        dict(name="compact churn", kind="compact", b=16, page=16, lo=64, hi=1024, fill=0.6, layers=4, heads=8, dim=128, q8=False, slots=True),
        # a cache of nine gigabytes, half of it free, before its upper half is given to something else
        dict(name="compact pool", kind="compact", b=64, page=32, lo=512, hi=8192, fill=0.5, layers=4, heads=8, dim=128, q8=False, slots=False),
        # latency: one request
        dict(name="decode one", kind="decode", groups=0, b=1, fan=1, lo=1001, hi=1001, tail=0, hq=32, hkv=8, dim=128, page=16),
        # a large batch of ragged contexts, nothing shared
        dict(name="decode batch", kind="decode", groups=0, b=256, fan=1, lo=256, hi=4096, tail=0, hq=32, hkv=8, dim=128, page=16),
        # samples of a few prompts
        dict(name="decode samples", kind="decode", groups=4, b=0, fan=16, lo=1024, hi=8192, tail=512, hq=32, hkv=8, dim=128, page=16),
        # beams of a batch, small heads, pages of one token
        dict(name="decode beams", kind="decode", groups=48, b=0, fan=4, lo=256, hi=4096, tail=64, hq=16, hkv=4, dim=64, page=1),
        # many samples of two long documents
        dict(name="decode long", kind="decode", groups=2, b=0, fan=32, lo=32768, hi=131072, tail=300, hq=64, hkv=8, dim=128, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    while True:
        kind = rng.choice(["fork", "release", "compact", "decode", "decode"])
        heads, dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64])
        if kind == "fork":
            c = dict(kind=kind, b=_log(rng, 1, 64), fan=_log(rng, 1, 32), page=page, lo=1, hi=_log(rng, 1, 131072), layers=_log(rng, 1, 32), heads=heads, dim=dim, q8=rng.random() < 0.5,
                     slots=rng.random() < 0.5)
            n = c["b"] * c["fan"]
            pool = (c["b"] * (c["hi"] // page + 1) + n) * c["layers"] * 2 * page * heads * dim * (1 if c["q8"] else 2)
            if n * c["hi"] > 64 * 131072 or pool > 10e9:
                continue
        elif kind == "release":
            c = dict(kind=kind, b=_log(rng, 1, 512), page=page, lo=0, hi=_log(rng, 1, 8192), new_lo=0, new_hi=_log(rng, 1, 16384))
            if c["b"] * (c["hi"] + c["new_hi"]) > 256 * 16384:
                continue
        elif kind == "compact":
            c = dict(kind=kind, b=_log(rng, 1, 64), page=page, lo=1, hi=_log(rng, 1, 8192), fill=round(rng.uniform(0.3, 0.95), 2), layers=_log(rng, 1, 8), heads=heads, dim=dim,
                     q8=rng.random() < 0.5, slots=rng.random() < 0.5)
            pages = c["b"] * (c["hi"] / 2 / page + 1) / c["fill"]
            if pages * c["layers"] * 2 * page * heads * dim * (1 if c["q8"] else 2) > 9e9:
                continue
        else:
            shared = rng.random() < 0.7
            g = _log(rng, 1, 64) if shared else 0
            c = dict(kind=kind, groups=g, b=0 if shared else _log(rng, 1, 256), fan=_log(rng, 1, 32) if shared else 1, lo=0, hi=_log(rng, 1, 131072), tail=_log(rng, 1, 1024) if shared else 0,
                     hq=heads * rng.choice([1, 2, 3, 4, 6, 8]), hkv=heads, dim=dim, page=rng.choice([1, 16, 32, 64]))
            keys = (g or c["b"]) * c["hi"] + g * c["fan"] * c["tail"]
            if keys * heads * dim > 1.1e9 or g * c["fan"] > 256 or g * c["fan"] * c["hi"] * c["hq"] * dim > 5e10:
                continue
        return c


def _between(case, what, lo, hi, count):
    r = random.Random("%s %s" % (what, sorted((k, v) for k, v in case.items() if k != "name")))
    return [r.randint(lo, hi) for _ in range(count)]


def _contexts(case, count, lo=None, hi=None):
    """Tokens of each request (or group): they are part of the case, not of the seed."""
    lo, hi = case["lo"] if lo is None else lo, case["hi"] if hi is None else hi
    return [lo, hi] if count == 2 and hi > lo else _between(case, "contexts", lo, hi, count)


def _decode_shape(case):
    """(shared tokens of each group, members of each group, tokens of each request)."""
    if not case["groups"]:
        return [], [], _contexts(case, case["b"])
    page = case["page"]
    shared = [x // page * page for x in _contexts(case, case["groups"])]
    fans = [case["fan"]] * 2 if case["groups"] == 2 else _between(case, "fan", (case["fan"] + 1) // 2, case["fan"], case["groups"])
    tails = iter(_between(case, "tail", 1, case["tail"], sum(fans)))
    return shared, fans, [s + next(tails) for s, f in zip(shared, fans) for _ in range(f)]


def _pages(x, page):
    return -(-x // page)


def _pair(case):
    """Requests of a compacted cache that share their first pages with the request before them, and how many."""
    lens, page = _contexts(case, case["b"]), case["page"]
    return [min(lens[r], lens[r - 1]) // 2 // page if r % 4 == 1 else 0 for r in range(case["b"])]


def work(case):
    kind = case["kind"]
    if kind == "fork":
        lens, page, fan = _contexts(case, case["b"]), case["page"], case["fan"]
        entries = sum(_pages(x, page) for x in lens) * fan
        whole = sum(x // page for x in lens)
        tails = sum(x % page > 0 for x in lens) * fan
        size = case["layers"] * 2 * (page * case["dim"] * (1 if case["q8"] else 2) + (1 if case["q8"] else 0)) * case["heads"]
        # pages copied; table entries read and written by the fork, read by the release; counts up and down; slots; lists
        return {"bytes": tails * (2 * size + 8 + 8) + 12 * entries + 16 * whole + (4 * sum(lens) * fan if case["slots"] else 0) + 24 * len(lens) * fan, "flops": 0}
    if kind == "release":
        lens, new = _contexts(case, case["b"]), _between(case, "new", case["new_lo"], case["new_hi"], case["b"])
        pages = sum(_pages(x + n, case["page"]) - _pages(x, case["page"]) for x, n in zip(lens, new))
        # an id, an entry, a slot and a position a token taken; an entry and a count read, an id written given back
        return {"bytes": 24 * case["b"] + 8 * pages + 8 * sum(new) + 12 * pages, "flops": 0}
    if kind == "compact":
        lens, page = _contexts(case, case["b"]), case["page"]
        entries = sum(_pages(x, page) for x in lens)
        live = entries - sum(_pair(case))
        total = int(live / case["fill"]) + 2
        moves = live * (total - live) / total
        size = case["layers"] * 2 * (page * case["dim"] * (1 if case["q8"] else 2) + (1 if case["q8"] else 0)) * case["heads"]
        return {"bytes": moves * (2 * size + 8) + 8 * entries + 16 * total + (4 * sum(lens) if case["slots"] else 0), "flops": 0}
    shared, fans, lens = _decode_shape(case)
    keys = sum(shared) + sum(lens) - sum(s * f for s, f in zip(shared, fans))
    row = case["hkv"] * case["dim"] * 4
    return {"bytes": keys * row + 4 * _pages(keys, case["page"]) + len(lens) * case["hq"] * (case["dim"] * 4 + 4), "flops": 4 * case["dim"] * case["hq"] * sum(lens)}


# ------------------------------------------------------------------ inputs

def _i32(v, dev="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _pools(case, pages, gen, dev):
    """K and V pages of every layer: bf16 slots, or e4m3 bytes with a scale byte for each page and head.  They are only
    moved, so the slots' bits ("k_bits", "v_bits") have to be equal."""
    layers, page, heads, dim = case["layers"], case["page"], case["heads"], case["dim"]
    if not case["q8"]:
        s = {x: torch.randn(layers, pages * page, heads, dim, generator=gen, device=dev, dtype=torch.bfloat16) for x in ("k", "v")}
        return {**s, "k_bits": s["k"].view(torch.int16), "v_bits": s["v"].view(torch.int16)}
    s = {x: torch.randint(0, 127, (layers, pages, heads, page, dim), generator=gen, device=dev, dtype=torch.uint8) for x in ("k", "v")}
    s.update({x: torch.randint(100, 130, (layers, pages, heads), generator=gen, device=dev, dtype=torch.uint8) for x in ("ks", "vs")})
    return s


def _fill(table, row, ids):
    table[row, : ids.numel()] = ids


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    kind, page = case["kind"], case["page"]
    s = dict(case=case, kind=kind, page=page)
    perm = lambda n: torch.randperm(n, generator=gen, device=dev).to(torch.int32)  # noqa: E731
    fixed = lambda shape, v=-1: torch.full(shape, v, dtype=torch.int32, device=dev)  # noqa: E731
    if kind == "fork":
        b, fan = case["b"], case["fan"]
        lens = _contexts(case, b)
        n, held = b * fan, sum(_pages(x, page) for x in lens)
        total = held + n + 5
        ids, rows = perm(total), perm(b + n + 2)
        s["table"] = fixed((b + n + 2, max(_pages(x, page) for x in lens) + 1))
        at = 0
        for r, x in enumerate(lens):
            _fill(s["table"], int(rows[r]), ids[at : at + _pages(x, page)])
            at += _pages(x, page)
        s.update(n=n, parents=rows[:b].repeat_interleave(fan).contiguous(), children=rows[b : b + n].contiguous(), lens=_i32([x for x in lens for _ in range(fan)]), counts=fixed((total,), 0),
                 free=ids[held:].contiguous(), n_free=_i32([n + 3]), slot_table=fixed((b + n + 2, s["table"].shape[1] * page)) if case["slots"] else None,
                 tails=sum(x % page > 0 for x in lens) * fan, src=fixed((n,)), dst=fixed((n,)), copies=fixed((1,)), left=fixed((1,)), back=fixed((1,)), most=max(lens))
        s.update(_pools(case, total, gen, dev))
    elif kind == "release":
        b = case["b"]
        lens, new = _contexts(case, b), _between(case, "new", case["new_lo"], case["new_hi"], b)
        need = sum(_pages(x + n, page) - _pages(x, page) for x, n in zip(lens, new))
        held = sum(_pages(x, page) for x in lens)
        total = held + need + 100
        ids, rows = perm(total), perm(b + 3)
        s["table"] = fixed((b + 3, max(_pages(x + n, page) for x, n in zip(lens, new)) + 1))
        counts = torch.tensor([_pages(x, page) for x in lens], device=dev)
        start, col = counts.cumsum(0) - counts, torch.arange(s["table"].shape[1], device=dev)
        s["table"][rows[:b].long()] = torch.where(col < counts[:, None], ids[(start[:, None] + col).clamp(max=total - 1)], -1)
        s.update(b=b, rows=rows[:b].contiguous(), lens=_i32(lens), new=_i32(new), after=_i32([x + n for x, n in zip(lens, new)]), counts=fixed((total,), 0), free=ids[held:].contiguous(),
                 n_free=_i32([need + 90]), cu=fixed((b + 1,)), map=fixed((max(1, sum(new)),)), pos=fixed((max(1, sum(new)),)), left=fixed((1,)), back=fixed((1,)), total=sum(new), most=max(new), slots=total * page)
    elif kind == "compact":
        b, lens, pair = case["b"], _contexts(case, case["b"]), _pair(case)
        live = sum(_pages(x, page) for x in lens) - sum(pair)
        total = int(live / case["fill"]) + 2
        ids, rows = perm(total), perm(b + 2)
        width = max(_pages(x, page) for x in lens) + 1
        s["table"], s["counts"] = fixed((b + 2, width)), fixed((total,), 0)
        at = 0
        for r, x in enumerate(lens):
            mine = ids[at : at + _pages(x, page) - pair[r]]
            at += mine.numel()
            if pair[r]:
                theirs = s["table"][int(rows[r - 1]), : pair[r]]
                s["counts"][theirs.long()] += 1
                mine = torch.cat([theirs, mine])
            _fill(s["table"], int(rows[r]), mine)
        s.update(b=b, rows=rows[:b].contiguous(), lens=_i32(lens), free=ids[live:].contiguous(), n_free=_i32([total - live]), slot_table=fixed((b + 2, width * page)) if case["slots"] else None,
                 new_table=fixed((b + 2, width)), new_slots=fixed((b + 2, width * page)) if case["slots"] else None, new_counts=fixed((total,)), new_free=fixed((total - live,)), left=fixed((1,)),
                 src=fixed((total - live,)), dst=fixed((total - live,)), moves=fixed((1,)), most=max(lens))
        s.update(_pools(case, total, gen, dev))
    else:
        hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
        shared, fans, lens = _decode_shape(case)
        b = len(lens)
        common = [x // page for x, f in zip(shared, fans) for _ in range(f)] if fans else [0] * b
        total = sum(x // page for x in shared) + sum(_pages(x, page) - c for x, c in zip(lens, common)) + 3
        ids, rows = perm(total), perm(b + 3)
        mine = torch.tensor([_pages(x, page) for x in lens], device=dev)
        ahead = torch.tensor(common, device=dev)
        group = [j for j, f in enumerate(fans) for _ in range(f)] if fans else [0] * b
        firsts = torch.tensor([0] + [x // page for x in shared], device=dev).cumsum(0)
        more = (mine - ahead).cumsum(0) + firsts[-1] - (mine - ahead)
        col = torch.arange(max(_pages(x, page) for x in lens) + 1, device=dev)
        at = torch.where(col < ahead[:, None], firsts[torch.tensor(group, device=dev)][:, None] + col, more[:, None] + col - ahead[:, None])
        table = fixed((b + 3, col.numel()))
        table[rows[:b].long()] = torch.where(col < mine[:, None], ids[at.clamp(0, total - 1)], -1)
        qkv = torch.randn(b, hq + 2 * hkv, dim, generator=gen, device=dev).to(torch.bfloat16)  # one packed projection's rows
        s.update(b=b, hq=hq, hkv=hkv, dim=dim, table=table, rows=rows[:b].contiguous(), lens=_i32(lens), most=max(lens), q=qkv[:, :hq], fans=fans, most_shared=max(shared + [0]),
                 starts=_i32([0] + fans).cumsum(0).to(torch.int32) if fans else None, shared=_i32(shared) if fans else None, tail=max([x - c * page for x, c in zip(lens, common)]),
                 out=torch.zeros(b, hq, dim, dtype=torch.bfloat16, device=dev), lse=torch.zeros(b, hq, dtype=torch.float32, device=dev))
        s.update({x: torch.randn(total * page, hkv, dim, generator=gen, device=dev, dtype=torch.bfloat16) for x in ("k", "v")})
    return s


# -------------------------------------------------------------------- runs

def run(s):
    if own:
        return _RUN_OWN[s["kind"]](s)
    return _RUN_PLAIN[s["kind"]](s)


def _answer(s, *names):
    return {x: s[x + "_bits" if x + "_bits" in s else x] for x in names if s.get(x) is not None}


_FORK = ("table", "counts", "src", "dst", "copies", "left", "free", "back", "slot_table", "k", "v", "ks", "vs")
_RELEASE = ("table", "counts", "free", "left", "back", "cu", "map", "pos")
_COMPACT = ("new_table", "new_slots", "new_counts", "new_free", "left", "src", "dst", "moves", "k", "v", "ks", "vs")


def _workspace(ops, s, *sizes):
    if "ws" not in s:
        s["ws"] = ops.Workspace(max(ops.spec_workspace_size(*x) for x in sizes))
    return s["ws"]


def _layers(ops, s):
    if "layered" not in s:
        s["layered"] = [ops.LayerList(s[x].unbind(0)) if x in s else None for x in ("k", "v", "ks", "vs")]
    return s["layered"]


def _own_fork(s):
    from accept_select_top_gb300 import ops
    n, page = s["n"], s["page"]
    ws = _workspace(ops, s, *((op, n, 1, 1, s["counts"].numel(), 0, 0, s["most"]) for op in (ops.OP_FORK_PAGES, ops.OP_COPY_PAGES, ops.OP_RELEASE_PAGES)))
    ops.spec_fork_pages(n, page, s["parents"], s["children"], s["lens"], s["counts"], s["free"], s["n_free"], s["table"], s["slot_table"], s["src"], s["dst"], s["copies"], s["left"], ws)
    ops.spec_copy_pages(page, *_layers(ops, s), s["src"], s["dst"], s["copies"], ws)
    ops.spec_release_pages(n, page, s["children"], s["lens"], None, s["counts"], s["free"], s["left"], s["table"], s["back"], ws)
    return _answer(s, *_FORK)


def _own_release(s):
    from accept_select_top_gb300 import ops
    ws = _workspace(ops, s, *((op, s["b"], 1, 1, s["counts"].numel()) for op in (ops.OP_ALLOC_SLOTS, ops.OP_RELEASE_PAGES)))
    ops.spec_alloc_slots(s["b"], s["page"], s["rows"], s["lens"], s["new"], s["most"], s["free"], s["n_free"], s["slots"], s["table"], None, s["cu"], s["map"], s["pos"], s["left"], ws)
    ops.spec_release_pages(s["b"], s["page"], s["rows"], s["after"], s["lens"], s["counts"], s["free"], s["left"], s["table"], s["back"], ws)
    return _answer(s, *_RELEASE)


def _own_compact(s):
    from accept_select_top_gb300 import ops
    ws = _workspace(ops, s, *((op, s["b"], 1, 1, s["counts"].numel(), 0, 0, s["most"]) for op in (ops.OP_COMPACT_PAGES, ops.OP_COPY_PAGES)))
    ops.spec_compact_pages(s["b"], s["page"], s["rows"], s["lens"], 0, s["counts"], s["free"], s["n_free"], s["table"], s["slot_table"], s["new_counts"], s["new_free"], s["left"], s["new_table"],
                           s["new_slots"], s["src"], s["dst"], s["moves"], ws)
    ops.spec_copy_pages(s["page"], *_layers(ops, s), s["src"], s["dst"], s["moves"], ws)
    return _answer(s, *_COMPACT)


def _own_decode(s):
    from accept_select_top_gb300 import ops
    ws = _workspace(ops, s, (ops.OP_DECODE_ATTENTION, s["b"], 1, 1, 1, s["hq"], s["hkv"], s["most"]))
    ops.spec_decode_attention(s["b"], s["hq"], s["hkv"], s["dim"], s["page"], s["q"], s["k"], s["v"], s["table"], s["rows"], s["lens"], s["most"], s["starts"], s["shared"],
                              1 / math.sqrt(s["dim"]), s["out"], s["lse"], ws)
    return _answer(s, "out", "lse")


def _ceil(a, m):
    return torch.div(a + (m - 1), m, rounding_mode="floor")


def _plain_copy(s, src, dst):
    """Pages src of every layer copied to dst."""
    for x in ("k", "v", "ks", "vs"):
        if x in s:
            pages = s[x] if s[x].shape[1] == s["counts"].numel() else s[x].view(s[x].shape[0], -1, s["page"], *s[x].shape[2:])
            pages[:, dst] = pages[:, src]


def _plain_release(s, rows, keep, lens, n_free, back):
    """The pages of the rows behind `keep` tokens: a holder less; those without one go back, first given up last."""
    page, table = s["page"], s["table"]
    first, last = _ceil(keep, page), _ceil(lens, page)
    col = torch.arange(table.shape[1], device=table.device)
    mine = ((col >= first[:, None]) & (col < last[:, None])).view(-1)
    ids = torch.where(mine, table[rows].view(-1).long(), s["counts"].numel())
    total = s["counts"].numel()
    given = torch.zeros(total + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, ids, torch.ones_like(ids))[:total]
    at = torch.arange(ids.numel(), device=ids.device)
    opened = torch.full((total + 1,), ids.numel(), device=ids.device).scatter_reduce_(0, ids, at, "amin")
    freed = given > s["counts"]
    goes = mine & (opened[ids] == at) & torch.nn.functional.pad(freed, (0, 1))[ids]
    count = goes.sum()
    rank = goes.cumsum(0) - 1
    to = torch.where(goes, n_free.long() + count - 1 - rank, s["free"].numel())
    s["free"].copy_(torch.nn.functional.pad(s["free"], (0, 1)).scatter_(0, to, ids.int())[:-1])
    s["counts"].copy_(torch.where(given > 0, (s["counts"] - given).clamp(min=0), s["counts"]))
    back.copy_(n_free + count)


def _plain_fork(s):
    page, table = s["page"], s["table"]
    parents, children, lens = s["parents"].long(), s["children"].long(), s["lens"].long()
    whole, part = lens // page, lens % page > 0
    j = part.cumsum(0) - part.long()
    fresh = s["free"][(s["n_free"].long() - 1 - j).clamp(0, s["free"].numel() - 1)]
    col = torch.arange(table.shape[1], device=table.device)
    theirs, shared = table[parents], col < whole[:, None]
    at = whole.clamp(max=table.shape[1] - 1)[:, None]
    now = torch.where(shared, theirs, table[children])
    now = torch.where((col == whole[:, None]) & part[:, None], fresh[:, None], now)
    table[children] = now
    total = s["counts"].numel()
    ids = torch.where(shared, theirs.long(), total).view(-1)
    s["counts"] += torch.zeros(total + 1, dtype=torch.int32, device=ids.device).scatter_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))[:total]
    if s["slot_table"] is not None:
        pos = torch.arange(s["slot_table"].shape[1], device=ids.device)
        slots = now[:, pos // page] * page + pos % page
        s["slot_table"][children] = torch.where(pos < lens[:, None], slots.int(), s["slot_table"][children])
    to = torch.where(part, j, s["n"])
    for name, what in (("src", theirs.gather(1, at)[:, 0]), ("dst", fresh)):
        s[name].copy_(torch.nn.functional.pad(s[name], (0, 1)).scatter_(0, to, what)[:-1])
    s["copies"].copy_(part.sum())
    s["left"].copy_(s["n_free"] - part.sum())
    if s["tails"]:
        _plain_copy(s, s["src"][: s["tails"]].long(), s["dst"][: s["tails"]].long())
    _plain_release(s, children, torch.zeros_like(lens), lens, s["left"], s["back"])
    return _answer(s, *_FORK)


def _plain_take(s):
    """Pages for the new tokens from the free list, their slots and positions."""
    page, lens, new = s["page"], s["lens"].long(), s["new"].long()
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    first, last = _ceil(lens, page), _ceil(lens + new, page)
    need = last - first
    before = need.cumsum(0) - need
    col = torch.arange(s["table"].shape[1], device=lens.device)[None]
    fresh = (col >= first[:, None]) & (col < last[:, None])
    at = s["n_free"].long() - 1 - (before[:, None] + col - first[:, None])
    rows = s["rows"].long()
    s["table"][rows] = torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], s["table"][rows])
    token = torch.arange(s["total"], device=lens.device)
    req = torch.searchsorted(cu, token, right=True) - 1
    pos = lens[req] + token - cu[req]
    s["cu"].copy_(cu)
    s["pos"][: s["total"]] = pos.int()
    s["map"][: s["total"]] = (s["table"][rows[req], pos // page].long() * page + pos % page).int()
    s["left"].copy_(s["n_free"] - need.sum())


def _plain_both(s):
    _plain_take(s)
    _plain_release(s, s["rows"].long(), s["lens"].long(), s["after"].long(), s["left"], s["back"])
    return _answer(s, *_RELEASE)


def _plain_compact(s):
    page, total = s["page"], s["counts"].numel()
    ids = torch.arange(total, device="cuda")
    idle = torch.zeros(total, dtype=torch.bool, device=ids.device)
    idle[s["free"].long()] = torch.arange(s["free"].numel(), device=ids.device) < s["n_free"]
    live = total - idle.sum()
    dst, src = torch.nonzero(idle & (ids < live)).view(-1), torch.nonzero(~idle & (ids >= live)).view(-1)
    to = ids.clone()
    to[src] = dst
    moves = src.numel()
    s["src"][:moves], s["dst"][:moves] = src.int(), dst.int()
    s["moves"].fill_(moves)
    s["new_counts"].copy_(s["counts"])
    s["new_counts"][dst] = s["counts"][src]
    s["new_counts"][src] = 0
    left = total - live
    at = torch.arange(s["new_free"].numel(), device=ids.device)
    s["new_free"].copy_(torch.where(at < left, total - 1 - at, s["new_free"]))
    s["left"].copy_(left)
    rows, lens = s["rows"].long(), s["lens"].long()
    col = torch.arange(s["table"].shape[1], device=ids.device)
    now = to[s["table"][rows].long().clamp(min=0)].int()
    s["new_table"][rows] = torch.where(col < _ceil(lens, page)[:, None], now, s["new_table"][rows])
    if s["new_slots"] is not None:
        pos = torch.arange(s["new_slots"].shape[1], device=ids.device)
        s["new_slots"][rows] = torch.where(pos < lens[:, None], now[:, pos // page] * page + (pos % page).int(), s["new_slots"][rows])
    _plain_copy(s, src, dst)
    return _answer(s, *_COMPACT)


def _plain_decode(s):
    b, hq, hkv, dim, page = (s[x] for x in ("b", "hq", "hkv", "dim", "page"))
    g, dev, lens, rows = hq // hkv, s["lens"].device, s["lens"].long(), s["rows"].long()
    q = s["q"].float().view(b, hkv, g, dim) / math.sqrt(dim)
    width = s["table"].shape[1] - 1

    def held(pool, row, pos, seen):
        slot = s["table"][row[:, None], (pos // page).clamp(max=width)].long() * page + pos % page
        return pool[torch.where(seen, slot, 0)].float().permute(0, 2, 3, 1)  # requests, heads, dim, keys

    base, scores, sums = torch.zeros_like(lens), [], []
    if s["starts"] is not None:  # the shared tokens, a group at a time
        starts, shared = s["starts"].long(), s["shared"].long()
        most = max(s["fans"])
        group = torch.searchsorted(starts, torch.arange(b, device=dev), right=True) - 1
        member = torch.arange(b, device=dev) - starts[group]
        base = shared[group]
        if s["most_shared"]:
            pos = torch.arange(s["most_shared"], device=dev)[None].expand(shared.numel(), -1)
            seen = pos < shared[:, None]
            padded = torch.zeros(shared.numel(), most, hkv, g, dim, device=dev)
            padded[group, member] = q
            x = padded.transpose(1, 2).reshape(shared.numel(), hkv, most * g, dim) @ held(s["k"], rows[starts[:-1]], pos, seen)
            scores.append(x.masked_fill_(~seen[:, None, None], -math.inf))
            values = held(s["v"], rows[starts[:-1]], pos, seen).transpose(2, 3)
            sums.append(lambda x: (x @ values).view(-1, hkv, most, g, dim)[group, :, member])
    pos = base[:, None] + torch.arange(max(1, s["tail"]), device=dev)
    seen = pos < lens[:, None]
    tail = (q @ held(s["k"], rows, pos, seen)).masked_fill_(~seen[:, None, None], -math.inf)
    top = tail.amax(dim=-1)
    if scores:
        first = scores[0].amax(dim=-1).view(-1, hkv, most, g)[group, :, member]
        top = torch.maximum(top, first)
    safe = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(tail - safe[..., None])
    z, o = p.sum(dim=-1), p @ held(s["v"], rows, pos, seen).transpose(2, 3)
    if scores:
        ref = torch.zeros(shared.numel(), hkv, most, g, device=dev)
        ref[group, :, member] = safe
        p = torch.exp(scores[0] - ref.view(-1, hkv, most * g, 1))
        z += p.sum(dim=-1).view(-1, hkv, most, g)[group, :, member]
        o += sums[0](p)
    s["out"].copy_((o / torch.where(z > 0, z, 1.0)[..., None]).view(b, hq, dim))
    s["lse"].copy_((torch.log(z) + top).view(b, hq))
    return _answer(s, "out", "lse")


_RUN_OWN = {"fork": _own_fork, "release": _own_release, "compact": _own_compact, "decode": _own_decode}
_RUN_PLAIN = {"fork": _plain_fork, "release": _plain_both, "compact": _plain_compact, "decode": _plain_decode}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    if case["kind"] != "decode":
        return None  # whole numbers, and bytes that are only moved
    s = prepare(case, seed)
    b, hq, hkv, dim, page = (s[x] for x in ("b", "hq", "hkv", "dim", "page"))
    out = torch.zeros(b, hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    rows, lens = s["rows"].tolist(), s["lens"].tolist()
    for r in range(b):
        if not lens[r]:
            continue
        pos = torch.arange(lens[r], device="cuda")
        slots = s["table"][rows[r]].long()[pos // page] * page + pos % page
        for h in range(hkv):
            mine = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = s["q"][r, mine].double() @ s["k"][slots, h].double().T * dim ** -0.5
            lse[r, mine] = torch.logsumexp(x, dim=-1)
            out[r, mine] = torch.softmax(x, dim=-1) @ s["v"][slots, h].double()
    return {"out": out, "lse": lse}
