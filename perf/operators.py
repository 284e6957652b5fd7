"""Measured cases of the operators around the 8-bit paged KV cache and the
token log probabilities of a verify step:

  alloc      pages for new tokens from the free list: block table, slot map, positions
  commit     accepted (or prefilled) bf16 K/V rows quantised into e4m3 pages, one
             power-of-two scale for each (page, kv head)
  attention  tree-masked verify attention over the e4m3 pages and the step's own
             bf16 K/V rows (one token a request is plain decoding)
  logprobs   log probability of given tokens, entropy and the k best alternatives of
             verify rows

``run`` computes them in elementary torch operations where ``own`` is false, and
through ``accept_select_top_gb300.ops`` where it is true.
"""
import math
import random

import torch

own = False

EXP_BIAS = 127
EXP_MIN = 16  # smallest scale exponent byte: 2^-111
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one verify step of a large batch of short chains: a few slots a request
        dict(name="alloc chain step", kind="alloc", b=256, page=16, lo=256, hi=4096, new_lo=1, new_hi=4),
        # admission of a batch of prompts: every slot of every prompt
        dict(name="alloc prompts", kind="alloc", b=64, page=16, lo=0, hi=0, new_lo=1, new_hi=16384),
        # accepted path of a 64-node tree, 32 requests, eight layers of a GQA model
        dict(name="commit tree step", kind="commit", b=32, n=64, width=7, layers=8, heads=8, dim=128, page=16, lo=2048, hi=2048, prompt=False),
        # a chain step of a large batch, ragged contexts
        dict(name="commit chain step", kind="commit", b=256, n=4, width=4, layers=2, heads=8, dim=128, page=16, lo=256, hi=4096, prompt=False),
        # prompts written into the cache, one chunk behind a cached prefix
        dict(name="commit prompts", kind="commit", b=5, n=1, width=4099, layers=4, heads=8, dim=128, page=64, lo=0, hi=1000, prompt=True),
        # latency: one request, one token
        dict(name="attention one token", kind="attention", b=1, n=1, hq=32, hkv=8, dim=128, page=16, lo=1001, hi=1001),
        # chains of four over ragged contexts, a large batch
        dict(name="attention chains", kind="attention", b=256, n=4, hq=32, hkv=8, dim=128, page=16, lo=256, hi=4096),
        # trees of 64 nodes
        dict(name="attention trees", kind="attention", b=32, n=64, hq=32, hkv=8, dim=128, page=16, lo=2048, hi=2048),
        # two long contexts, trees of 64 nodes
        dict(name="attention long", kind="attention", b=2, n=64, hq=64, hkv=8, dim=128, page=64, lo=32768, hi=131072),
        # latency: the rows of one chain, rows that are not whole 16-byte vectors
        dict(name="logprobs one chain", kind="logprobs", b=1, n=4, width=4, vocab=50257, bf16=True, k=5, rows="all", tempered=False),
        # the accepted rows of a sampled tree step
        dict(name="logprobs accepted", kind="logprobs", b=32, n=64, width=7, vocab=128256, bf16=True, k=8, rows="accepted", tempered=True),
        # every row of a chain step in fp32 with many alternatives
        dict(name="logprobs all rows", kind="logprobs", b=256, n=4, width=4, vocab=129280, bf16=False, k=20, rows="all", tempered=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = {"alloc": 1 << 19, "commit": 2.5e8, "attention": 1.2e9, "logprobs": 5e8}
    while True:
        kind = rng.choice(["alloc", "commit", "attention", "logprobs"])
        if kind == "alloc":
            c = dict(kind=kind, b=_log(rng, 1, 1024), page=rng.choice([1, 16, 32, 64]), lo=0, hi=_log(rng, 1, 8192), new_lo=0, new_hi=_log(rng, 1, 16384))
            cost = c["b"] * c["new_hi"] / 2
        elif kind == "commit":
            prompt = rng.random() < 0.4
            n = 1 if prompt else _log(rng, 1, 64)
            c = dict(kind=kind, b=_log(rng, 1, 8 if prompt else 256), n=n, width=_log(rng, 5, 4099) if prompt else rng.randint(1, min(n, 9)), layers=_log(rng, 1, 16),
                     heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64]), lo=0, hi=_log(rng, 1, 4096), prompt=prompt)
            cost = c["b"] * (c["hi"] + c["width"]) * c["layers"] * c["heads"] * c["dim"] * 2
        elif kind == "attention":
            hkv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
            c = dict(kind=kind, b=_log(rng, 1, 256), n=_log(rng, 1, 64), hq=hkv * rng.choice([1, 2, 3, 4, 6, 8]), hkv=hkv, dim=dim, page=rng.choice([16, 32, 64]), lo=0, hi=_log(rng, 1, 131072))
            cost = c["b"] * c["hi"] * (hkv * dim + c["n"] * c["hq"] * dim / 64)
        else:
            accepted = rng.random() < 0.5
            n = _log(rng, 1, 64)
            c = dict(kind=kind, b=_log(rng, 1, 256), n=n, width=rng.randint(1, min(n, 9)) if accepted else n, vocab=_log(rng, 1000, 200000), bf16=rng.random() < 0.5,
                     k=rng.randint(0, 20), rows="accepted" if accepted else "all", tempered=rng.random() < 0.5)
            cost = c["b"] * c["n"] * c["vocab"] * (2 if c["bf16"] else 4)
        if cost <= most[kind]:
            return c


def _rng(case, what):
    return random.Random("%s %s" % (what, sorted((k, v) for k, v in case.items() if k != "name")))


def _between(case, what, lo, hi, count):
    r = _rng(case, what)
    return [r.randint(lo, hi) for _ in range(count)]


def _contexts(case):
    """Tokens in the cache of each request: they are part of the case, not of the seed."""
    lens = _between(case, "contexts", case["lo"], case["hi"], case["b"])
    if case["b"] == 2 and case["hi"] > case["lo"]:
        lens = [case["lo"], case["hi"]]
    return lens


def _parents(case):
    """A tree of n nodes for each request (parent of node 0 is -1)."""
    r = _rng(case, "tree")
    return [[-1] + [r.randint(max(0, i - 9), i - 1) for i in range(1, case["n"])] for _ in range(case["b"])]


def _masks(parents):
    masks = []
    for p in parents:
        row = []
        for i, a in enumerate(p):
            row.append((row[a] if a >= 0 else 0) | (1 << i))
        masks.append(row)
    return masks


def _accepted(case):
    """Accepted path lengths (root included), at least one row a request."""
    return _between(case, "accepted", 1, case["width"], case["b"])


def work(case):
    kind, b = case["kind"], case["b"]
    if kind == "alloc":
        ctx, new = _contexts(case), _between(case, "new", case["new_lo"], case["new_hi"], b)
        pages = sum(-(-(c + x) // case["page"]) - -(-c // case["page"]) for c, x in zip(ctx, new))
        # lengths and rows read, offsets written; a page: id read, table entry written; a token: slot and position written
        return {"bytes": 12 * b + 4 * (b + 1) + 8 * pages + 8 * sum(new), "flops": 0}
    if kind == "commit":
        ctx, new = _contexts(case), _between(case, "new", max(1, case["width"] // 2), case["width"], b) if case["prompt"] else _accepted(case)
        pages = sum(-(-(c + x) // case["page"]) - c // case["page"] for c, x in zip(ctx, new))
        row = case["heads"] * case["dim"]
        return {"bytes": case["layers"] * 2 * (sum(new) * row * 3 + pages * case["heads"]) + 4 * (sum(new) + pages + 4 * b), "flops": 0}
    if kind == "attention":
        ctx, n = _contexts(case), case["n"]
        seen = sum(n * c for c in ctx) + sum(bin(m).count("1") for row in _masks(_parents(case)) for m in row)
        pages = sum(-(-c // case["page"]) for c in ctx)
        kv = sum(ctx) * case["hkv"] * case["dim"] * 2 + b * n * case["hkv"] * case["dim"] * 4 + pages * (2 * case["hkv"] + 4)
        return {"bytes": kv + b * n * case["hq"] * (case["dim"] * 4 + 4) + b * n * 8, "flops": 4 * case["dim"] * case["hq"] * seen}
    rows = sum(_accepted(case)) if case["rows"] == "accepted" else b * case["n"]
    return {"bytes": rows * (case["vocab"] * (2 if case["bf16"] else 4) + 16 + 8 * case["k"]), "flops": 0}


# ------------------------------------------------------------------ inputs

def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _tables(lens, page, gen, dev, spare=3):
    """A block table over scattered pages for requests of `lens` tokens, at scattered rows; pages in all."""
    need = [-(-x // page) for x in lens]
    width, rows = max(need + [1]) + 1, len(lens) + spare
    total = sum(need) + spare
    ids = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    where = torch.randperm(rows, generator=gen, device=dev)[: len(lens)].to(torch.int32)
    counts = torch.tensor(need, device=dev)
    start = torch.cumsum(counts, 0) - counts
    col = torch.arange(width, device=dev)
    mine = col[None] < counts[:, None]
    table = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
    table[where.long()] = torch.where(mine, ids[torch.clamp(start[:, None] + col, max=total - 1)], -1)
    return table, where, total


def _cache(pages, heads, page, dim, gen, dev, spread):
    """e4m3 pages and their scale exponents as a cache holds them: rows of unit normals, each (page, head) of its own magnitude."""
    x = torch.randn(pages, heads, page, dim, generator=gen, device=dev)
    e = (torch.frexp(x.abs().amax(dim=(2, 3)) / E4M3_MAX).exponent + EXP_BIAS).clamp(min=EXP_MIN)
    x *= torch.exp2((EXP_BIAS - e).float())[:, :, None, None]
    shift = torch.randint(-spread, spread + 1, e.shape, generator=gen, device=dev)
    return x.to(torch.float8_e4m3fn), (e + shift).to(torch.uint8)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    b, kind = case["b"], case["kind"]
    s = dict(case=case, kind=kind, b=b)
    empty = lambda shape, dt: torch.zeros(shape, dtype=dt, device=dev)  # noqa: E731
    if kind == "alloc":
        ctx, new = _contexts(case), _between(case, "new", case["new_lo"], case["new_hi"], b)
        page = case["page"]
        table, where, used = _tables(ctx, page, gen, dev)
        width = max(-(-(c + x) // page) for c, x in zip(ctx, new)) + 1
        s["table"] = torch.full((table.shape[0], width), -1, dtype=torch.int32, device=dev)
        most = min(width, table.shape[1])
        s["table"][:, :most] = table[:, :most]
        need = sum(-(-(c + x) // page) - -(-c // page) for c, x in zip(ctx, new))
        s["free"] = (torch.randperm(need + 100, generator=gen, device=dev) + used).to(torch.int32)
        s.update(page=page, rows=where, lens=_i32(ctx, dev), new=_i32(new, dev), n_free=_i32([need + 90], dev), slots=(used + need + 100) * page,
                 cu=empty(b + 1, torch.int32), slot_map=empty(max(1, sum(new)), torch.int32), positions=empty(max(1, sum(new)), torch.int32), left=empty(1, torch.int32),
                 total=sum(new), most=max(new))
    elif kind == "commit":
        ctx = _contexts(case)
        new = _between(case, "new", max(1, case["width"] // 2), case["width"], b) if case["prompt"] else _accepted(case)
        page, heads, dim, layers = case["page"], case["heads"], case["dim"], case["layers"]
        table, where, pages = _tables([c + x for c, x in zip(ctx, new)], page, gen, dev)
        k, ks = _cache(layers * pages, heads, page, dim, gen, dev, 1)
        v, vs = _cache(layers * pages, heads, page, dim, gen, dev, 1)
        rows = sum(new) if case["prompt"] else b * case["n"]
        # the K and V columns of the projection's packed output
        kv = torch.randn(layers, rows, 2, heads, dim, generator=gen, device=dev).to(torch.bfloat16)
        s.update(page=page, heads=heads, dim=dim, layers=layers, width=case["width"], table=table, rows=where, lens=_i32(ctx, dev), new=_i32(new, dev), k=k.view(layers, pages, heads, page, dim),
                 v=v.view(layers, pages, heads, page, dim), ks=ks.view(layers, pages, heads), vs=vs.view(layers, pages, heads), k_new=kv[:, :, 0], v_new=kv[:, :, 1],
                 after=empty(b, torch.int32), index=None, start=None)
        if case["prompt"]:
            s["start"] = _i32([0] + new, dev).cumsum(0)[:-1].to(torch.int32)
        else:
            # increasing node indices, node 0 first, as an accepted path has them
            pick = torch.rand(b, case["n"], generator=gen, device=dev)
            pick[:, 0] = -1
            path = pick.argsort(dim=1)[:, : case["width"]].sort(dim=1).values + torch.arange(b, device=dev)[:, None] * case["n"]
            s["index"] = torch.where(torch.arange(case["width"], device=dev)[None] < s["new"][:, None], path, -1).to(torch.int32)
    elif kind == "attention":
        ctx, n = _contexts(case), case["n"]
        page, hq, hkv, dim = case["page"], case["hq"], case["hkv"], case["dim"]
        table, where, pages = _tables(ctx, page, gen, dev)
        k, ks = _cache(pages, hkv, page, dim, gen, dev, 1)
        v, vs = _cache(pages, hkv, page, dim, gen, dev, 2)
        # the step's rows come out of one packed projection
        qkv = torch.randn(b * n, hq + 2 * hkv, dim, generator=gen, device=dev).to(torch.bfloat16)
        masks = torch.tensor([m - (1 << 64) if m >> 63 else m for row in _masks(_parents(case)) for m in row], dtype=torch.int64, device=dev)
        s.update(n=n, page=page, hq=hq, hkv=hkv, dim=dim, table=table, rows=where, lens=_i32(ctx, dev), most=max(ctx), k=k, v=v, ks=ks, vs=vs, q=qkv[:, :hq], k_new=qkv[:, hq : hq + hkv],
                 v_new=qkv[:, hq + hkv :], masks=masks, out=empty((b * n, hq, dim), torch.bfloat16), lse=empty((b * n, hq), torch.float32))
    else:
        n, width, k = case["n"], case["width"], case["k"]
        x = torch.randn(b * n, case["vocab"], generator=gen, device=dev) * 2
        # confident rows and, on every third row, a grammar's mask over most of the vocabulary
        top = torch.randint(0, case["vocab"], (b * n, 1), generator=gen, device=dev)
        x.scatter_add_(1, top, torch.rand(b * n, 1, generator=gen, device=dev) * 16)
        x[2::3, case["vocab"] // 16 :] = -math.inf
        s.update(n=n, width=width, k=k, logits=x.to(torch.bfloat16) if case["bf16"] else x, index=None)
        if case["rows"] == "accepted":
            new = _i32(_accepted(case), dev)
            pick = torch.rand(b, n, generator=gen, device=dev)
            pick[:, 0] = -1
            path = pick.argsort(dim=1)[:, :width].sort(dim=1).values + torch.arange(b, device=dev)[:, None] * n
            s["index"] = torch.where(torch.arange(width, device=dev)[None] < new[:, None], path, -1).to(torch.int32)
        at = torch.arange(b * n, device=dev).view(b, n)[:, :width] if s["index"] is None else s["index"].long().clamp(min=0)
        likely = top.view(-1)[at]
        other = torch.randint(0, max(1, case["vocab"] // 16), (b, width), generator=gen, device=dev)
        s["tokens"] = torch.where(torch.rand(b, width, generator=gen, device=dev) < 0.7, likely, other).to(torch.int32)
        if s["index"] is not None:
            s["tokens"] = torch.where(s["index"] < 0, -1, s["tokens"])
        s["temps"] = (torch.rand(b, generator=gen, device=dev) * 0.9 + 0.5) if case["tempered"] else None
        s.update(logprobs=empty((b, width), torch.float32), entropy=empty((b, width), torch.float32), top_ids=empty((b, width, k), torch.int32) if k else None,
                 top_logprobs=empty((b, width, k), torch.float32) if k else None)
    return s


# -------------------------------------------------------------------- runs

def run(s):
    if own:
        return _RUN_OWN[s["kind"]](s)
    return _RUN_PLAIN[s["kind"]](s)


def _workspace(ops, s, *size):
    if "ws" not in s:
        s["ws"] = ops.Workspace(ops.spec_workspace_size(*size))
    return s["ws"]


def _own_alloc(s):
    from accept_select_top_gb300 import ops
    ws = _workspace(ops, s, ops.OP_ALLOC_SLOTS, s["b"], 1, 1, 1)
    ops.spec_alloc_slots(s["b"], s["page"], s["rows"], s["lens"], s["new"], s["most"], s["free"], s["n_free"], s["slots"], s["table"], None, s["cu"], s["slot_map"],
                         s["positions"], s["left"], ws)
    return {"table": s["table"], "cu": s["cu"], "slots": s["slot_map"], "positions": s["positions"], "left": s["left"]}


def _own_commit(s):
    from accept_select_top_gb300 import ops
    ws = _workspace(ops, s, ops.OP_COMMIT_KV_Q8, s["b"], 1, 1, 1)
    if "layered" not in s:
        s["layered"] = [ops.LayerList(s[x].unbind(0)) for x in ("k_new", "v_new", "k", "v", "ks", "vs")]
    ops.spec_commit_kv_q8(s["b"], s["heads"], s["dim"], s["page"], *s["layered"], s["table"], s["rows"], s["lens"], s["index"], s["start"], s["new"], s["width"],
                          s["after"], ws)
    return {"k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"], "lens": s["after"]}


def _own_attention(s):
    from accept_select_top_gb300 import ops
    ws = _workspace(ops, s, ops.OP_VERIFY_ATTENTION_Q8, s["b"], s["n"], 1, 1, s["hq"], s["hkv"], s["most"])
    ops.spec_verify_attention_q8(s["b"], s["n"], s["hq"], s["hkv"], s["dim"], s["page"], s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["ks"], s["vs"], s["table"],
                                 s["rows"], s["lens"], s["most"], s["masks"], 1 / math.sqrt(s["dim"]), s["out"], s["lse"], ws)
    return {"out": s["out"], "lse": s["lse"]}


def _own_logprobs(s):
    from accept_select_top_gb300 import ops
    ws = _workspace(ops, s, ops.OP_TOKEN_LOGPROBS, s["b"], s["width"], max(1, s["k"]), s["logits"].shape[1])
    ops.spec_token_logprobs(s["b"], s["n"], s["width"], s["logits"], s["index"], s["tokens"], s["temps"], s["k"], s["logprobs"], s["entropy"], s["top_ids"],
                            s["top_logprobs"], ws)
    return {"logprobs": s["logprobs"], "entropy": s["entropy"], "top_ids": s["top_ids"], "top_logprobs": s["top_logprobs"]}


def _ceil(a, m):
    return torch.div(a + (m - 1), m, rounding_mode="floor")


def _plain_alloc(s):
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
    s["positions"][: s["total"]] = pos.int()
    s["slot_map"][: s["total"]] = (s["table"][rows[req], pos // page].long() * page + pos % page).int()
    s["left"].copy_(s["n_free"] - need.sum())
    return {"table": s["table"], "cu": s["cu"], "slots": s["slot_map"], "positions": s["positions"], "left": s["left"]}


def _scale(e):
    return (e.int() << 23).view(torch.float32)


def _plain_write(cache, exps, rows, kept, filled, page_ids):
    """The pages of `page_ids` after `rows` (fp32, where `filled`) were written behind the rows they hold (`kept`)."""
    old = cache[:, page_ids].float() * kept[None, :, None, :, None]
    amax = (rows * filled[None, :, None, :, None]).abs().amax(dim=(3, 4))
    f = torch.frexp(amax)
    need = (f.exponent - 9 + (f.mantissa > 0.875).int() + EXP_BIAS).clamp(min=EXP_MIN)
    need = torch.where(amax > 0, need, EXP_MIN)
    had = exps[:, page_ids].int()
    e = torch.where(kept.any(dim=1)[None, :, None], torch.maximum(had, need), need)
    moved = old * torch.exp2((had - e).float())[..., None, None]
    fresh = rows * _scale(2 * EXP_BIAS - e)[..., None, None]
    held = cache[:, page_ids].float()
    now = torch.where(filled[None, :, None, :, None], fresh, torch.where(kept[None, :, None, :, None], moved, held))
    cache.view(torch.uint8)[:, page_ids] = now.to(torch.float8_e4m3fn).view(torch.uint8)
    exps[:, page_ids] = e.to(torch.uint8)


def _plain_commit(s):
    page, lens, new, b = s["page"], s["lens"].long(), s["new"].long(), s["b"]
    width = (s["width"] + page - 2) // page + 1
    index = lens[:, None] // page + torch.arange(width, device=lens.device)[None]
    used = index * page < (lens + new)[:, None]
    req = torch.arange(b, device=lens.device)[:, None].expand(b, width)[used]
    index = index[used]
    page_ids = s["table"][s["rows"].long()[req], index].long()
    pos = index[:, None] * page + torch.arange(page, device=lens.device)[None]
    kept = pos < lens[req][:, None]
    filled = ~kept & (pos < (lens + new)[req][:, None])
    j = (pos - lens[req][:, None]).clamp(0, s["width"] - 1)
    src = (s["start"].long()[req][:, None] + j) if s["index"] is None else s["index"].long()[req[:, None], j]
    src = torch.where(filled, src, 0)
    _plain_write(s["k"], s["ks"], s["k_new"][:, src].float().transpose(2, 3), kept, filled, page_ids)
    _plain_write(s["v"], s["vs"], s["v_new"][:, src].float().transpose(2, 3), kept, filled, page_ids)
    s["after"].copy_(s["lens"] + s["new"])
    return {"k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"], "lens": s["after"]}


def _plain_attention(s):
    b, n, hq, hkv, dim, page = (s[x] for x in ("b", "n", "hq", "hkv", "dim", "page"))
    g, dev = hq // hkv, s["lens"].device
    pos = torch.arange(max(1, s["most"]), device=dev)
    seen = pos[None] < s["lens"][:, None]
    ids = torch.where(seen, s["table"][s["rows"].long()][:, (pos // page).clamp(max=s["table"].shape[1] - 1)], 0).long()

    def rows(cache, exps, fresh):
        held = cache.view(torch.uint8)[ids, :, pos % page].view(torch.float8_e4m3fn).float() * _scale(exps[ids])[..., None]
        return torch.cat([held, fresh.float().view(b, n, hkv, dim)], dim=1).transpose(1, 2)

    q = s["q"].float().view(b, n, hkv, g, dim).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, dim)
    x = q @ rows(s["k"], s["ks"], s["k_new"]).transpose(2, 3) / math.sqrt(dim)
    tree = (s["masks"].view(b, n, 1) >> torch.arange(n, device=dev)) & 1
    see = torch.cat([seen[:, None].expand(b, n, pos.numel()), tree.bool()], dim=2)
    x = x.view(b, hkv, g, n, -1).masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    z = x.sum(dim=-1, keepdim=True)
    out = (x.view(b, hkv, g * n, -1) @ rows(s["v"], s["vs"], s["v_new"])).view(b, hkv, g, n, dim) / torch.where(z > 0, z, 1.0)
    lse = (torch.log(z) + top).squeeze(-1)
    s["out"].copy_(out.permute(0, 3, 1, 2, 4).reshape(b * n, hq, dim))
    s["lse"].copy_(lse.permute(0, 3, 1, 2).reshape(b * n, hq))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_logprobs(s):
    b, n, width, k = s["b"], s["n"], s["width"], s["k"]
    dev = s["logits"].device
    at = torch.arange(b * n, device=dev).view(b, n)[:, :width] if s["index"] is None else s["index"].long()
    used = at >= 0
    x = s["logits"][at.clamp(min=0)]
    y = x.float() if s["temps"] is None else x.float() / s["temps"][:, None, None]
    y = y - y.amax(dim=-1, keepdim=True)
    p = torch.exp(y)
    z = p.sum(dim=-1, keepdim=True)
    logp = y - torch.log(z)
    entropy = torch.log(z).squeeze(-1) - (p * torch.where(p > 0, y, 0.0)).sum(dim=-1) / z.squeeze(-1)
    asked = used & (s["tokens"] >= 0)
    mine = torch.gather(logp, 2, s["tokens"].long().clamp(min=0)[..., None]).squeeze(-1)
    s["logprobs"].copy_(torch.where(asked, mine, 0.0))
    s["entropy"].copy_(torch.where(used, entropy, 0.0))
    if k:
        ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :k]
        s["top_ids"].copy_(torch.where(used[..., None], ids, -1))
        s["top_logprobs"].copy_(torch.where(used[..., None], torch.gather(logp, 2, ids), 0.0))
    return {"logprobs": s["logprobs"], "entropy": s["entropy"], "top_ids": s["top_ids"], "top_logprobs": s["top_logprobs"]}


_RUN_OWN = {"alloc": _own_alloc, "commit": _own_commit, "attention": _own_attention, "logprobs": _own_logprobs}
_RUN_PLAIN = {"alloc": _plain_alloc, "commit": _plain_commit, "attention": _plain_attention, "logprobs": _plain_logprobs}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    return {"alloc": _exact_alloc, "commit": _exact_commit, "attention": _exact_attention, "logprobs": _exact_logprobs}[case["kind"]](s)


def _exact_alloc(s):
    return None  # whole numbers only


def _to_e4m3(x):
    """Nearest e4m3 value of float64 `x` within +-448: three mantissa bits, quantum 2^-9 below 2^-6, ties to even."""
    ulp = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / ulp) * ulp


def _exact_commit(s):
    """Token by token of each request, in float64: a page's scale is 2^x with the smallest x at which its largest new
    value fits 448, never below the scale of the rows already in it."""
    page, table = s["page"], s["table"].tolist()
    lens, new, rows = s["lens"].tolist(), s["new"].tolist(), s["rows"].tolist()
    index = None if s["index"] is None else s["index"].tolist()
    start = None if s["start"] is None else s["start"].tolist()
    got = {}
    for name, exps, fresh in (("k", "ks", "k_new"), ("v", "vs", "v_new")):
        held, e = s[name].double(), s[exps].double()
        for r in range(s["b"]):
            for p in range(lens[r] // page, -(-(lens[r] + new[r]) // page)):
                pid, lo, hi = table[rows[r]][p], max(lens[r], p * page), min(lens[r] + new[r], (p + 1) * page)
                src = [start[r] + t - lens[r] if index is None else index[r][t - lens[r]] for t in range(lo, hi)]
                x = s[fresh][:, src[0] : src[-1] + 1] if index is None else s[fresh][:, src]
                x = x.double().transpose(1, 2)  # layers, heads, tokens, dim
                amax = x.abs().amax(dim=(2, 3))
                need = torch.where(amax > 0, torch.ceil(torch.log2(amax.clamp(min=1e-40) / E4M3_MAX)) + EXP_BIAS, float(EXP_MIN)).clamp(min=EXP_MIN)
                old = lo - p * page
                now = torch.maximum(need, e[:, pid]) if old else need
                if old:
                    held[:, pid, :, :old] = _to_e4m3(held[:, pid, :, :old] * torch.exp2(e[:, pid] - now)[..., None, None])
                held[:, pid, :, old : hi - p * page] = _to_e4m3(x * torch.exp2(EXP_BIAS - now)[..., None, None])
                e[:, pid] = now
        got[name] = held
    return {"k": got["k"], "v": got["v"]}


def _exact_attention(s):
    b, n, hq, hkv, dim, page = (s[x] for x in ("b", "n", "hq", "hkv", "dim", "page"))
    g = hq // hkv
    out = torch.zeros(b * n, hq, dim, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(b * n, hq, dtype=torch.float64, device=s["q"].device)
    lens, rows = s["lens"].tolist(), s["rows"].tolist()
    bits = torch.arange(n, device=out.device)
    for r in range(b):
        mine = slice(r * n, (r + 1) * n)
        ids = s["table"][rows[r], : -(-lens[r] // page)].long()
        see = torch.cat([torch.ones(n, lens[r], dtype=torch.bool, device=out.device), ((s["masks"][mine][:, None] >> bits) & 1).bool()], dim=1)
        for h in range(hkv):
            def keys(cache, exps, fresh):
                held = cache.view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double() * torch.exp2(exps[ids, h].double() - EXP_BIAS)[:, None, None]
                return torch.cat([held.reshape(-1, dim)[: lens[r]], fresh[mine, h].double()])

            q = s["q"][mine, h * g : (h + 1) * g].double()
            x = torch.einsum("ngd,kd->ngk", q, keys(s["k"], s["ks"], s["k_new"])) * dim ** -0.5
            x = torch.where(see[:, None], x, -math.inf)
            lse[mine, h * g : (h + 1) * g] = torch.logsumexp(x, dim=-1)
            out[mine, h * g : (h + 1) * g] = torch.softmax(x, dim=-1) @ keys(s["v"], s["vs"], s["v_new"])
    return {"out": out, "lse": lse}


def _exact_logprobs(s):
    b, n, width, k = s["b"], s["n"], s["width"], s["k"]
    got = {"logprobs": torch.zeros(b, width, dtype=torch.float64), "entropy": torch.zeros(b, width, dtype=torch.float64), "top_ids": None,
           "top_logprobs": torch.zeros(b, width, k, dtype=torch.float64) if k else None}
    for r in range(b):
        at = torch.arange(r * n, r * n + width, device=s["logits"].device) if s["index"] is None else s["index"][r].long()
        at = at[at >= 0]
        m = at.numel()
        x = s["logits"][at].double()
        if s["temps"] is not None:
            x = x / s["temps"][r].double()
        logp = torch.log_softmax(x, dim=-1)
        tokens = s["tokens"][r, :m].long()
        got["logprobs"][r, :m] = logp.gather(1, tokens[:, None])[:, 0].cpu()
        got["entropy"][r, :m] = torch.special.entr(logp.exp()).sum(dim=-1).cpu()
        if k:
            got["top_logprobs"][r, :m] = logp.topk(k, dim=-1).values.cpu()
    return got
