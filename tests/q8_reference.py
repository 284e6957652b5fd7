"""Plain 64-bit forms of the 8-bit cache operators and the token log
probabilities, request by request and token by token (test infrastructure,
CPU tensors only)."""
import math

import torch

E4M3 = torch.float8_e4m3fn
BIAS, EXP_MIN = 127, 16


def e4m3_values(byte):
    """float64 values of e4m3 bytes (sign, 4 exponent bits of bias 7, 3 mantissa bits; S.1111.111 is NaN)."""
    b = byte.to(torch.int64)
    e, m = (b >> 3) & 15, b & 7
    v = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    v = torch.where((b & 127) == 127, math.nan, v)
    return torch.where((b & 128) > 0, -v, v)


def e4m3_bytes(x):
    """Nearest e4m3 bytes of float64 x (ties to even mantissa; +-448 beyond; NaN to NaN with its sign dropped)."""
    mag = x.abs().clamp(max=448.0)
    grid = e4m3_values(torch.arange(0, 127))  # ascending, 0 to 448
    mag0 = torch.nan_to_num(mag, nan=0.0)
    hi = torch.searchsorted(grid, mag0).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = mag0 - grid[lo], grid[hi] - mag0
    near = torch.where(dl < dh, lo, torch.where(dl > dh, hi, torch.where(lo % 2 == 0, lo, hi)))
    out = near + 128 * torch.signbit(x).long()
    return torch.where(torch.isnan(x), 127, out).to(torch.uint8)


def need_exp(x):
    """The smallest e >= EXP_MIN with max |x| <= 448 * 2^(e - 127), over the finite values of float64 x."""
    a = x.abs()
    a = float(a[torch.isfinite(a)].max()) if torch.isfinite(a).any() else 0.0
    e = EXP_MIN
    while a > 448.0 * 2.0 ** (e - BIAS):
        e += 1
    return e


def alloc(page, rows, lens, new, free, n_free, table, slot_table=None):
    """(cu, slots, positions, left) and the tables changed in place; lists of ints and CPU tensors."""
    cu, slots, positions, top = [0], [], [], n_free
    for r, L, m in zip(rows, lens, new):
        for p in range(-(-L // page), -(-(L + m) // page)):
            top -= 1
            table[r, p] = free[top]
        for x in range(L, L + m):
            slots.append(int(table[r, x // page]) * page + x % page)
            positions.append(x)
            if slot_table is not None:
                slot_table[r, x] = slots[-1]
        cu.append(cu[-1] + m)
    return cu, slots, positions, top


def commit(page, table, rows, lens, src, fresh, pages, scales):
    """src[b]: the row indices of request b's new tokens; pages [num_pages, Hkv, page, D] bytes and
    scales [num_pages, Hkv] bytes of one pool, changed in place."""
    for b, idx in enumerate(src):
        L = lens[b]
        for p in range(L // page, -(-(L + len(idx)) // page)):
            if not idx:
                break
            pid, lo, hi = int(table[rows[b], p]), max(L, p * page), min(L + len(idx), (p + 1) * page)
            for h in range(scales.shape[1]):
                x = fresh[idx[lo - L:hi - L], h].double()
                e, held = need_exp(x), lo - p * page
                if held:
                    had = int(scales[pid, h])
                    e = max(e, had)
                    if e > had:
                        pages[pid, h, :held] = e4m3_bytes(e4m3_values(pages[pid, h, :held]) * 2.0 ** (had - e))
                pages[pid, h, held:held + hi - lo] = e4m3_bytes(x * 2.0 ** (BIAS - e))
                scales[pid, h] = e


def attention(n, page, q, k_new, v_new, k_pages, v_pages, k_scales, v_scales, table, rows, lens, masks, scale):
    """(out, lse, size, dx): out and lse in float64; size = sum p |v| / l, by which a relative error
    of P moves out; dx = the largest scale * sum |q| |k| of a row, by which fp32 products move x."""
    Hq, D = q.shape[1:]
    Hkv = k_new.shape[1]
    G, b = Hq // Hkv, len(lens)
    out = torch.zeros(b * n, Hq, D, dtype=torch.float64)
    size = torch.zeros_like(out)
    lse = torch.full((b * n, Hq), -math.inf, dtype=torch.float64)
    dx = torch.zeros(b * n, Hq, dtype=torch.float64)
    for r in range(b):
        ids = [int(table[rows[r], x // page]) for x in range(lens[r])]
        off = [x % page for x in range(lens[r])]
        for h in range(Hkv):
            def keys(pages, scales, fresh):
                if not ids:
                    return fresh[r * n:(r + 1) * n, h].double()
                held = e4m3_values(pages[ids, h, off]) * torch.exp2(scales[ids, h].double() - BIAS)[:, None]
                return torch.cat([held, fresh[r * n:(r + 1) * n, h].double()])
            k, v = keys(k_pages, k_scales, k_new), keys(v_pages, v_scales, v_new)
            for i in range(n):
                see = torch.tensor([True] * lens[r] + [bool(int(masks[r * n + i]) >> j & 1) for j in range(n)])
                if not see.any():
                    continue
                kk, vv = k[see], v[see]
                for g in range(G):
                    at = (r * n + i, h * G + g)
                    x = scale * (kk @ q[at].double())
                    lse[at] = torch.logsumexp(x, 0)
                    p = torch.exp(x - lse[at])
                    out[at] = p @ vv
                    size[at] = p @ vv.abs()
                    dx[at] = scale * (kk.abs() @ q[at].double().abs()).max()
    return out, lse, size, dx


def logprobs(n, W, logits, index, tokens, temps, k):
    """(logprobs, entropy, ids, top) of [b, W] rows, float64; index rows of -1 give 0 and -1."""
    b, V = tokens.shape[0], logits.shape[1]
    lp, ent = torch.zeros(b, W, dtype=torch.float64), torch.zeros(b, W, dtype=torch.float64)
    ids, top = torch.full((b, W, k), -1, dtype=torch.int64), torch.zeros(b, W, k, dtype=torch.float64)
    for r in range(b):
        for j in range(W):
            i = r * n + j if index is None else int(index[r, j])
            if i < 0:
                continue
            x = logits[i].double()
            x = torch.where(torch.isnan(x), -math.inf, x)
            T = 1.0 if temps is None else float(temps[i // n])
            y = x / T if T > 0 else x
            if torch.isinf(x).all() and (x < 0).all():
                p = torch.zeros(V, dtype=torch.float64)
                y = torch.full((V,), -math.inf, dtype=torch.float64)
            else:
                y = y - y.max()  # first: at -3.4e38, a sum of logarithms would vanish in float64 too
                y = y - torch.logsumexp(y, 0)
                p = torch.exp(y)
            ent[r, j] = -(p * torch.where(p > 0, y, 0.0)).sum()
            if int(tokens[r, j]) >= 0:
                lp[r, j] = y[int(tokens[r, j])]
            order = sorted(range(V), key=lambda v: (-float(x[v]), v))[:k] if V <= 4096 else \
                torch.sort(x, descending=True, stable=True).indices[:k].tolist()
            ids[r, j] = torch.tensor(order, dtype=torch.int64)
            top[r, j] = y[order]
    return lp, ent, ids, top
