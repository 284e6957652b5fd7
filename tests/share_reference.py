"""Plain forms of the calls that let requests share pages: lists and loops, one page at a time.  Each changes the
lists (and tensors) that it is given, as the calls change theirs."""


def fork(page, parents, children, lens, counts, free, n_free, table, slots=None):
    """(copies, left): the pairs to copy and the free pages left."""
    copies = []
    for p, c, L in zip(parents, children, lens):
        for i in range(-(-L // page)):
            pid = table[p][i]
            if (i + 1) * page <= L:
                counts[pid] += 1
            else:
                n_free -= 1
                copies.append((pid, free[n_free]))
                pid = free[n_free]
            table[c][i] = pid
            if slots is not None:
                for x in range(i * page, min(L, (i + 1) * page)):
                    slots[c][x] = pid * page + x % page
    return copies, n_free


def release(page, rows, lens, keep, counts, free, n_free, table):
    """The new number of free pages."""
    given, order = {}, []
    for r, L, k in zip(rows, lens, keep):
        for i in range(-(-k // page), -(-L // page)):
            pid = table[r][i]
            given[pid] = given.get(pid, 0) + 1
            if given[pid] == 1:
                order.append(pid)
    freed = [pid for pid in order if given[pid] > counts[pid]]
    for pid in order:
        counts[pid] = max(0, counts[pid] - given[pid])
    for pid in reversed(freed):
        free[n_free] = pid
        n_free += 1
    return n_free


def compact(page, rows, lens, limit, counts, free, n_free, table, slots=None):
    """(moves, left); table, slots, counts and free are changed in place."""
    idle = set(free[:n_free])
    total = len(counts)
    limit = min(total, max(limit, total - len(idle)))
    holes = [p for p in range(limit) if p in idle]
    moves = list(zip([p for p in range(limit, total) if p not in idle], holes))
    to = dict(moves)
    for src, dst in moves:
        counts[dst], counts[src] = counts[src], 0
        idle.remove(dst)
        idle.add(src)
    for j, p in enumerate(sorted(idle, reverse=True)):
        free[j] = p
    for r, L in zip(rows, lens):
        for i in range(-(-L // page)):
            table[r][i] = to.get(table[r][i], table[r][i])
            if slots is not None:
                for x in range(i * page, min(L, (i + 1) * page)):
                    slots[r][x] = table[r][i] * page + x % page
    return moves, len(idle)
