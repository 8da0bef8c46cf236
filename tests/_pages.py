"""The page calls on the host, page by page."""

import random


def free_pages(refs):
    return [p for p, r in enumerate(refs) if r <= 0]


def resize(table, lens, refs, page):
    for n, row in enumerate(table):
        for e in range(-(-lens[n] // page), len(row)):
            if row[e] >= 0:
                refs[row[e]] -= 1
            row[e] = -1
    free = iter(free_pages(refs))
    enough = True
    for n, row in enumerate(table):
        for e in range(-(-lens[n] // page)):
            if row[e] < 0:
                row[e] = next(free, -1)
                if row[e] >= 0:
                    refs[row[e]] = 1
                else:
                    enough = False
    return enough


def fork(table, lens, refs, parent, page):
    """Returns the new table, lens, the list, and whether there were enough pages."""
    width = len(table[0])
    new, new_lens, wants, seen = [], [], [], set()
    for n, p in enumerate(parent):
        L = lens[p] if p >= 0 else 0
        held = -(-L // page)
        row = (table[p][:held] if p >= 0 else []) + [-1] * (width - held)
        if p >= 0 and L % page and p in seen:
            wants.append((n, held - 1, row[held - 1]))
            row[held - 1] = -1
        seen.add(p)
        new.append(row)
        new_lens.append(L)
    for row in table:
        for v in row:
            if v >= 0:
                refs[v] -= 1
    for row in new:
        for v in row:
            if v >= 0:
                refs[v] += 1
    free, pairs, enough = iter(free_pages(refs)), [], True
    for n, e, src in wants:
        got = next(free, -1)
        if got < 0:
            new_lens[n] = e * page
            enough = False
            continue
        new[n][e] = got
        refs[got] = 1
        pairs.append((src, got))
    return new, new_lens, pairs, enough


def compact(table, refs):
    used = sum(r > 0 for r in refs)
    movers = [p for p, r in enumerate(refs) if r > 0 and p >= used]
    holes = [p for p, r in enumerate(refs) if r <= 0 and p < used]
    assert len(movers) == len(holes)
    place = dict(zip(movers, holes))
    new = [[place.get(v, v) for v in row] for row in table]
    for s, d in place.items():
        refs[d], refs[s] = refs[s], 0
    return new, list(zip(movers, holes))


def some_state(seed, n_seqs, width, n_pages, page, fill):
    """A table in use: prefixes shared between rows, pages that the caller keeps, pages held
    past a row's length."""
    r = random.Random(seed)
    order = list(range(n_pages))
    r.shuffle(order)
    order = order[:int(n_pages * fill)]
    refs = [0] * n_pages
    for p in order[:len(order) // 10]:
        refs[p] = 1
    order = order[len(order) // 10:]
    table, lens = [], []
    for n in range(n_seqs):
        row, L = [-1] * width, r.randint(0, width * page)
        held = -(-L // page)
        shared = 0
        if n and r.random() < 0.4:
            m = r.randrange(n)
            shared = min(lens[m] // page, L // page)
            row[:shared] = table[m][:shared]
        for e in range(shared, min(width, held + (r.random() < 0.3))):
            if not order:
                break
            row[e] = order.pop()
        there = next((e for e in range(width) if row[e] < 0), width)
        lens.append(min(L, there * page))
        table.append(row)
    for row in table:
        for v in row:
            if v >= 0:
                refs[v] += 1
    return table, lens, refs, r
