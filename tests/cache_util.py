"""The page operators as loops over plain lists."""


def pages_of(n, size):
    return -(-n // size)


def resize(table, lens, new_lens, refs, size, window=0, first=0):
    """The table and counts after a resize; the fresh entries that no page was left for are -1."""
    table, refs = [list(r) for r in table], list(refs)
    free = [p for p, n in enumerate(refs) if n == 0]
    for row, a, b in zip(table, lens, new_lens):
        for i in range(pages_of(a, size), pages_of(b, size)):
            row[i] = free.pop(0) if free else -1
            if row[i] >= 0:
                refs[row[i]] = 1
    for row, a, b in zip(table, lens, new_lens):
        n0, n1 = pages_of(a, size), pages_of(b, size)
        for i in range(n0):
            dead = window and i < n1 and (i + 1) * size <= b - window and i * size >= first
            if i >= n1 or dead:
                if row[i] >= 0:
                    refs[row[i]] -= 1
                row[i] = -1
    return table, refs


def fork(table, lens, refs, parents, size):
    """(new table, new lengths, copies, counts)"""
    before, refs = list(refs), list(refs)
    free = [p for p, n in enumerate(before) if n == 0]
    width = len(table[0])
    for row, n in zip(table, lens):
        for p in row[:pages_of(n, size)]:
            if p >= 0:
                refs[p] -= 1
    new, new_lens, copies, served = [], [], [], set()
    for r in parents:
        n = lens[r] if r >= 0 else 0
        row = list(table[r][:pages_of(n, size)]) if r >= 0 else []
        copy = [-1, -1, 0]
        if n % size and row[-1] >= 0 and (before[row[-1]] != 1 or r in served):
            fresh = free.pop(0) if free else -1
            if fresh >= 0:
                copy = [row[-1], fresh, n % size]
            row[-1] = fresh
        served.add(r)
        for p in row:
            if p >= 0:
                refs[p] += 1
        new.append(row + [-1] * (width - len(row)))
        new_lens.append(n)
        copies.append(copy)
    return new, new_lens, copies, refs
