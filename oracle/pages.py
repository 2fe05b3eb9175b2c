"""The bookkeeping of a paged cache's pages and the copies within it, in plain loops and
from their definitions. TEST INFRASTRUCTURE ONLY (see oracle/attention.py).

Tables, counts and lengths are numpy integer arrays that the calls change; what is out
of range is left out and counted as a fault."""
from __future__ import annotations

import numpy as np


def _take(refs, free):
    """The lowest free page from number `free` on, now held once; -1: none."""
    while free < len(refs) and refs[free] != 0:
        free += 1
    if free == len(refs):
        return -1, free
    refs[free] = 1
    return free, free


def release(refs, table, size, first, last) -> int:
    faults = 0
    for b in range(len(table)):
        for e in range(table.shape[1]):
            page = table[b, e]
            if not (max(first[b], 0) <= e * size and (e + 1) * size <= last[b]) or page < 0:
                continue
            table[b, e] = -1
            if page >= len(refs) or refs[page] <= 0:
                faults += 1
            else:
                refs[page] -= 1
    return faults


def fork(refs, table, size, lens, src, dst):
    """Returns (from, to, faults)."""
    n, room = len(src), table.shape[1] * size
    old, new, faults = np.full(n, -1), np.full(n, -1), 0
    good = []
    for i in range(n):
        ok = 0 <= src[i] < len(table) and 0 <= dst[i] < len(table)
        ok = ok and dst[i] not in list(src) and dst[i] not in list(dst[:i])
        ok = ok and 0 <= lens[src[i]] <= room
        good.append(ok)
        faults += not ok
    for i in range(n):
        if not good[i]:
            continue
        a, b = src[i], dst[i]
        whole = lens[a] // size
        for e in range(table.shape[1]):
            page = table[a, e] if e < whole else -1
            if page >= len(refs):
                page, faults = -1, faults + 1
            if page >= 0:
                refs[page] += 1
            table[b, e] = max(page, -1)
        lens[b] = lens[a]
    free = 0
    for i in range(n):
        if not good[i] or lens[src[i]] % size == 0:
            continue
        whole = lens[src[i]] // size
        part = table[src[i], whole]
        if not 0 <= part < len(refs):
            faults += part >= len(refs)
            continue
        page, free = _take(refs, free)
        table[dst[i], whole] = page
        if page < 0:
            faults += 1
        else:
            old[i], new[i] = part, page
    return old, new, faults


def reserve(refs, table, size, lens, new_lens) -> int:
    faults, free = 0, 0
    room = table.shape[1] * size
    for b in range(len(table)):
        if lens[b] < 0 or lens[b] > room or new_lens[b] > room:
            faults += 1
            continue
        for e in range(-(-lens[b] // size), -(-new_lens[b] // size)):
            if not 0 <= table[b, e] < len(refs):
                faults += table[b, e] >= len(refs)
                table[b, e], free = _take(refs, free)
                faults += table[b, e] < 0
    return faults


def copy(pages, old, new) -> int:
    """pages [n_pages, ...], changed in place."""
    faults = 0
    for a, b in zip(old, new):
        if a < 0 or b < 0:
            continue
        if a >= len(pages) or b >= len(pages):
            faults += 1
            continue
        pages[b] = pages[a]
    return faults


def gather(pages, size, table, places, cu, to_table=None, to_start=None) -> int:
    """pages [n_pages, size, ...], changed in place."""
    before, faults = pages.copy(), 0
    to = table if to_table is None else to_table
    for b in range(len(table)):
        for j, p in enumerate(places[max(cu[b], 0):cu[b + 1]]):
            z = (0 if to_start is None else to_start[b]) + j
            ok = 0 <= p < table.shape[1] * size and 0 <= z < to.shape[1] * size
            ok = ok and (to_table is not None or p >= z)
            if ok:
                x, y = table[b, p // size], to[b, z // size]
                ok = 0 <= x < len(pages) and 0 <= y < len(pages)
            if ok:
                pages[y, z % size] = before[x, p % size]
            faults += not ok
    return faults
