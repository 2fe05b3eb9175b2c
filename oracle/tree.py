"""What drafted tokens see of a cache, from the definition. TEST INFRASTRUCTURE ONLY (see
oracle/attention.py)."""
from __future__ import annotations


def seen(n_keys: int, n_new: int, i: int, mask=None, window=None, sinks: int = 0):
    """The keys that drafted token i of n_new sees, the last ones of n_keys. mask: an int
    whose bit x stands for drafted token x; None: a chain."""
    before = n_keys - n_new
    if mask is None:
        place = before + i
        mine = list(range(before, before + i + 1))
    else:
        mask &= (1 << n_new) - 1
        place = before - 1 + max(1, bin(mask).count("1"))
        mine = [before + x for x in range(n_new) if mask >> x & 1]

    def near(j):
        return window is None or j > place - window or j < sinks

    return [j for j in range(before) if near(j)] + [j for j in mine if mask is not None or near(j)]
