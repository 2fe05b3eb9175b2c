"""The cache's pages without a GPU: the oracle's own invariants, and what the binding and
the C ABI refuse."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import pages


@pytest.fixture(scope="module")
def eba():
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


def names(table, n):
    return np.bincount(table[(table >= 0) & (table < n)], minlength=n)


@pytest.mark.parametrize("seed", range(6))
def test_oracle_keeps_its_counts(seed):
    """After any turn of calls a page's count is the number of entries that name it,
    and a forked sequence reads what its source does."""
    r = np.random.default_rng(seed)
    size, B, wide, n = int(r.integers(1, 9)), 7, 6, 60
    lens = r.integers(0, wide * size - 2 * size, B).clip(0)
    table, refs = np.full((B, wide), -1), np.zeros(n, dtype=int)
    data = r.integers(0, 1000, (n, size))
    assert pages.reserve(refs, table, size, np.zeros(B, int), lens) == 0
    read = [[data[table[b, p // size], p % size] for p in range(lens[b])] for b in range(B)]
    zero, full = np.zeros(B, int), np.full(B, wide * size)
    for b in (1, 4):
        full_b = np.where(np.arange(B) == b, full, 0)
        assert pages.release(refs, table, size, zero, full_b) == 0
    old, new, faults = pages.fork(refs, table, size, lens, np.array([2, 2]), np.array([4, 1]))
    assert faults == 0 and pages.copy(data, old, new) == 0
    for b, a in ((4, 2), (1, 2), (0, 0), (3, 3)):
        assert lens[b] == lens[a]
        assert [data[table[b, p // size], p % size] for p in range(lens[b])] == read[a]
    assert pages.reserve(refs, table, size, lens, lens + size) == 0
    assert (refs == names(table, n)).all()
    assert pages.release(refs, table, size, zero, full) == 0
    assert (refs == 0).all() and (table == -1).all()


def test_oracle_gather_in_place_is_a_stable_selection():
    data = np.arange(40).reshape(10, 4)
    table = np.array([[3, 1, 7, -1]])
    places = np.array([5, 6, 9, 11])
    want = [data[table[0, p // 4], p % 4] for p in places]
    assert pages.gather(data, 4, table, places, np.array([0, 4]), to_start=np.array([5])) == 0
    assert [data[table[0, p // 4], p % 4] for p in range(5, 9)] == want
    # a later place, a place without a page, one outside the table
    assert pages.gather(data, 4, table, np.array([1, 13, 99]), np.array([0, 3]), to_start=np.array([2])) == 3


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_binding_refuses(eba):
    refs = torch.zeros(9, dtype=torch.int32)
    for bad in (refs.long(), refs[None], refs[::2], refs[:0], [0, 0]):
        with pytest.raises(ValueError):
            eba.PagePool(bad, 16)
    for size in (0, -1, 1 << 31):
        with pytest.raises(ValueError):
            eba.PagePool(refs, size)
    pool = eba.PagePool(refs, 16)
    table, lens = torch.full((3, 4), -1, dtype=torch.int32), i32(0, 1, 2)
    for args in ((pool, table.long(), lens, lens), (pool, table[0], lens, lens), (None, table, lens, lens),
                 (pool, table, lens[:2], lens), (pool, table, lens, lens.long()), (pool, table, lens, None),
                 (pool, table.t()[:3], lens, lens), (pool, table[:1].expand(3, 4), lens, lens),
                 (pool, table[:, :0], lens, lens)):
        with pytest.raises(ValueError):
            eba.pages_release(*args)
        with pytest.raises(ValueError):
            eba.pages_reserve(*args)
    for src, dst in ((i32(0), i32(1, 2)), (i32(0).long(), i32(1)), (i32(0)[None], i32(1)[None]), ([0], [1])):
        with pytest.raises(ValueError):
            eba.pages_fork(pool, table, lens, src, dst)
    # the last check: a pool on the CPU has no kernels
    with pytest.raises(ValueError, match="CUDA"):
        eba.pages_release(pool, table, lens, lens)
    with pytest.raises(ValueError, match="CUDA"):
        eba.pages_fork(pool, table, lens, i32(0), i32(1))
    kv = torch.zeros(2, 5, 16, 2, 64, dtype=torch.bfloat16)
    cache = eba.PagedCache(kv[0], kv[1])
    for a, b in ((i32(0), i32(1, 2)), (i32(0).long(), i32(1)), (i32(0)[None], i32(1)[None]), (None, i32(1))):
        with pytest.raises(ValueError):
            eba.cache_copy(cache, a, b)
    with pytest.raises(ValueError):
        eba.cache_copy(kv, i32(0), i32(1))
    cu = i32(0, 1, 1, 2)
    for args, more in (((kv, table, i32(0, 1), cu), {}), ((cache, table[0], i32(0, 1), cu), {}),
                       ((cache, table, i32(0, 1), cu[:3]), {}), ((cache, table, i32(0, 1).long(), cu), {}),
                       ((cache, table, i32(0, 1), cu.long()), {}), ((cache, table, None, cu), {}),
                       ((cache, table, i32(0, 1), cu), dict(to_table=table[:2])),
                       ((cache, table, i32(0, 1), cu), dict(to_table=table[:, :0])),
                       ((cache, table, i32(0, 1), cu), dict(to_start=lens[:2])),
                       ((cache, table, i32(0, 1), cu), dict(to_start=lens.long()))):
        with pytest.raises(ValueError):
            eba.cache_gather(*args, **more)
    with pytest.raises(ValueError, match="CUDA"):
        eba.cache_gather(cache, table, i32(0, 1), cu)


def test_abi_refuses(eba):
    """Argument errors come before anything touches CUDA (there is no GPU here)."""
    L = eba.lib()
    P = eba._PoolStruct
    one = ctypes.c_void_p(4096)

    def pool(**k):
        return P(**{**dict(refs=4096, scratch=4096, n_pages=8, page_size=16), **k})

    invalid, unsupported = 1, 2
    for p in (None, pool(refs=None), pool(scratch=None), pool(n_pages=0), pool(n_pages=(1 << 30) + 1), pool(page_size=0)):
        assert L.attn_pages_release(p, one, 4, 4, one, one, 2, None) == invalid
        assert L.attn_pages_reserve(p, one, 4, 4, one, one, 2, None) == invalid
        assert L.attn_pages_fork(p, one, 4, 4, one, 2, one, one, 1, one, one, None) == invalid
    p = pool()
    for table, stride, wide, n in ((None, 4, 4, 2), (one, 3, 4, 2), (one, -1, 4, 2), (one, 4, 0, 2), (one, 4, 4, 0),
                                   (one, 1 << 16, 1 << 16, 1 << 15)):
        assert L.attn_pages_release(p, table, stride, wide, one, one, n, None) == invalid
    assert L.attn_pages_release(p, one, 4, 4, None, one, 2, None) == invalid
    assert L.attn_pages_reserve(p, one, 4, 4, one, None, 2, None) == invalid
    for args in ((None, 2, one, one, 1, one, one), (one, 2, None, one, 1, one, one), (one, 2, one, one, 0, one, one),
                 (one, 2, one, one, 1, one, None)):
        assert L.attn_pages_fork(p, one, 4, 4, *args, None) == invalid
    c = eba._CacheStruct()
    c.k, c.v, c.n_pages, c.page_size, c.H_kv, c.d, c.type, c.k_scale, c.v_scale = 4096, 8192, 4, 16, 2, 64, 0, 1, 1
    c.k_strides[:] = c.v_strides[:] = (16 * 2 * 64, 2 * 64, 64)
    assert L.attn_cache_copy(None, one, one, 1, None) == invalid
    assert L.attn_cache_copy(c, None, one, 1, None) == invalid
    assert L.attn_cache_copy(c, one, one, 0, None) == invalid
    for args in ((None, 4, 4, 2, one, one, 3, None, 0, 0, None), (one, 4, 0, 2, one, one, 3, None, 0, 0, None),
                 (one, 4, 4, 0, one, one, 3, None, 0, 0, None), (one, 4, 4, 2, None, one, 3, None, 0, 0, None),
                 (one, 4, 4, 2, one, None, 3, None, 0, 0, None), (one, 4, 4, 2, one, one, 0, None, 0, 0, None),
                 (one, 4, 4, 2, one, one, 3, one, 4, 0, None), (one, 4, 4, 2, one, one, 3, one, -1, 4, None)):
        assert L.attn_cache_gather(c, *args, None) == invalid
    c.d = 96
    assert L.attn_cache_copy(c, one, one, 1, None) == unsupported
