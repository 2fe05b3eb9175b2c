"""Drafted tokens' attention without a GPU: the oracle's sets, and what the binding and the C
ABI refuse."""
import ctypes

import pytest
import torch

from oracle import tree


@pytest.fixture(scope="module")
def eba():
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


def test_sets():
    assert tree.seen(5, 2, 0) == [0, 1, 2, 3] and tree.seen(5, 2, 1) == [0, 1, 2, 3, 4]
    assert tree.seen(5, 2, 1, window=2) == [3, 4] and tree.seen(5, 2, 0, window=2, sinks=1) == [0, 2, 3]
    assert tree.seen(5, 3, 2, mask=0b101) == [0, 1, 2, 4]
    assert tree.seen(5, 3, 2, mask=0b101, window=2) == [2, 4]  # at place 3
    assert tree.seen(5, 3, 2, mask=0b1000) == [0, 1]           # bits of no token
    assert tree.seen(5, 3, 2, mask=0, window=1, sinks=1) == [0]
    assert tree.seen(2, 2, 1, mask=0) == []


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_binding_refuses(eba):
    kv = torch.zeros(2, 5, 16, 2, 64, dtype=torch.bfloat16)
    cache = eba.PagedCache(kv[0], kv[1])
    table, lens, cu = torch.zeros(2, 4, dtype=torch.int32), i32(9, 9), i32(0, 2, 5)
    q, mask = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, dtype=torch.int64)

    def layout(cache=cache, q=q, table=table, lens=lens, cu=cu, mask=mask, window=None, sinks=0):
        import unittest.mock as m
        # the device check of the query comes first: everything else is looked at on the CPU
        with m.patch.object(eba, "_rows", lambda t, name, nd: [t.stride(0), t.stride(1)]):
            return eba._tree_layout(cache, q, table, lens, cu, mask, window, sinks)

    assert layout()[3:] == (2, 5, 4, 64, 2, 2, eba.decode_tree_workspace_size(cache, 5, 2, 4))
    assert layout(mask=mask[:, 0])[7:9] == (2, 1)
    for bad in (dict(cache=kv), dict(q=q[:, :3]), dict(q=q[:0]), dict(q=torch.zeros(5, 4, 128)), dict(cu=i32(0, 5)),
                dict(cu=None), dict(cu=cu.long()), dict(mask=mask.int()), dict(mask=mask[:4]), dict(mask=mask[:, :0]),
                dict(mask=torch.zeros(5, 17, dtype=torch.int64)), dict(mask=mask.t().contiguous().t()), dict(mask=[1] * 5),
                dict(window=0), dict(window=-2), dict(sinks=-3), dict(window=4, sinks=-1), dict(lens=lens[:1]),
                dict(table=table[:1])):
        with pytest.raises(ValueError):
            layout(**bad)
    with pytest.raises(ValueError, match="CUDA"):
        eba.decode_tree(cache, q, table, lens, cu)


def test_abi_refuses(eba):
    L = eba.lib()
    one, c = ctypes.c_void_p(4096), eba._CacheStruct()
    c.k, c.v, c.n_pages, c.page_size, c.H_kv, c.d, c.type, c.k_scale, c.v_scale = 4096, 8192, 4, 16, 2, 64, 0, 1, 1
    c.k_strides[:] = c.v_strides[:] = (16 * 2 * 64, 2 * 64, 64)
    st = (ctypes.c_longlong * 2)(256, 64)
    need = L.attn_decode_tree_workspace_size(5, 2, 4, 2, 64)
    assert need > 0 and L.attn_decode_tree_workspace_size(5, 2, 3, 2, 64) == 0
    assert L.attn_decode_tree_workspace_size(0, 2, 4, 2, 64) == 0 and L.attn_decode_tree_workspace_size(5, 2, 4, 2, 96) == 0

    def call(cache=c, q=one, st=st, table=one, stride=4, wide=4, lens=one, B=2, cu=one, T=5, H=4, mask=one, mst=2, words=2,
             window=0, sinks=0, scale=0.125, o=one, lse=one, ws=one, n=need):
        return L.attn_decode_tree(cache, q, st, table, stride, wide, lens, B, cu, T, H, mask, mst, words, window, sinks, scale,
                                  o, lse, ws, n, None)

    for bad in (dict(cache=None), dict(q=None), dict(st=None), dict(table=None), dict(wide=0), dict(lens=None), dict(B=0),
                dict(T=0), dict(cu=None), dict(H=3), dict(H=0), dict(words=0), dict(mst=-1), dict(window=-1), dict(sinks=-1),
                dict(scale=0.0), dict(scale=float("nan")), dict(o=None), dict(T=1 << 30), dict(wide=1 << 30, T=1 << 20)):
        assert call(**bad) == 1, bad
    assert call(words=17) == 2
    assert call(q=ctypes.c_void_p(4100)) == 3 and call(ws=ctypes.c_void_p(4100)) == 3
    assert call(st=(ctypes.c_longlong * 2)(256, 63)) == 3
    assert call(ws=None) == 6 and call(n=need - 1) == 6
