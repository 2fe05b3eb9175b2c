"""Windowed decode without a GPU: refusals of the binding and the C ABI, and its workspace."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def eba():
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


def test_binding_refuses(eba):
    kv = torch.zeros(2, 5, 16, 2, 64, dtype=torch.bfloat16)
    cache = eba.PagedCache(kv[0], kv[1])
    # (sizes are checked before devices: nothing of this needs a GPU)
    for window, sinks in ((0, 0), (-3, 0), (1.5, 0), ("8", 0), (8, -1), (8, 1.0), (1 << 31, 0), (8, 1 << 31), (None, -1), (None, 2.0)):
        with pytest.raises(ValueError, match="window|sinks"):
            eba._window(window, sinks)
    assert eba._window(None, 0) == eba._window(None, 7) == (None, 0) and eba._window(8, 4) == (8, 4)
    with pytest.raises(ValueError):
        eba.decode(cache, torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32),
                   torch.zeros(1, dtype=torch.int32), window=0)


def test_abi_refuses(eba):
    L = eba.lib()
    one, c = ctypes.c_void_p(4096), eba._CacheStruct()
    c.k, c.v, c.n_pages, c.page_size, c.H_kv, c.d, c.type, c.k_scale, c.v_scale = 4096, 8192, 4, 16, 2, 64, 0, 1, 1
    c.k_strides[:] = c.v_strides[:] = (16 * 2 * 64, 2 * 64, 64)
    st = (ctypes.c_longlong * 2)(256, 64)
    for window, sinks in ((0, 0), (-1, 0), (5, -1)):
        assert L.attn_decode_window(c, one, st, one, 4, 4, one, 1, 4, window, sinks, 0.125, None, None, 0, one, one, None, 0, None) == 1
        assert L.attn_decode_window_workspace_size(1, 4, 2, 64, 0, 64, window, sinks) == 0
    assert L.attn_decode_window(c, one, st, one, 4, 4, one, 1, 3, 8, 0, 0.125, None, None, 0, one, one, None, 0, None) == 1


def test_workspace_goes_by_the_window(eba):
    kv = torch.zeros(2, 2, 16, 2, 128, dtype=torch.bfloat16)
    cache = eba.PagedCache(kv[0], kv[1])
    assert eba.decode_workspace_size(cache, 1, 8, 8192) > 0
    assert eba.decode_workspace_size(cache, 1, 8, 8192, window=512, sinks=4) == 0  # one cluster an item
    assert eba.decode_workspace_size(cache, 1, 8, 8192, window=1 << 20) > 0
