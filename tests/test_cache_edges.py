"""The rotation and the cache without a GPU, where they are most easily wrong: the
exact bits of a rotation's table, arguments of another type, gradients that are not
asked for."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def eba():
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


def test_scales_that_no_factor_holds_are_refused(eba):
    c, L, at = eba._CacheStruct(), eba.lib(), 1 << 20  # an address that is never used
    c.k = c.v = at
    c.k_strides[:] = c.v_strides[:] = [2048, 128, 64]
    c.n_pages, c.page_size, c.H_kv, c.d, c.k_scale, c.v_scale = 10, 16, 2, 64, 1.0, 1.0
    strides = (ctypes.c_longlong * 2)(128, 64)
    for c.type in (0, 1):
        assert L.attn_decode(c, at, strides, at, 4, 4, at, 3, 2, 3e38, None, None, 0, at, at, at, 1 << 30, None) == 1
