"""The rotation and the cache without a GPU, where they are most easily wrong: the
exact bits of a rotation's table, arguments of another type, gradients that are not
asked for."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch


@pytest.fixture(scope="module")
def eba():
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


def two_pi():
    """2 pi to 1300 bits: 8 (4 atan(1/5) - atan(1/239)), the arctangents' series in integers."""
    one = 1 << 1330

    def atan_inverse(n):
        term, total, k = one // n, 0, 0
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term //= n * n
            k += 1
        return total

    return Fraction(8 * (4 * atan_inverse(5) - atan_inverse(239)), one)


@pytest.mark.parametrize("freq", [
    [1.0, 0.5, -1.0, 0.0, 2 * math.pi, 100.0, 1e-12, -1e-30],
    [10000.0 ** (-i / 64) for i in range(64)], [500000.0 ** (-i / 22) for i in range(24)],
    [-3.7, 12345.678, -1e6, 1e9, -1e15, 1e22, 5e-324, -5e-324]], ids=["mixed", "text", "axis", "far"])
def test_rope_table_holds_all_its_bits(eba, freq):
    # a step is 2^-64 turns; the two-part 1 / (2 pi) adds |f| 2^-107 turns
    table = eba.Rope((len(freq),), frequencies=freq)._struct.turns
    turn = two_pi()
    for f, t in zip(freq, table):
        exact = Fraction(f) / turn * 2 ** 64
        off = (t - exact) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        assert off <= 1 + Fraction(abs(f)) / 2 ** 43, (f, float(off))


def test_far_positions_are_as_exact_as_near_ones(eba):
    # the fixed-point angle, as the kernels form it, within 2^-31 turns at every position
    freq = [10000.0 ** (-i / 64) for i in range(64)]
    table = eba.Rope((64,), frequencies=freq)._struct.turns
    turn = two_pi()
    for p in (1, 12345, 2 ** 31 - 1, -2 ** 31):
        for f, t in zip(freq, table):
            angle = (p * t) % 2 ** 64 >> 32
            off = (angle - Fraction(f) * p / turn * 2 ** 32) % 2 ** 32
            assert min(off, 2 ** 32 - off) <= 2, (p, f)


def test_positions_that_are_no_tensor_are_refused(eba):
    pages = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    cache, plan = eba.PagedCache(pages, pages.clone()), eba.Rope((32,))
    for positions in ([1, 2, 3], 7, "123"):
        with pytest.raises(ValueError):
            cache._turn(plan, positions, 3)


def test_scales_that_no_factor_holds_are_refused(eba):
    c, L, at = eba._CacheStruct(), eba.lib(), 1 << 20  # an address that is never used
    c.k = c.v = at
    c.k_strides[:] = c.v_strides[:] = [2048, 128, 64]
    c.n_pages, c.page_size, c.H_kv, c.d, c.k_scale, c.v_scale = 10, 16, 2, 64, 1.0, 1.0
    strides = (ctypes.c_longlong * 2)(128, 64)
    for c.type in (0, 1):
        assert L.attn_decode(c, at, strides, at, 4, 4, at, 3, 2, 3e38, None, None, 0, at, at, at, 1 << 30, None) == 1


@pytest.mark.parametrize("again", [False, True], ids=["once", "create_graph"])
@pytest.mark.parametrize("trained", ["q", "k", "qk"])
def test_gradients_nobody_asks_for_are_not_computed(eba, monkeypatch, trained, again):
    calls = []

    def turn(q, k, positions, plan, inverse):
        calls.append((inverse, q, k))
        return q * 1.0, None if k is None else k * 1.0

    monkeypatch.setattr(eba, "_rope", turn)
    q, k = torch.ones(3, 2, 4, requires_grad="q" in trained), torch.ones(3, 1, 4, requires_grad="k" in trained)
    qo, ko = eba.rope(q, k, torch.arange(3), None)
    inputs = [x for x in (q, k) if x.requires_grad]
    grads = torch.autograd.grad((qo * ko).sum(), inputs, create_graph=again)
    assert [g.shape for g in grads] == [x.shape for x in inputs]
    inverse, dq, dk = calls[1]
    assert inverse and len(calls) == 2
    assert dq.shape == inputs[0].shape and (dk is None) == (trained != "qk")
