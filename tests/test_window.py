"""Windowed attention without a GPU: the oracle against closed forms, automatic and finite
differences, and what the binding and the C ABI refuse."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import window


@pytest.fixture(scope="module")
def eba():
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


def data(seed, B, H, Hkv, Lq, Lk, d):
    r = np.random.default_rng(seed)
    return [r.standard_normal(s) for s in ((B, H, Lq, d), (B, Hkv, Lk, d), (B, Hkv, Lk, d), (B, H, Lq, d))]


def test_visible_pairs():
    see = window.visible(4, 6, 1, 0, 1)  # places 2 to 5
    assert [list(np.flatnonzero(r)) for r in see] == [[0, 1, 2], [0, 2, 3], [0, 3, 4], [0, 4, 5]]
    see = window.visible(5, 3, 0, 1, 2)  # places -2 to 2
    assert [list(np.flatnonzero(r)) for r in see] == [[], [0], [0, 1], [0, 1, 2], [0, 1, 2]]
    assert window.visible(3, 4, None, None, 0).all()
    assert (window.visible(4, 4, None, 0, 3) == np.tri(4, dtype=bool)).all()


def test_no_ends_is_plain_attention():
    q, k, v, do = data(1, 1, 4, 2, 7, 9, 8)
    for mine, plain in ((window.forward(q, k, v, None, None, 3, 0.3), oracle.gqa_forward(q, k, v, 0.3)),
                        (window.backward(q, k, v, do, None, None, 3, 0.3), oracle.gqa_backward(q, k, v, do, 0.3))):
        for a, b in zip(mine, plain):
            assert np.abs(a - b).max() < 1e-13


@pytest.mark.parametrize("Lq,Lk,left,right,sinks", [(6, 6, 2, 0, 1), (5, 9, 1, 1, 0), (9, 5, 3, 0, 2), (4, 4, None, 0, 0), (6, 8, 0, None, 4)])
def test_gradients(Lq, Lk, left, right, sinks):
    """The formulas against torch's automatic differentiation of a masked softmax and
    against central differences."""
    q, k, v, do = data(Lq * 10 + Lk, 1, 2, 1, Lq, Lk, 4)
    seen = torch.from_numpy(window.visible(Lq, Lk, left, right, sinks))
    t = [torch.from_numpy(x).requires_grad_(True) for x in (q, k, v)]
    x = (t[0] @ t[1].transpose(-1, -2) * 0.5).masked_fill(~seen, -1e300)
    o = (torch.softmax(x, -1) * seen) @ t[2]
    grads = torch.autograd.grad(o, t, torch.from_numpy(do))
    got = window.backward(q, k, v, do, left, right, sinks, 0.5)
    assert np.abs(window.forward(q, k, v, left, right, sinks, 0.5)[0] - o.detach().numpy()).max() < 1e-13
    for a, b in zip(got, grads):
        assert np.abs(a - b.numpy()).max() < 1e-12
    r = np.random.default_rng(0)
    for n, x in enumerate((q, k, v)):
        step = r.standard_normal(x.shape)

        def loss(h):
            args = [q, k, v]
            args[n] = x + h * step
            return (window.forward(*args, left, right, sinks, 0.5)[0] * do).sum()

        assert abs((loss(1e-5) - loss(-1e-5)) / 2e-5 - (got[n] * step).sum()) < 1e-7


def test_binding_refuses(eba):
    for left, right, sinks in ((-1, 0, 0), (1.0, 0, 0), (0, -1, 0), (0, "1", 0), (0, 0, -1), (0, 0, None), (1 << 31, 0, 0)):
        with pytest.raises(ValueError):
            eba._sides(left, right, sinks)
    assert eba._sides(None, None, 3) == [-1, -1, 3]
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    for f in (eba.fwd_window, eba.attention_window):
        with pytest.raises(ValueError, match="CUDA"):
            f(q, q, q, 4)


def test_abi_refuses(eba):
    L = eba.lib()
    one = ctypes.c_void_p(4096)
    off = ctypes.c_void_p(4100)

    def fwd(B=1, H=4, Hkv=2, Lq=9, Lk=9, d=64, left=3, right=0, sinks=0, scale=0.1, q=one, rest=None):
        return L.attn_fwd_window(q, one, one, one, rest, one, B, H, Hkv, Lq, Lk, d, left, right, sinks, scale, None)

    def bwd(B=1, H=4, Hkv=2, Lq=9, Lk=9, d=64, left=3, right=0, sinks=0, scale=0.1, q=one, ws=one, n=1 << 40, rest=None):
        return L.attn_bwd_window(q, one, one, one, rest, one, one, one, one, one, B, H, Hkv, Lq, Lk, d, left, right, sinks, scale, ws, n, None)

    for f in (fwd, bwd):
        for bad in (dict(B=0), dict(H=0), dict(Lq=0), dict(Lk=0), dict(Hkv=3), dict(Hkv=0), dict(left=-2), dict(right=-2),
                    dict(sinks=-1), dict(scale=0.0), dict(scale=float("inf")), dict(q=None), dict(Lq=(1 << 29) + 1),
                    dict(Lk=(1 << 29) + 1)):
            assert f(**bad) == 1, bad
        assert f(d=96) == 2 and f(q=off) == 3 and f(rest=off) == 3
    assert bwd(ws=None) == 6 and bwd(n=100) == 6 and bwd(ws=off) == 3


def test_workspace(eba):
    size = eba.bwd_window_workspace_size
    plain = eba.bwd_workspace_size(1, 16, 12544, 12544, 128)
    assert size(1, 16, 4, 12544, 12544, 128, 1567) == plain
    assert size(1, 16, 4, 12544, 12544, 128, None, 0, 16) == plain  # every query sees them anyway
    # the first tokens' key tile in pieces of 15 query tiles: 7 of them for 98
    assert size(1, 16, 4, 12544, 12544, 128, 1567, 0, 16) == plain + 4 * 7 * 2 * 128 * 128 * 4
    assert eba.lib().attn_bwd_window_workspace_size(1, 4, 3, 9, 9, 64, 1, 1, 0) == 0
