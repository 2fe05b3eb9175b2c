"""Rotation, cache append and decode without a GPU: what the C ABI and the Python
binding refuse before anything is launched, the rotation's fixed-point table,
and the oracle's own pins."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle

A16 = 1 << 20        # a fake, 16-byte aligned address; never dereferenced
MIS = (1 << 20) + 8  # a fake misaligned address; never dereferenced


@pytest.fixture(scope="module")
def eba():
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


def ll(*x):
    return (ctypes.c_longlong * len(x))(*x)


def test_rope_init_refuses(eba):
    L = eba.lib()

    def init(pairs=8, axes=1, axis=None, freq=None, r=None):
        n = max(pairs, 1)
        return L.attn_rope_init(r or eba._RopeStruct(), pairs, axes,
                                (ctypes.c_int * n)(*(axis or [0] * n)),
                                (ctypes.c_double * n)(*(freq or [1.0] * n)), 0)

    assert init() == 0
    assert init(pairs=0) == 1 and init(pairs=12) == 1 and init(pairs=72) == 2
    assert init(axes=0) == 1 and init(axes=5) == 2
    assert init(axis=[0] * 7 + [1]) == 1 and init(axis=[0] * 7 + [-1]) == 1
    assert init(freq=[1.0] * 7 + [math.nan]) == 1 and init(freq=[math.inf] + [1.0] * 7) == 1
    assert L.attn_rope_init(None, 8, 1, (ctypes.c_int * 8)(), (ctypes.c_double * 8)(), 0) == 1


def test_rope_table_is_turns_in_fixed_point(eba):
    freq = [1.0, 0.5, -1.0, 0.0, 2 * math.pi, 100.0, 1e-12, -1e-30]
    plan = eba.Rope((8,), frequencies=freq)
    for f, t in zip(freq, plan._struct.turns):
        exact = f / (2 * math.pi) % 1.0
        off = abs(t / 2.0 ** 64 - exact)
        assert min(off, 1 - off) <= 2.0 ** -52 * max(1.0, abs(f))
    plan = eba.Rope((8, 12, 12))
    assert plan.n_axes == 3 and list(plan._struct.axis)[:32] == [0] * 8 + [1] * 12 + [2] * 12
    assert plan.frequencies[8] == 1.0 and plan.frequencies[9] == 10000.0 ** (-1 / 12)


@pytest.mark.parametrize("kw", [
    dict(axis_pairs=()), dict(axis_pairs=(4,)), dict(axis_pairs=(0, 8)), dict(axis_pairs=(72,)),
    dict(axis_pairs=(8,) * 5), dict(axis_pairs=(8,), theta=0), dict(axis_pairs=(8,), theta=math.inf),
    dict(axis_pairs=(8,), pairing="quarter"), dict(axis_pairs=(8,), frequencies=[1.0] * 7),
    dict(axis_pairs=(8,), frequencies=[math.nan] * 8)], ids=str)
def test_rope_plan_refuses(eba, kw):
    with pytest.raises(ValueError):
        eba.Rope(**kw)


def test_rope_call_refuses(eba):
    L, plan = eba.lib(), eba.Rope((32,))

    def call(q=A16, qs=(0, 64, 128), k=A16, ks=(0, 64, 128), pos=A16, B=1, H=2, Hk=2, n=4, d=64,
             r=plan._struct, qo=A16):
        return L.attn_rope(r, q, ll(*qs), qo, ll(0, 64, 128), k, ll(*ks), A16, ll(0, 64, 128), pos,
                           ll(0, 0), B, H, Hk, n, d, 0, None)

    assert call(q=None) == 1 and call(pos=None) == 1 and call(k=None) == 1 and call(r=None) == 1
    assert call(B=0) == 1 and call(H=0) == 1 and call(Hk=-1) == 1 and call(n=0) == 1
    assert call(d=96) == 2 and call(H=70000) == 1
    assert call(q=MIS) == 3 and call(qo=MIS) == 3 and call(qs=(0, 64, 100)) == 3
    assert call(ks=(0, -64, 128)) == 1
    assert call(r=eba.Rope((64,))._struct) == 1      # 128 elements of 64
    assert call(r=eba._RopeStruct()) == 1            # never filled in


def cache_struct(eba, **kw):
    s = eba._CacheStruct()
    s.k = s.v = A16
    s.k_strides[:] = s.v_strides[:] = [16 * 2 * 64, 2 * 64, 64]
    s.n_pages, s.page_size, s.H_kv, s.d, s.type, s.k_scale, s.v_scale = 10, 16, 2, 64, 0, 1, 1
    for n, x in kw.items():
        setattr(s, n, x)
    return s


BAD_CACHES = [(dict(k=None), 1), (dict(v=MIS), 3), (dict(n_pages=0), 1), (dict(n_pages=1 << 31), 1),
              (dict(page_size=0), 1), (dict(H_kv=0), 1), (dict(d=96), 2), (dict(type=2), 2),
              (dict(k_scale=0.5), 1), (dict(type=1, v_scale=0.0), 1), (dict(type=1, k_scale=math.nan), 1),
              (dict(type=1, k_scale=1e-45), 1), (dict(k_strides=(ctypes.c_longlong * 3)(2048, 128, 60)), 3),
              (dict(type=1, k_strides=(ctypes.c_longlong * 3)(2048, 128, 72)), 3),
              (dict(v_strides=(ctypes.c_longlong * 3)(-2048, 128, 64)), 1)]


@pytest.mark.parametrize("kw,code", BAD_CACHES, ids=str)
def test_caches_refused(eba, kw, code):
    L, c = eba.lib(), cache_struct(eba, **kw)
    assert L.attn_cache_append(c, A16, ll(128, 64), A16, ll(128, 64), A16, 4, 4, A16, 3, None, 3, None,
                               None, 0, None) == code
    assert L.attn_decode(c, A16, ll(128, 64), A16, 4, 4, A16, 3, 2, 0.1, None, None, 0, A16, A16, A16,
                         1 << 30, None) == code


def test_append_refuses(eba):
    L, c = eba.lib(), cache_struct(eba)
    one, three = eba.Rope((32,))._struct, eba.Rope((8, 12, 12))._struct

    def call(cache=c, k=A16, ks=(128, 64), v=A16, table=A16, stride=4, wide=4, lens=A16, n=3, cu=None,
             T=3, rope=None, pos=None):
        return L.attn_cache_append(cache, k, ll(*ks), v, ll(128, 64), table, stride, wide, lens, n, cu, T,
                                   rope, pos, 0, None)

    assert call(cache=None) == 1 and call(k=None) == 1 and call(v=MIS) == 3 and call(ks=(128, 60)) == 3
    assert call(table=None) == 1 and call(lens=None) == 1 and call(wide=0) == 1 and call(stride=-1) == 1
    assert call(n=0) == 1 and call(T=4) == 1 and call(T=0, cu=A16) == 1
    assert call(rope=three) == 1                          # several axes need positions
    assert call(rope=eba.Rope((64,))._struct, pos=A16) == 1


def test_decode_refuses(eba):
    L, c = eba.lib(), cache_struct(eba)
    need = L.attn_decode_workspace_size(3, 6, 2, 64, 0, 2000 * 16)
    assert need > 0
    assert L.attn_decode_workspace_size(3, 6, 2, 64, 0, 64) == 0  # short: none

    def call(cache=c, q=A16, qs=(384, 64), wide=2000, B=3, H=6, scale=0.1, rope=None, pos=None, o=A16,
             lse=A16, ws=A16, size=need):
        return L.attn_decode(cache, q, ll(*qs), A16, 4, wide, A16, B, H, scale, rope, pos, 0, o, lse, ws,
                             size, None)

    assert call(cache=None) == 1 and call(q=None) == 1 and call(o=MIS) == 3 and call(lse=None) == 1
    assert call(qs=(384, 62)) == 3 and call(qs=(-384, 64)) == 1
    assert call(B=0) == 1 and call(H=0) == 1 and call(H=5) == 1 and call(wide=0) == 1
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=scale) == 1
    assert call(rope=eba.Rope((8, 12, 12))._struct) == 1
    assert call(ws=None) == 6 and call(size=need - 1) == 6 and call(ws=MIS) == 3
    for bad in ((0, 6, 2, 64, 0, 32000), (3, 0, 2, 64, 0, 32000), (3, 6, 0, 64, 0, 32000),
                (3, 6, 4, 64, 0, 32000), (3, 6, 2, 96, 0, 32000), (3, 6, 2, 64, 2, 32000), (3, 6, 2, 64, 0, 0)):
        assert L.attn_decode_workspace_size(*bad) == 0
    # a table of more tiles than can be counted
    assert call(cache=cache_struct(eba, page_size=1 << 30), wide=1 << 30, B=1000, size=1 << 40) == 1


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_paged_cache_handle_refuses(eba):
    ok = z(4, 16, 2, 64)
    eba.PagedCache(ok, ok.clone())
    eba.PagedCache(z(4, 2, 16, 64).transpose(1, 2), z(4, 2, 16, 64).transpose(1, 2))
    f8 = ok.to(torch.float8_e4m3fn)
    eba.PagedCache(f8, f8.clone(), 0.1, 2.0)
    both = z(4, 2, 16, 2, 64)  # keys and values of a page side by side
    eba.PagedCache(both[:, 0], both[:, 1])
    for k, v, kw in [
        (ok, z(4, 16, 2, 128), {}), (ok, f8, {}), (ok[0], ok[0], {}), (ok, ok, {}),
        (z(4, 16, 2, 96), z(4, 16, 2, 96), {}), (z(0, 16, 2, 64), z(0, 16, 2, 64), {}),
        (ok.float(), ok.float(), {}), (ok, ok.clone(), dict(k_scale=2.0)),
        (f8, f8.clone(), dict(v_scale=0.0)), (f8, f8.clone(), dict(k_scale=math.inf)),
        (z(4, 16, 2, 128)[..., ::2], z(4, 16, 2, 64), {}),           # rows with gaps
        (z(4, 16, 2, 68)[..., :64], z(4, 16, 2, 68)[..., :64], {}),   # rows off 16-byte boundaries
        (z(1, 16, 2, 64).expand(4, 16, 2, 64), ok, {}),              # pages on top of one another
    ]:
        with pytest.raises(ValueError):
            eba.PagedCache(k, v, **kw)


def test_binding_refuses_before_the_library(eba, monkeypatch):
    plan, plan3 = eba.Rope((32,)), eba.Rope((8, 12, 12))

    def no_library():
        raise AssertionError("the library was called")

    monkeypatch.setattr(eba, "lib", no_library)
    ok = z(4, 16, 2, 64)
    cache = eba.PagedCache(ok, ok.clone())
    i32 = dict(dtype=torch.int32)
    for call in [
        lambda: eba.rope_fwd(z(3, 2, 64), None, z(3, **i32), plan),            # CPU tensors
        lambda: eba.rope(z(1, 2, 3, 64), None, z(3, **i32), plan),
        lambda: eba.rope_fwd("q", None, z(3, **i32), plan),
        lambda: eba.cache_append(cache, z(3, 2, 64), z(3, 2, 64), z(3, 4, **i32), z(3, **i32)),
        lambda: eba.cache_append(ok, z(3, 2, 64), z(3, 2, 64), z(3, 4, **i32), z(3, **i32)),
        lambda: eba.decode(cache, z(3, 2, 64), z(3, 4, **i32), z(3, **i32)),
        lambda: eba.decode(None, z(3, 2, 64), z(3, 4, **i32), z(3, **i32)),
    ]:
        with pytest.raises(ValueError):
            call()
    # the checks behind the device's, on CPU tensors
    cpu = torch.device("cpu")
    assert eba._rows(z(3, 2, 64), "q", 3, "cpu") == [128, 64]
    assert eba._rows(z(1, 2, 64).expand(3, 2, 64), "q", 3, "cpu") == [0, 64]
    for bad in (z(3, 2, 64).float(), z(2, 64), z(3, 2, 96), z(3, 2, 128)[..., ::2], z(3, 2, 68)[..., 4:],
                z(3, 2, 68)[..., :64], z(400)[4:388].view(3, 2, 64)):
        with pytest.raises(ValueError):
            eba._rows(bad, "q", 3, "cpu")
    assert plan._positions(z(5, **i32), cpu, (5,)) == 0
    assert plan._positions(z(1, 5, **i32), cpu, (5,)) == 5
    assert plan3._positions(z(3, 5, **i32), cpu, (5,)) == 5
    for p, bad in ((plan, z(4, **i32)), (plan, z(5)), (plan, z(2, 5, **i32)), (plan3, z(5, **i32)),
                   (plan3, z(3, 10, **i32)[:, ::2]), (plan, z(5, dtype=torch.int64)), (plan, None)):
        with pytest.raises(ValueError):
            p._positions(bad, cpu, (5,))
    assert cache._batch(z(3, 4, **i32), z(3, **i32)) == 3
    for table, lens in ((z(2, 4, **i32), z(3, **i32)), (z(3, 0, **i32), z(3, **i32)), (z(0, 4, **i32), z(0, **i32)),
                        (z(3, **i32), z(3, **i32)), (z(3, 4, dtype=torch.int64), z(3, **i32)),
                        (z(4, 3, **i32).t(), z(3, **i32)), (z(3, 4, **i32), z(6, **i32)[::2])):
        with pytest.raises(ValueError):
            cache._batch(table, lens)
    assert cache._turn(None, None, 3) == (None, None, 0)
    for rope, pos in ((None, z(3, **i32)), (plan3, None), (plan3, z(3, **i32)), ("r", z(3, **i32)),
                      (eba_rope_128(plan), z(3, **i32))):
        with pytest.raises(ValueError):
            cache._turn(rope, pos, 3)


def eba_rope_128(plan):
    """A copy of a plan that claims 64 pairs: too many for heads of 64."""
    other = object.__new__(type(plan))
    other.__dict__.update(plan.__dict__, n_pairs=64)
    return other


# ---------------------------------------------------------------------------
# The oracle's pins
# ---------------------------------------------------------------------------

def test_oracle_rope_is_the_rotation_of_complex_numbers():
    r = np.random.default_rng(0)
    x, pos = r.normal(size=(5, 2, 12)), r.integers(-9, 9, size=(2, 5))
    axis, freq = [0, 0, 1, 1], [1.0, 0.3, 0.7, 0.01]
    for inter in (False, True):
        y = oracle.rope(x, pos, axis, freq, inter)
        first, second = (np.arange(0, 8, 2), np.arange(1, 8, 2)) if inter else (np.arange(4), np.arange(4, 8))
        z = (x[..., first] + 1j * x[..., second]) * np.exp(1j * pos[axis].T * freq)[:, None]
        assert np.allclose(y[..., first], z.real) and np.allclose(y[..., second], z.imag)
        assert np.array_equal(y[..., 8:], x[..., 8:])


def test_oracle_rope_scores_depend_on_differences_and_gradient_is_the_transpose():
    r = np.random.default_rng(1)
    q, k = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8))
    args = ([0, 0, 1, 1], [1.0, 0.1, 1.0, 0.1], False)

    def score(p, s):
        return (oracle.rope(q, np.array(p)[:, None], *args) * oracle.rope(k, np.array(s)[:, None], *args)).sum()

    assert abs(score((5, 2), (3, 7)) - score((105, 52), (103, 57))) < 1e-12
    # the gradient of sum(rope(x) g) by differences
    x, g, pos = r.normal(size=(3, 2, 8)), r.normal(size=(3, 2, 8)), r.integers(0, 50, size=(2, 3))
    dx = oracle.rope(g, pos, *args, inverse=True)
    for i in np.ndindex(3, 2, 8):
        e = np.zeros_like(x)
        e[i] = 1e-4
        diff = ((oracle.rope(x + e, pos, *args) - oracle.rope(x - e, pos, *args)) * g).sum() / 2e-4
        assert abs(diff - dx[i]) < 1e-9


def test_oracle_decode_is_the_forward_of_one_query():
    r = np.random.default_rng(2)
    q = r.normal(size=(2, 4, 16))
    keys, values = [[r.normal(size=(n, 2, 16)) for n in (7, 0)] for _ in range(2)]
    o, lse = oracle.decode(q, keys, values, 0.25)
    ro, rl = oracle.gqa_forward(q[:1, :, None], keys[0].swapaxes(0, 1)[None], values[0].swapaxes(0, 1)[None], 0.25)
    assert np.allclose(o[0], ro[0, :, 0]) and np.allclose(lse[0], rl[0, :, 0])
    assert (o[1] == 0).all() and np.isneginf(lse[1]).all()
    pages = r.normal(size=(4, 3, 2, 16))
    assert np.array_equal(oracle.gather(pages, [2, 0], 5), np.concatenate([pages[2], pages[0, :2]]))
