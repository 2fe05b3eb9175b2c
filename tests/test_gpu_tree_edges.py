"""Drafted tokens' attention where a cache, a query or the offsets hold what they should not."""
import math

import numpy as np
import pytest
import torch

import oracle
from cache_util import Paged, bf16, np64
from oracle import tree
from test_gpu_tree import tolerances

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eba():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


@pytest.fixture(autouse=True)
def status_is_clean(eba):
    eba.poll_device_status()
    yield
    assert eba.poll_device_status() == 0


def test_offsets_that_fall(eba):
    """They are recorded; sequences that share no row with others are as ever."""
    p = Paged([300, 50, 40], 16, 1, 64, seed=7)
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(6), 9, 2, 64).cuda()
    call = lambda *cu: eba.decode_tree(cache, q, p.gtable, p.glens, torch.tensor(cu, dtype=torch.int32).cuda())  # noqa: E731
    o, lse = call(0, 3, 6, 9)
    for cu, rows in (((0, 3, 6, 0), range(6)), ((0, 3, 1, 1), range(3)), ((0, 3, -1, 0), range(3)), ((9, 9, 9, 0), ())):
        x, y = call(*cu)
        assert eba.poll_device_status() == 7
        rows = torch.tensor(list(rows), dtype=torch.long, device="cuda")
        # (within the rounding of both, should the list be cut elsewhere)
        assert ((x - o).float().abs() <= 2.0 ** -7 * o.float().abs() + 2.0 ** -16)[rows].all()
        assert ((y - lse).abs() <= 1e-5)[rows].all()


def test_offsets_that_fall_too_often(eba):
    """The sequences they name have more tiles together than an int can count, 4000 times all 2048
    tokens of 64 heads over 131072 keys: no row is computed."""
    p = Paged([300], 128, 8, 64, seed=8)
    cache = p.on_gpu(eba)
    B, T = 8000, 2048
    table = p.gtable[:, :1].expand(1, 1024).contiguous().expand(B, 1024)
    lens = torch.full((B,), 1024 * 128, dtype=torch.int32, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    q = bf16(torch.Generator().manual_seed(9), T, 64, 64).cuda()
    o, lse = eba.decode_tree(cache, q, table, lens, cu)
    assert eba.poll_device_status() == 7
    assert (o == 0).all() and torch.isneginf(lse).all()


# one tile; items that are not cut; cut in few parts, and in many
LENS = [[100, 90], [700] * 40, [2000, 1500], [20000]]


@pytest.mark.parametrize("d,e4m3,page", [(128, False, 16), (64, False, 20), (64, True, 16), (128, True, 7)])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: f"{len(x)}x{x[0]}")
def test_nan_and_infinities_that_are_seen(eba, lens, d, e4m3, page):
    """By K/V head: 0 a NaN key, 1 a NaN in one element of a value, 2 a key of score +inf or
    -inf (by the query's sign), 3 only keys of such scores, 4 plain, with a NaN query in its
    first head and an all-NaN one in its second (e4m3 holds no infinities: 2 and 3 plain)."""
    hk, H, news = 5, 10, [3] * len(lens)
    p = Paged(lens, page, hk, d, e4m3=e4m3, seed=d, **(dict(k_scale=0.05, v_scale=0.5) if e4m3 else {}))
    kk, vv = p.pages(p.k).float(), p.pages(p.v).float()
    for b, n in enumerate(lens):
        rows = torch.tensor(p.rows[b])
        at = n // 2
        page_, slot = rows[at // page], at % page
        kk[page_, slot, 0, 1] = math.nan
        vv[page_, slot, 1, 5] = math.nan
        if not e4m3:
            kk[page_, slot, 2, 0] = math.inf
            every = torch.arange(n)
            kk[rows[every // page], every % page, 3, 0] = math.inf
    p.k, p.v = ((x.transpose(1, 2) if p.heads_first else x).to(p.k.dtype) for x in (kk, vv))
    cache = p.on_gpu(eba)
    T = sum(news)
    q = bf16(torch.Generator().manual_seed(7), T, H, d)
    q[:, :, 0] = torch.where(q[:, :, 0] == 0, torch.ones_like(q[:, :, 0]), q[:, :, 0])
    q[1::3, 8, 3] = math.nan
    q[2::3, 9] = math.nan
    cu = torch.arange(0, T + 1, 3, dtype=torch.int32).cuda()
    o, lse = eba.decode_tree(cache, q.cuda(), p.gtable, p.glens, cu)
    o, lse = np64(o), np64(lse)
    up = np64(q)[:, :, 0] > 0
    assert np.isnan(o[:, :2]).all() and np.isnan(lse[:, :2]).all()
    assert np.isnan(o[:, 2:4, 5]).all() and np.isfinite(o[:, 2:4, 6:]).all() and np.isfinite(lse[:, 2:4]).all()
    if not e4m3:
        pos, neg = up[:, 4:6], ~up[:, 4:6]
        assert np.isnan(o[:, 4:6][pos]).all() and np.isnan(lse[:, 4:6][pos]).all()
        assert np.isfinite(o[:, 4:6][neg]).all() and np.isfinite(lse[:, 4:6][neg]).all()
        pos, neg = up[:, 6:8], ~up[:, 6:8]
        assert np.isnan(o[:, 6:8][pos]).all() and np.isnan(lse[:, 6:8][pos]).all()
        assert (o[:, 6:8][neg] == 0).all() and np.isneginf(lse[:, 6:8][neg]).all()
    bad = np.zeros((T, 2), dtype=bool)
    bad[1::3, 0] = bad[2::3, 1] = True
    assert np.isnan(o[:, 8:][bad]).all() and np.isnan(lse[:, 8:][bad]).all()
    keys, values = p.contents()
    sets = [(b, tree.seen(n, 3, i)) for b, n in enumerate(lens) for i in range(3)]
    ks, vs = [keys[b][s][:, 4:] for b, s in sets], [values[b][s][:, 4:] for b, s in sets]
    clean = torch.where(torch.isnan(q[:, 8:]), torch.zeros_like(q[:, 8:]), q[:, 8:])
    ro, rl = oracle.decode(clean, ks, vs, 1 / math.sqrt(d))
    to, tl = tolerances(clean, ks, vs, 1 / math.sqrt(d), ro, rl, e4m3)
    assert (np.abs(o[:, 8:] - ro) <= to)[~bad].all() and (np.abs(lse[:, 8:] - rl) <= tl)[~bad].all()
