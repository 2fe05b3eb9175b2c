"""Single-token decode within a sliding window and to the first tokens, against the
float64 oracle over the keys that are seen. Keys, pages and table entries that are not
seen are poisoned: NaN, and page numbers of no page."""
import math

import numpy as np
import pytest
import torch

import oracle
from cache_util import Paged, bf16, decode_tolerances, np64, rope_exact

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


def seen(n, window, sinks):
    return [j for j in range(n) if j >= n - window or j < sinks]


def hide(p, window, sinks):
    """Poison what no token sees; returns the seen keys and values of each sequence."""
    keys, values = p.contents()
    out_k, out_v = [], []
    kk, vv = p.pages(p.k).float(), p.pages(p.v).float()  # (views of copies: put back below)
    for b, n in enumerate(p.lens):
        mine = seen(n, window, sinks)
        out_k.append(keys[b][mine])
        out_v.append(values[b][mine])
        there = {j // p.page_size for j in mine}
        for e in range(-(-n // p.page_size)):
            if e not in there:
                p.table[b, e] = (1 << 30) + e if e % 2 else -1 - e
        hidden = torch.tensor(sorted(set(range(n)) - set(mine)), dtype=torch.long)
        rows = torch.tensor(p.rows[b], dtype=torch.long)
        if len(hidden):
            at = rows[hidden // p.page_size], hidden % p.page_size
            kk[at] = float("nan")
            vv[at] = float("nan")
    if p.heads_first:
        kk, vv = kk.transpose(1, 2).contiguous(), vv.transpose(1, 2).contiguous()
    p.k, p.v = kk.to(p.k.dtype), vv.to(p.v.dtype)
    return out_k, out_v


def check(eba, p, q, window, sinks, q_exact=None, **more):
    keys, values = hide(p, window, sinks)
    cache = p.on_gpu(eba)
    B, H, d = q.shape
    need = eba.decode_workspace_size(cache, B, H, p.table.shape[1], window, sinks)
    ws = torch.full((need,), 255, device="cuda", dtype=torch.uint8)
    o, lse = eba.decode(cache, q.cuda(), p.gtable, p.glens, workspace=ws, window=window, sinks=sinks, **more)
    scale = 1 / math.sqrt(d)
    q = q if q_exact is None else q_exact
    ro, rl = oracle.decode(q, keys, values, scale)
    to, tl = decode_tolerances(q, keys, values, scale, ro, rl, p.k.dtype != torch.bfloat16)
    o, lse = np64(o), np64(lse)
    assert np.isfinite(o).all()
    empty = np.isneginf(rl)
    assert (np.isneginf(lse) == empty).all() and (o[empty] == 0).all()
    assert (np.abs(o - ro) <= to).all(), np.max(np.abs(o - ro) - to)
    assert (np.abs(lse[~empty] - rl[~empty]) <= tl[~empty]).all()


# lengths, H, H_kv, d, page size, e4m3, heads first, windows and sinks
CASES = [
    ([1, 0, 2], 2, 1, 64, 16, False, False, [(1, 0), (1, 1), (5, 3)]),
    ([333], 32, 8, 128, 16, False, False, [(1, 0), (16, 1), (17, 4), (100, 40), (332, 1), (333, 0), (400, 500), (2**31 - 1, 0)]),
    ([63, 64, 65, 200, 0, 31], 8, 2, 128, 16, False, False, [(32, 4), (33, 16), (47, 17), (64, 0), (64, 2**31 - 1)]),
    ([700, 129, 1], 6, 3, 64, 7, True, False, [(128, 5), (20, 100), (500, 0)]),       # pages of 7: one key at a time
    ([20000], 2, 2, 128, 128, False, False, [(4096, 4), (15000, 300), (1, 0)]),       # one sequence over all CTAs
    ([30001, 200], 8, 1, 64, 64, True, False, [(10000, 1), (150, 50)]),
    ([9000, 50, 4000], 40, 2, 128, 16, False, True, [(2000, 4), (8999, 1)]),          # groups of 20
    ([5000, 4999, 0, 12], 16, 16, 64, 48, False, False, [(1000, 4), (3001, 65)]),     # heads in fours
    ([3000, 3, 0, 0, 64, 65, 31, 32], 64, 8, 64, 33, True, True, [(1024, 4), (40, 8)]),
    ([2500, 1, 65, 0, 100, 700, 32, 33], 24, 8, 128, 16, True, False, [(500, 33), (64, 1)]),
    ([3000, 2999, 1, 2], 32, 16, 128, 40, True, True, [(1111, 22)]),
]


@pytest.mark.parametrize("lens,H,hk,d,page,e4m3,heads_first,windows", CASES, ids=lambda x: str(x).replace(" ", ""))
def test_matches_oracle(eba, lens, H, hk, d, page, e4m3, heads_first, windows):
    scales = dict(k_scale=0.03, v_scale=0.5) if e4m3 else {}
    q = bf16(torch.Generator().manual_seed(1), len(lens), H, d)
    for i, (window, sinks) in enumerate(windows):
        p = Paged(lens, page, hk, d, e4m3=e4m3, heads_first=heads_first, seed=sum(lens) + H + i, **scales)
        check(eba, p, q, window, sinks)


@pytest.mark.parametrize("H,hk,d,e4m3,page", [(6, 2, 64, False, 16), (8, 8, 64, True, 16), (16, 8, 128, True, 24), (3, 1, 128, False, 5)])
def test_many_sequences(eba, H, hk, d, e4m3, page):
    r = np.random.default_rng(d)
    lens = [int(x) for x in r.integers(0, 200, size=333)]
    q = bf16(torch.Generator().manual_seed(2), len(lens), H, d)
    check(eba, Paged(lens, page, hk, d, e4m3=e4m3, seed=3), q, 37, 6)


def test_rotated_on_the_way(eba):
    """The default position stays the token's place in its whole sequence."""
    plan = eba.Rope((32,))
    lens = [500, 70]
    p = Paged(lens, 16, 2, 64, seed=9)
    q = bf16(torch.Generator().manual_seed(4), 2, 4, 64)
    turned, _ = eba.rope_fwd(q.cuda(), None, torch.tensor([n - 1 for n in lens], dtype=torch.int32).cuda(), plan)
    exact = rope_exact(np64(q), np.array([n - 1 for n in lens]), plan)
    assert np.abs(np64(turned) - exact).max() < 0.05
    check(eba, p, q, 100, 4, q_exact=turned.cpu(), rope=plan)


def test_a_window_of_everything_is_plain_decode(eba):
    """The same keys in the same order: bit for bit."""
    p = Paged([900, 333, 0], 16, 2, 128, seed=6)
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(5), 3, 8, 128).cuda()
    for window, sinks in ((10**6, 0), (900, 7)):
        a, b = eba.decode(cache, q, p.gtable, p.glens), eba.decode(cache, q, p.gtable, p.glens, window=window, sinks=sinks)
        assert all((np64(x) - np64(y) == 0)[np.isfinite(np64(x))].all() for x, y in zip(a, b))


def test_absent_pages_within_the_window(eba):
    """A page of no number among the seen ones: its keys are left out, and it is reported."""
    p = Paged([300], 16, 1, 64, seed=7)
    keys, values = p.contents()
    p.table[0, 17] = -1  # keys 272 to 287
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(6), 1, 2, 64)
    o, lse = eba.decode(cache, q.cuda(), p.gtable, p.glens, window=60, sinks=2)
    mine = [j for j in seen(300, 60, 2) if not 272 <= j < 288]
    ro, rl = oracle.decode(q, [keys[0][mine]], [values[0][mine]], 0.125)
    to, tl = decode_tolerances(q, [keys[0][mine]], [values[0][mine]], 0.125, ro, rl, False)
    assert (np.abs(np64(o) - ro) <= to).all() and (np.abs(np64(lse) - rl) <= tl).all()
    assert eba.poll_device_status() == 7


def test_captured_call_follows_lengths(eba):
    p = Paged([1000, 700], 16, 2, 128, seed=8)
    keys, values = p.contents()
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(7), 2, 4, 128)
    gq, lens = q.cuda(), p.glens.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o, lse = eba.decode(cache, gq, p.gtable, lens, window=200, sinks=3)
    for n in ([1000, 700], [12, 0], [201, 500]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        mine = [seen(x, 200, 3) for x in n]
        ks, vs = ([c[b][m] for b, m in enumerate(mine)] for c in (keys, values))
        ro, rl = oracle.decode(q, ks, vs, 1 / math.sqrt(128))
        to, tl = decode_tolerances(q, ks, vs, 1 / math.sqrt(128), ro, rl, False)
        assert (np.abs(np64(o) - ro) <= to).all()
        ok = np.isfinite(rl)
        assert (np.isneginf(np64(lse)) == ~ok).all() and (np.abs(np64(lse) - rl)[ok] <= tl[ok]).all()
