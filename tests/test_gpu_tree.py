"""Drafted tokens' attention over the paged cache against the float64 oracle, element by
element: trees and chains, windows, every type, head group, layout and length at which it
can go wrong. What no token sees is poisoned (NaN, page numbers of no page), as is the
workspace."""
import math

import numpy as np
import pytest
import torch

import oracle
from cache_util import Paged, bf16, np64
from oracle import tree

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


def tolerances(q, keys, values, scale, o, lse, e4m3):
    """Bounds of |O - exact| [T, H, d] and |lse - exact| [T, H] by arithmetic, token t over
    keys[t], values[t].

    Scores: d products added in fp32, off by at most d 2^-24 sum |q k| scale, and as much
    again for the scaling, the base-2 reference and the exponential's own 2^-20. The weights
    enter the product with V as bf16 (half a step, 2^-8) or, with an e4m3 cache, fp16
    (2^-11), which moves O by at most that of P |v|, and once more through the sum they are
    divided by; so do the scores' error and the fp32 sums over n keys (n / 16 + 64
    roundings). The bf16 output is off by half a step of its own."""
    q = np64(q)
    to, tl = np.zeros_like(o), np.zeros_like(lse)
    for t in range(len(keys)):
        n, hk = keys[t].shape[:2]
        for h in range(q.shape[1] if n else 0):
            g = h // (q.shape[1] // hk)
            big = (np.abs(keys[t][:, g]) @ np.abs(q[t, h])).max() * scale
            score = 2 * q.shape[2] * 2.0 ** -24 * big + 2.0 ** -20
            weight = score + (2.0 ** -11 if e4m3 else 2.0 ** -8) + (n / 16 + 64) * 2.0 ** -24
            p, _ = oracle.softmax_weights(q[t, h][None], keys[t][:, g], scale)
            to[t, h] = 2.0 ** -8 * np.abs(o[t, h]) + 2 * weight * (p @ np.abs(values[t][:, g]))[0]
            tl[t, h] = score + (n / 16 + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[t, h])
    return to, tl


def random_masks(r, news):
    """Trees of any shape, a token's own bit and its ancestors'."""
    out = []
    for n in news:
        mine = []
        for i in range(n):
            p = int(r.integers(-1, i)) if i else -1
            mine.append((mine[p] if p >= 0 else 0) | 1 << i)
        out.append(mine)
    return out


def words_of(masks, words):
    rows = [[m >> 64 * w & (1 << 64) - 1 for w in range(words)] for mine in masks for m in mine]
    return torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in rows], dtype=torch.int64)


def hide_between(p, sets, news):
    """Poison what no token of a sequence sees of its context: keys, and table entries of whole
    pages."""
    kk, vv = p.k.float(), p.v.float()
    for b, n in enumerate(p.lens):
        mine = set().union(*sets[b], range(n - news[b], n)) if n else set()
        there = {j // p.page_size for j in mine}
        rows = torch.tensor(p.rows[b], dtype=torch.long)
        hidden = torch.tensor(sorted(set(range(n)) - mine), dtype=torch.long)
        if len(hidden):
            at = rows[hidden // p.page_size], hidden % p.page_size
            p.pages(kk)[at] = float("nan")
            p.pages(vv)[at] = float("nan")
        for e in range(-(-n // p.page_size)):
            if e not in there:
                p.table[b, e] = (1 << 30) + e if e % 2 else -1 - e
    p.k, p.v = kk.to(p.k.dtype), vv.to(p.v.dtype)


def check(eba, p, news, H, masks=None, words=1, window=None, sinks=0, scale=None, seed=1, poison=True, q=None, before=0):
    """decode_tree of a Paged batch, sequence b's last news[b] keys drafted; masks[b][i] an
    int. `before`: rows of q before the first sequence's."""
    hk, d = p.pages(p.k).shape[2:]
    g = torch.Generator().manual_seed(seed)
    T = sum(news)
    cu = [before]
    for n in news:
        cu.append(cu[-1] + n)
    keys, values = p.contents()
    empty = [p.lens[b] == 0 for b in range(len(news))]
    sets = [[[] if empty[b] else tree.seen(p.lens[b], n, i, None if masks is None else masks[b][i], window, sinks) for i in range(n)]
            for b, n in enumerate(news)]
    if poison:
        hide_between(p, sets, news)
    cache = p.on_gpu(eba)
    total = T + before + (5 if before else 0)
    if q is None:
        q = bf16(g, max(total, 1), H, d)
    mask = None
    if masks is not None:
        mask = torch.full((total, words), -1, dtype=torch.int64)
        mask[before:before + T] = words_of(masks, words)
        mask = (mask if words > 1 else mask[:, 0]).cuda()
    ws = torch.full((eba.decode_tree_workspace_size(cache, total, len(news), H),), 255, device="cuda", dtype=torch.uint8)
    o, lse = eba.decode_tree(cache, q.cuda(), p.gtable, p.glens, torch.tensor(cu, dtype=torch.int32).cuda(), mask=mask,
                             window=window, sinks=sinks, scale=scale, workspace=ws)
    scale = 1 / math.sqrt(d) if scale is None else scale
    ks = [keys[b][s] for b in range(len(news)) for s in sets[b]]
    vs = [values[b][s] for b in range(len(news)) for s in sets[b]]
    mine = q[before:before + T]
    ro, rl = oracle.decode(mine, ks, vs, scale)
    to, tl = tolerances(mine, ks, vs, scale, ro, rl, p.k.dtype != torch.bfloat16)
    o, lse = np64(o)[before:before + T], np64(lse)[before:before + T]
    assert np.isfinite(o).all()
    blind = np.isneginf(rl)
    assert (np.isneginf(lse) == blind).all() and (o[blind] == 0).all()
    assert (np.abs(o - ro) <= to).all(), np.max(np.abs(o - ro) - to)
    assert (np.abs(lse[~blind] - rl[~blind]) <= tl[~blind]).all()
    # as a whole: two independent roundings to bf16 at most, each of rms 2^-8 / sqrt(3)
    if ro.size > 4000:
        assert np.linalg.norm(o - ro) <= 2.0 ** -8 * np.linalg.norm(ro)


# lengths, drafted tokens, H, H_kv, d, page size, e4m3, heads first
CASES = [
    ([1], [1], 1, 1, 64, 16, False, False),
    ([1], [1], 8, 1, 128, 1, True, False),
    ([3, 2], [3, 1], 4, 2, 128, 16, False, False),             # no context at all
    ([16, 17, 0], [4, 5, 0], 4, 2, 64, 8, False, True),
    ([127, 128, 129], [1, 2, 3], 8, 2, 128, 16, False, False),
    ([256, 257, 130], [16, 17, 64], 6, 3, 64, 7, True, False),
    ([300, 140, 20], [60, 64, 20], 10, 2, 128, 48, False, False),  # groups of 5: rows of a token in two items
    ([333], [16], 32, 8, 128, 16, False, False),
    ([1000, 333], [40, 3], 9, 1, 128, 100, False, False),
    ([500, 31], [33, 31], 16, 1, 64, 32, True, True),
    ([777, 40], [8, 1], 17, 1, 128, 64, False, True),
    ([700], [9], 66, 2, 64, 20, True, False),                  # groups of 33
    ([400], [2], 300, 1, 128, 16, False, False),               # a group of 300: a token in three items
    ([5000, 4999, 12], [12, 1, 12], 2, 1, 64, 33, False, False),
    ([20000], [24], 8, 2, 128, 128, False, False),             # one sequence over all CTAs
    ([30001, 5], [12, 5], 16, 1, 128, 64, True, False),
    ([9000, 50, 4000], [7, 50, 64], 40, 2, 64, 16, True, False),
    ([700] * 30 + [90] * 20, [13] * 50, 16, 4, 128, 32, False, False),   # many items cut or not
    ([650] * 20 + [64] * 40, [4, 9] * 30, 8, 8, 64, 24, True, True),
]


@pytest.mark.parametrize("lens,news,H,hk,d,page,e4m3,heads_first", CASES, ids=lambda x: str(x).replace(" ", "")[:24])
def test_trees_and_chains(eba, lens, news, H, hk, d, page, e4m3, heads_first):
    scales = dict(k_scale=0.03, v_scale=0.5) if e4m3 else {}
    r = np.random.default_rng(len(lens) + H)
    for masks in (random_masks(r, news), None):
        p = Paged(lens, page, hk, d, e4m3=e4m3, heads_first=heads_first, seed=sum(lens) % 1000 + H, **scales)
        check(eba, p, news, H, masks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (64, 4), (100, 130), (333, 1), (500, 500), (2**31 - 1, 0)])
@pytest.mark.parametrize("d,e4m3", [(128, False), (64, True)])
def test_windows(eba, window, sinks, d, e4m3):
    lens, news = [700, 333, 140, 20, 0, 12], [20, 3, 33, 20, 0, 5]
    r = np.random.default_rng(window % 1000)
    for masks in (random_masks(r, news), None):
        p = Paged(lens, 16, 2, d, e4m3=e4m3, seed=window % 97, k_scale=0.05 if e4m3 else 1.0)
        check(eba, p, news, 8, masks, window=window, sinks=sinks)


def test_any_mask(eba):
    """Bits that make no tree: later tokens, none at all, bits of no token; two and four words."""
    r = np.random.default_rng(5)
    for words, most in ((1, 64), (2, 128), (4, 200)):
        news = [most, 9, most // 2 + 1]
        lens = [300, 9, 500]
        masks = [[int.from_bytes(r.bytes(8 * words), "little") for _ in range(n)] for n in news]
        masks[0][3] = masks[1][0] = masks[1][5] = 0
        masks[2][1] = 1 << (64 * words - 1)
        for window in (None, 40):
            check(eba, Paged(lens, 16, 2, 64, seed=words), news, 4, masks, words, window, 2 if window else 0)


def test_prompt_of_many_tokens(eba):
    """A chain of more than a thousand tokens over a context, windowed and not."""
    for window in (None, 200):
        check(eba, Paged([1500, 700], 16, 1, 64, seed=3), [1100, 700], 2, None, window=window, sinks=5 if window else 0)


@pytest.mark.parametrize("seed,window", [(0, None), (1, None), (2, 300), (3, None)])
def test_long_runs_over_many_ends(eba, seed, window):
    """So many tiles that an item's end counts in the split of the list: runs that begin at
    ends, of items of one tile and of many, and items cut in several."""
    r = np.random.default_rng(seed + 40)
    lens = [int(n) for n in r.choice([1, 2, 127, 128, 129, 700, 3000, 6100], 48)] + [9000]
    if window:
        lens = [min(3 * n, 700) for n in lens] * 4
    news = [int(r.integers(1, min(n, 3) + 1)) for n in lens]
    assert window or sum(-(-n // 128) for n in lens) * 8 >= 12 * 152
    check(eba, Paged(lens, 16, 8, 64, seed=seed), news, 8, random_masks(r, news), window=window, sinks=3 if window else 0)


def test_rows_of_no_sequence_stay(eba):
    r = np.random.default_rng(6)
    news = [3, 0, 5]
    check(eba, Paged([40, 30, 200], 16, 2, 128, seed=2), news, 4, random_masks(r, news), before=4)
    # written where they belong only: the call writes into fresh tensors, so look at the ABI
    p = Paged([40, 200], 16, 2, 64, seed=2)
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(3), 12, 4, 64).cuda()
    cu = torch.tensor([2, 5, 9], dtype=torch.int32).cuda()
    o, lse = torch.full_like(q, 7.0), torch.full((12, 4), 7.0, device="cuda")
    n = eba.decode_tree_workspace_size(cache, 12, 2, 4)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    eba._launch(q.device, eba.lib().attn_decode_tree, cache._at(), q.data_ptr(), eba._Strides2(256, 64), p.gtable.data_ptr(),
                p.gtable.stride(0), p.gtable.shape[1], p.glens.data_ptr(), 2, cu.data_ptr(), 12, 4, None, 0, 0, 0, 0, 0.125,
                o.data_ptr(), lse.data_ptr(), ws.data_ptr(), n)
    out = torch.tensor([0, 1, 9, 10, 11])
    assert (o[out] == 7).all() and (lse[out] == 7).all() and (lse[2:9] != 7).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_sharp_and_flat_softmax(eba, e4m3):
    p = Paged([300, 77], 16, 1, 128, e4m3=e4m3, seed=5, k_scale=0.02 if e4m3 else 1.0)
    q = bf16(torch.Generator().manual_seed(3), 12, 4, 128)
    q = q * torch.tensor([1.0, 2.0 ** -20, 64.0, 0.0])[:, None].to(torch.bfloat16)
    check(eba, p, [9, 3], 4, scale=0.5, q=q)
    check(eba, p, [9, 3], 4, scale=1e-3, q=q)


def test_one_token_each_is_decode(eba):
    """Within the rounding of both."""
    p = Paged([900, 333, 0, 64], 16, 2, 128, seed=6)
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(5), 4, 8, 128).cuda()
    for window, sinks in ((None, 0), (None, 6), (100, 4)):
        a = eba.decode(cache, q, p.gtable, p.glens, window=window, sinks=sinks)
        b = eba.decode_tree(cache, q, p.gtable, p.glens, window=window, sinks=sinks)
        assert (a[0].float() - b[0].float()).abs().max() <= 2.0 ** -7
        assert (torch.isneginf(a[1]) == torch.isneginf(b[1])).all()
        ok = ~torch.isneginf(a[1])
        assert (a[1] - b[1])[ok].abs().max() <= 1e-5


def test_the_same_call_twice_is_the_same(eba):
    r = np.random.default_rng(8)
    news = [int(x) for x in r.integers(1, 30, 40)]
    lens = [int(n + x) for n, x in zip(news, r.integers(0, 3000, 40))]
    p = Paged(lens, 32, 4, 128, seed=4)
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(9), sum(news), 16, 128).cuda()
    cu = torch.tensor(np.cumsum([0] + news), dtype=torch.int32).cuda()
    mask = words_of(random_masks(r, news), 1)[:, 0].cuda()
    a = eba.decode_tree(cache, q, p.gtable, p.glens, cu, mask=mask)
    for _ in range(5):
        b = eba.decode_tree(cache, q, p.gtable, p.glens, cu, mask=mask)
        assert all((x == y).all() for x, y in zip(a, b))


def test_views(eba):
    """A query that is a view, a mask that is a column of a wider one, a table of wider rows."""
    r = np.random.default_rng(10)
    news = [5, 9]
    p = Paged([200, 77], 16, 2, 64, seed=4)
    masks = random_masks(r, news)
    cache = p.on_gpu(eba)
    wide = bf16(torch.Generator().manual_seed(9), 14, 12, 64).cuda()
    m3 = torch.stack([words_of(masks, 1)[:, 0]] * 3, 1).cuda()
    cu = torch.tensor([0, 5, 14], dtype=torch.int32).cuda()
    a = eba.decode_tree(cache, wide[:, 4:8], p.gtable, p.glens, cu, mask=m3[:, 1])
    b = eba.decode_tree(cache, wide[:, 4:8].contiguous(), p.gtable, p.glens, cu, mask=m3[:, 1].contiguous())
    assert all((x == y).all() for x, y in zip(a, b))


def test_faults_are_reported(eba):
    p = Paged([300, 50, 40], 16, 1, 64, seed=7)
    keys, values = p.contents()
    q = bf16(torch.Generator().manual_seed(6), 9, 2, 64)
    cu = torch.tensor([0, 3, 6, 9], dtype=torch.int32).cuda()
    # an absent page: its keys are left out
    p.table[0, 7] = -1
    cache = p.on_gpu(eba)
    o, lse = eba.decode_tree(cache, q.cuda(), p.gtable, p.glens, cu)
    sets = [[j for j in tree.seen(300, 3, i) if not 112 <= j < 128] for i in range(3)]
    ro, rl = oracle.decode(q[:3], [keys[0][s] for s in sets], [values[0][s] for s in sets], 0.125)
    to, tl = tolerances(q[:3], [keys[0][s] for s in sets], [values[0][s] for s in sets], 0.125, ro, rl, False)
    assert (np.abs(np64(o)[:3] - ro) <= to).all() and (np.abs(np64(lse)[:3] - rl) <= tl).all()
    assert eba.poll_device_status() == 7
    # lengths and offsets out of range
    for lens in ([300, 2, 40], [-5, 50, 40], [1 << 30, 50, 40]):
        o, lse = eba.decode_tree(cache, q.cuda(), p.gtable, torch.tensor(lens, dtype=torch.int32).cuda(), cu)
        assert eba.poll_device_status() == 7
        if lens[1] == 2:
            assert (o[3:6] == 0).all() and torch.isneginf(lse[3:6]).all()
        if lens[0] < 0:
            assert (o[:3] == 0).all() and torch.isneginf(lse[:3]).all()
    for bad in ([0, 6, 3, 9], [-4, 3, 6, 9], [0, 3, 6, 1 << 30], [9, 9, 9, 0]):
        eba.decode_tree(cache, q.cuda(), p.gtable, p.glens, torch.tensor(bad, dtype=torch.int32).cuda())
        assert eba.poll_device_status() == 7
    # an empty slot is none
    p.table[0, 7] = p.rows[0][7]
    cache = p.on_gpu(eba)
    o, lse = eba.decode_tree(cache, q.cuda(), p.gtable, torch.tensor([300, 0, 40], dtype=torch.int32).cuda(), cu)
    assert (o[3:6] == 0).all() and torch.isneginf(lse[3:6]).all()


def test_captured_call_follows_its_batch(eba):
    r = np.random.default_rng(11)
    p = Paged([900, 700], 16, 2, 128, seed=8)
    keys, values = p.contents()
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(7), 20, 4, 128)
    gq, lens, cu = q.cuda(), p.glens.clone(), torch.tensor([0, 10, 20], dtype=torch.int32).cuda()
    mask = torch.zeros(20, dtype=torch.int64).cuda()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o, lse = eba.decode_tree(cache, gq, p.gtable, lens, cu, mask=mask)
    for n, news in (([900, 700], [10, 10]), ([40, 699], [1, 15]), ([8, 130], [8, 4])):
        masks = random_masks(r, news)
        T = sum(news)
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        cu.copy_(torch.tensor([0, news[0], T], dtype=torch.int32))
        mask[:T] = words_of(masks, 1)[:, 0].cuda()
        graph.replay()
        sets = [(b, tree.seen(n[b], news[b], i, masks[b][i])) for b in range(2) for i in range(news[b])]
        ks, vs = [keys[b][s] for b, s in sets], [values[b][s] for b, s in sets]
        ro, rl = oracle.decode(q[:T], ks, vs, 1 / math.sqrt(128))
        to, tl = tolerances(q[:T], ks, vs, 1 / math.sqrt(128), ro, rl, False)
        assert (np.abs(np64(o)[:T] - ro) <= to).all() and (np.abs(np64(lse)[:T] - rl) <= tl).all()


def test_a_step_of_speculative_decoding(eba):
    """Reserve, append, verify and gather: afterwards the cache holds the accepted path, and the
    next token sees what it would without the drafts."""
    r = np.random.default_rng(12)
    size, hk, H, d, B = 16, 2, 8, 64, 3
    ctx = [37, 64, 200]
    p = Paged(ctx, size, hk, d, seed=9, spare_pages=12)
    keys, values = p.contents()
    cache = p.on_gpu(eba)
    refs = torch.zeros(p.n_pages, dtype=torch.int32)
    for row in p.rows:
        refs[row] = 1
    pool = eba.PagePool(refs.cuda(), size)
    table = torch.full((B, 18), -1, dtype=torch.int32)
    for b, row in enumerate(p.rows):
        table[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
    table, lens = table.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda()
    news = [20, 7, 30]
    masks = random_masks(r, news)
    T = sum(news)
    g = torch.Generator().manual_seed(10)
    q, k, v = bf16(g, T, H, d), bf16(g, T, hk, d), bf16(g, T, hk, d)
    cu = torch.tensor(np.cumsum([0] + news), dtype=torch.int32).cuda()
    more = lens + torch.tensor(news, dtype=torch.int32).cuda()
    eba.pages_reserve(pool, table, lens, more)
    eba.cache_append(cache, k.cuda(), v.cuda(), table, more, cu)
    o, lse = eba.decode_tree(cache, q.cuda(), table, more, cu, mask=words_of(masks, 1)[:, 0].cuda())
    # the whole path of some token is accepted
    paths = [[x for x in range(n) if m[pick] >> x & 1] for n, m, pick in zip(news, masks, (19, 3, 29))]
    places = torch.tensor([c + x for c, path in zip(ctx, paths) for x in path], dtype=torch.int32).cuda()
    kept = torch.tensor(np.cumsum([0] + [len(x) for x in paths]), dtype=torch.int32).cuda()
    eba.cache_gather(cache, table, places, kept, to_start=lens)
    now = lens + torch.tensor([len(x) for x in paths], dtype=torch.int32).cuda()
    end = torch.full((B,), 18 * size, dtype=torch.int32).cuda()
    eba.pages_release(pool, table, now, end)
    at = np.cumsum([0] + news)
    ks = [np.concatenate([keys[b], np64(k)[[at[b] + x for x in paths[b]]]]) for b in range(B)]
    vs = [np.concatenate([values[b], np64(v)[[at[b] + x for x in paths[b]]]]) for b in range(B)]
    q1 = bf16(g, B, H, d)
    o1, l1 = eba.decode(cache, q1.cuda(), table, now)
    ro, rl = oracle.decode(q1, ks, vs, 0.125)
    to, tl = tolerances(q1, ks, vs, 0.125, ro, rl, False)
    assert (np.abs(np64(o1) - ro) <= to).all() and (np.abs(np64(l1) - rl) <= tl).all()
    # what the path's last token saw is that sequence
    last = [at[b] + paths[b][-1] for b in range(B)]
    ro, rl = oracle.decode(q[last], ks, vs, 0.125)
    to, tl = tolerances(q[last], ks, vs, 0.125, ro, rl, False)
    assert (np.abs(np64(o)[last] - ro) <= to).all() and (np.abs(np64(lse)[last] - rl) <= tl).all()
    held = [-(-(c + len(x)) // size) for c, x in zip(ctx, paths)]
    assert (table.cpu() >= 0).sum(1).tolist() == held and int(pool.refs.sum()) == sum(held)


def test_two_calls_at_once(eba):
    """Calls on streams of their own, at the same time and behind one another."""
    r = np.random.default_rng(12)
    calls = []
    for seed, (d, e4m3) in enumerate(((64, False), (128, True), (128, False))):
        news = [int(n) for n in r.integers(1, 20, 9)]
        p = Paged([int(n) + 20 for n in r.integers(1, 4000, 9)], 32, 4, d, e4m3=e4m3, seed=seed)
        q = bf16(torch.Generator().manual_seed(seed), sum(news), 8, d).cuda()
        cu = torch.tensor([0, *np.cumsum(news)], dtype=torch.int32).cuda()
        mask = words_of(random_masks(r, news), 1)[:, 0].cuda()
        calls.append((p.on_gpu(eba), q, p.gtable, p.glens, cu, mask))
    alone = [eba.decode_tree(*c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]
    for _ in range(20):
        for c, s, out in zip(calls, streams, got):
            with torch.cuda.stream(s):
                out.append(eba.decode_tree(*c))
    torch.cuda.synchronize()
    for (o, lse), outs in zip(alone, got):
        assert all(torch.equal(o, x) and torch.equal(lse, y) for x, y in outs)
