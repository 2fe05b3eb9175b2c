"""One new token's attention over the paged cache against the float64 oracle:
every size, head group, page size, layout and type at which it can go wrong,
with the unused part of the cache poisoned (see cache_util)."""
import math

import numpy as np
import pytest
import torch

import oracle
from cache_util import Paged, bf16, decode_tolerances, np64

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


def poisoned(eba, cache, B, H, max_pages):
    n = eba.decode_workspace_size(cache, B, H, max_pages)
    return torch.full((n,), 255, device="cuda", dtype=torch.uint8)  # NaN as fp32


def check(eba, p, q, scale=None, q_gpu=None):
    """decode() of a Paged batch against the oracle, element by element."""
    cache = p.on_gpu(eba)
    B, H, d = q.shape
    q_gpu = q.cuda() if q_gpu is None else q_gpu
    o, lse = eba.decode(cache, q_gpu, p.gtable, p.glens, scale,
                        workspace=poisoned(eba, cache, B, H, p.table.shape[1]))
    scale = 1 / math.sqrt(d) if scale is None else scale
    keys, values = p.contents()
    ro, rl = oracle.decode(q, keys, values, scale)
    to, tl = decode_tolerances(q, keys, values, scale, ro, rl, p.k.dtype != torch.bfloat16)
    o, lse = np64(o), np64(lse)
    assert np.isfinite(o).all()
    empty = np.isneginf(rl)
    assert (np.isneginf(lse) == empty).all() and (o[empty] == 0).all()
    assert (np.abs(o - ro) <= to).all(), np.max(np.abs(o - ro) - to)
    assert (np.abs(lse[~empty] - rl[~empty]) <= tl[~empty]).all()


# lengths, H, H_kv, d, page size, e4m3, heads first
CASES = [
    ([1], 1, 1, 64, 16, False, False),
    ([1], 8, 1, 128, 1, True, False),
    ([15], 4, 4, 128, 16, False, False),
    ([16, 17], 4, 2, 64, 8, False, True),
    ([63, 64, 65], 8, 2, 128, 16, False, False),
    ([127, 128, 129, 0], 6, 3, 64, 7, True, False),
    ([0, 1, 0, 200, 0], 10, 2, 128, 48, False, False),     # empty slots; groups of 5
    ([0, 0], 4, 4, 64, 16, False, False),                  # nothing at all
    ([333], 32, 8, 128, 16, False, False),
    ([333, 1000], 9, 1, 128, 100, False, False),           # a group of 9: two column sets
    ([500, 31], 16, 1, 64, 32, True, True),
    ([777, 40], 17, 1, 128, 64, False, True),              # a group in two blocks
    ([260, 5], 40, 2, 64, 20, True, False),                # groups of 20
    ([70, 300], 66, 2, 128, 256, False, False),            # groups of 33; pages beyond the length
    ([2500, 1, 900], 4, 1, 128, 3, True, False),           # many pages
    ([5000, 4999, 12], 2, 1, 64, 33, False, False),
    ([20000], 2, 2, 128, 128, False, False),               # one sequence over all CTAs
    ([30001], 8, 1, 64, 64, True, False),
    ([9000, 50], 40, 2, 128, 16, False, False),            # a group in two blocks, over all CTAs
    ([6000, 700], 80, 4, 64, 24, True, False),
    # short rows, heads in fours
    ([5000, 4999, 0, 12], 16, 16, 64, 48, False, False),
    ([3000, 3, 0, 0, 64, 65, 31, 32], 64, 8, 64, 33, True, True),
    ([2500, 1, 65, 0, 100, 700, 32, 33], 24, 8, 128, 16, True, False),
    ([2000, 0, 100, 1], 80, 16, 64, 16, True, False),
    ([4100, 31] + [5] * 6, 16, 8, 64, 20, False, True),
    ([3000, 2999, 1, 2], 32, 16, 128, 40, True, True),
    # the same few items as single heads, cut into many parts
    ([9000, 3], 32, 4, 64, 33, True, True),
    ([7000], 24, 8, 128, 16, True, False),
]


@pytest.mark.parametrize("lens,H,hk,d,page,e4m3,heads_first", CASES, ids=lambda x: str(x).replace(" ", ""))
def test_decode_matches_oracle(eba, lens, H, hk, d, page, e4m3, heads_first):
    scales = dict(k_scale=0.03, v_scale=0.5) if e4m3 else {}
    p = Paged(lens, page, hk, d, e4m3=e4m3, heads_first=heads_first, seed=sum(lens) + H, **scales)
    check(eba, p, bf16(torch.Generator().manual_seed(1), len(lens), H, d))


@pytest.mark.parametrize("H,hk,d,e4m3,page", [(6, 2, 64, False, 16), (6, 2, 128, True, 16), (8, 8, 64, True, 16),
                                              (16, 8, 128, True, 24), (24, 8, 64, False, 32), (3, 1, 128, False, 5)])
def test_many_sequences_of_mixed_lengths(eba, H, hk, d, e4m3, page):
    r = np.random.default_rng(d)
    lens = [int(x) for x in r.integers(0, 200, size=333)]
    p = Paged(lens, page, hk, d, e4m3=e4m3, seed=3)
    check(eba, p, bf16(torch.Generator().manual_seed(2), len(lens), H, d))


@pytest.mark.parametrize("e4m3", [False, True])
def test_sharp_and_flat_softmax(eba, e4m3):
    # scores of +-60 (one key takes all), then tiny ones (all keys alike), and
    # queries of very different sizes in one group
    p = Paged([300, 77], 16, 1, 128, e4m3=e4m3, seed=5, k_scale=0.02 if e4m3 else 1.0)
    q = bf16(torch.Generator().manual_seed(3), 2, 4, 128)
    q = q * torch.tensor([1.0, 2.0 ** -20, 64.0, 0.0])[:, None].to(torch.bfloat16)
    check(eba, p, q, scale=0.5)
    check(eba, p, q, scale=1e-3)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_long_tail_of_small_weights_counts(eba, e4m3):
    # one key outweighs each of 40000 others by 2^18, which together hold a
    # seventh of the weight: the tail must not be rounded away
    d, n = 64, 40001
    k = torch.zeros(n, 1, d)
    k[0, 0, 0] = 16.0
    v = torch.ones(n, 1, d)
    v[0] = -1.0
    p = Paged([n], 64, 1, d, e4m3=e4m3, data=[(k.to(torch.bfloat16), v.to(torch.bfloat16))])
    q = torch.zeros(1, 2, d, dtype=torch.bfloat16)
    q[0, :, 0] = 1.0
    check(eba, p, q, scale=18 * math.log(2) / 16)


def test_query_views_and_wider_tables(eba):
    p = Paged([100, 300], 16, 2, 64, seed=9)
    g = torch.Generator().manual_seed(4)
    big = bf16(g, 2, 3, 8, 64).cuda()  # e.g. q, k, v of one projection
    view = big[:, 1]
    wide = torch.full((2, 40), -1, dtype=torch.int32)
    wide[:, 5:5 + p.table.shape[1]] = p.table
    cache = p.on_gpu(eba)
    o, lse = eba.decode(cache, view.contiguous(), p.gtable, p.glens)
    o2, lse2 = eba.decode(cache, view, wide.cuda()[:, 5:5 + p.table.shape[1]], p.glens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check(eba, p, view.cpu(), q_gpu=view)


def test_special_values(eba):
    # per K/V head: 0 all scores -inf (no weight: O = 0), 1 one NaN key, 2 one
    # +inf score, 3 one key of score -inf among others, 4 an infinite value
    n, d = 150, 64
    g = torch.Generator().manual_seed(6)
    k, v = bf16(g, n, 5, d), bf16(g, n, 5, d)
    q = torch.rand(1, 10, d, generator=g).add(0.5).to(torch.bfloat16)
    k[:, 0] = -math.inf
    k[70, 1] = math.nan
    k[71, 2] = math.inf
    k[72, 3] = -math.inf
    v[73, 4] = math.inf
    p = Paged([n], 16, 5, d, data=[(k, v)])
    o, lse = eba.decode(p.on_gpu(eba), q.cuda(), p.gtable, p.glens)
    o, lse = np64(o)[0], np64(lse)[0]
    assert (o[0:2] == 0).all() and np.isneginf(lse[0:2]).all()
    assert np.isnan(o[2:6]).all() and np.isnan(lse[2:6]).all()
    keys, values = p.contents()
    keep = np.arange(n) != 72  # weight 0
    ro, rl = oracle.decode(np64(q)[:, 6:8], [keys[0][keep][:, 3:4]], [values[0][keep][:, 3:4]], 0.125)
    to, tl = decode_tolerances(np64(q)[:, 6:8], [keys[0][keep][:, 3:4]], [values[0][keep][:, 3:4]],
                               0.125, ro, rl, False)
    assert (np.abs(o[6:8] - ro[0]) <= to[0]).all() and (np.abs(lse[6:8] - rl[0]) <= tl[0]).all()
    assert np.isposinf(o[8:10]).all() and np.isfinite(lse[8:10]).all()


def test_bad_pages_and_lengths_are_reported_and_absent(eba):
    p = Paged([200, 90, 64], 16, 2, 128, seed=11)
    q = bf16(torch.Generator().manual_seed(7), 3, 4, 128)
    cache = p.on_gpu(eba)
    ref = eba.decode(cache, q.cuda(), p.gtable, p.glens)
    for bad in (p.n_pages, -1, -2 ** 31, 2 ** 31 - 1):  # each by itself
        table = p.gtable.clone()
        table[2, 1] = bad
        eba.decode(cache, q.cuda(), table, p.glens)
        assert eba.poll_device_status() == 7
    table = p.gtable.clone()
    table[0, 3], table[0, 7] = p.n_pages, -1   # two pages of sequence 0
    o, lse = eba.decode(cache, q.cuda(), table, p.glens)
    assert eba.poll_device_status() == 7
    assert "page" in eba.status_string(7)
    keys, values = p.contents()
    keep = [i for i in range(200) if i // 16 not in (3, 7)]
    keys[0], values[0] = keys[0][keep], values[0][keep]
    ro, rl = oracle.decode(q, keys, values, 1 / math.sqrt(128))
    to, tl = decode_tolerances(q, keys, values, 1 / math.sqrt(128), ro, rl, False)
    assert (np.abs(np64(o) - ro) <= to).all() and (np.abs(np64(lse) - rl) <= tl).all()
    assert torch.equal(o[1:], ref[0][1:]) and torch.equal(lse[1:], ref[1][1:])
    # a negative length holds nothing; one beyond the table is cut to it
    cut = p.gtable[:, :4].contiguous()   # 64 keys
    lens = torch.tensor([1 << 30, -5, 64], device="cuda", dtype=torch.int32)
    o, lse = eba.decode(cache, q.cuda(), cut, lens)
    assert eba.poll_device_status() == 7
    keys, values = p.contents()
    keys = [keys[0][:64], keys[1][:0], keys[2]]
    values = [values[0][:64], values[1][:0], values[2]]
    ro, rl = oracle.decode(q, keys, values, 1 / math.sqrt(128))
    to, tl = decode_tolerances(q, keys, values, 1 / math.sqrt(128), ro, rl, False)
    assert np.isneginf(np64(lse)[1]).all() and (np64(o)[1] == 0).all()
    assert (np.abs(np64(o) - ro) <= to).all()
    assert (np.abs(np64(lse)[[0, 2]] - rl[[0, 2]]) <= tl[[0, 2]]).all()


def test_cache_past_four_gigabytes(eba):
    # pages whose byte offsets pass 2^32 and element offsets 2^31
    d, hk, size = 128, 8, 64
    n_pages = (9 << 28) // (d * hk * size)  # 2.25 Gi elements, 4.5 GiB, each of k and v
    k = torch.empty((n_pages, size, hk, d), device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    k[-4:] = torch.randn(k[-4:].shape, generator=g, device="cuda").to(torch.bfloat16)
    v[-4:] = torch.randn(v[-4:].shape, generator=g, device="cuda").to(torch.bfloat16)
    assert k.numel() > 2 ** 31
    q = torch.randn((1, 16, d), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([230], device="cuda", dtype=torch.int32)
    table = torch.tensor([[n_pages - 1 - i for i in range(4)]], device="cuda", dtype=torch.int32)
    o, lse = eba.decode(eba.PagedCache(k, v), q, table, lens)
    small = eba.PagedCache(k[-4:].clone(), v[-4:].clone())
    o2, lse2 = eba.decode(small, q, table - (n_pages - 4), lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("hk", [1, 8])
@pytest.mark.parametrize("d,e4m3,page", [(64, False, 16), (128, True, 16), (64, True, 20), (128, False, 32),
                                         (64, True, 16)])
def test_values_of_one_sequence_never_reach_another(eba, d, e4m3, page, hk):
    # every other sequence holds NaN values; those between end inside a tile that
    # the same block loaded NaN into before, or have a page that is none in it
    lens = [200, 3, 130, 17] * (150 if hk == 1 else 40)
    g = torch.Generator().manual_seed(21)
    nan = lambda n: (bf16(g, n, hk, d), torch.full((n, hk, d), math.nan, dtype=torch.bfloat16))
    p = Paged(lens, page, hk, d, e4m3=e4m3, seed=21,
              data=[nan(n) if n > 100 else (bf16(g, n, hk, d), bf16(g, n, hk, d)) for n in lens])
    cache = p.on_gpu(eba)
    q = bf16(g, len(lens), 2 * hk, d).cuda()
    o, _ = eba.decode(cache, q, p.gtable, p.glens)
    finite = torch.isfinite(o).all(2).all(1).cpu()
    assert finite.tolist() == [n < 100 for n in lens]
    table = p.gtable.clone()
    table[3::4, 0] = -1  # the first keys of each 17
    o2, _ = eba.decode(cache, q, table, p.glens)
    assert eba.poll_device_status() == 7
    assert torch.isfinite(o2[3::4]).all() and torch.equal(o2[1::4], o[1::4])


@pytest.mark.parametrize("lens,hk", [([4000, 100, 2500], 2), ([4000, 100] * 2, 16), ([500, 100], 8)],
                         ids=["list", "four_heads", "cluster"])
def test_same_call_same_bits(eba, lens, hk):
    p = Paged(lens, 16, hk, 64, seed=13)
    cache = p.on_gpu(eba)
    B, H = len(lens), 2 * hk
    q = bf16(torch.Generator().manual_seed(8), B, H, 64).cuda()
    a = eba.decode(cache, q, p.gtable, p.glens)
    for _ in range(5):
        b = eba.decode(cache, q, p.gtable, p.glens, workspace=poisoned(eba, cache, B, H, p.table.shape[1]))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("longest,H,hk,d", [(2500, 8, 2, 128), (300, 8, 2, 128), (2500, 32, 32, 64)],
                         ids=["list", "cluster", "four_heads"])
def test_captured_call_follows_lengths_and_tables(eba, longest, H, hk, d):
    p = Paged([longest - 70, longest, 64], 16, hk, d, seed=17)
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(9), 3, H, d).cuda()
    lens, table = p.glens.clone(), p.gtable.clone()
    eba.decode(cache, q, table, lens)  # loads the kernels before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = eba.decode(cache, q, table, lens)
        o2, lse2 = eba.decode(cache, q, table, lens)  # two calls in one graph
    for new in ([longest - 70, longest, 64], [1, 0, 63], [0, 0, 0], [longest - 71, longest // 2, 2]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        q.copy_(q.roll(1, 1))
        graph.replay()
        ref = eba.decode(cache, q, table, lens)
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
        assert torch.equal(o2, ref[0]) and torch.equal(lse2, ref[1])


def test_two_streams_at_once(eba):
    ps = [Paged([3000, 800], 16, 2, 64, seed=s) for s in (1, 2)]
    caches = [p.on_gpu(eba) for p in ps]
    qs = [bf16(torch.Generator().manual_seed(s), 2, 8, 64).cuda() for s in (3, 4)]
    refs = [eba.decode(c, q, p.gtable, p.glens) for c, q, p in zip(caches, qs, ps)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(eba.decode(caches[i], qs[i], ps[i].gtable, ps[i].glens))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, refs[i][0]) and torch.equal(lse, refs[i][1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("axes,pairing,d", [((64,), "half", 128), ((10, 11, 11), "interleaved", 64),
                                            ((8, 16), "half", 128)])
@pytest.mark.parametrize("H,hk,longest", [(18, 2, 300), (32, 16, 3000)])
def test_query_rotated_on_the_way(eba, H, hk, longest, axes, pairing, d, e4m3):
    # bit for bit the rotation kernel's query
    p = Paged([longest, 0, 45, 1], 16, hk, d, e4m3=e4m3, seed=19)
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(10), 4, H, d).cuda()
    plan = eba.Rope(axes, pairing=pairing)
    pos = torch.randint(-1000, 10 ** 6, (len(axes), 4), device="cuda", dtype=torch.int32)
    turned, _ = eba.rope_fwd(q, None, pos, plan)
    ref = eba.decode(cache, turned, p.gtable, p.glens)
    got = eba.decode(cache, q, p.gtable, p.glens, rope=plan, positions=pos)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    if len(axes) == 1:  # no positions: the last token's
        turned, _ = eba.rope_fwd(q, None, p.glens - 1, plan)
        ref = eba.decode(cache, turned, p.gtable, p.glens)
        got = eba.decode(cache, q, p.gtable, p.glens, rope=plan)
        assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


def test_two_captured_calls_share_a_workspace(eba):
    # one workspace for all layers: what a call leaves there does not matter to the
    # next, in whatever order the graphs are replayed
    ps = [Paged([3000, 17, 900], 16, 2, 64, seed=s) for s in (31, 32)]
    caches = [p.on_gpu(eba) for p in ps]
    qs = [bf16(torch.Generator().manual_seed(s), 3, 8, 64).cuda() for s in (5, 6)]
    refs = [eba.decode(c, q, p.gtable, p.glens) for c, q, p in zip(caches, qs, ps)]
    ws = poisoned(eba, caches[0], 3, 8, ps[0].table.shape[1])
    graphs, outs = [], []
    for c, q, p in zip(caches, qs, ps):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(eba.decode(c, q, p.gtable, p.glens, workspace=ws))
    for i in (0, 1, 1, 0, 0, 1):
        graphs[i].replay()
        assert torch.equal(outs[i][0], refs[i][0]) and torch.equal(outs[i][1], refs[i][1])


def test_keys_and_values_side_by_side_and_shared_pages(eba):
    # one tensor [pages, 2, slots, heads, d]; two sequences that begin with the same pages
    g = torch.Generator().manual_seed(33)
    both = bf16(g, 40, 2, 16, 2, 128).cuda()
    k, v = both[:, 0], both[:, 1]
    table = torch.randperm(40, generator=g)[:36].view(2, 18).to(torch.int32)
    table[1, :10] = table[0, :10]
    lens = torch.tensor([280, 170], dtype=torch.int32)
    q = bf16(g, 2, 4, 128)
    o, lse = eba.decode(eba.PagedCache(k, v), q.cuda(), table.cuda(), lens.cuda())
    keys = [oracle.gather(np64(k), r, n) for r, n in zip(table.tolist(), lens.tolist())]
    values = [oracle.gather(np64(v), r, n) for r, n in zip(table.tolist(), lens.tolist())]
    ro, rl = oracle.decode(q, keys, values, 1 / math.sqrt(128))
    to, tl = decode_tolerances(q, keys, values, 1 / math.sqrt(128), ro, rl, False)
    assert (np.abs(np64(o) - ro) <= to).all() and (np.abs(np64(lse) - rl) <= tl).all()


@pytest.mark.parametrize("hk,d", [(1, 128), (8, 64)])
def test_thousands_of_sequences(eba, hk, d):
    # many more sequences than counting threads and CTAs, most of them empty or short
    r = np.random.default_rng(3)
    lens = np.where(r.random(3001) < 0.5, 0, r.integers(1, 40, size=3001))
    lens[[0, 1500, 3000]] = 0, 2000, 33
    p = Paged([int(x) for x in lens], 16, hk, d, seed=35)
    check(eba, p, bf16(torch.Generator().manual_seed(36), 3001, hk, d))
