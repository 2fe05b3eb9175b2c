"""The rotation, the paged cache and the decode where they are most easily wrong:
absent pages, special values and far-out sizes on every path of the decode, exact
roundings of an e4m3 cache, and several threads at once."""
import concurrent.futures
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


def compare(o, lse, q, keys, values, scale, e4m3):
    """o, lse against the oracle over the given keys and values, element by element."""
    ro, rl = oracle.decode(q, keys, values, scale)
    to, tl = decode_tolerances(q, keys, values, scale, ro, rl, e4m3)
    o, lse = np64(o), np64(lse)
    empty = np.isneginf(rl)
    assert (np.isneginf(lse) == empty).all() and (o[empty] == 0).all()
    assert (np.abs(o - ro) <= to).all(), np.max(np.abs(o - ro) - to)
    assert (np.abs(lse[~empty] - rl[~empty]) <= tl[~empty]).all()


# sequences, keys, H, H_kv, d, page, e4m3: what the calls are cut into
PATHS = {
    "cluster": (1, 700, 16, 4, 128, 16, False),
    "many_parts": (3, 20000, 4, 2, 128, 16, False),
    "few_parts": (5, 4000, 16, 8, 128, 32, False),
    "few_parts_odd_pages": (5, 4000, 16, 8, 128, 20, False),
    "two_column_sets_e4m3": (3, 20000, 32, 2, 128, 64, True),
    "two_blocks": (3, 6000, 40, 2, 64, 16, False),
    "four_heads": (5, 3000, 16, 16, 64, 48, False),
    "four_heads_odd_pages_e4m3": (5, 3000, 32, 16, 64, 40, True),
}


@pytest.mark.parametrize("path", PATHS)
def test_tiles_without_a_key(eba, path):
    # whole tiles whose pages are none, between tiles that hold keys: their masks are
    # empty, and their zeros and the keys around them must not count or be lost. In the
    # first sequence the tiles of 128 keys take turns at random, the second holds none
    # at all, the third begins with a long run of none (parts without weight), the others
    # are whole.
    B, n, H, hk, d, page, e4m3 = PATHS[path]
    scales = dict(k_scale=0.03, v_scale=0.5) if e4m3 else {}
    p = Paged([n] * min(B, 3) + [n - 77] * (B - 3), page, hk, d, e4m3=e4m3, seed=n + H, **scales)
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(n), B, H, d)
    r = np.random.default_rng(n)
    first = np.arange(len(p.rows[0])) * page // 128  # of each page: its tile of 128 keys
    absent = [r.random(first.max() + 1)[first] < 0.5]
    if B > 1:
        absent += [np.ones(len(first), bool), np.arange(len(first)) < 0.7 * len(first)]
    table = p.table.clone()
    keys, values = p.contents()
    for b, gone in enumerate(absent):
        table[b, :len(gone)][torch.tensor(gone)] = torch.tensor([p.n_pages, -1])[b % 2].int()
        held = ~gone[np.arange(n) // page]
        keys[b], values[b] = keys[b][held], values[b][held]
    o, lse = eba.decode(cache, q.cuda(), table.cuda(), p.glens)
    assert eba.poll_device_status() == 7
    for _ in range(3):
        o2, lse2 = eba.decode(cache, q.cuda(), table.cuda(), p.glens)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert eba.poll_device_status() == 7
    compare(o, lse, q, keys, values, 1 / math.sqrt(d), e4m3)


E4M3_PATHS = {
    "cluster": (1, 700, 16, 4, 128, 16),
    "two_column_sets": (2, 6000, 32, 2, 64, 64),
    "few_parts": (5, 4000, 16, 8, 128, 20),
    "four_heads": (5, 3000, 32, 16, 64, 40),
}


@pytest.mark.parametrize("power", [-130, -100, -50, 0, 99, 116, 127])
@pytest.mark.parametrize("path", E4M3_PATHS)
def test_queries_of_any_size_on_an_e4m3_cache(eba, path, power):
    # from bf16's smallest to its largest numbers, with keys so scaled that the scores
    # are ordinary numbers; the odd heads are 2^10 smaller than the even ones
    B, n, H, hk, d, page = E4M3_PATHS[path]
    p = Paged([n] * B, page, hk, d, e4m3=True, seed=n)
    p.k_scale = 2.0 ** min(max(-power, -126), 126)
    g = torch.Generator().manual_seed(power + 200)
    q = (torch.rand(B, H, d, generator=g) * 1.5 + 0.49) * torch.randn(B, H, d, generator=g).sign()
    q = (q.double() * 2.0 ** power).float()
    if power > -100:
        q[:, 1::2] *= 2.0 ** -10
    q = q.to(torch.bfloat16)
    assert torch.isfinite(q).all() and (q != 0).all()
    o, lse = eba.decode(p.on_gpu(eba), q.cuda(), p.gtable, p.glens)
    compare(o, lse, q, *p.contents(), 1 / math.sqrt(d), True)


@pytest.mark.parametrize("e4m3,k_scale,scale,size", [
    (True, 1.0, 2.0 ** 40, 2.0 ** 126), (True, 2.0 ** 100, 2.0 ** 100, 1.0), (False, 1.0, 2.0 ** 127, 0.0)], ids=str)
def test_scores_of_zero_are_zero_at_any_scale(eba, e4m3, k_scale, scale, size):
    # the factors of the scores, together or the scale alone, are beyond fp32's largest number
    d, n = 64, 100
    zero, v = torch.zeros(n, 1, d, dtype=torch.bfloat16), bf16(torch.Generator().manual_seed(1), n, 1, d)
    p = Paged([n], 16, 1, d, e4m3=e4m3, k_scale=k_scale, data=[(zero, v)])
    q = torch.full((1, 2, d), size, dtype=torch.bfloat16)
    o, lse = eba.decode(p.on_gpu(eba), q.cuda(), p.gtable, p.glens, scale)
    compare(o, lse, q, *p.contents(), scale, e4m3)


@pytest.mark.parametrize("scale", [0.03, 7.0, 0.3, 0.02, 1.0, 1.9999999, 3e-10, 2.0 ** -120, 2.0 ** 127])
def test_append_to_e4m3_multiplies_by_the_reciprocal(eba, scale):
    # every bf16 number that is one, bit for bit: times the fp32 reciprocal of the scale, rounded to e4m3
    x = torch.arange(2 ** 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.where(torch.isnan(x), torch.zeros_like(x), x).view(-1, 1, 64)
    T = x.shape[0]
    p = Paged([T], 32, 1, 64, e4m3=True, k_scale=scale, v_scale=scale)
    cache = p.on_gpu(eba)
    cu = torch.tensor([0, T], device="cuda", dtype=torch.int32)
    eba.cache_append(cache, x.cuda(), x.flip(0).cuda(), p.gtable, p.glens, cu)
    with np.errstate(over="ignore"):
        exact = x.float().numpy() * (np.float32(1) / np.float32(scale))
    want = torch.tensor(np.clip(exact, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    for pages, w in ((p.gk, want), (p.gv, want.flip(0))):
        got = pages.cpu().view(torch.uint8)[torch.tensor(p.rows[0])].view(-1, 1, 64)[:T]
        assert torch.equal(got, w), int((got != w).sum())


SPECIAL_PATHS = {
    "cluster": (1, 300, 8, 64, 16),
    "few_parts": (4, 3000, 8, 128, 16),
    "many_parts": (1, 9000, 8, 128, 20),
    "four_heads": (8, 2000, 16, 64, 16),
    "four_heads_many_parts": (4, 9000, 16, 64, 48),
}


@pytest.mark.parametrize("group", [2, 9])
@pytest.mark.parametrize("path", SPECIAL_PATHS)
def test_special_values_on_every_path(eba, path, group):
    # per K/V head: 0 all scores -inf (no weight at all: O = 0), 1 one NaN key, 2 one
    # +inf score, 3 keys of score -inf among others, 4 an infinite value, 5 -inf scores
    # for the first two thirds (parts without weight), 6 one NaN value; the others plain
    B, n, hk, d, page = SPECIAL_PATHS[path]
    H, at = group * hk, n // 2
    g = torch.Generator().manual_seed(n + group)
    data = []
    for _ in range(B):
        k, v = bf16(g, n, hk, d), bf16(g, n, hk, d)
        k[:, 0] = -math.inf
        k[at, 1] = math.nan
        k[at + 1, 2] = math.inf
        k[at + 2::7, 3] = -math.inf
        v[at + 3, 4] = math.inf
        k[:2 * n // 3, 5] = -math.inf
        v[at + 4, 6, 3] = math.nan
        data.append((k, v))
    q = torch.rand(B, H, d, generator=g).add(0.5).to(torch.bfloat16)  # positive
    p = Paged([n] * B, page, hk, d, data=data)
    o, lse = eba.decode(p.on_gpu(eba), q.cuda(), p.gtable, p.glens)
    o4, l4 = np64(o).reshape(B, hk, group, d), np64(lse).reshape(B, hk, group)
    assert (o4[:, 0] == 0).all() and np.isneginf(l4[:, 0]).all()
    assert np.isnan(o4[:, 1:3]).all() and np.isnan(l4[:, 1:3]).all()
    assert np.isposinf(o4[:, 4]).all() and np.isfinite(l4[:, 4]).all()
    assert np.isnan(o4[:, 6, :, 3]).all() and np.isfinite(l4[:, 6]).all()
    keys, values = p.contents()
    dropped = np.arange(n) >= at + 2
    dropped &= (np.arange(n) - at - 2) % 7 == 0
    for head, keep in ((3, ~dropped), (5, np.arange(n) >= 2 * n // 3), (7, np.ones(n, bool)), (4, None), (6, None)):
        mine = slice(head * group, (head + 1) * group)
        ks, vs = ([x[:, head:head + 1] if keep is None else x[keep][:, head:head + 1] for x in y]
                  for y in (keys, values))
        if keep is None:  # the scores do not know of the value; the other columns neither
            vs = [np.where(np.isfinite(x), x, 0) for x in vs]
            good = np.isfinite(o4[0, head, 0])
            ro, rl = oracle.decode(np64(q)[:, mine], ks, vs, 1 / math.sqrt(d))
            to, tl = decode_tolerances(np64(q)[:, mine], ks, vs, 1 / math.sqrt(d), ro, rl, False)
            assert (np.abs(l4[:, head] - rl) <= tl).all()
            assert (np.abs(o4[:, head] - ro) <= to)[..., good].all()
        else:
            compare(o[:, mine], lse[:, mine], q[:, mine], ks, vs, 1 / math.sqrt(d), False)


@pytest.mark.parametrize("path", E4M3_PATHS)
def test_special_values_on_an_e4m3_cache(eba, path):
    # e4m3 has NaN and no infinities: infinite scores come from the query. Keys' first
    # elements are positive. K/V head 0: plain; 1: one NaN key; 2 (where there are so
    # many): one NaN value. Query heads of each: 0 an element of -inf (all scores -inf:
    # O = 0), 1 one of +inf (NaN), 2 (where there is one) plain.
    B, n, H, hk, d, page = E4M3_PATHS[path]
    group, at = H // hk, n // 2
    g = torch.Generator().manual_seed(n)
    data = []
    for _ in range(B):
        k, v = bf16(g, n, hk, d), bf16(g, n, hk, d)
        k[..., 0] = k[..., 0].abs() + 0.5
        k[at, 1, 5] = math.nan
        if hk > 2:
            v[at, 2, 7] = math.nan
        data.append((k, v))
    p = Paged([n] * B, page, hk, d, e4m3=True, data=data)
    q = bf16(g, B, hk, group, d)
    q[:, :, 0, 0], q[:, :, 1, 0] = -math.inf, math.inf
    q = q.view(B, H, d)
    o, lse = eba.decode(p.on_gpu(eba), q.cuda(), p.gtable, p.glens)
    o4, l4 = np64(o).reshape(B, hk, group, d), np64(lse).reshape(B, hk, group)
    plain = [h for h in range(hk) if h not in (1, 2)]
    assert (o4[:, plain, 0] == 0).all() and np.isneginf(l4[:, plain, 0]).all()
    assert np.isnan(o4[:, plain, 1]).all() and np.isnan(l4[:, plain, 1]).all()
    assert np.isnan(o4[:, 1]).all() and np.isnan(l4[:, 1]).all()
    keys, values = p.contents()
    if hk > 2 and group > 2:
        assert np.isnan(o4[:, 2, 2:, 7]).all() and np.isfinite(l4[:, 2, 2:]).all()
    for head in plain[:2]:
        if group > 2:
            mine = slice(head * group + 2, (head + 1) * group)
            one = slice(head, head + 1)
            compare(o[:, mine], lse[:, mine], q[:, mine], [x[:, one] for x in keys], [x[:, one] for x in values],
                    1 / math.sqrt(d), True)


@pytest.mark.parametrize("lens,H,hk,e4m3", [([333], 32, 8, False), ([40, 0, 700, 5] * 16, 8, 2, False),
                                            ([900, 3], 32, 2, True)], ids=["one", "many", "e4m3"])
def test_a_table_far_wider_than_the_lengths(eba, lens, H, hk, e4m3):
    # as a captured call holds it for the longest sequence it may ever see: another way of
    # cutting up the work, the same attention
    p = Paged(lens, 16, hk, 128, e4m3=e4m3, seed=7, k_scale=0.03 if e4m3 else 1.0)
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(12), len(lens), H, 128)
    wide = torch.full((len(lens), 8192), -1, dtype=torch.int32)
    wide[:, :p.table.shape[1]] = p.table
    for table in (p.gtable, wide.cuda()):
        o, lse = eba.decode(cache, q.cuda(), table, p.glens)
        compare(o, lse, q, *p.contents(), 1 / math.sqrt(128), e4m3)


def test_threads_at_once(eba):
    # each with a stream of its own, one plan and one read-only cache for all of them
    plan, n = eba.Rope((64,)), 4
    shared = Paged([2500, 100], 16, 2, 128, seed=50)
    common = shared.on_gpu(eba)
    own = [Paged([900 + 50 * i, 64], 16, 2, 128, seed=51 + i) for i in range(n)]
    caches = [p.on_gpu(eba) for p in own]
    pos = torch.tensor([5, 6], device="cuda", dtype=torch.int32)
    start = [bf16(torch.Generator().manual_seed(60 + i), 2, 4, 128).cuda() for i in range(n)]
    torch.cuda.synchronize()

    def run(i):
        outs, x = [], start[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(25):
                x, _ = eba.rope_fwd(x, None, pos, plan)
                eba.cache_append(caches[i], x[:, :2], x[:, 2:], own[i].gtable, own[i].glens, rope=plan)
                outs.append(eba.decode(caches[i], x, own[i].gtable, own[i].glens, rope=plan)[0])
                outs.append(eba.decode(common, x, shared.gtable, shared.glens)[0])
            torch.cuda.current_stream().synchronize()
        return torch.stack(outs)

    alone = [run(i) for i in range(n)]
    with concurrent.futures.ThreadPoolExecutor(n) as pool:
        for a, b in zip(alone, pool.map(run, range(n))):
            assert torch.equal(a, b)


def test_rotation_refuses_forward_mode_and_vmap(eba):
    plan, pos = eba.Rope((32,)), torch.arange(6, device="cuda", dtype=torch.int32)
    x = bf16(torch.Generator().manual_seed(1), 3, 6, 2, 64).cuda()
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda y: eba.rope(y, None, pos, plan)[0])(x)
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda y: eba.rope(y, None, pos, plan)[0], (x[0],), (x[1],))


def test_one_of_two_inputs_trained(eba):
    # the other's gradient is not asked for: the trained one's is as with both
    g = torch.Generator().manual_seed(14)
    plan, pos = eba.Rope((8, 12, 12)), torch.randint(0, 99, (3, 20), generator=g).to(torch.int32).cuda()
    q, k = bf16(g, 20, 4, 64).cuda(), bf16(g, 20, 2, 64).cuda()
    gq, gk = bf16(g, 20, 4, 64).cuda(), bf16(g, 20, 2, 64).cuda()
    want = eba.rope_bwd(gq, gk, pos, plan)
    for i, trained in enumerate((q, k)):
        trained.requires_grad_()
        outs = eba.rope(q, k, pos, plan)
        got, = torch.autograd.grad(outs, trained, (gq, gk))
        trained.requires_grad_(False)
        assert torch.equal(got, want[i])
