"""The rotation, the paged cache and the decode where they are most easily wrong:
absent pages, special values and far-out sizes on every path of the decode, exact
roundings of an e4m3 cache, and several threads at once."""
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
