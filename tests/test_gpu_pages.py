"""The cache's pages on the GPU: counts, tables and copies against plain loops, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import pages

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
PAGE_FAULT = 7


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


def gpu(x):
    return torch.as_tensor(np.asarray(x)).to(torch.int32).cuda()


def same(t, x):
    assert (t.cpu().numpy() == np.asarray(x)).all()


class Batch:
    """Sequences with pages, as numpy arrays and on the GPU. wide tables are views of
    wider ones, so that a write behind a row shows."""

    def __init__(self, eba, B, wide, size, n_pages, seed, fill=0.6):
        r = self.r = np.random.default_rng(seed)
        self.size, self.lens = size, r.integers(0, max(1, int(wide * size * fill)) + 1, B)
        self.table, self.refs = np.full((B, wide), -1), np.zeros(n_pages, dtype=np.int64)
        order = r.permutation(n_pages)
        for b in range(B):
            k = -(-self.lens[b] // size)
            self.table[b, :k], order = order[:k], order[k:]
            self.refs[self.table[b, :k]] = 1
        self.room = torch.full((B, wide + 3), -77, dtype=torch.int32, device="cuda")
        self.gtable = self.room[:, :wide]
        self.gtable.copy_(gpu(self.table))
        self.grefs, self.glens = gpu(self.refs), gpu(self.lens)
        self.pool = eba.PagePool(self.grefs, size)

    def check(self):
        same(self.gtable, self.table)
        same(self.grefs, self.refs)
        same(self.glens, self.lens)
        assert (self.room[:, self.table.shape[1]:] == -77).all()


# sequences, table columns, page size, pages
SIZES = [(1, 1, 1, 1), (1, 3, 16, 4), (3, 7, 20, 31), (40, 33, 8, 1500), (300, 5, 16, 1601), (7, 2500, 4, 20011),
         (700, 40, 3, 60000)]


@pytest.mark.parametrize("B,wide,size,n", SIZES)
def test_turns(eba, B, wide, size, n):
    """Release, fork and reserve, one behind the other, several times."""
    s = Batch(eba, B, wide, size, n, seed=B + wide)
    r = s.r
    for turn in range(4):
        first = r.integers(-3, wide * size + 5, B)
        last = first + r.integers(-5, wide * size, B)
        gone = r.random(B) < 0.3  # these end
        first, last = np.where(gone, 0, first), np.where(gone, wide * size, last)
        assert pages.release(s.refs, s.table, size, first, last) == 0
        eba.pages_release(s.pool, s.gtable, gpu(first), gpu(last))
        s.check()
        slots = r.permutation(B)
        k = B // 3
        dst, src = slots[:k], slots[k:][r.integers(0, B - k, k)]
        pages.release(s.refs, s.table, size, np.zeros(B, int), np.where(np.isin(np.arange(B), dst), wide * size, 0))
        s.gtable.copy_(gpu(s.table))
        s.grefs.copy_(gpu(s.refs))
        old, new, faults = pages.fork(s.refs, s.table, size, s.lens, src, dst)
        gold, gnew = eba.pages_fork(s.pool, s.gtable, s.glens, gpu(src), gpu(dst))
        same(gold, old)
        same(gnew, new)
        s.check()
        assert (eba.poll_device_status() == PAGE_FAULT) == (faults > 0)
        more = np.minimum(s.lens + r.integers(-2, 4 * size, B), wide * size)
        faults = pages.reserve(s.refs, s.table, size, s.lens, more)
        eba.pages_reserve(s.pool, s.gtable, s.glens, gpu(more))
        s.check()
        assert (eba.poll_device_status() == PAGE_FAULT) == (faults > 0)


def test_out_of_pages(eba):
    s = Batch(eba, 6, 9, 4, 20, seed=1, fill=0.3)
    more = np.full(6, 36)
    faults = pages.reserve(s.refs, s.table, 4, s.lens, more)
    eba.pages_reserve(s.pool, s.gtable, s.glens, gpu(more))
    s.check()
    assert faults > 0 and eba.poll_device_status() == PAGE_FAULT
    s.lens[:] = 5  # every source's last page is part full, and no page is free
    s.glens.copy_(gpu(s.lens))
    old, new, faults = pages.fork(s.refs, s.table, 4, s.lens, np.array([0, 1]), np.array([2, 3]))
    gold, gnew = eba.pages_fork(s.pool, s.gtable, s.glens, gpu([0, 1]), gpu([2, 3]))
    same(gold, old)
    same(gnew, new)
    s.check()
    assert faults > 0 and eba.poll_device_status() == PAGE_FAULT


def test_faults(eba):
    """Indexes, lengths, pages and pairs out of range: left out, recorded, the rest done."""
    s = Batch(eba, 8, 6, 16, 100, seed=2)
    src, dst = np.array([0, -1, 1, 9, 2, 0, 3, 4]), np.array([5, 5, 8, 6, 2, 5, 0, 7])
    want = pages.fork(s.refs, s.table, 16, s.lens, src, dst)
    got = eba.pages_fork(s.pool, s.gtable, s.glens, gpu(src), gpu(dst))
    same(got[0], want[0])
    same(got[1], want[1])
    s.check()
    assert want[2] == 6 and eba.poll_device_status() == PAGE_FAULT
    s.lens[:3] = -4, 97, 1 << 30
    s.glens.copy_(gpu(s.lens))
    want = pages.fork(s.refs, s.table, 16, s.lens, np.array([0, 1, 2]), np.array([5, 6, 7]))
    eba.pages_fork(s.pool, s.gtable, s.glens, gpu([0, 1, 2]), gpu([5, 6, 7]))
    s.check()
    assert want[2] == 3 and eba.poll_device_status() == PAGE_FAULT
    more = np.array([3, 4, 2000000000, 97, 96, -5, 0, 96])
    assert pages.reserve(s.refs, s.table, 16, s.lens, more) > 0
    eba.pages_reserve(s.pool, s.gtable, s.glens, gpu(more))
    s.check()
    assert eba.poll_device_status() == PAGE_FAULT
    # a page number of no page, a page that nobody holds
    s.table[4, 0], s.table[5, 0], s.refs[50] = 100, 50, 0
    s.gtable.copy_(gpu(s.table))
    s.grefs.copy_(gpu(s.refs))
    zero, full = np.zeros(8, int), np.full(8, 2**31 - 1)
    assert pages.release(s.refs, s.table, 16, zero, full) > 0
    eba.pages_release(s.pool, s.gtable, gpu(zero), gpu(full))
    s.check()
    assert eba.poll_device_status() == PAGE_FAULT and (s.table == -1).all()


def cache_of(eba, n, size, hkv, d, e4m3, heads_first, seed=0):
    g = torch.Generator().manual_seed(seed)
    shape = (2, n, hkv, size, d) if heads_first else (2, n, size, hkv, d)
    raw = torch.randint(-2**15, 2**15, shape, generator=g).to(torch.int16)  # any bits, NaN among them
    raw = raw.to(torch.int8).view(E4M3) if e4m3 else raw.view(torch.bfloat16)
    t = raw.cuda()
    k, v = (x.transpose(1, 2) if heads_first else x for x in t)
    bits = (lambda x: x.view(torch.int8) if e4m3 else x.view(torch.int16))
    return eba.PagedCache(k, v, *((0.5, 0.25) if e4m3 else ())), [bits(x) for x in (k, v)]


FORMS = [(16, 8, 128, False, False), (20, 3, 64, False, True), (1, 1, 64, True, False), (48, 5, 128, True, True),
         (7, 40, 64, True, False)]


@pytest.mark.parametrize("size,hkv,d,e4m3,heads_first", FORMS)
def test_copy(eba, size, hkv, d, e4m3, heads_first):
    cache, bits = cache_of(eba, 30, size, hkv, d, e4m3, heads_first)
    old, new = np.array([3, -1, 7, 3, 9, 12, 30]), np.array([4, 5, -1, 6, 9, 31, 1])
    want = [b.cpu().numpy().copy() for b in bits]
    faults = [pages.copy(w, old, new) for w in want]
    eba.cache_copy(cache, gpu(old), gpu(new))
    for b, w in zip(bits, want):
        same(b, w)
    assert faults == [2, 2] and eba.poll_device_status() == PAGE_FAULT


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("size,hkv,d,e4m3,heads_first", FORMS)
def test_gather(eba, size, hkv, d, e4m3, heads_first, in_place):
    """Sequences of no, one, few and many tokens; places that repeat and go back and forth."""
    r = np.random.default_rng(size)
    lens = [0, 1, 5, 700 // size * size + 3, 333, 2]
    wide = -(-max(lens) // size)
    n = 2 * len(lens) * wide + 2
    order = r.permutation(n)
    table = order[:len(lens) * wide].reshape(len(lens), wide)
    new = order[len(lens) * wide:2 * len(lens) * wide].reshape(len(lens), wide)
    start = [0, 0, 2, 40, 0, 0]
    places = []
    for x, s in zip(lens, start):
        mine = [max(p, s + j) for j, p in enumerate(sorted(r.choice(np.arange(s, max(x, s + 1)), size=max(0, (x - s) // 2))))]
        places.append([p if r.random() < 0.9 else min(x - 1, p + 1) for p in mine])
    cu = np.cumsum([2] + [len(p) for p in places])  # two entries before the first sequence's are not used
    flat = np.array([10**6, 0] + sum(places, []) + [0, -1])
    cache, bits = cache_of(eba, n, size, hkv, d, e4m3, heads_first)
    want = [b.cpu().numpy().copy() for b in bits]
    for w in want:
        assert pages.gather(w, size, table, flat, cu, None if in_place else new, start) == 0
    eba.cache_gather(cache, gpu(table), gpu(flat), gpu(cu), to_table=None if in_place else gpu(new), to_start=gpu(start))
    for b, w in zip(bits, want):
        same(b, w)


def test_gather_faults(eba):
    cache, bits = cache_of(eba, 12, 4, 2, 64, False, False)
    table, new = np.array([[3, 1, 40, -1], [5, 6, 7, 8]]), np.array([[0, 9], [10, -3]])
    places, cu = np.array([5, 8, 12, 16, -1, 2, 0, 1, 2, 3, 4, 5, 6, 7, 8]), np.array([0, 6, 15])
    for to, start in ((None, [1, 0]), (None, [3, 3]), (new, [0, 0]), (new, [-1, 6])):
        want = [b.cpu().numpy().copy() for b in bits]
        assert min(pages.gather(w, 4, table, places, cu, to, start) for w in want) > 0
        eba.cache_gather(cache, gpu(table), gpu(places), gpu(cu), to_table=None if to is None else gpu(to),
                         to_start=gpu(start))
        for b, w in zip(bits, want):
            same(b, w)
        assert eba.poll_device_status() == PAGE_FAULT
    # offsets that decrease, or lie outside places: nothing out of range is read
    for cu in ([9, 3, 5], [-5, 4, 10**9]):
        eba.cache_gather(cache, gpu(table), gpu(places), gpu(cu))
        eba.cache_gather(cache, gpu(table), gpu(places), gpu(cu), to_table=gpu(new))
        eba.poll_device_status()


def test_nothing_to_do(eba):
    s = Batch(eba, 4, 5, 8, 40, seed=3)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    old, new = eba.pages_fork(s.pool, s.gtable, s.glens, none, none)
    assert old.shape == new.shape == (0,)
    cache, bits = cache_of(eba, 40, 8, 2, 64, False, False)
    before = [b.clone() for b in bits]
    eba.cache_copy(cache, none, none)
    eba.cache_gather(cache, s.gtable, none, gpu([0] * 5))
    eba.pages_reserve(s.pool, s.gtable, s.glens, s.glens)
    eba.pages_release(s.pool, s.gtable, s.glens, s.glens)
    s.check()
    assert all((a == b).all() for a, b in zip(bits, before))


def test_captured_turn_follows_its_tables(eba):
    """A turn in a CUDA graph, replayed on other tables, on a stream of its own."""
    s = Batch(eba, 50, 12, 16, 900, seed=4)
    first, last, src, dst, more = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (50, 50, 9, 9, 50))

    def turn():
        eba.pages_release(s.pool, s.gtable, first, last)
        out = eba.pages_fork(s.pool, s.gtable, s.glens, src, dst)
        eba.pages_reserve(s.pool, s.gtable, s.glens, more)
        return out

    stream = torch.cuda.Stream()
    dst.copy_(gpu(np.arange(9) + 1))
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            old, new = turn()
    torch.cuda.synchronize()
    for seed in (11, 12, 13):
        t = Batch(eba, 50, 12, 16, 900, seed=seed)
        r = np.random.default_rng(seed)
        slots = r.permutation(50)
        d, a = slots[:9], r.choice(slots[9:], 9)
        f, e = np.zeros(50, int), np.where(np.isin(np.arange(50), d), 12 * 16, 0)
        for to, x in ((s.gtable, t.table), (s.grefs, t.refs), (s.glens, t.lens), (first, f), (last, e), (src, a), (dst, d)):
            to.copy_(gpu(x))
        pages.release(t.refs, t.table, 16, f, e)
        want = pages.fork(t.refs, t.table, 16, t.lens, a, d)
        grow = np.minimum(t.lens + 20, 12 * 16)
        more.copy_(gpu(grow))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert pages.reserve(t.refs, t.table, 16, t.lens, grow) == 0 and want[2] == 0
        for g, x in ((s.gtable, t.table), (s.grefs, t.refs), (s.glens, t.lens), (old, want[0]), (new, want[1])):
            same(g, x)


def test_pages_behind_2_to_the_31_elements(eba):
    """Offsets in the cache that pass 32 bits."""
    n = (1 << 31) // (64 * 4 * 64) + 300
    k = torch.zeros(n, 64, 4, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(n, 64, 4, 64, dtype=torch.bfloat16, device="cuda")
    cache = eba.PagedCache(k, v)
    k[n - 1], v[n - 1] = 3, 4
    eba.cache_copy(cache, gpu([n - 1]), gpu([n - 2]))
    assert (k[n - 2] == 3).all() and (v[n - 2] == 4).all() and (k[n - 3] == 0).all()
    eba.cache_gather(cache, gpu([[n - 1, n - 5]]), gpu([3, 9]), gpu([0, 2]), to_table=gpu([[n - 7]]), to_start=gpu([5]))
    assert (k[n - 7, 5:7] == 3).all() and (v[n - 7, 5:7] == 4).all()
    assert (k[n - 7, :5] == 0).all() and (k[n - 7, 7:] == 0).all()


def test_a_pool_that_goes_leaves_its_scratch_to_its_stream(eba):
    """Memory of a pool used on another stream is not handed out while that one may run."""
    batch = Batch(eba, 8, 40, 16, 4096, 3)
    pool = eba.PagePool(batch.grefs, 16)
    at, side = pool._scratch.data_ptr(), torch.cuda.Stream()
    more = np.minimum(batch.lens + 50, 640)
    gmore = gpu(more)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        eba.pages_reserve(pool, batch.gtable, batch.glens, gmore)
    del pool
    held = [torch.empty(4096, dtype=torch.int32, device="cuda") for _ in range(64)]
    assert not side.query() and all(x.data_ptr() != at for x in held)
    side.synchronize()
    pages.reserve(batch.refs, batch.table, 16, batch.lens, more)
    batch.check()
