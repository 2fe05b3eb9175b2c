"""The pages' bookkeeping at the ends of its arguments' ranges, against plain loops."""
import numpy as np
import pytest
import torch

from oracle import pages
from test_gpu_pages import PAGE_FAULT, Batch, gpu, same

pytestmark = pytest.mark.gpu
TOP = 2**31 - 1


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


@pytest.mark.parametrize("size", [1, 2, 16])
def test_release_of_bounds_beyond_the_table(eba, size):
    """Bounds outside the table count as its ends: from the largest number on there is nothing
    to give back."""
    s = Batch(eba, 5, 700, size, 5000, seed=7)
    first = np.array([TOP, TOP - 1, TOP - 300, 700 * size, 3])
    for last in (np.full(5, TOP), np.full(5, -TOP - 1), np.array([TOP, 0, TOP, TOP, TOP])):
        assert pages.release(s.refs, s.table, size, first, last) == 0
        eba.pages_release(s.pool, s.gtable, gpu(first), gpu(last))
        s.check()
    assert (s.table[4, 3:] == -1).all() and (s.table[:4] >= 0).any()


def test_release_at_the_end_of_the_widest_table(eba):
    """One sequence with 2^31 - 1 entries, the last few of which hold pages."""
    row = torch.full((1, TOP), -1, dtype=torch.int32, device="cuda")
    row[0, -5:] = gpu([3, 1, 4, 0, 2])
    refs = gpu([1, 1, 1, 1, 1])
    pool = eba.PagePool(refs, 1)
    eba.pages_release(pool, row, gpu([TOP - 3]), gpu([TOP]))
    same(row[0, -5:], [3, 1, -1, -1, -1])
    same(refs, [0, 1, 0, 1, 0])
    eba.pages_release(pool, row, gpu([TOP - 4000]), gpu([TOP - 4]))
    same(row[0, -5:], [-1, 1, -1, -1, -1])
    same(refs, [0, 1, 0, 0, 0])


@pytest.mark.parametrize("size", [1, 2, 16])
def test_reserve_of_lengths_beyond_the_table(eba, size):
    """A length beyond the table is out of range also where nothing is wanted: the sequence
    gets no page and the status says so."""
    s = Batch(eba, 6, 30, size, 400, seed=8, fill=0.3)
    more = np.minimum(s.lens + 3 * size, 30 * size)
    s.lens[:3] = TOP, TOP - 40, 30 * size + 1
    s.glens.copy_(gpu(s.lens))
    for grow in (more, np.full(6, -5), np.where(np.arange(6) < 3, TOP, 0)):
        assert pages.reserve(s.refs, s.table, size, s.lens, grow) == 3
        eba.pages_reserve(s.pool, s.gtable, s.glens, gpu(grow))
        s.check()
        assert eba.poll_device_status() == PAGE_FAULT


def test_reserve_at_the_end_of_the_widest_table(eba):
    """One sequence with 2^31 - 1 entries grows to its last ones."""
    row = torch.full((1, TOP), -1, dtype=torch.int32, device="cuda")
    row[0, -2] = 7
    refs = gpu([0, 1, 0, 0, 1, 0, 0, 1])
    pool = eba.PagePool(refs, 1)
    eba.pages_reserve(pool, row, gpu([TOP - 4]), gpu([TOP]))
    same(row[0, -5:], [-1, 0, 2, 7, 3])
    same(refs, [1, 1, 1, 1, 1, 0, 0, 1])


def test_fork_records_a_last_page_out_of_range(eba):
    """A source whose last, partly filled page has no page's number: the fork lacks its last
    tokens, and the status says so."""
    s = Batch(eba, 4, 6, 16, 100, seed=5)
    s.lens[:] = 20, 33, 16, 7
    s.table[:], s.refs[:] = -1, 0
    s.table[0, :2], s.table[1, :3], s.table[2, 0], s.table[3, 0] = (4, 100), (5, 6, 2**31 - 1), 7, 8
    s.refs[4:9] = 1
    s.glens.copy_(gpu(s.lens))
    s.gtable.copy_(gpu(s.table))
    s.grefs.copy_(gpu(s.refs))
    for src, dst in ((0, 2), (1, 3)):
        want = pages.fork(s.refs, s.table, 16, s.lens, np.array([src]), np.array([dst]))
        got = eba.pages_fork(s.pool, s.gtable, s.glens, gpu([src]), gpu([dst]))
        same(got[0], want[0])
        same(got[1], want[1])
        s.check()
        assert want[2] == 1 and eba.poll_device_status() == PAGE_FAULT


def test_reserve_replaces_pages_out_of_range(eba):
    """An entry with no page's number holds none: it gets one, and the status says so."""
    s = Batch(eba, 3, 6, 4, 40, seed=6)
    s.lens[:] = 5, 0, 3
    s.table[:], s.refs[:] = -1, 0
    s.table[0, :4], s.table[2, 0] = (0, 1, 40, 2), 3
    s.refs[:4] = 1
    s.glens.copy_(gpu(s.lens))
    s.gtable.copy_(gpu(s.table))
    s.grefs.copy_(gpu(s.refs))
    more = np.array([20, 3, 3])
    assert pages.reserve(s.refs, s.table, 4, s.lens, more) == 1
    eba.pages_reserve(s.pool, s.gtable, s.glens, gpu(more))
    s.check()
    assert eba.poll_device_status() == PAGE_FAULT
    assert (s.table[0, :5] == [0, 1, 4, 2, 5]).all() and s.table[1, 0] == 6
