"""Drafted tokens' attention where a cache, a query or the offsets hold what they should not."""
import pytest
import torch

from cache_util import Paged, bf16

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


def test_offsets_that_fall_compute_nothing(eba):
    """Also where the sequences they name would have more tiles together than an int can count:
    4000 times all 2048 tokens of 64 heads over 131072 keys."""
    p = Paged([300, 50, 40], 16, 1, 64, seed=7)
    cache = p.on_gpu(eba)
    q = bf16(torch.Generator().manual_seed(6), 9, 2, 64).cuda()
    for bad in ([0, 6, 3, 9], [9, 9, 9, 0], [0, 3, -1, 9], [0, 1 << 30, 3, 9]):
        o, lse = eba.decode_tree(cache, q, p.gtable, p.glens, torch.tensor(bad, dtype=torch.int32).cuda())
        assert eba.poll_device_status() == 7
        assert (o == 0).all() and torch.isneginf(lse).all()
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
