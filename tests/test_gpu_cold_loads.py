"""Query tiles without a second one beside them, over keys that come from HBM (the caches were
written over): the loads then land in any order, and each reader of the ring has to wait for
its own. All launches give the same bits, near the plain form in 64 bits, and no wait runs out."""
import math

import pytest
import torch

from cache_util import bf16

pytestmark = pytest.mark.gpu

U = 2.0 ** -8  # a bf16 rounding, relative


@pytest.fixture(scope="module")
def eba():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


def plain(q, k, v, seen, scale):
    """[H, Lq, d] in float64."""
    k, v = (x.repeat_interleave(q.shape[0] // k.shape[0], 0) for x in (k, v))
    s = (q.double() @ k.double().transpose(1, 2) * scale).masked_fill(~seen, -math.inf)
    return s.softmax(-1) @ v.double(), (s.softmax(-1) @ v.double().abs())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,Lk,left,right", [(100, 3000, None, None), (823, 823, 435, 27), (300, 1700, None, None), (1100, 1100, 700, 0)])
def test_same_bits_from_cold_memory(eba, Lq, Lk, left, right, d):
    H, Hkv = 32, 16
    g = torch.Generator().manual_seed(Lq + d)
    q, k, v = (bf16(g, 1, h, n, d).cuda() for h, n in ((H, Lq), (Hkv, Lk), (Hkv, Lk)))
    flush = torch.empty(64 << 20, device="cuda", dtype=torch.int32)
    i, j = torch.arange(Lq, device="cuda")[:, None] + Lk - Lq, torch.arange(Lk, device="cuda")
    seen = (j >= i - (Lk if left is None else left)) & (j <= i + (Lk if right is None else right))
    scale = 1 / math.sqrt(d)
    want, size = plain(q[0], k[0], v[0], seen, scale)
    eba.poll_device_status()
    forms = [lambda: eba.fwd_window(q, k, v, left, right, 0)]
    if left is None:
        forms.append(lambda: eba.fwd(q, k, v))
    for form in forms:
        first = None
        for turn in range(60):
            flush.fill_(turn)
            o, lse = form()
            if first is None:
                first = o, lse
            assert torch.equal(o, first[0]) and torch.equal(lse, first[1]), turn
        assert eba.poll_device_status() == 0
        # weights as bf16, their sum, and O's own rounding; fp32 sums are far below
        assert ((o[0].double() - want).abs() <= 2.1 * U * size + U * want.abs()).all()
