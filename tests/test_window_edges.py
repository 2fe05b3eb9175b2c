"""Windowed attention's host side without a GPU: what a training step keeps, and the bytes of
the backward's workspace."""
import numpy as np
import pytest

from oracle.window import visible


@pytest.fixture(scope="module")
def eba():
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


@pytest.mark.parametrize("Lq,Lk,left,right,sinks,few", [
    (9000, 9000, 255, 256, 0, True), (9000, 9000, 256, 256, 0, False), (9000, 9000, 50, 46, 415, True),
    (9000, 9000, 50, 46, 416, False), (9000, 9000, 100, 9, 4000, False), (512, 512, -1, -1, 0, True),
    (513, 513, -1, -1, 0, False), (400, 400, -1, 0, 4000, True), (300, 300, 2**31 - 1, 2**31 - 1, 2**31 - 1, True),
    # the first rows see few: causal ones; the last ones: the other way round
    (9000, 9000, 1023, 0, 0, True), (9000, 9000, 1024, 0, 0, False), (1024, 1024, -1, 0, 0, True),
    (1025, 1025, -1, 0, 0, False), (9000, 9000, 0, 1023, 0, True), (1024, 1024, 0, -1, 0, True), (9000, 9000, 96, 0, 928, False),
    (9000, 9000, 95, 0, 928, True), (900, 900, 600, 6, 0, True), (900, 900, 600, 7, 0, False),
    (1024, 1024, 7, -1, 0, False), (1024, 1024, 6, -1, 0, True), (20, 900, -1, 0, 0, False), (893, 900, -1, 0, 0, False),
    (894, 900, -1, 0, 0, True), (1500, 900, -1, 100, 0, True), (1500, 900, -1, -1, 0, False)])
def test_few_keys_a_row(eba, Lq, Lk, left, right, sinks, few):
    """What rounding took from o is kept where no row sees more than 512 keys, sinks among them, or
    some fewer than 8 and none more than 1024."""
    assert eba._few_keys(Lq, Lk, left, right, sinks) == few


def test_few_keys_is_what_the_rows_see(eba):
    """Against the visible pairs themselves."""
    r = np.random.default_rng(0)
    for _ in range(300):
        Lq, Lk = (int(x) for x in r.integers(1, 1300, 2))
        left, right = (None if r.random() < 0.3 else int(r.choice([0, 3, 40, 700]) + r.integers(0, 5)) for _ in range(2))
        sinks = int(r.choice([0, 0, 2, 300]))
        n = visible(Lq, Lk, left, right, sinks).sum(1)
        few = eba._few_keys(Lq, Lk, *(-1 if x is None else x for x in (left, right)), sinks)
        # (a window that no row has room for may count for more than any row sees)
        most = min(Lk, (Lk if left is None else left) + (Lk if right is None else right) + 1 + sinks)
        assert n.max() <= most
        fewest = min(n[n > 0].min(), 8) if (n > 0).any() else 8
        assert few == (most <= (1024 if fewest < 8 else 512)), (Lq, Lk, left, right, sinks)


@pytest.mark.parametrize("H,Hkv,L,left,sinks", [
    (8, 8, 131072, 511, 64), (8, 8, 131072, 511, 4096), (8, 8, 131072, 511, 9000), (1, 1, 1 << 20, 100, 60000),
    (1, 1, 1 << 20, 100, 77000), (600, 600, 60000, 100, 1), (304, 304, 60000, 100, 200), (64, 1, 1 << 22, 20, 4),
    (1, 1, 1 << 22, 20, 70000)])
@pytest.mark.parametrize("d", [64, 128])
def test_parts_are_bounded(eba, H, Hkv, L, left, sinks, d):
    """The parts of the first tokens' gradients: at most 1216, dK and dV of 128 keys each, in
    fp32."""
    more = eba.bwd_window_workspace_size(1, H, Hkv, L, L, d, left, 0, sinks) - eba.bwd_workspace_size(1, H, L, L, d)
    assert 0 <= more <= 2 * 4 * 152 * 2 * 128 * d * 4
    assert more <= 160 * 10 ** 6


def test_window_as_wide_as_the_longest_sequences(eba):
    """Both sides together pass an int: every tile of queries sees every tile of keys, and
    nothing is cut."""
    L = 1 << 29
    plain = eba.bwd_workspace_size(1, 1, L, L, 64)
    assert plain > 0
    for side in (L - 1, L, 2 * L - 2, 2 * L - 1):
        assert eba.bwd_window_workspace_size(1, 1, 1, L, L, 64, side, side, 5) == plain
