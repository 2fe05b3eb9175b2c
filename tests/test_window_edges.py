"""Windowed attention's host side without a GPU: what a training step keeps, and the bytes of
the backward's workspace."""
import pytest


@pytest.fixture(scope="module")
def eba():
    from exact_blockwise_attention_gb300 import _build

    _build.build()
    import exact_blockwise_attention_gb300 as m

    return m


@pytest.mark.parametrize("Lk,left,right,sinks,few", [
    (9000, 511, 0, 0, True), (9000, 512, 0, 0, False), (9000, 255, 256, 0, True), (9000, 256, 256, 0, False),
    (9000, 96, 0, 415, True), (9000, 96, 0, 416, False), (9000, 100, 0, 4000, False), (9000, 0, 0, 511, True),
    (512, -1, -1, 0, True), (513, -1, 0, 0, False), (400, -1, 0, 4000, True), (513, 0, -1, 0, False),
    (300, 2**31 - 1, 2**31 - 1, 2**31 - 1, True)])
def test_few_keys_counts_the_sinks(eba, Lk, left, right, sinks, few):
    """What rounding took from o is kept where no row sees more than 512 keys."""
    assert eba._few_keys(Lk, left, right, sinks) == few


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
