"""Drafted tokens' sets without a GPU: a window over a mask and over its chain."""
import pytest

from oracle import tree


@pytest.mark.parametrize("window", [1, 2, 4, 7, 40])
@pytest.mark.parametrize("n_keys,n_new", [(8, 8), (20, 8), (30, 5)])
@pytest.mark.parametrize("sinks", [0, 3])
def test_masks_without_far_ancestors_are_the_window(n_keys, n_new, window, sinks):
    """A chain's mask without the bits of the ancestors `window` or more places back sees what the
    chain does, but for drafted sinks."""
    for i in range(n_new):
        mask = sum(1 << x for x in range(max(0, i - window + 1), i + 1))
        chain = tree.seen(n_keys, n_new, i, window=window, sinks=sinks)
        first = n_keys - n_new
        far = [j for j in chain if j >= first and j <= first + i - window]  # sinks that are drafted themselves
        assert tree.seen(n_keys, n_new, i, mask, window, sinks) == [j for j in chain if j not in far]
