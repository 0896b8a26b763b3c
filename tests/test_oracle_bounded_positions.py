"""Pins of oracle.bounded.visible: entries in order, enumeration, and an eviction."""
import numpy as np
import pytest

from oracle import bounded as B


@pytest.mark.parametrize("prefix", [0, 10, 33])
def test_in_order_it_is_the_count(prefix):
    for n in (0, 1, 7):
        for shift in (0, 3):
            pos = 4 * (np.arange(n) + shift) + 3
            for t in range(-2, 50):
                assert list(B.visible(pos, t, prefix)) == list(range(B.visible_count(n, shift, t, prefix)))


def test_scattered_entries_by_enumeration():
    pos = 4 * np.random.default_rng(3).permutation(12)[:7] + 3
    for t in range(-1, 50):
        for prefix in (0, 18):
            sees = set(range(max(t + 1, prefix if t < prefix else 0))) if t >= 0 else set()
            assert list(B.visible(pos, t, prefix)) == [j for j, p in enumerate(pos) if set(range(p - 3, p + 1)) <= sees]


def test_no_token_sees_what_comes_after_it_once_entries_were_evicted():
    """150 entries cut to 120: the newest of them fill holes, so an index tells nothing about a position."""
    w = np.random.default_rng(4).random(150)
    pos = 4 * np.arange(150) + 3
    holes, movers = B.evict(w, pos, 0, 120, 4, 16)
    order = np.arange(150)
    order[holes] = movers
    pos = pos[order[:120]]
    assert int(np.argmax(pos)) < 119
    for t in range(592, 600):
        seen = pos[B.visible(pos, t)]
        assert seen.max() <= t and len(seen) == int((pos <= t).sum())
    # going by index, the token at 592 would see the entry that ends at 599
    assert pos[:B.visible_count(120, 30, 592)].max() == 599
