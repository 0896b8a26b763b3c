"""Pins of the bounded-cache oracle (oracle/bounded.py): library routines, closed
forms and brute force on tiny inputs."""
import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import bounded as B


def test_visible_count_by_enumeration():
    for n in (0, 1, 7):
        for shift in (0, 3):
            for t in range(-1, 50):
                for prefix in (0, 10, 33):
                    sees = range(0, max(t + 1, prefix if t < prefix else 0)) if t >= 0 else range(0)
                    want = sum(all(4 * (j + shift) + k in sees for k in range(4)) for j in range(n))
                    assert B.visible_count(n, shift, t, prefix) == want


def test_attention_is_the_library_attention():
    g = np.random.default_rng(1)
    q, k = g.standard_normal((5, 16)), g.standard_normal((23, 16))
    x = B.logits(q, k, 0.25, 90, np.arange(23))
    o, lse = B.attention(x, k)
    t = lambda a: torch.from_numpy(a)[None, None]  # noqa: E731
    want = torch.nn.functional.scaled_dot_product_attention(t(q), t(k), t(k), scale=0.25)[0, 0].numpy()
    assert np.allclose(o, want, atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(torch.from_numpy(x), 1).numpy(), atol=1e-12)
    o2, lse2 = A.softmax_attention(q, k, 0.25)
    assert np.allclose(o, o2, atol=1e-12) and np.allclose(lse, lse2, atol=1e-12)


def test_no_key_gives_zeros_and_minus_infinity():
    o, lse = B.attention(np.zeros((3, 0)), np.zeros((0, 8)))
    assert not o.any() and np.all(np.isneginf(lse))


def test_cap_and_bias():
    g = np.random.default_rng(2)
    q, k = 40 * g.standard_normal((4, 8)), g.standard_normal((9, 8))
    pos = np.array([3, 7, 11, 15, 19, 23, 27, 31, 35])
    plain = B.logits(q, k, 1.0, 20, pos)
    capped = B.logits(q, k, 1.0, 20, pos, cap=5.0)
    assert np.all(np.abs(capped) <= 5.0) and np.all(np.sign(capped) == np.sign(plain))
    # 1 >= tanh(y) / y >= 1 - y^2 / 3
    y = 1e-4 * np.abs(plain).max() / 5
    assert np.allclose(B.logits(1e-4 * q, k, 1.0, 20, pos, cap=5.0), 1e-4 * plain, rtol=y * y / 3, atol=1e-15)
    assert np.allclose(capped, torch.tanh(torch.from_numpy(plain / 5)).numpy() * 5)
    biased = B.logits(q, k, 1.0, 20, pos, slopes=np.array([0.0, 0.5, 1.0, 2.0]))
    assert np.array_equal(biased[0], plain[0])
    for h, s in enumerate((0.0, 0.5, 1.0, 2.0)):
        assert np.allclose((plain - biased)[h], [s * abs(20 - p) for p in pos])


@pytest.mark.parametrize("n,keep,sink,recent", [(9, 4, 1, 2), (9, 9, 0, 0), (5, 9, 1, 1), (12, 1, 0, 0), (12, 6, 3, 3)])
def test_evict_by_brute_force(n, keep, sink, recent):
    g = np.random.default_rng(n * 31 + keep)
    for trial in range(40):
        shift = int(g.integers(0, 4))
        entries = g.permutation(n + shift)[:n]
        entries = np.concatenate([entries[entries < n + shift - recent],
                                  entries[entries >= n + shift - recent]])
        pos = 4 * entries + 3
        w = g.integers(0, 4, n).astype(np.float64)       # many ties
        holes, movers = B.evict(w, pos, shift, keep, sink, recent)
        assert len(holes) == len(movers)
        if n <= keep:
            assert len(holes) == 0
            continue
        stay = [j for j in range(keep) if j not in set(holes)] + list(movers)
        assert len(stay) == keep and all(h < keep for h in holes) and all(m >= keep for m in movers)
        gone = [j for j in range(n) if j not in set(stay)]
        rank = lambda j: (entries[j] < sink or entries[j] >= n + shift - recent, w[j], -j)  # noqa: E731
        safe = lambda j: entries[j] < sink or entries[j] >= n + shift - recent  # noqa: E731
        assert not any(safe(j) for j in gone)
        for a in stay:
            for b in gone:
                assert safe(a) or rank(a)[1:] > rank(b)[1:]
        assert list(holes) == sorted(holes) and list(movers) == sorted(movers)
