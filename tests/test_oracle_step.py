"""Pins of oracle.step: library routines, closed forms and brute force (no GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import compress as OC
from oracle import formats as F
from oracle import step as O


def test_fp8_blocks_against_torch_casts():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(9, 400, generator=g) * torch.exp(2 * torch.randn(9, 1, generator=g))
    codes, scales = O.pack_fp8_blocks(x.numpy())
    for k in range(4):
        blk = x[:, 128 * k:128 * k + 128]
        a = blk.abs().amax(dim=1)
        assert np.array_equal(scales[:, k], (a / torch.tensor(448.0)).numpy())
        q = (blk * (torch.tensor(448.0) / a).unsqueeze(1)).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert np.array_equal(codes[:, 128 * k:128 * k + 128], q.view(torch.uint8).numpy())
    # every value within half a step (2^-4) of itself, or of the smallest normal code
    back = O.unpack_fp8_blocks(codes, scales)
    top = scales.astype(np.float64)[:, np.arange(400) // 128]
    assert np.all(np.abs(back - x.double().numpy()) <= (np.abs(x.double().numpy()) + 2.0 ** -6 * top) * (2.0 ** -4 + 2.0 ** -22))


def test_product_of_values():
    g = np.random.RandomState(1)
    a, b = g.randint(0, 127, (5, 200)).astype(np.uint8), g.randint(0, 127, (130, 200)).astype(np.uint8)
    sa, sb = g.rand(5, 2), g.rand(2, 2)
    C, mag = O.matmul_fp8(a, sa, b, sb)
    m, n = 3, 129
    want = sum(F.e4m3_decode_code(int(a[m, k])) * F.e4m3_decode_code(int(b[n, k])) * sa[m, k // 128] * sb[1, k // 128] for k in range(200))
    assert abs(C[m, n] - want) <= 1e-12 * mag[m, n] and mag[m, n] == pytest.approx(C[m, n])


def test_rope_is_the_cached_keys_rotation():
    """Half pairs at the end of the head, plain frequencies: what the compression does to its entries."""
    g = np.random.RandomState(2)
    x, pos = g.randn(7, 64), np.array([0, 3, 7, 1000, 4003, 65535, 1048575])
    ref = OC.rope(x, pos, 16, 10000.0)
    got = O.rope(x[:, None], pos, O.rope_frequencies(16), 48)[:, 0]
    assert np.max(np.abs(got - ref)) <= 2.0 ** -24 * np.max(np.abs(x)) * 2


def test_rope_pairs_norm_and_relative_position():
    g = np.random.RandomState(3)
    x = g.randn(2, 3, 24)
    th = O.rope_frequencies(8)
    for layout in ("half", "interleaved"):
        y = O.rope(x, [5, 9], th, 4, layout)
        assert np.array_equal(y[:, :, :4], x[:, :, :4]) and np.array_equal(y[:, :, 12:], x[:, :, 12:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose(O.rope(y, [5, 9], th, 4, layout, inverse=True), x)
        q, k = x[:1], x[1:]
        dot = lambda p, s: (O.rope(q, [p], th, 4, layout) * O.rope(k, [s], th, 4, layout)).sum()  # noqa: E731
        assert dot(100, 40) == pytest.approx(dot(160, 100))
    # interleaved pairs are half pairs of the channels in another order
    order = np.r_[0:4, 4 + np.r_[0:8:2, 1:8:2], 12:24]
    assert np.allclose(O.rope(x[:, :, order], [5, 9], th, 4, "half"), O.rope(x, [5, 9], th, 4, "interleaved")[:, :, order])


def test_scaled_frequencies():
    th = O.rope_frequencies(64)
    assert np.allclose(O.rope_frequencies(64, scaling="linear", factor=8.0), th / 8)
    ntk = O.rope_frequencies(64, scaling="ntk", factor=8.0)
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(th[-1] / 8)        # the slowest pair is stretched by the factor
    y = O.rope_frequencies(64, scaling="yarn", factor=40.0)
    turns = 4096 * th / (2 * math.pi)
    assert np.allclose(y[turns > 40], th[turns > 40]) and np.allclose(y[turns < 0.7], th[turns < 0.7] / 40)
    assert np.all(np.diff(y / th) <= 1e-12)
    assert np.allclose(O.rope_frequencies(64, scaling="yarn", factor=1.0), th)


def test_tree_plan_by_hand():
    parent = np.array([[-1, 0, 0, 2, -1, -2, 4], [-1, 0, 5, 2, -2, 4, 0]])
    q, path, bad_i, bad_c = O.tree_plan(parent, [10, 7], 3)
    assert q[0].tolist() == [10, 11, 11, 12, 10, -1, 11] and path[0, 3].tolist() == [0, 2, 3] and path[0, 6].tolist() == [4, 6, -1]
    assert q[1].tolist() == [7, 8, -1, -1, -1, -1, 8] and bad_i and not bad_c


def test_tree_window_by_masks():
    """Against a mask over all positions: committed ones that the buffer holds, and the line's own."""
    for t, W, ctx, pos0, cap, line in ((12, 8, 10, 4, 6, [3, 5, 9]), (5, 128, 4, -100, 104, [0, 1]), (30, 4, 25, 20, 5, list(range(6)))):
        old, new = O.tree_window(t, W, ctx, pos0, cap, line)
        seen = [p for p in range(t + 1) if t - p < W]
        assert old == [p - pos0 for p in seen if p < ctx and pos0 <= p < pos0 + cap]
        assert new == [line[p - ctx] for p in seen if p >= ctx]


def test_attention_against_torch():
    g = torch.Generator().manual_seed(4)
    Q, keys = torch.randn(3, 64, generator=g, dtype=torch.float64), torch.randn(50, 64, generator=g, dtype=torch.float64)
    o, lse, mag, qk = O.attention(Q.numpy(), keys.numpy(), 0.125)
    want = torch.nn.functional.scaled_dot_product_attention(Q[None], keys[None], keys[None])[0]
    assert np.allclose(o, want.numpy()) and np.allclose(lse, torch.logsumexp(Q @ keys.t() / 8, dim=1).numpy())
    assert np.all(mag >= np.abs(o)) and np.all(qk >= np.abs(Q.numpy() @ keys.numpy().T / 8).max(axis=1))
    o, lse, _, _ = O.attention(Q.numpy(), np.zeros((0, 64)), 0.125)
    assert np.all(o == 0) and np.all(np.isneginf(lse))


def test_pages_by_hand():
    table = np.array([[4, 5, 9, 9], [6, 9, 9, 9], [9, 9, 9, 9]])
    out = O.page_plan([600, 100, 0], [-400, 200, 300], [3, 1, 0], table, np.array([0, 1, 2, 3, -1, -1, -1]), 2, Tq=300, max_new=80)
    # sequence 0 keeps one page (50 entries) and gives 5 and 9 back; the others pop 9, 5 and 1, 0
    assert out["held"].tolist() == [1, 2, 2] and out["table"][1, :2].tolist() == [6, 9] and out["table"][2, :2].tolist() == [5, 1]
    assert out["n_free"] == 1 and out["free"][0] == 0 and out["n_entries"].tolist() == [50, 75, 75]
    assert out["slots"][2, 64] == 64 and out["slots"][2, 75] == -1 and out["q_pos"][1, 199] == 299 and out["q_pos"][1, 200] == -1
