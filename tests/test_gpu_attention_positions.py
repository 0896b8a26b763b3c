"""Sparse attention at the ends of the position range, and drafted trees without a window there."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build
from oracle import formats as F
from oracle import step as O

pytestmark = pytest.mark.gpu

FIRST, LAST = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def fp8_rows(n, d, g):
    x = torch.randn(n, d, generator=g).numpy()
    s = (np.abs(x).max(axis=1) / 448).astype(np.float32)
    c = F.e4m3_encode_array((x / s[:, None]).astype(np.float32))
    return torch.tensor(c).cuda(), torch.tensor(s).cuda(), F.bf16_round((F.E4M3_TABLE[c] * s.astype(np.float64)[:, None]).astype(np.float32))


class Window:
    """One sequence without entries: tokens at `positions` over a window buffer of `cap` rows from `pos0` on."""

    def __init__(self, positions, pos0, cap, W, d, Hq=5, seed=0):
        g = torch.Generator().manual_seed(seed)
        T = len(positions)
        self.positions, self.pos0, self.cap, self.W, self.d, self.Hq = positions, pos0, cap, W, d, Hq
        self.codes, self.scales, self.rows = fp8_rows(cap, d, g)
        self.Q = torch.randn(1, T, Hq, d, generator=g).bfloat16()
        self.page = torch.zeros(64 * d, dtype=torch.uint8, device="cuda")
        self.table, self.n, self.p0 = i32([[0]]), i32([0]), i32([pos0])
        self.dims = abi.Dims(B=1, Tq=T, d=d, r=64, Hq=Hq, Hi=8, Di=128, idx_dtype=abi.CSA2_BF16, K=4, W=W, max_pages=1, swa_cap=cap,
                             kv_format=abi.CSA2_KV_MXFP4)
        self.cache = abi.Cache(kv_codes=self.page.data_ptr(), kv_scales=self.page.data_ptr(), page_table=self.table.data_ptr(),
                               n_entries=self.n.data_ptr(), n_pages=1)
        self.win = abi.Window(codes=self.codes.data_ptr(), scales=self.scales.data_ptr(), pos0=self.p0.data_ptr())
        self.q_pos, self.idx, self.cnt = i32([positions]), i32(np.full((1, T, 4), -1)), i32(np.zeros((1, T)))
        self.O, self.lse = torch.full((1, T, Hq, d), 9.0, device="cuda"), torch.full((1, T, Hq), 9.0, device="cuda")

    def check(self):
        tau = 1.0 / np.sqrt(self.d)
        abi.csa2_sparse_attn(self.dims, self.cache, self.win, self.Q.cuda(), self.q_pos, self.idx, self.cnt, tau, self.O, self.lse)
        torch.cuda.synchronize()
        assert abi.csa2_get_status() == 0
        got, lse = self.O.double().cpu().numpy(), self.lse.double().cpu().numpy()
        for i, t in enumerate(self.positions):
            held = [p - self.pos0 for p in range(max(0, t - self.W + 1), t + 1) if 0 <= p - self.pos0 < self.cap]
            if not held:
                assert np.all(got[0, i] == 0) and np.all(np.isneginf(lse[0, i])), t
                continue
            o, z, mag, qk = O.attention(self.Q[0, i].double().numpy(), self.rows[held], tau)
            # a logit: d additions of at most 2^-23 of sum |q k| tau; P rounded to fp16: 2^-11, and 2^-25 of the
            # reference below its normal range; O's fp32 sums: 2^-16
            e = (self.d + 3) * 2.0 ** -23 * qk[:, None]
            tol = (2 * e + 2.0 ** -11 + 2.0 ** -16) * mag + len(held) * 2.0 ** -25 * np.abs(self.rows).max()
            assert np.all(np.abs(got[0, i] - o) <= tol), t
            assert np.all(np.abs(lse[0, i] - z) <= e[:, 0] + (np.abs(z) + 12) * 2.0 ** -20), t


@pytest.mark.parametrize("d", [512, 64])
@pytest.mark.parametrize("pos0", [0, -20, 7, FIRST, FIRST + 100, LAST - 30])
def test_tokens_before_the_first_position_see_nothing(pos0, d):
    Window([-1, -5, FIRST, FIRST + 1, FIRST + 15, FIRST + 16, 3, 1000, LAST], pos0, 40, 16, d).check()


@pytest.mark.parametrize("d", [512, 64])
@pytest.mark.parametrize("pos0", [LAST - 10, LAST - 39, LAST - 38, LAST])
def test_a_buffer_that_ends_behind_the_last_position(pos0, d):
    Window([LAST, LAST - 1, LAST - 12], pos0, 40, 16, d).check()


@pytest.mark.parametrize("d", [512, 64])
def test_a_tree_without_a_window_at_the_last_position(d):
    """W = 0: a drafted token sees no window row, its own and its ancestors' among them."""
    B, T, Hq = 1, 5, 3
    g = torch.Generator().manual_seed(d)
    codes, scales, _ = fp8_rows(T, d, g)
    ctx, parent = i32([LAST - 4]), i32([[-1, 0, 1, 2, 3]])
    q_pos, path = torch.empty(B, T, dtype=torch.int32, device="cuda"), torch.empty(B, T, T, dtype=torch.int32, device="cuda")
    dims = abi.Dims(B=B, Tq=T, d=d, r=64, Hq=Hq, Hi=8, Di=128, idx_dtype=abi.CSA2_BF16, K=4, W=0, max_pages=1, swa_cap=0,
                    kv_format=abi.CSA2_KV_MXFP4)
    abi.csa2_tree_plan(dims, parent, ctx, q_pos, path)
    page, table, n = torch.zeros(64 * d, dtype=torch.uint8, device="cuda"), i32([[0]]), i32([0])
    cache = abi.Cache(kv_codes=page.data_ptr(), kv_scales=page.data_ptr(), page_table=table.data_ptr(), n_entries=n.data_ptr(), n_pages=1)
    tree = abi.Tree(codes=codes.data_ptr(), scales=scales.data_ptr(), ctx_len=ctx.data_ptr(), path=path.data_ptr(), max_depth=T)
    Q = torch.randn(B, T, Hq, d, generator=g).bfloat16().cuda()
    out, lse = torch.full((B, T, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((B, T, Hq), 9.0, device="cuda")
    idx, cnt = i32(np.full((B, T, 4), -1)), i32(np.zeros((B, T)))
    abi.csa2_tree_attn(dims, cache, None, tree, Q, q_pos, idx, cnt, 0.1, out, lse)
    torch.cuda.synchronize()
    assert abi.csa2_get_status() == 0
    assert q_pos.tolist() == [[LAST - 4, LAST - 3, LAST - 2, LAST - 1, LAST]]
    assert bool((out == 0).all()) and bool(lse.isneginf().all())
