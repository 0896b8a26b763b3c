"""The query side of a step with drafted tokens, one operator after the other as a program runs them: pages for the
committed tokens, FP8 projection of the drafted tokens' hidden states, rotation at tree positions, selection by the
indexer, attention of the tree, rotation back, and pages given back when drafts are rejected."""
import math

import numpy as np
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build
from oracle import formats as F
from oracle import step as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Step:
    """Two sequences of a pool, T drafted tokens each; every buffer made once."""

    def __init__(self, T=6, Hq=16, H=256, K=32, W=64):
        g = torch.Generator().manual_seed(0)
        self.B, self.T, self.Hq, self.H, self.K, self.W, self.d, self.r = 2, T, Hq, H, K, W, 512, 64
        B, d = 2, 512
        self.n_pages, self.max_pages = 40, 16
        self.len0 = np.array([1501, 403])
        self.held = i32([0, 0])
        self.table = torch.zeros(B, self.max_pages, dtype=torch.int32, device="cuda")
        self.free, self.n_free = i32(np.random.RandomState(0).permutation(self.n_pages)), i32([self.n_pages])
        self.seq_len = i32([0, 0])
        self.n_entries, self.first_entry, self.granted = i32([0, 0]), i32([0, 0]), i32([0, 0])
        self.dims = abi.Dims(B=B, Tq=T, d=d, r=self.r, Hq=Hq, Hi=8, Di=128, idx_dtype=abi.CSA2_BF16, K=K, W=W,
                             max_pages=self.max_pages, n_pool_blocks=0, pool_block=8, swa_cap=W, kv_format=abi.CSA2_KV_MXFP4)
        self.pool = abi.PagePool(page_table=self.table.data_ptr(), held=self.held.data_ptr(), free_pages=self.free.data_ptr(),
                                 n_free=self.n_free.data_ptr(), n_pages=self.n_pages)
        self.plan_ws = torch.empty(abi.csa2_page_plan_workspace_size(self.dims), dtype=torch.uint8, device="cuda")
        ns = self.n_pages * 64
        rows = torch.randn(ns, d, generator=g)
        self.codes, self.scales = torch.empty(ns, d // 2, dtype=torch.uint8, device="cuda"), torch.empty(ns, d // 16, dtype=torch.uint8, device="cuda")
        abi.csa2_pack_mxfp4_f32(rows.cuda(), self.codes, self.scales)
        self.idx_k = torch.randn(ns, 128, generator=g).bfloat16().cuda()
        self.cache = abi.Cache(kv_codes=self.codes.data_ptr(), kv_scales=self.scales.data_ptr(), idx_k=self.idx_k.data_ptr(),
                               page_table=self.table.data_ptr(), n_entries=self.n_entries.data_ptr(), n_pages=self.n_pages)
        fp8 = lambda n: (torch.empty(n, d, dtype=torch.uint8, device="cuda"), torch.empty(n, device="cuda"))  # noqa: E731
        self.wc, self.wsc = fp8(B * W)
        abi.csa2_pack_swa_fp8(torch.randn(B * W, d, generator=g).cuda(), self.wc, self.wsc)
        self.nc, self.nsc = fp8(B * T)
        self.pos0 = i32(self.len0 - W)
        self.window = abi.Window(codes=self.wc.data_ptr(), scales=self.wsc.data_ptr(), pos0=self.pos0.data_ptr())
        self.parent = i32([[-1, 0, 0, 1, -1, 4][:T]] * B)
        self.path = torch.empty(B, T, T, dtype=torch.int32, device="cuda")
        self.q_pos = torch.empty(B, T, dtype=torch.int32, device="cuda")
        self.tree = abi.Tree(codes=self.nc.data_ptr(), scales=self.nsc.data_ptr(), ctx_len=self.seq_len.data_ptr(),
                             path=self.path.data_ptr(), max_depth=T)
        n_out = Hq * d + 8 * 128                              # queries and indexer queries from one product
        W0 = (0.05 * torch.randn(n_out, H, generator=g)).numpy()
        wb = np.abs(W0.reshape(-1, 128, H // 128, 128)).max(axis=(1, 3)) / 448
        self.w_scales = torch.tensor(wb.astype(np.float32)).cuda()
        q = W0.reshape(-1, 128, H // 128, 128) / wb.astype(np.float32)[:, None, :, None]
        self.w_codes = torch.tensor(F.e4m3_encode_array(q.reshape(n_out, H))).cuda()
        self.hidden = torch.randn(B * T, H, generator=g).bfloat16().cuda()
        self.latent = torch.randn(B * T, d, generator=g).cuda()
        self.h_codes, self.h_scales = torch.empty(B * T, H, dtype=torch.uint8, device="cuda"), torch.empty(B * T, H // 128, device="cuda")
        self.proj = torch.empty(B * T, n_out, dtype=torch.bfloat16, device="cuda")
        self.mm_ws = torch.empty(max(16, abi.csa2_matmul_fp8_workspace_size(B * T, n_out, H)), dtype=torch.uint8, device="cuda")
        self.rope = torch.empty(self.r // 2, dtype=torch.int64, device="cuda")
        abi.csa2_rope_table(abi.RopeSpec(scaling=abi.ROPE_PLAIN, base=10000.0, factor=1.0), self.r, self.rope)
        self.Q = torch.empty(B * T, Hq, d, dtype=torch.bfloat16, device="cuda")
        self.idx_q = torch.empty(B * T, 8, 128, dtype=torch.bfloat16, device="cuda")
        self.idx_w = torch.randn(B, T, 8, generator=g).cuda()
        self.idx, self.cnt = torch.empty(B, T, K, dtype=torch.int32, device="cuda"), torch.empty(B, T, dtype=torch.int32, device="cuda")
        self.topk_ws = torch.empty(abi.csa2_index_topk_workspace_size(self.dims, 1024), dtype=torch.uint8, device="cuda")
        self.O, self.lse = torch.empty(B, T, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, T, Hq, device="cuda")

    def pages(self, n_new):
        abi.csa2_page_plan(self.dims, self.pool, self.seq_len, n_new, self.seq_len, self.n_entries, self.first_entry, self.plan_ws,
                           granted=self.granted)

    def run(self):
        abi.csa2_tree_plan(self.dims, self.parent, self.seq_len, self.q_pos, self.path)
        abi.csa2_pack_swa_fp8(self.latent, self.nc, self.nsc)
        abi.csa2_pack_fp8_blocks(self.hidden, self.h_codes, self.h_scales)
        abi.csa2_matmul_fp8(self.h_codes, self.h_scales, self.w_codes, self.w_scales, self.proj, self.mm_ws)
        n = self.Hq * self.d
        pos = self.q_pos.view(-1)
        abi.csa2_rope(self.proj[:, :n].unflatten(1, (self.Hq, self.d)), self.Q, pos, self.rope, start=self.d - self.r)
        abi.csa2_rope(self.proj[:, n:].unflatten(1, (8, 128)), self.idx_q, pos, self.rope, start=64)
        abi.csa2_index_topk(self.dims, self.cache, self.idx_q, self.idx_w, self.q_pos, self.idx, self.cnt, 1024, self.topk_ws)
        abi.csa2_tree_attn(self.dims, self.cache, self.window, self.tree, self.Q, self.q_pos, self.idx, self.cnt,
                           1.0 / math.sqrt(self.d), self.O, self.lse)
        abi.csa2_rope(self.O.view(-1, self.Hq, self.d), self.O.view(-1, self.Hq, self.d), pos, self.rope, start=self.d - self.r,
                      inverse=True)


def check(s):
    """Every operator's output against the oracle of its own inputs."""
    B, T, Hq, d, r = s.B, s.T, s.Hq, s.d, s.r
    ctx = s.seq_len.cpu().numpy()
    q_pos, lines, bi, bc = O.tree_plan(s.parent.cpu().numpy(), ctx, T)
    assert not bi and not bc
    np.testing.assert_array_equal(s.q_pos.cpu().numpy(), q_pos)
    hc, hs = O.pack_fp8_blocks(s.hidden.float().cpu().numpy())
    np.testing.assert_array_equal(s.h_codes.cpu().numpy(), hc)
    C, mag = O.matmul_fp8(hc, hs, s.w_codes.cpu().numpy(), s.w_scales.cpu().numpy())
    proj = s.proj.double().cpu().numpy()
    tol = (130 + hs.shape[1]) * 2.0 ** -23 * mag
    assert np.all(np.abs(proj - C) <= tol + (np.abs(C) + tol) * 2.0 ** -8)
    theta = O.rope_frequencies(r)
    x = proj[:, :Hq * d].reshape(-1, Hq, d)
    Q = s.Q.double().cpu().numpy()
    ref = O.rope(x, q_pos.reshape(-1), theta, d - r)
    tol = 2.0 ** -20 * np.abs(x).max(axis=-1, keepdims=True)
    assert np.all(np.abs(Q - ref) <= tol + (np.abs(ref) + tol) * 2.0 ** -8)
    # attention over the GPU's own selection (whose entries must be distinct and visible)
    idx, cnt, table = s.idx.cpu().numpy(), s.cnt.cpu().numpy(), s.table.cpu().numpy()
    rows = F.mxfp4_unpack(s.codes.cpu().numpy(), s.scales.cpu().numpy())
    value = lambda c, w: F.bf16_round((F.E4M3_TABLE[c.cpu().numpy()] * w.double().cpu().numpy()[:, None]).astype(np.float32))  # noqa: E731
    win, new = value(s.wc, s.wsc), value(s.nc, s.nsc)
    n_ent, pos0 = s.n_entries.cpu().numpy(), s.pos0.cpu().numpy()
    got = s.O.double().cpu().numpy()
    for b in range(B):
        assert n_ent[b] == ctx[b] // 4
        for i in range(T):
            t = q_pos[b, i]
            assert cnt[b, i] == min(s.K, n_ent[b], (t + 1) // 4)
            j = idx[b, i, :cnt[b, i]]
            assert len(set(j.tolist())) == cnt[b, i] and j.max() < n_ent[b]
            old, mine = O.tree_window(t, s.W, ctx[b], pos0[b], s.W, [n for n in lines[b, i] if n >= 0])
            keys = np.concatenate([rows[table[b, j // 64] * 64 + j % 64], win[b * s.W + np.array(old)], new[b * T + np.array(mine)]])
            o, _, mag, qk = O.attention(Q[b * T + i], keys, 1.0 / math.sqrt(d))
            o = O.rope(o[None], [t], theta, d - r, inverse=True)[0]
            e = 515 * 2.0 ** -23 * qk[:, None]
            tol = (2 * e + 2.0 ** -11 + 2.0 ** -16) * mag + len(keys) * 2.0 ** -25 * np.abs(keys).max()
            tol += (np.abs(o) + tol) * 2.0 ** -8
            # the rotation back mixes two channels, each rounded to bf16 before and after
            tol[:, d - r:] = (tol[:, d - r:] + np.roll(tol[:, d - r:], r // 2, axis=1)) * 1.01 + 2.0 ** -8 * np.abs(o[:, d - r:]) + \
                2.0 ** -8 * np.abs(np.roll(o[:, d - r:], r // 2, axis=1))
            assert np.all(np.abs(got[b, i] - o) <= tol), (b, i)


@pytest.mark.parametrize("captured", [False, True])
def test_a_step_with_drafted_tokens(captured):
    s = Step()
    s.pages(i32(s.len0))
    if captured:
        s.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.run()
        s.O.zero_()
        graph.replay()
    else:
        s.run()
    torch.cuda.synchronize()
    assert abi.csa2_get_status() == 0
    assert s.granted.tolist() == [1, 1] and s.seq_len.tolist() == s.len0.tolist()
    assert s.held.tolist() == [-(-(n // 4) // 64) for n in s.len0.tolist()]
    check(s)
    # three drafts of the first sequence are accepted, the second ends: its pages come back
    s.pages(i32([3, -403]))
    torch.cuda.synchronize()
    assert abi.csa2_get_status() == 0
    assert s.seq_len.tolist() == [1504, 0] and s.n_entries.tolist() == [376, 0] and s.first_entry.tolist() == [375, 0]
    assert int(s.n_free[0]) == s.n_pages - 6 and s.held.tolist() == [6, 0]
