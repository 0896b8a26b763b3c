"""Drafted trees against oracle.step: positions and paths (exact), and attention with bounds from the operands.

Attention: fp16 operands are exact, so a logit is off by the fp32 accumulation alone: 512 (64) additions of at most
2^-23 of sum |q k| tau each, and three roundings of its scaling.  With that error e, weights are off by a factor of
1 +- 2 e; P's rounding to fp16 adds 2^-11, below 2^-14 of the reference 2^-25 of it per key; O's own sums 2^-16 and
its rounding to bf16 2^-8 of O.  lse is off by e, and log2 and exp2 by 2^-20 of what they return."""
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


def status():
    torch.cuda.synchronize()
    return abi.csa2_get_status()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def random_parents(r, B, T, live=None, chain=False):
    p = np.full((B, T), -2, dtype=np.int64)
    for b in range(B):
        for i in range(T if live is None else live[b]):
            p[b, i] = i - 1 if chain else max(-1, i - 1 - int(r.geometric(0.4)))
    return p


def plan(parent, ctx, depth):
    B, T = parent.shape
    q_pos, path = torch.full((B, T), -9, dtype=torch.int32, device="cuda"), torch.full((B, T, depth), -9, dtype=torch.int32, device="cuda")
    abi.csa2_tree_plan(abi.Dims(B=B, Tq=T), i32(parent), i32(ctx), q_pos, path)
    return q_pos, path


@pytest.mark.parametrize("B,T,depth", [(1, 1, 1), (3, 8, 8), (5, 61, 20), (2, 1024, 1024), (70, 33, 40)])
def test_plan(B, T, depth):
    r = np.random.RandomState(T)
    parent = random_parents(r, B, T, live=r.randint(0, T + 1, B))
    if T > 8:      # a place without a node in the middle, nobody's parent
        parent[0, :] = np.where(parent[0] == 3, -1, parent[0])
        parent[0, 3] = -2
    ctx = r.randint(0, 1 << 20, B)
    q_pos, path = plan(parent, ctx, depth)
    want, lines, bad_i, bad_c = O.tree_plan(parent, ctx, depth)
    bits = (abi.STATUS_BAD_INDEX if bad_i else 0) | (abi.STATUS_BAD_COUNT if bad_c else 0)
    assert status() == bits
    np.testing.assert_array_equal(q_pos.cpu().numpy(), want)
    np.testing.assert_array_equal(path.cpu().numpy(), lines)


@pytest.mark.parametrize("parent,ctx,depth", [
    ([[-1, 0, 2, 1]], [5], 4),             # its own parent
    ([[-1, 5, 0, 1]], [5], 4),             # a parent behind it
    ([[-1, -2, 1, 2]], [5], 4),            # children of no node
    ([[-1, 0, 1, 2]], [5], 3),             # too deep
    ([[-1, 0, 1, 2]], [-1], 4),
    ([[-1, 0, 1, 2]], [2 ** 31 - 3], 4),   # past the last position
    ([[-1000, -1, 1, -1]], [0], 2),
])
def test_plan_of_bad_trees(parent, ctx, depth):
    parent = np.array(parent)
    q_pos, path = plan(parent, ctx, depth)
    want, lines, bad_i, bad_c = O.tree_plan(parent, ctx, depth)
    assert status() == (abi.STATUS_BAD_INDEX if bad_i else 0) | (abi.STATUS_BAD_COUNT if bad_c else 0)
    np.testing.assert_array_equal(q_pos.cpu().numpy(), want)
    np.testing.assert_array_equal(path.cpu().numpy(), lines)


class Case:
    def __init__(self, seed, lens, T, Hq=64, K=64, W=128, d=512, fp8=False, cap=None, late=0, chain=False, live=None, few=False,
                 depth=None, rest=None, big=False):
        g, r = torch.Generator().manual_seed(seed), np.random.RandomState(seed)
        B = len(lens)
        self.T, self.Hq, self.K, self.W, self.d, self.fp8, self.lens = T, Hq, K, W, d, fp8, list(lens)
        per = [-(-n // 64) for n in lens]
        self.pages = sum(per) + 2
        perm = r.permutation(self.pages)
        self.table = np.full((B, max(max(per), 1)), -5)
        at = 0
        for b in range(B):
            self.table[b, :per[b]] = perm[at:at + per[b]]
            at += per[b]
        ns = self.pages * 64
        rows = torch.randn(ns, d, generator=g).numpy()
        if fp8:
            s = (np.abs(rows).max(axis=1) / 448).astype(np.float32)
            self.codes, self.scales = F.e4m3_encode_array(rows / s[:, None]), s
            self.rows = self.window_value(self.codes, s)
        else:
            self.codes, self.scales = F.mxfp4_pack(rows)
            self.rows = F.mxfp4_unpack(self.codes, self.scales)
        self.ctx = 4 * np.array(lens) + (r.randint(0, 4, B) if rest is None else rest)
        self.cap = W if cap is None else cap
        self.pos0 = self.ctx - self.cap + late          # late: the buffer misses the oldest rows of the window
        self.depth = T if depth is None else depth
        self.parent = random_parents(r, B, T, live, chain)
        self.win = self.fp8_rows(torch.randn(max(1, B * self.cap), d, generator=g), big, r)
        self.new = self.fp8_rows(torch.randn(B * T, d, generator=g), big, r)
        self.Q = torch.randn(B, T, Hq, d, generator=g).bfloat16()
        self.idx, self.cnt = np.full((B, T, K), -1), np.zeros((B, T), dtype=np.int64)
        for b in range(B):
            for i in range(T):
                n = min(K, lens[b]) if not few else int(r.randint(0, min(K, lens[b]) + 1))
                self.idx[b, i, :n] = np.sort(r.permutation(lens[b])[:n])
                self.cnt[b, i] = n
        self.tau = 1.0 / np.sqrt(d)

    @staticmethod
    def window_value(codes, s):
        return F.bf16_round((F.E4M3_TABLE[codes] * np.asarray(s, dtype=np.float64)[:, None]).astype(np.float32))

    def fp8_rows(self, x, big, r):
        x = x.numpy()
        if big:      # scales from 2^-60 to 2^30: outside fp16's range
            x = x * np.exp2(r.randint(-60, 30, len(x)))[:, None].astype(np.float32)
        s = (np.abs(x).max(axis=1) / 448).astype(np.float32)
        c = F.e4m3_encode_array((x / s[:, None]).astype(np.float32))
        return c, s, self.window_value(c, s)

    def upload(self):
        B, d = len(self.lens), self.d
        up = lambda a, t: torch.tensor(np.ascontiguousarray(a)).to(t).cuda()  # noqa: E731
        self.t = {"codes": up(self.codes, torch.uint8), "scales": up(self.scales, torch.float32 if self.fp8 else torch.uint8),
                  "table": i32(self.table), "n": i32(self.lens), "wc": up(self.win[0], torch.uint8), "ws": up(self.win[1], torch.float32),
                  "nc": up(self.new[0], torch.uint8), "ns": up(self.new[1], torch.float32), "pos0": i32(self.pos0), "ctx": i32(self.ctx),
                  "Q": self.Q.cuda(), "idx": i32(self.idx), "cnt": i32(self.cnt), "parent": i32(self.parent)}
        p = {k: v.data_ptr() for k, v in self.t.items()}
        self.q_pos = torch.full((B, self.T), -9, dtype=torch.int32, device="cuda")
        self.path = torch.full((B, self.T, self.depth), -9, dtype=torch.int32, device="cuda")
        self.dims = abi.Dims(B=B, Tq=self.T, d=d, r=64, Hq=self.Hq, Hi=8, Di=128, idx_dtype=abi.CSA2_BF16, K=self.K, W=self.W,
                             max_pages=self.table.shape[1], swa_cap=self.cap, kv_format=abi.CSA2_KV_FP8 if self.fp8 else abi.CSA2_KV_MXFP4)
        self.cache = abi.Cache(kv_codes=p["codes"], kv_scales=p["scales"], page_table=p["table"], n_entries=p["n"], n_pages=self.pages)
        self.window = abi.Window(codes=p["wc"], scales=p["ws"], pos0=p["pos0"]) if self.cap else None
        self.tree = abi.Tree(codes=p["nc"], scales=p["ns"], ctx_len=p["ctx"], path=self.path.data_ptr(), max_depth=self.depth)
        n = B * self.T * self.Hq
        self.O_all = torch.full((n * d + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
        self.O = self.O_all[:n * d].view(B, self.T, self.Hq, d)
        self.lse = torch.full((B, self.T, self.Hq), 3.0, device="cuda")
        return self

    def run(self, lse=True):
        abi.csa2_tree_plan(self.dims, self.t["parent"], self.t["ctx"], self.q_pos, self.path)
        abi.csa2_tree_attn(self.dims, self.cache, self.window, self.tree, self.t["Q"], self.q_pos, self.t["idx"], self.t["cnt"],
                           self.tau, self.O, self.lse if lse else None)

    def check(self, tokens=None, bad=()):
        B, T, d = len(self.lens), self.T, self.d
        want, lines, _, _ = O.tree_plan(self.parent, self.ctx, self.depth)
        np.testing.assert_array_equal(self.q_pos.cpu().numpy(), want)
        got, lse = self.O.double().cpu().numpy(), self.lse.double().cpu().numpy()
        win, new = self.win[2].reshape(-1, d), self.new[2].reshape(B, T, d)
        Q = self.Q.double().numpy()
        for b, i in tokens or [(b, i) for b in range(B) for i in range(T)]:
            t = want[b, i]
            if t < 0:
                assert np.all(got[b, i] == 0) and np.all(np.isneginf(lse[b, i]))
                continue
            line = [n for n in lines[b, i] if n >= 0]
            j = self.idx[b, i, :self.cnt[b, i]]
            j = np.array([x for x in j if x < min(self.lens[b], (t + 1) // 4) and (b, x // 64) not in bad], dtype=np.int64)
            page = self.table[b, j // 64]
            old, mine = O.tree_window(t, self.W, self.ctx[b], self.pos0[b], self.cap, line)
            keys = np.concatenate([self.rows[page * 64 + j % 64], win[b * self.cap + np.array(old, dtype=np.int64)],
                                   new[b, np.array(mine, dtype=np.int64)]])
            ro, rl, mag, qk = O.attention(Q[b, i], keys, self.tau)
            if len(keys) == 0:
                assert np.all(got[b, i] == 0) and np.all(np.isneginf(lse[b, i]))
                continue
            e = (d + 3) * 2.0 ** -23 * qk[:, None]
            top = np.abs(keys).max(axis=0)[None, :]
            # below 2^-14 of the reference, which is at most the maximum, a weight's step is 2^-25 of it
            tol = (2 * e + 2.0 ** -11 + 2.0 ** -16) * mag + len(keys) * 2.0 ** -25 * top
            tol += (np.abs(ro) + tol) * 2.0 ** -8
            err = np.abs(got[b, i] - ro)
            assert np.all(err <= tol), (b, i, float((err / tol).max()))
            assert np.all(np.abs(lse[b, i] - rl) <= e[:, 0] + (np.abs(rl) + 12) * 2.0 ** -20), (b, i)
        assert bool((self.O_all[self.O.numel():] == 3).all())


@pytest.mark.parametrize("kw", [
    dict(lens=[300], T=1),                                               # a single token
    dict(lens=[0], T=1, rest=[0], K=1),                                  # the first token of all
    dict(lens=[1, 0, 40], T=5, K=16),
    dict(lens=[500, 70], T=8, K=128, few=True),
    dict(lens=[300] * 3, T=61, K=64, live=[61, 1, 0]),                   # padded trees, one without a node
    dict(lens=[257, 1000], T=7, Hq=40, K=200, W=200),
    dict(lens=[600], T=9, Hq=128, K=512),
    dict(lens=[90], T=33, Hq=1, K=17, W=16),                             # a window shorter than the tree is deep
    dict(lens=[90], T=40, Hq=3, K=17, W=7, chain=True),
    dict(lens=[100, 300], T=6, W=0, K=64),                               # no window: entries alone
    dict(lens=[100, 300], T=6, W=64, cap=0, K=64),                       # no committed rows: ancestors alone
    dict(lens=[100, 300], T=6, W=64, late=30, K=64),                     # the buffer begins inside the window
    dict(lens=[100, 300], T=6, W=64, cap=80, late=25, K=64),             # and ends behind the committed text
    dict(lens=[100, 300], T=6, W=64, cap=40, late=-10, K=64),            # and ends before it
    dict(lens=[3, 5], T=12, W=128, K=4),                                 # the window reaches before the first token
    dict(lens=[700, 40, 3], T=8, fp8=True, K=300),
    dict(lens=[700, 40, 3], T=6, fp8=True, K=64, big=True),
    dict(lens=[400], T=10, K=64, big=True),
    dict(lens=[3000], T=2, K=2048, W=1024),                              # the longest key list
], ids=lambda k: "-".join(f"{a}{str(v).replace(' ', '')}" for a, v in k.items()))
def test_attention(kw):
    c = Case(len(str(kw)), **kw).upload()
    c.run()
    assert status() == 0
    c.check()


@pytest.mark.parametrize("kw", [dict(lens=[15, 200], T=2, K=2048, W=5), dict(lens=[700], T=3, K=1024, W=3), dict(lens=[2000, 0], T=1, K=2048, W=9),
                                dict(lens=[512], T=8, K=512), dict(lens=[511], T=4, K=512), dict(lens=[900, 33], T=5, K=1000, W=100, few=True),
                                dict(lens=[600], T=2, K=600, W=1, fp8=True)])
def test_shares_of_a_split_token(kw):
    """Few tokens: the keys that are there go over several CTAs, whatever K and W would allow."""
    c = Case(24, **kw).upload()
    c.run()
    assert status() == 0
    c.check()


@pytest.mark.parametrize("kw", [dict(lens=[300, 20], T=9, K=64, Hq=7), dict(lens=[60], T=20, K=16, W=5, Hq=4, chain=True),
                                dict(lens=[100, 3], T=6, W=64, cap=40, late=-10, K=64, Hq=17), dict(lens=[90], T=6, K=20, W=0),
                                dict(lens=[90, 4], T=6, K=20, cap=0, live=[6, 2]), dict(lens=[90], T=6, K=20, big=True)])
def test_attention_d64(kw):
    c = Case(3, d=64, **kw).upload()
    c.run()
    assert status() == 0
    c.check()


@pytest.mark.parametrize("d", [512, 64])
def test_the_last_positions(d):
    """Trees that end at position 2^31 - 1, the buffer's rows in front of them."""
    c = Case(19, lens=[50, 70], T=5, K=20, W=30, d=d, chain=True)
    c.ctx = np.array([2 ** 31 - 5, 2 ** 31 - 40])
    c.pos0 = c.ctx - c.cap
    c.upload()
    c.run()
    assert status() == 0
    c.check()


def test_two_streams_at_once():
    cs = [Case(20 + k, lens=[300 + k, 40], T=6, K=64).upload() for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                c.run()
    assert status() == 0
    for c in cs:
        c.check()


def test_many_tokens():
    """More tokens than SMs: one CTA per token."""
    c = Case(11, lens=[1000 + 37 * b for b in range(24)], T=8, K=512).upload()
    c.run()
    assert status() == 0
    c.check(tokens=[(b, i) for b in (0, 5, 23) for i in range(8)])


@pytest.mark.parametrize("d", [512, 64])
def test_a_chain_equals_sparse_attention(d):
    """A tree that is a chain is what csa2_sparse_attn does over a window that holds the chain's rows."""
    c = Case(12, lens=[333, 80], T=6, K=64, W=50, chain=True, d=d).upload()
    c.run()
    B, T = 2, 6
    cap = c.cap + T
    codes = torch.cat([c.t["wc"].view(B, c.cap, d), c.t["nc"].view(B, T, d)], dim=1).contiguous()
    scales = torch.cat([c.t["ws"].view(B, c.cap), c.t["ns"].view(B, T)], dim=1).contiguous()
    win = abi.Window(codes=codes.data_ptr(), scales=scales.data_ptr(), pos0=c.t["pos0"].data_ptr())
    dims = abi.Dims.from_buffer_copy(c.dims)
    dims.swa_cap = cap
    Of, lf = torch.empty(B, T, c.Hq, d, device="cuda"), torch.empty(B, T, c.Hq, device="cuda")
    abi.csa2_sparse_attn(dims, c.cache, win, c.t["Q"], c.q_pos, c.t["idx"], c.t["cnt"], c.tau, Of, lf)
    assert status() == 0
    assert torch.equal(Of.bfloat16(), c.O) and torch.equal(lf, c.lse)


def test_no_lse():
    c = Case(13, lens=[200], T=4).upload()
    c.run()
    first = c.O.clone()
    c.O.fill_(1)
    c.run(lse=False)
    assert status() == 0 and torch.equal(first, c.O)


def test_bad_pages_indices_and_counts():
    c = Case(14, lens=[400, 200], T=5, K=64)
    c.table[0, 2] = c.pages
    c.upload()
    c.run()
    assert status() == abi.STATUS_BAD_PAGE
    c.check(bad={(0, 2)})
    c = Case(15, lens=[400, 200], T=5, K=64)
    c.idx[1, 2, 3], c.idx[0, 1, 0] = 10 ** 9, -4          # entries that are not there are left out
    c.upload()
    c.run()
    assert status() == abi.STATUS_BAD_INDEX
    c.idx[1, 2, 3] = c.idx[0, 1, 0] = 10 ** 9
    c.check()


def test_broken_paths_leave_their_keys_out():
    c = Case(16, lens=[200], T=6, K=32, chain=True).upload()
    c.run()
    whole = c.O.clone()
    c.path[0, 4, 1], c.path[0, 5, 2] = 6, -3
    abi.csa2_tree_attn(c.dims, c.cache, c.window, c.tree, c.t["Q"], c.q_pos, c.t["idx"], c.t["cnt"], c.tau, c.O, c.lse)
    assert status() == abi.STATUS_BAD_INDEX
    assert torch.equal(whole[0, :4], c.O[0, :4]) and not torch.equal(whole[0, 4], c.O[0, 4])
    assert bool(c.O.isfinite().all())


def test_nan_in_a_sibling_reaches_nobody_else():
    c = Case(17, lens=[200], T=4, K=32)
    c.parent[0] = [-1, -1, 0, 1]                          # two branches
    c.upload()
    c.run()
    whole = c.O.clone()
    c.t["ns"][1] = float("nan")                           # node 1's row: seen by 1 and 3
    c.run()
    assert status() == 0
    assert torch.equal(whole[0, 0], c.O[0, 0]) and torch.equal(whole[0, 2], c.O[0, 2])


def test_same_bits_and_replayed():
    c = Case(18, lens=[900, 50, 333], T=8, K=256).upload()
    c.run()
    first, lse = c.O.clone(), c.lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.O.fill_(0)
    graph.replay()
    assert status() == 0
    assert torch.equal(first, c.O) and torch.equal(lse, c.lse)
    c.parent = random_parents(np.random.RandomState(5), 3, 8)
    c.t["parent"].copy_(i32(c.parent))
    graph.replay()
    assert status() == 0
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[700, 90], [300 + b for b in range(40)]])
def test_rows_that_start_on_16_bytes_only(lens, fp8):
    """Codes 16 bytes behind a 32-byte boundary give the same bits."""
    c = Case(23, lens=lens, T=5, K=256, fp8=fp8, Hq=8).upload()
    c.run()
    first, lse = c.O.clone(), c.lse.clone()
    moved = {}
    for k in ("codes", "wc", "nc"):
        t = c.t[k].view(-1)
        buffer = torch.full((t.numel() + 48,), 0x55, dtype=torch.uint8, device="cuda")
        at = (16 - buffer.data_ptr()) % 32
        moved[k] = buffer[at:at + t.numel()]
        moved[k].copy_(t)
        assert moved[k].data_ptr() % 32 == 16
        c.t[k].fill_(0)
    c.cache.kv_codes, c.window.codes, c.tree.codes = (moved[k].data_ptr() for k in ("codes", "wc", "nc"))
    c.O.fill_(0)
    c.run()
    assert status() == 0
    assert torch.equal(first, c.O) and torch.equal(lse, c.lse)
