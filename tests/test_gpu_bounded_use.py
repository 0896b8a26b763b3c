"""A bounded cache as it is used: compress, attend, weigh, evict, compress again, with the other calls beside
them; captured graphs, other streams, calls that overlap, tiles cut into slabs."""
import numpy as np
import pytest
import torch

from bounded_case import Case
from compressed_sparse_attention_05_gb300 import abi, build
from oracle import bounded as OB

pytestmark = pytest.mark.gpu

H, DI, EPS, BASE = 128, 128, 1e-6, 1e4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def status():
    torch.cuda.synchronize()
    return abi.csa2_get_status()


class Cache(Case):
    """A Case whose rows come from csa2_compress_pack_bounded and whose host copies follow the device's."""

    def __init__(self, seed, B=2, room=192, **kw):
        super().__init__(seed=seed, B=B, lens=(room,), window=False, scrambled=True, shift=[0], **kw)
        g = torch.Generator().manual_seed(seed + 1)
        rnd = lambda *s: (torch.randn(*s, generator=g) / (4 * H) ** 0.5).to(torch.bfloat16).cuda()  # noqa: E731
        self.W_c, self.W_i = rnd(self.d, 4 * H), rnd(DI, 4 * H)
        self.gamma = torch.ones(self.d, device="cuda")
        self.g = g
        ns = self.n_pages * 64
        self.idx_k = torch.zeros(ns, DI, dtype=torch.bfloat16, device="cuda")
        self.weight = torch.full((ns,), -3.0, device="cuda")
        self.t["pos"].fill_(-999)
        self.t["n"].zero_()
        self.lens = [0] * B
        self.page_slots = [self.table[b, np.arange(room) // 64].astype(np.int64) * 64 + np.arange(room) % 64
                           for b in range(B)]
        self.room = room

    def structs(self):
        cache, bounded, win, mods = super().structs()
        cache.idx_k = self.idx_k.data_ptr()
        bounded.weight = self.weight.data_ptr()
        return cache, bounded, win, mods

    def dims(self, **kw):
        dm = super().dims()
        dm.r, dm.Hi, dm.Di, dm.K = 64, 8, DI, 256
        for k, v in kw.items():
            setattr(dm, k, v)
        return dm

    def compress(self, entries, hidden=None):
        """Appends `entries` entries to every sequence; returns the hidden rows."""
        if hidden is None:
            hidden = torch.randn(self.B, 4 * entries, H, generator=self.g).to(torch.bfloat16).cuda()
        cache, bounded, _, _ = self.structs()
        ws = torch.empty(max(16, abi.lib().csa2_compress_workspace_size(self.B, 4 * entries, H, self.d, DI)),
                         dtype=torch.uint8, device="cuda")
        abi.csa2_compress_pack_bounded(hidden, self.W_c, self.gamma, EPS, BASE, self.W_i, self.t["n"], self.dims(),
                                       cache, bounded, ws)
        torch.cuda.synchronize()
        self.t["n"] += entries
        return hidden

    def evict(self, keep, sinks, recent, ws=None, stream=None):
        cache, bounded, _, _ = self.structs()
        if ws is None:
            ws = torch.full((abi.csa2_evict_workspace_size(self.dims(), self.room),), 0xFF, dtype=torch.uint8,
                            device="cuda")
        abi.csa2_evict(self.dims(), cache, bounded, self.t["n"], keep, sinks, recent, self.room, ws, stream=stream)

    def pull(self):
        """Host copies of the device's state; the query is the newest token of each sequence."""
        torch.cuda.synchronize()
        self.codes, self.scales = self.t["codes"].cpu(), self.t["scales"].cpu()
        self.entry_pos = self.t["pos"].cpu()
        self.lens, self.shift = self.t["n"].tolist(), self.t["shift"].tolist()
        self.slots = [s[:n] for s, n in zip(self.page_slots, self.lens)]
        self.max_entries = self.room

    def ask(self):
        """New queries, those of the newest token of each sequence."""
        self.pull()
        self.q_pos = np.array([[4 * (self.lens[b] + self.shift[b]) - 1] for b in range(self.B)])
        self.Q = torch.randn(self.B, 1, self.Hq, self.d, generator=self.g).to(torch.bfloat16)
        self.t["Q"] = self.Q.cuda()
        self.t["q_pos"] = torch.tensor(self.q_pos, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("shift", [(0, 0), (37, 5)], ids=["unshifted", "shifted"])
def test_compress_writes_the_rows_of_the_plain_call(shift):
    """Entry first + i of a bounded cache has the bytes that csa2_compress_pack writes at first + shift + i."""
    c = Cache(1)
    c.t["shift"].copy_(torch.tensor(shift, dtype=torch.int32))
    first = [10, 64]
    c.t["n"].copy_(torch.tensor(first, dtype=torch.int32))
    before = [c.t["codes"].clone(), c.t["scales"].clone(), c.idx_k.clone(), c.t["pos"].clone(), c.weight.clone()]
    n = 50
    hidden = c.compress(n)
    assert status() == 0
    # the plain call, into another pool with pages in order
    pages = 4
    table = torch.arange(2 * pages, dtype=torch.int32, device="cuda").reshape(2, pages)
    ns = 2 * pages * 64
    codes, scales = (torch.zeros(ns, w, dtype=torch.uint8, device="cuda") for w in (256, 32))
    keys = torch.zeros(ns, DI, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([f + s for f, s in zip(first, shift)], dtype=torch.int32, device="cuda")
    cache = abi.Cache(kv_codes=codes.data_ptr(), kv_scales=scales.data_ptr(), idx_k=keys.data_ptr(),
                      page_table=table.data_ptr(), n_entries=at.data_ptr(), n_pages=2 * pages)
    ws = torch.empty(max(16, abi.lib().csa2_compress_workspace_size(2, 4 * n, H, 512, DI)), dtype=torch.uint8, device="cuda")
    abi.csa2_compress_pack(hidden, c.W_c, c.gamma, EPS, BASE, c.W_i, at, c.dims(max_pages=pages), cache, ws)
    assert status() == 0
    for b in range(2):
        mine = torch.from_numpy(c.page_slots[b][first[b]:first[b] + n]).cuda()
        his = torch.arange(n, device="cuda") + b * pages * 64 + first[b] + shift[b]
        assert torch.equal(c.t["codes"][mine], codes[his]) and torch.equal(c.t["scales"][mine], scales[his])
        assert torch.equal(c.idx_k[mine].view(torch.int16), keys[his].view(torch.int16))
        assert c.t["pos"][mine].tolist() == [4 * (first[b] + shift[b] + i) + 3 for i in range(n)]
        assert not c.weight[mine].any()
    rest = torch.ones(c.n_pages * 64, dtype=torch.bool, device="cuda")
    for b in range(2):
        rest[torch.from_numpy(c.page_slots[b][first[b]:first[b] + n]).cuda()] = False
    for now, old in zip([c.t["codes"], c.t["scales"], c.idx_k.view(torch.int16), c.t["pos"], c.weight],
                        [before[0], before[1], before[2].view(torch.int16), before[3], before[4]]):
        assert torch.equal(now[rest], old[rest])


def test_a_cache_in_use():
    """Prompt, then rounds of decode, weights, eviction and new entries; every stage against the oracle, and the
    sparse path over the same cache against the dense one."""
    c = Cache(2)
    c.compress(150)
    for keep in (120, 130, 64):
        c.ask()
        c.attend()
        assert status() == 0
        c.check_attention()
        before = c.weight.clone()
        c.weigh(c.lse, c.weight, c.weight, decay=0.9)
        assert status() == 0
        c.check_weights(c.lse, before, c.weight, decay=0.9)
        _sparse_agrees(c)
        c.pull()
        w, want = c.weight.cpu(), []
        for b in range(c.B):
            s = c.slots[b]
            if c.lens[b] > keep:
                holes, movers = OB.evict(w[s].numpy(), c.entry_pos[s].numpy(), c.shift[b], keep, 4, 16)
                order = np.arange(c.lens[b])
                order[holes] = movers
                want.append((s[order[:keep]], c.shift[b] + c.lens[b] - keep, keep))
            else:
                want.append((s, c.shift[b], c.lens[b]))
        old = [t.clone() for t in (c.t["codes"], c.t["scales"], c.idx_k.view(torch.int16), c.t["pos"], c.weight)]
        c.evict(keep, 4, 16)
        assert status() == 0
        c.pull()
        for b, (src, shift, n) in enumerate(want):
            assert (c.shift[b], c.lens[b]) == (shift, n)
            now = (c.t["codes"], c.t["scales"], c.idx_k.view(torch.int16), c.t["pos"], c.weight)
            for a, o in zip(now, old):
                assert torch.equal(a[torch.from_numpy(c.slots[b]).cuda()], o[torch.from_numpy(src).cuda()])
        c.compress(30)
        assert status() == 0
    c.ask()
    c.attend()
    c.check_attention()


def _sparse_agrees(c):
    """Top-K of everything and the sparse call, with q_pos less 4 shift, see what the dense call sees."""
    cache, _, _, _ = c.structs()
    n, B = max(c.lens), c.B
    dm = c.dims(swa_cap=1, W=1)
    local = torch.tensor(c.q_pos - 4 * np.array(c.shift)[:, None], dtype=torch.int32, device="cuda")
    idx = torch.full((B, 1, dm.K), -7, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    iq = torch.randn(B, 1, 8, DI, generator=c.g).to(torch.bfloat16).cuda()
    w = torch.ones(B, 1, 8, device="cuda")
    ws = torch.empty(abi.csa2_index_topk_workspace_size(dm, n), dtype=torch.uint8, device="cuda")
    abi.csa2_index_topk(dm, cache, iq, w, local, idx, cnt, n, ws)
    assert status() == 0
    assert cnt.flatten().tolist() == c.lens
    for b in range(B):
        assert sorted(idx[b, 0, :c.lens[b]].tolist()) == list(range(c.lens[b]))
    # the sparse call needs a window: one row of zeros, whose logit is 0
    codes = torch.zeros(B, 1, 512, dtype=torch.uint8, device="cuda")
    scales = torch.ones(B, 1, device="cuda")
    pos0 = local[:, 0].clone()
    win = abi.Window(codes=codes.data_ptr(), scales=scales.data_ptr(), pos0=pos0.data_ptr())
    O, lse = torch.empty(B, 1, 64, 512, device="cuda"), torch.empty(B, 1, 64, device="cuda")
    abi.csa2_sparse_attn(dm, cache, win, c.t["Q"], local, idx, cnt, c.tau, O, lse)
    assert status() == 0
    # the sparse sums are the dense ones plus exp(0)
    z = c.lse.double()
    z2 = torch.logaddexp(z, torch.zeros_like(z))
    # Each kernel's lse is off by at most 2^-20 mag + 2^-21 (|l| + mag) + 2^-20 + 2^-23 |z|, mag the sum of
    # |q| |k| tau over the channels: below 512 * 0.64 * 1.1 / sqrt(512) < 16.5 on average, and 25 bounds it.
    e = 2.0 ** -20 * 25 + 2.0 ** -21 * 50 + 2.0 ** -20 + 2.0 ** -23 * 50
    assert (lse.double() - z2).abs().max() < 2 * e
    want = c.O.double() * torch.exp(z - z2)[..., None]
    # Each kernel's O: P rounded to fp16 and two logit errors, times |v|; the dense one is rounded to bf16.
    v = max(float(np.abs(c.keys(b)[0]).max()) for b in range(B))
    assert (O.double() - want).abs().max() < 2.0 ** -8 * c.O.abs().max() + 2 * v * (2.0 ** -11 + 2 * e)


def _graph_case():
    c = Case(seed=21, B=3, Tq=2, lens=(700, 90, 1300), cap=20.0, slopes=[0.01])
    ws = torch.empty(max(16, abi.csa2_dense_attn_workspace_size(c.dims(), c.max_entries),
                         abi.csa2_entry_weights_workspace_size(c.dims(), c.max_entries)), dtype=torch.uint8, device="cuda")
    w = torch.zeros(c.n_pages * 64, device="cuda")
    return c, ws, w


def test_captured_calls_on_a_side_stream_share_a_workspace():
    """Two graphs over one workspace, replayed in turn with new lengths and queries between the replays."""
    c, ws, w = _graph_case()
    s = torch.cuda.Stream()

    def step():
        c.attend(ws=ws, stream=s)
        c.weigh(c.lse, None, w, ws=ws, stream=s)

    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        graphs.append(g)
    rng = torch.Generator().manual_seed(3)
    all_slots = c.slots
    for k in range(4):
        c.Q = torch.randn(c.Q.shape, generator=rng).to(torch.bfloat16)
        c.t["Q"].copy_(c.Q)
        n = [[700, 90, 1300], [64, 0, 1], [699, 65, 128], [1, 90, 1000]][k]
        c.lens = n
        c.slots = [x[:m] for x, m in zip(all_slots, n)]
        c.t["n"].copy_(torch.tensor(n, dtype=torch.int32))
        c.O.fill_(float("nan"))
        w.fill_(-1.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[k & 1].replay()
        torch.cuda.synchronize()
        assert status() == 0
        c.check_attention()
        c.check_weights(c.lse, None, w)


def test_overlapping_calls_with_their_own_workspaces():
    a, b = (Case(seed=s, B=2, lens=(3000, 500)) for s in (31, 32))
    want = []
    for c in (a, b):
        c.attend()
        want.append((c.O.clone(), c.lse.clone()))
        c.O.fill_(0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.attend(stream=s)
    assert status() == 0
    for c, (O, lse) in zip((a, b), want):
        assert torch.equal(c.O.view(torch.int16), O.view(torch.int16)) and torch.equal(c.lse, lse)


def test_weights_of_tiles_in_slabs():
    """max_entries so large that the sums of the tiles need more than one slab of the workspace."""
    c = Case(seed=41, Tq=64, lens=(300,), W=8, docs=[[(7 * i) % 900 for i in range(64)]])
    c.attend()
    w_in = torch.rand(c.n_pages * 64, device="cuda")
    out = torch.zeros_like(w_in)
    small = w_in.clone()
    c.weigh(c.lse, small, small, decay=0.5)
    c.max_entries = 1_300_000
    assert abi.csa2_entry_weights_workspace_size(c.dims(), c.max_entries) < 300 << 20
    c.weigh(c.lse, w_in, out, decay=0.5)
    assert status() == 0
    c.check_weights(c.lse, w_in, out, decay=0.5)
    s = torch.from_numpy(c.slots[0]).cuda()
    assert torch.equal(out[s], small[s])     # the tiles' sums are added in the same order


def test_weights_of_more_tiles_than_a_slab_holds():
    """32 tiles of 128 rows whose sums take more than twice the slab."""
    c = Case(seed=42, Tq=64, lens=(300,), W=8, docs=[[(7 * i) % 900 for i in range(64)]])
    c.attend()
    c.max_entries = 5_000_000
    assert 32 * c.max_entries * 4 > 2 * 256 << 20
    assert abi.csa2_entry_weights_workspace_size(c.dims(), c.max_entries) < 300 << 20
    w_in = torch.rand(c.n_pages * 64, device="cuda")
    out = torch.zeros_like(w_in)
    c.weigh(c.lse, w_in, out, decay=0.5)
    assert status() == 0
    c.check_weights(c.lse, w_in, out, decay=0.5)


def test_one_slot_of_a_page_at_the_end_of_a_large_pool():
    """Byte offsets past 2^32: the last page of a pool whose codes take more than 4 GB."""
    n_pages = (1 << 32) // (64 * 256) + 3
    free, _ = torch.cuda.mem_get_info()
    assert free > 6 << 30
    c = Case(seed=51, lens=(70,), W=4)
    far = n_pages - 1 - np.arange(2)
    codes = torch.empty(n_pages * 64, 256, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n_pages * 64, 32, dtype=torch.uint8, device="cuda")
    for k, page in enumerate(far):
        old = int(c.table[0, k])
        codes[page * 64:page * 64 + 64] = c.t["codes"][old * 64:old * 64 + 64]
        scales[page * 64:page * 64 + 64] = c.t["scales"][old * 64:old * 64 + 64]
    c.attend()
    O, lse = c.O.clone(), c.lse.clone()
    w = c.weigh(lse, None, torch.zeros(c.n_pages * 64, device="cuda"))
    near_slots = torch.from_numpy(c.slots[0]).cuda()
    c.t["codes"], c.t["scales"], c.n_pages = codes, scales, n_pages
    c.t["table"][0, :2] = torch.tensor(far.astype(np.int32), device="cuda")
    c.attend()
    far_w = c.weigh(lse, None, torch.zeros(n_pages * 64, device="cuda"))
    assert status() == 0
    assert torch.equal(c.O.view(torch.int16), O.view(torch.int16)) and torch.equal(c.lse, lse)
    far_slots = torch.from_numpy(far[np.arange(70) // 64] * 64 + np.arange(70) % 64).cuda()
    assert torch.equal(far_w[far_slots], w[near_slots])
