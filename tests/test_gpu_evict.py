"""Eviction against oracle.bounded: which entries leave, where the others go, and that nothing else moves."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build
from oracle import bounded as OB

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def status():
    torch.cuda.synchronize()
    return abi.csa2_get_status()


class Pool:
    def __init__(self, seed, lens, d=512, fmt="mxfp4", idx="bf16", Di=128, shift=None, weights="tail", scrambled=True,
                 room=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.d, self.fmt, self.Di, self.idx = list(lens), d, fmt, Di, idx
        B = len(lens)
        per = [(n + 63) // 64 for n in lens]
        self.n_pages = sum(per) + 2
        perm = torch.randperm(self.n_pages, generator=g)
        self.table = torch.full((B, max(max(per), 1) + room), -5, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :per[b]] = perm[at:at + per[b]].int()
            at += per[b]
        ns = self.n_pages * 64
        byte = lambda w: torch.randint(0, 256, (ns, w), dtype=torch.uint8, generator=g)  # noqa: E731
        self.codes = byte(d if fmt == "fp8" else d // 2)
        self.scales = byte(4 if fmt == "fp8" else d // 16)
        self.idx_k = byte(Di * (4 if idx == "fp32" else 2)) if idx else None
        w = torch.randn(ns, generator=g)
        if weights == "tail":
            w = torch.exp(1.5 * w)
        elif weights == "ties":
            w = torch.randint(-1, 3, (ns,), generator=g).float()
            w[torch.rand(ns, generator=g) < 0.2] = -0.0
        elif weights == "equal":
            w = torch.full((ns,), 0.5)
        self.weight = w
        self.shift = [0] * B if shift is None else list(shift)
        self.pos = torch.full((ns,), -77, dtype=torch.int32)
        self.slots = []
        for b in range(B):
            n, total = lens[b], lens[b] + self.shift[b]
            s = self.table[b, torch.arange(n) // 64].long() * 64 + torch.arange(n) % 64
            self.slots.append(s)
            ids = torch.randperm(total, generator=g)[:n] if scrambled else torch.arange(total - n, total)
            self.pos[s] = (4 * ids + 3).int()
        self.t = {k: getattr(self, k).cuda() for k in ("codes", "scales", "weight", "pos", "table")}
        self.t["idx_k"] = None if self.idx_k is None else self.idx_k.cuda()
        self.t["n"] = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.t["shift"] = torch.tensor(self.shift, dtype=torch.int32, device="cuda")

    def evict(self, keep, sink=0, recent=0, max_entries=None, stream=None, ws=None):
        p = lambda k: None if self.t[k] is None else self.t[k].data_ptr()  # noqa: E731
        m = max(self.lens) if max_entries is None else max_entries
        dm = abi.Dims(B=len(self.lens), Tq=1, d=self.d, Di=self.Di, max_pages=self.table.shape[1],
                      idx_dtype=abi.CSA2_F32 if self.idx == "fp32" else abi.CSA2_BF16,
                      kv_format=abi.CSA2_KV_FP8 if self.fmt == "fp8" else abi.CSA2_KV_MXFP4)
        c = abi.Cache(kv_codes=p("codes"), kv_scales=p("scales"), idx_k=p("idx_k"), page_table=p("table"),
                      n_entries=p("n"), n_pages=self.n_pages)
        bd = abi.Bounded(entry_pos=p("pos"), weight=p("weight"), shift=p("shift"))
        if ws is None:
            ws = torch.full((max(16, abi.csa2_evict_workspace_size(dm, m)),), 0xFF, dtype=torch.uint8, device="cuda")
        abi.csa2_evict(dm, c, bd, self.t["n"], keep, sink, recent, m, ws, stream=stream)

    def expect(self, keep, sink=0, recent=0, untouched=()):
        """Applies the oracle's moves to the host copies and compares every byte."""
        for b, n in enumerate(self.lens):
            if b in untouched or n <= keep:
                continue
            s = self.slots[b]
            holes, movers = OB.evict(self.weight[s].numpy(), self.pos[s].numpy(), self.shift[b], keep, sink, recent)
            for k in ("codes", "scales", "idx_k", "weight", "pos"):
                a = getattr(self, k)
                if a is not None:
                    a[s[holes]] = a[s[movers]].clone()
            self.shift[b] += n - keep
            self.lens[b] = keep
            self.slots[b] = s[:keep]
        assert self.t["n"].tolist() == self.lens and self.t["shift"].tolist() == self.shift
        for k in ("codes", "scales", "idx_k", "pos"):
            if getattr(self, k) is not None:
                assert torch.equal(self.t[k].cpu(), getattr(self, k)), k
        assert torch.equal(self.t["weight"].cpu().view(torch.int32), self.weight.view(torch.int32))


CASES = {
    "one_over": dict(lens=[65], keep=64),
    "keep_one": dict(lens=[1, 2, 200], keep=1),
    "step": dict(lens=[4160] * 3, keep=4096, sink=4, recent=64),
    "half": dict(lens=[3000, 2999], keep=1500, sink=16, recent=100),
    "ragged": dict(lens=[10, 0, 700, 64, 65, 5000], keep=64, sink=3, recent=20),
    "all_protected": dict(lens=[300, 301], keep=100, sink=40, recent=60),
    "ties": dict(lens=[2500, 130, 4097], keep=120, weights="ties"),
    "equal": dict(lens=[1030, 9000], keep=777, weights="equal"),
    "negative": dict(lens=[1500], keep=333, weights="normal"),
    "shifted": dict(lens=[900, 500], keep=400, sink=8, recent=50, shift=[100, 3]),
    "in_order": dict(lens=[900], keep=300, sink=8, recent=50, shift=[5], scrambled=False),
    "clusters": dict(lens=[2048, 2049, 16384, 20001], keep=2000, sink=1, recent=1),
    "past_shared_memory": dict(lens=[400000], keep=1000, sink=10, recent=10),
    "most_stay": dict(lens=[70000], keep=69000),
    "fp8": dict(lens=[500, 70], keep=60, fmt="fp8"),
    "d64_fp32_keys": dict(lens=[500, 70], keep=60, d=64, idx="fp32", Di=32),
    "no_keys": dict(lens=[500, 70], keep=60, idx=None),
}


@pytest.mark.parametrize("name", CASES)
def test_evict_matches_oracle(name):
    kw = dict(CASES[name])
    keep, sink, recent = kw.pop("keep"), kw.pop("sink", 0), kw.pop("recent", 0)
    p = Pool(len(name), **kw)
    p.evict(keep, sink, recent)
    assert status() == 0
    p.expect(keep, sink, recent)


def test_again_and_again():
    """Three evictions in a row from the same cache, the last of them with nothing to do."""
    p = Pool(3, [3000, 1200])
    for keep in (2000, 900, 900):
        p.evict(keep, 5, 30, max_entries=3000)
        assert status() == 0
        p.expect(keep, 5, 30)


def test_bad_counts_leave_the_sequence_alone():
    p = Pool(4, [300, 300, 300, 300], shift=[0, 0, -2, 0], scrambled=False)
    p.lens[0], p.lens[1] = -1, 100000
    p.t["n"][0], p.t["n"][1] = -1, 100000
    p.evict(100, max_entries=300)
    assert status() == abi.STATUS_BAD_COUNT
    lens = list(p.lens)
    p.expect(100, untouched=(0, 1, 2))
    assert p.lens == [lens[0], lens[1], lens[2], 100]


def test_count_past_the_page_table_is_refused():
    p = Pool(5, [300, 300])
    p.lens[0] = 64 * p.table.shape[1] + 1
    p.t["n"][0] = p.lens[0]
    p.evict(100, max_entries=4096)
    assert status() == abi.STATUS_BAD_COUNT
    p.expect(100, untouched=(0,))


def test_runs_of_a_captured_graph():
    p = Pool(6, [5000, 800])
    first = {k: v.clone() for k, v in p.t.items() if v is not None}
    s = torch.cuda.Stream()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(s):
        p.evict(700, 4, 64, max_entries=5000, stream=s, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        p.evict(700, 4, 64, max_entries=5000, stream=s, ws=ws)
    for _ in range(2):
        for k, v in first.items():
            p.t[k].copy_(v)
        graph.replay()
    assert status() == 0
    p.expect(700, 4, 64)
