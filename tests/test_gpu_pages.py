"""The page plan against oracle.step: pages, positions, slots, who waits, and that nothing else changes."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build
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


class Plan:
    """A pool with sequences of random lengths, on the host."""

    def __init__(self, seed, B, max_len, step, shift=False, free=None, ends=0.1, extra_held=False):
        r = np.random.RandomState(seed)
        self.len = np.round(np.exp(r.uniform(0, np.log(max_len), B))).astype(np.int64) - 1
        self.shift = np.where(r.rand(B) < 0.5, self.len // 4 // 2, 0) if shift else None
        s = self.shift if shift else 0
        self.new = r.randint(0, step + 1, B)
        u = r.rand(B)
        self.new = np.where(u < ends, 4 * s - self.len, self.new)
        self.new = np.where((u > 0.8), -np.minimum(r.randint(0, 9, B), self.len - 4 * s), self.new)
        self.max_pages = (max_len + step) // 256 + 3
        self.held = -(-(self.len // 4 - s) // 64)
        if extra_held:                                # pages taken ahead of the entries, or left behind by an eviction
            self.held = np.minimum(self.held + r.randint(0, 3, B), self.max_pages)
        self.n_free = int(self.held.sum()) // 2 + 3 if free is None else free
        self.n_pages = int(self.held.sum()) + self.n_free + 2
        perm = r.permutation(self.n_pages)
        self.table = r.randint(-9, self.n_pages + 9, (B, self.max_pages))     # anything behind the held pages
        at = 0
        for b in range(B):
            self.table[b, :self.held[b]] = perm[at:at + self.held[b]]
            at += self.held[b]
        self.free = np.full(self.n_pages, -7)
        self.free[:self.n_free] = perm[at:at + self.n_free]
        self.Tq, self.max_new = step, step // 4 + 1

    def upload(self):
        self.d = {k: i32(getattr(self, k)) for k in ("len", "new", "held", "table", "free")}
        self.d["n_free"] = i32([self.n_free])
        self.d["shift"] = i32(self.shift) if self.shift is not None else None
        B = len(self.len)
        self.dims = abi.Dims(B=B, Tq=self.Tq, max_pages=self.max_pages)
        self.pool = abi.PagePool(page_table=self.d["table"].data_ptr(), held=self.d["held"].data_ptr(),
                                 free_pages=self.d["free"].data_ptr(), n_free=self.d["n_free"].data_ptr(), n_pages=self.n_pages)
        self.out = {k: torch.full(n, -99, dtype=torch.int32, device="cuda")
                    for k, n in (("n_entries", (B,)), ("first_entry", (B,)), ("granted", (B,)), ("q_pos", (B, self.Tq)))}
        self.out["slots"] = torch.full((B, self.max_new), -99, dtype=torch.int64, device="cuda")
        self.ws = torch.full((max(16, abi.csa2_page_plan_workspace_size(self.dims)),), 0xA5, dtype=torch.uint8, device="cuda")
        return self

    def call(self, len_out=None, **kw):
        o = self.out
        args = dict(shift=self.d["shift"], q_pos=o["q_pos"], slots=o["slots"], granted=o["granted"])
        args.update(kw)
        abi.csa2_page_plan(self.dims, self.pool, self.d["len"], self.d["new"], self.d["len"] if len_out is None else len_out,
                           o["n_entries"], o["first_entry"], self.ws, **args)

    def oracle(self):
        return O.page_plan(self.len, self.new, self.held, self.table, self.free, self.n_free, self.shift, self.Tq, self.max_new)

    def check(self, ref, skip=()):
        got = {"seq_len": self.d["len"], "held": self.d["held"], "table": self.d["table"], "free": self.d["free"], **self.out}
        for k, t in got.items():
            if k not in skip:
                np.testing.assert_array_equal(t.cpu().numpy(), ref[k], err_msg=k)
        assert int(self.d["n_free"][0]) == ref["n_free"]


@pytest.mark.parametrize("B,max_len,step,shift,free,ends,extra", [
    (1, 2, 1, False, None, 0.0, False),          # one token
    (1, 300, 256, False, 0, 0.0, False),         # nothing free
    (2, 70000, 8, True, None, 0.0, True),
    (33, 5000, 8, True, 1, 0.3, True),
    (64, 3000, 700, False, 20, 0.5, False),      # the columns of two kernels
    (257, 1000, 255, True, None, 0.2, True),
    (1024, 600, 4, False, 30, 0.2, False),
    (1025, 600, 4, True, 30, 0.2, True),         # more sequences than threads
    (2500, 300, 33, True, 100, 0.4, True),
    (3, 200000, 100000, False, None, 0.3, False),
])
def test_matches_oracle(B, max_len, step, shift, free, ends, extra):
    p = Plan(B + step, B, max_len, step, shift, free, ends, extra).upload()
    ref = p.oracle()
    assert ref["bad"] == []
    p.call()
    assert status() == 0
    p.check(ref)


def test_who_waits():
    """The third sequence does not fit; the fourth would, but does not overtake; those that need nothing go on."""
    p = Plan(3, 6, 2, 4096)
    p.len, p.held = np.array([0, 100, 0, 0, 256, 3]), np.array([0, 1, 0, 0, 1, 0])
    p.new = np.array([256 * 3, 100, 256 * 9, 256, -256, 0])
    p.n_free, p.n_pages, p.max_pages = 4, 9, 16
    p.table = np.arange(6 * 16).reshape(6, 16) % 9
    p.table[1, 0], p.table[4, 0] = 7, 8
    p.free = np.array([0, 1, 2, 3, -7, -7, -7, -7, -7])
    p.upload()
    ref = p.oracle()
    assert ref["granted"].tolist() == [1, 1, 0, 0, 1, 1] and ref["n_free"] == 2
    assert ref["table"][0, :3].tolist() == [8, 3, 2]      # the released page first
    p.call()
    assert status() == 0
    p.check(ref)


def test_impossible_sequences_wait():
    p = Plan(5, 12, 3000, 64, shift=True, extra_held=False, ends=0.0)
    p.shift[:] = 0
    p.new = np.full(12, 40)
    p.held = -(-(p.len // 4) // 64)
    p.len[0] = -1
    p.len[1], p.held[1], p.new[1] = 100, 1, -101
    p.shift[2] = -1
    p.len[3], p.held[3], p.shift[3] = 400, 2, 101         # evicted more than there was
    p.len[4], p.held[4] = 1024, 3                         # fewer pages than entries
    p.held[5] = -2
    p.held[6] = p.max_pages + 1
    p.new[7] = 65                                         # more than Tq
    p.len[8], p.held[8], p.new[8] = 2 ** 31 - 10, 1, 60   # past the last position
    p.upload()
    ref = p.oracle()
    assert ref["bad"] == list(range(9)) and all(ref["granted"][9:])
    p.call()
    assert status() == abi.STATUS_BAD_COUNT
    p.check(ref)


@pytest.mark.parametrize("n_free", [-1, 10 ** 6, "too many"])
def test_impossible_pool(n_free):
    p = Plan(6, 20, 3000, 64)
    p.n_free = p.n_pages - 1 if n_free == "too many" else n_free
    p.new[:] = 8
    p.new[3] = -p.len[3]
    p.len[3], p.held[3], p.new[3] = 800, 4, -800
    p.upload()
    ref = p.oracle()
    assert ref["bad"] == "pool"
    p.call()
    assert status() == abi.STATUS_BAD_COUNT
    p.check(ref)


def test_bad_page_ids_get_no_slot():
    p = Plan(7, 4, 1000, 300, free=30, ends=0.0)
    p.new[:] = 300
    p.free[p.n_free - 1], p.free[p.n_free - 2] = -3, p.n_pages
    p.upload()
    ref = p.oracle()
    p.call()
    assert status() == abi.STATUS_BAD_PAGE
    p.check(ref)


def test_outputs_that_are_not_wanted():
    p = Plan(8, 50, 2000, 64).upload()
    ref = p.oracle()
    after = torch.full((50,), -5, dtype=torch.int32, device="cuda")
    before = p.d["len"].clone()
    p.call(len_out=after, q_pos=None, slots=None, granted=None)
    assert status() == 0
    np.testing.assert_array_equal(after.cpu().numpy(), ref["seq_len"])
    assert torch.equal(p.d["len"], before)
    p.check({**ref, "seq_len": p.len}, skip=("q_pos", "slots", "granted"))
    for k in ("q_pos", "slots", "granted"):
        assert bool((p.out[k] == -99).all())


def test_many_steps_give_every_page_back():
    """A pool in use for 60 steps: no page is held twice or lost, and the plan equals the oracle's at every step."""
    r = np.random.RandomState(1)
    p = Plan(9, 40, 2, 64)
    p.len[:], p.held[:], p.shift = 0, 0, np.zeros(40, dtype=np.int64)
    p.n_pages, p.n_free, p.max_pages, p.Tq, p.max_new = 60, 60, 20, 200, 51
    p.table, p.free = np.zeros((40, 20), dtype=np.int64), r.permutation(60)
    p.upload()
    waited = 0
    for _ in range(60):
        p.new = np.where(r.rand(40) < 0.15, 4 * p.shift - p.len, r.randint(-5, 200, 40))
        p.new = np.maximum(p.new, 4 * p.shift - p.len)
        p.new = np.minimum(p.new, 20 * 256 + 4 * p.shift - p.len)
        p.d["new"].copy_(i32(p.new))
        p.d["shift"].copy_(i32(p.shift))
        ref = p.oracle()
        assert ref["bad"] == []
        p.call()
        p.check(ref)
        waited += int((ref["granted"] == 0).sum())
        p.len, p.held, p.table, p.free, p.n_free = (ref[k] for k in ("seq_len", "held", "table", "free", "n_free"))
        pages = np.concatenate([p.free[:p.n_free]] + [p.table[b, :p.held[b]] for b in range(40)])
        assert sorted(pages.tolist()) == list(range(60))
        cut = r.rand(40) < 0.1                          # entries evicted between the steps
        p.shift = np.where(cut, p.shift + (p.len // 4 - p.shift) // 2, p.shift)
    assert status() == 0 and waited > 20


@pytest.mark.parametrize("step", [8, 700])
def test_captured_and_replayed(step):
    """Two plans with pools and workspaces of their own in one graph, on two streams at once."""
    ps = [Plan(20 + k, 60, 3000, step, shift=True).upload() for k in range(2)]
    refs = [p.oracle() for p in ps]
    start = [{k: v.clone() for k, v in p.d.items()} for p in ps]
    side = [torch.cuda.Stream() for _ in ps]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for p, s in zip(ps, side):
            s.wait_stream(main)
            with torch.cuda.stream(s):
                p.call()
            main.wait_stream(s)
    for _ in range(3):
        for p, st in zip(ps, start):
            for k, v in st.items():
                p.d[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for p, ref in zip(ps, refs):
            p.check(ref)
    assert status() == 0
