"""Calls at the edges of what the entry points of a bounded cache accept."""
import pytest
import torch

from bounded_case import SENTINEL, Case
from compressed_sparse_attention_05_gb300 import abi, build
from test_gpu_bounded_use import Cache
from test_gpu_evict import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def status():
    torch.cuda.synchronize()
    return abi.csa2_get_status()


@pytest.mark.parametrize("d", [512, 64])
def test_no_query_tokens_leave_the_weights(d):
    c = Case(seed=21, Tq=1, Hq=8, d=d, lens=(90,))
    dm = c.dims()
    dm.Tq = 0
    cache, bounded, _, mods = c.structs()
    w_in = torch.rand(c.n_pages * 64, device="cuda")
    out = torch.full_like(w_in, SENTINEL)
    launches = abi.lib().csa2_launch_count()
    abi.csa2_entry_weights(dm, cache, None, None, None, c.tau, 0.5, w_in, out, 90, None, mods=mods, bounded=bounded)
    assert status() == 0
    assert abi.lib().csa2_launch_count() == launches and torch.all(out == SENTINEL)


def test_a_token_at_the_most_negative_position_sees_no_window():
    """In one tile with a token at the largest position, from which t - p wraps around."""
    top = 2 ** 31 - 1
    c = Case(seed=22, Tq=2, Hq=8, lens=(0,), W=8, q_pos=[[top - 3, top]])
    c.q_pos[0, 0] = -2 ** 31
    c.t["q_pos"][0, 0] = -2 ** 31
    c.attend()
    assert status() == 0
    assert not c.O[0, 0].any() and torch.all(c.lse[0, 0] == float("-inf"))
    c.check_attention([(0, 1)])


def test_entries_whose_position_does_not_fit_are_not_written():
    """Sequence 0's last 20 entries would lie past position 2^31 - 1; sequence 1's shift is negative."""
    c = Cache(23)
    c.t["shift"].copy_(torch.tensor([2 ** 29 - 40, -3], dtype=torch.int32))
    c.t["n"].copy_(torch.tensor([10, 64], dtype=torch.int32))
    names = ("codes", "scales", "pos")
    before = [c.t[k].clone() for k in names] + [c.idx_k.clone(), c.weight.clone()]
    c.compress(50)
    assert status() == abi.STATUS_BAD_COUNT
    wrote = torch.from_numpy(c.page_slots[0][10:40]).cuda()
    assert c.t["pos"][wrote].tolist() == [4 * (2 ** 29 - 40 + e) + 3 for e in range(10, 40)]
    assert not c.weight[wrote].any() and not torch.equal(c.t["codes"][wrote], before[0][wrote])
    rest = torch.ones(c.n_pages * 64, dtype=torch.bool, device="cuda")
    rest[wrote] = False
    for now, old in zip([c.t[k] for k in names] + [c.idx_k, c.weight], before):
        assert torch.equal(now[rest], old[rest])


@pytest.mark.parametrize("lens,keep,page", [([300, 280], 200, 0), ([300, 280], 200, 4), ([9000, 20000], 5000, 60)],
                         ids=["below_keep", "above_keep", "cluster"])
def test_a_bad_page_leaves_the_sequence_alone(lens, keep, page):
    """No survivor may be lost to a hole that cannot be written."""
    p = Pool(24, lens)
    p.t["table"][0, page] = p.n_pages
    p.evict(keep, 4, 10)
    assert status() == abi.STATUS_BAD_PAGE
    p.expect(keep, 4, 10, untouched=(0,))
    assert p.lens == [lens[0], keep]
