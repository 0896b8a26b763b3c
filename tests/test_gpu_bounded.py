"""Attention over the whole cache and the entries' weights against oracle.bounded."""
import numpy as np
import pytest
import torch

from bounded_case import SENTINEL, Case
from compressed_sparse_attention_05_gb300 import abi, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def status():
    torch.cuda.synchronize()
    return abi.csa2_get_status()


CASES = {
    # one token: no entry, no key at all, one entry, page and tile edges
    "empty_window_only": dict(lens=(0,)),
    "nothing_visible": dict(lens=(0,), window=False),
    "one_entry": dict(lens=(1,), W=1),
    "edges_63_64_65": dict(B=3, lens=(63, 64, 65)),
    "edges_127_128_129": dict(B=3, lens=(127, 128, 129), W=16),
    "edges_255_257": dict(B=2, lens=(255, 257), window=False),
    "split_long": dict(lens=(5001,)),
    "ragged": dict(B=5, lens=(1, 700, 0, 64, 3000)),
    # several chunks for every SM, tiles that begin and end inside an SM's share
    "many_chunks": dict(B=3, Tq=96, lens=(1500, 1100, 77)),
    "one_long": dict(lens=(150000,)),
    # heads and tokens
    "hq1": dict(Tq=70, Hq=1, lens=(300,), W=20),
    "hq8_tokens": dict(B=2, Tq=11, Hq=8, lens=(400, 90)),
    "hq40_tokens": dict(B=2, Tq=5, Hq=40, lens=(333,)),
    "hq65": dict(Tq=3, Hq=65, lens=(200,)),
    "hq128": dict(B=2, Tq=2, Hq=128, lens=(150, 640)),
    "prompt_from_zero": dict(Tq=256, Hq=16, lens=(64,), q_pos=list(range(256)), W=32),
    "window_1024": dict(Tq=2, lens=(900,), W=1024),
    # scores and masks
    "cap": dict(B=2, lens=(500,), cap=2.0, q_scale=3.0),
    "cap_small_logits": dict(lens=(300,), cap=50.0, q_scale=0.05),
    "cap_saturated": dict(lens=(300,), cap=5.0, q_scale=30.0),
    "slopes": dict(B=2, Tq=2, lens=(1500, 40), slopes=[0.5, 0.01, 0.0, 2.0 ** -8]),
    "slopes_cap_hq8": dict(Tq=9, Hq=8, lens=(700,), slopes=[1.0, 0.003], cap=30.0),
    "docs": dict(B=2, Tq=4, Hq=16, lens=(300,), W=64, docs=[[0, 41, 1198, 1200], [7, 7, 800, 1203]]),
    "docs_hide_all": dict(Tq=3, Hq=32, lens=(100,), window=False, docs=[[400, 0, 4000]]),
    "prefix": dict(B=2, Tq=64, Hq=8, lens=(40,), q_pos=[list(range(100, 164))] * 2, prefix=[130, 3], W=16),
    "prefix_slopes": dict(Tq=8, Hq=64, lens=(64,), q_pos=[list(range(200, 208))], prefix=[256], slopes=[0.02]),
    "shifted": dict(B=2, Tq=3, lens=(200, 333), shift=[50, 7]),
    "shifted_docs": dict(Tq=2, Hq=40, lens=(300,), shift=[50], docs=[[333, 800]], W=8),
    "scrambled": dict(B=2, Tq=3, Hq=40, lens=(200, 333), shift=[50, 1], scrambled=True, slopes=[0.01, 0.2]),
    "scrambled_docs": dict(Tq=2, Hq=64, lens=(260,), shift=[30], scrambled=True, docs=[[300, 801]], W=8),
    "tokens_far_apart": dict(Tq=4, Hq=8, lens=(600,), q_pos=[[40, 700, 1500, 2403]], W=16),
    "before_the_first_token": dict(B=2, Tq=2, Hq=16, lens=(80,), q_pos=[[-1, 0], [-7, 320]], W=4),
    # values
    "large_q": dict(lens=(300,), q_scale=3e4, tau=1e-6),
    "large_k": dict(lens=(300,), k_scale=300.0, tau=1e-3),
    "peaked": dict(lens=(2000,), q_scale=40.0),
}
SMALL = {"d64_" + k: dict(CASES[k], d=64) for k in ("empty_window_only", "nothing_visible", "ragged", "hq40_tokens",
                                                   "docs", "prefix", "scrambled", "slopes_cap_hq8")}
ALL = {**CASES, **SMALL}


@pytest.mark.parametrize("name", ["one_long", "many_chunks"])
def test_repeated_calls_give_the_same_bits(name):
    """No result depends on which copy, product or warp was first."""
    c = Case(seed=5, **CASES[name])
    O, lse = (t.clone() for t in c.attend())
    w = c.weigh(lse, None, torch.zeros(c.n_pages * 64, device="cuda")).clone()
    for _ in range(30):
        c.attend()
        again = c.weigh(lse, None, torch.zeros(c.n_pages * 64, device="cuda"))
        assert torch.equal(c.O.view(torch.int16), O.view(torch.int16)) and torch.equal(c.lse, lse)
        assert torch.equal(again, w)
    assert status() == 0


@pytest.mark.parametrize("name", ALL)
def test_attention_matches_oracle(name):
    c = Case(seed=len(name) * 7 + 1, **ALL[name])
    c.attend()
    assert status() == 0
    c.check_attention([(0, 0), (0, 95), (1, 40), (2, 0), (2, 1), (2, 95)] if name == "many_chunks" else None)


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
def test_weights_match_oracle(name, in_place):
    c = Case(seed=len(name) * 5 + 2, **ALL[name])
    c.attend()
    g = torch.Generator().manual_seed(9)
    w_in = torch.rand(c.n_pages * 64, generator=g).cuda()
    foreign = torch.ones(c.n_pages * 64, dtype=torch.bool)
    for s in c.slots:
        foreign[s] = False
    w_in[foreign.cuda()] = SENTINEL
    before = w_in.clone()
    out = w_in if in_place else torch.full_like(w_in, SENTINEL)
    c.weigh(c.lse, w_in, out, decay=0.75)
    assert status() == 0
    owned = c.check_weights(c.lse, before, out, decay=0.75)
    assert torch.all(out.cpu()[torch.from_numpy(~owned)] == SENTINEL)   # slots of nobody stay as they were


def test_weights_without_input_and_sum_rule():
    """Every row's weights over entries and window add up to one, so without a window the entries' sum is the
    number of rows."""
    c = Case(seed=3, B=2, Tq=3, lens=(500, 33), window=False)
    c.attend()
    out = torch.zeros(c.n_pages * 64, device="cuda")
    c.weigh(c.lse, None, out)
    assert status() == 0
    c.check_weights(c.lse, None, out)
    total = float(out.double().sum())
    assert abs(total - 2 * 3 * 64) < 2 * 3 * 64 * 1e-4


def test_max_entries_bounds_what_is_read():
    """More entries than max_entries: flagged, and only the first max_entries are read and written."""
    c = Case(seed=4, B=2, lens=(300, 20), max_entries=200)
    c.attend()
    assert status() == abi.STATUS_BAD_COUNT
    c.q_pos = c.q_pos.copy()
    c.check_attention()
    out = torch.full((c.n_pages * 64,), SENTINEL, device="cuda")
    c.weigh(c.lse, None, out)
    assert status() == abi.STATUS_BAD_COUNT
    owned = c.check_weights(c.lse, None, out)
    assert torch.all(out.cpu()[torch.from_numpy(~owned)] == SENTINEL)


def test_bad_pages_hide_their_entries():
    c = Case(seed=5, B=1, lens=(640,))
    for page, bad in ((2, -1), (5, c.n_pages), (9, 1 << 30)):
        c.t["table"][0, page] = bad
    hidden = [j for p in (2, 5, 9) for j in range(64 * p, 64 * p + 64)]
    c.attend()
    assert status() == abi.STATUS_BAD_PAGE
    seen = c.seen
    c.seen = lambda b, i, pos: np.setdiff1d(seen(b, i, pos), hidden)
    c.check_attention()
    out = torch.full((c.n_pages * 64,), SENTINEL, device="cuda")
    c.weigh(c.lse, None, out)
    assert status() == abi.STATUS_BAD_PAGE
    keep = np.setdiff1d(np.arange(640), hidden)
    got = out.cpu().numpy()
    assert np.all(got[c.slots[0][hidden]] == SENTINEL) and np.all(got[c.slots[0][keep]] != SENTINEL)


def test_infinite_lse_rows_add_nothing():
    c = Case(seed=6, Tq=2, Hq=8, lens=(90,), window=False)
    c.attend()
    lse = c.lse.clone()
    lse[0, 0, 3] = float("inf")
    lse[0, 1, :] = float("-inf")
    out = torch.zeros(c.n_pages * 64, device="cuda")
    c.weigh(lse, None, out)
    assert status() == 0
    c.check_weights(lse, None, out)


@pytest.mark.parametrize("kw", [dict(B=3, lens=(4000, 90, 1300)), dict(Tq=40, Hq=24, lens=(700,), cap=20.0)],
                         ids=["decode", "chunk"])
def test_runs_give_the_same_bits(kw):
    c = Case(seed=7, **kw)
    c.attend()
    O, lse = c.O.clone(), c.lse.clone()
    w = torch.zeros(c.n_pages * 64, device="cuda")
    c.weigh(lse, None, w)
    first = w.clone()
    for _ in range(3):
        c.O.fill_(float("nan"))
        c.attend()
        c.weigh(lse, None, w)
        assert torch.equal(c.O.view(torch.int16), O.view(torch.int16)) and torch.equal(c.lse, lse)
        assert torch.equal(w, first)
    assert status() == 0


@pytest.mark.parametrize("entries", [0, 70])
def test_rows_that_no_token_sees_near_the_largest_position(entries):
    """A tile with fewer rows than it has room for, positions up to 2^31 - 2: window rows between the tokens'
    windows hold NaN and must not be taken for visible ones."""
    top = 2 ** 31 - 2
    c = Case(seed=8, Tq=2, Hq=8, lens=(entries,), W=8, q_pos=[[top - 18, top]], docs=[[0, top]])
    hidden = [int(p - c.pos0[0]) for p in range(top - 17, top)]
    c.t["wscales"][0, hidden] = float("nan")
    c.t["wcodes"][0, hidden] = 0x7F
    c.attend()
    assert status() == 0
    c.check_attention()


@pytest.mark.parametrize("d", [512, 64])
@pytest.mark.parametrize("bad", ["entry", "window_scale", "window_code"])
def test_nan_keys_reach_only_the_tokens_that_see_them(d, bad):
    """Two tokens of one tile: a key with a NaN that the first sees and the second does not."""
    if d == 64 and bad != "entry":
        pytest.skip("the plain kernel reads only the window rows that its token sees")
    c = Case(seed=9, Tq=2, Hq=8, d=d, lens=(300,), W=16, q_pos=[[1170, 1199]], docs=[[0, 1180]])
    if bad == "entry":
        c.t["scales"][int(c.slots[0][200]), 1] = 0x7F
        c.t["scales"][int(c.slots[0][201]), 2] = 0xFF
    elif bad == "window_scale":
        c.t["wscales"][0, 1165 - int(c.pos0[0])] = float("nan")
        c.t["wscales"][0, 1166 - int(c.pos0[0])] = float("inf")
    else:
        c.t["wcodes"][0, 1165 - int(c.pos0[0]), 5] = 0x7F
        c.t["wcodes"][0, 1165 - int(c.pos0[0]), 400] = 0xFF
    c.attend()
    assert status() == 0
    assert c.lse[0, 0].isnan().all() and c.O[0, 0].isnan().any()   # the first token's result says so
    c.check_attention([(0, 1)])
    out = torch.zeros(c.n_pages * 64, device="cuda")
    c.weigh(torch.where(c.lse.isfinite(), c.lse, float("inf")), None, out)
    assert status() == 0
    visible = torch.from_numpy(c.slots[0][295:]).cuda()   # of the second token's document: finite
    assert out[visible].isfinite().all() and (out[visible] > 0).all()
