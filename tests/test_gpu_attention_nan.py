"""A NaN among the keys that a token sees: its outputs and its lse are NaN, whatever the keys' split over CTAs, and no
other's."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build
from test_gpu_tree import Case, i32, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


@pytest.mark.parametrize("kw", [dict(lens=[300], T=4, K=64), dict(lens=[3000], T=4, K=1024), dict(lens=[0], T=4, K=1),
                                dict(lens=[300] * 50, T=4, K=64), dict(lens=[300], T=4, K=64, d=64, Hq=7), dict(lens=[0], T=4, K=1, d=64, Hq=7),
                                dict(lens=[400], T=4, K=200, fp8=True)])
def test_a_nan_row(kw):
    c = Case(31, **kw)
    c.parent[0] = [-1, -1, 0, 1]                       # two branches
    c.upload()
    c.run()
    whole, lse = c.O.clone(), c.lse.clone()
    c.t["ns"][1] = float("nan")                        # node 1's row: seen by 1 and 3
    c.run()
    assert status() == 0
    for i in (1, 3):
        assert bool(c.O[0, i].isnan().all()) and bool(c.lse[0, i].isnan().all()), i
    c.O[0, [1, 3]], whole[0, [1, 3]] = 0, 0
    c.lse[0, [1, 3]], lse[0, [1, 3]] = 0, 0
    assert torch.equal(c.O, whole) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("d", [512, 64])
def test_a_nan_head(d):
    """A NaN in one head's query stays in that head."""
    c = Case(32, lens=[500], T=3, K=128, Hq=9, d=d).upload()
    c.run()
    whole, lse = c.O.clone(), c.lse.clone()
    c.t["Q"][0, 1, 4, 17] = float("nan")
    c.run()
    assert status() == 0
    assert bool(c.O[0, 1, 4].isnan().all()) and bool(c.lse[0, 1, 4].isnan())
    c.O[0, 1, 4], whole[0, 1, 4], c.lse[0, 1, 4], lse[0, 1, 4] = 0, 0, 0, 0
    assert torch.equal(c.O, whole) and torch.equal(c.lse, lse)


def test_no_key_is_no_nan():
    c = Case(33, lens=[0], T=2, K=1, W=0, rest=[0]).upload()
    c.run()
    assert status() == 0
    assert bool((c.O == 0).all()) and bool(c.lse.isneginf().all())
    assert not np.isnan(c.lse.cpu().numpy()).any()


@pytest.mark.parametrize("kw", [dict(lens=[300, 20], T=4, K=64), dict(lens=[300] * 45, T=4, K=64), dict(lens=[300, 20], T=4, K=64, d=64, Hq=7)])
@pytest.mark.parametrize("where", ["row", "head"])
def test_sparse_attention(where, kw):
    """The same without a tree: a window row of NaN, a head of NaN."""
    c = Case(34, chain=True, **kw).upload()
    B, T, d = len(kw["lens"]), 4, c.d
    q_pos = i32(c.ctx[:, None] - T + np.arange(T))
    Of, lf = torch.empty(B, T, c.Hq, d, device="cuda"), torch.empty(B, T, c.Hq, device="cuda")
    go = lambda: abi.csa2_sparse_attn(c.dims, c.cache, c.window, c.t["Q"], q_pos, c.t["idx"], c.t["cnt"], c.tau, Of, lf)  # noqa: E731
    c.t["cnt"].fill_(1)                                # (the first entry: visible to all of these)
    c.t["idx"].fill_(0)
    go()
    whole, lse = Of.clone(), lf.clone()
    assert bool(whole.isfinite().all()) and bool(lse.isfinite().all())
    if where == "row":                                 # the row of token 2's position: seen by 2 and 3
        c.t["ws"][int(q_pos[0, 2]) - int(c.pos0[0])] = float("nan")
        bad = (0, [2, 3])
    else:
        c.t["Q"][0, 1, 2, 5] = float("nan")
        bad = (0, 1, 2)
    go()
    assert status() == 0
    assert bool(Of[bad].isnan().all()) and bool(lf[bad].isnan().all())
    Of[bad], whole[bad], lf[bad], lse[bad] = 0, 0, 0, 0
    assert torch.equal(Of, whole) and torch.equal(lf, lse)
