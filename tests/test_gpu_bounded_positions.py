"""What a token sees of a cache that entries were evicted from: the entries whose last token is at or before it,
wherever they lie."""
import numpy as np
import pytest
import torch

from bounded_case import SENTINEL, Case
from compressed_sparse_attention_05_gb300 import abi, build
from oracle import bounded as OB
from test_gpu_bounded_use import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def status():
    torch.cuda.synchronize()
    return abi.csa2_get_status()


class ByPosition(Case):
    """A Case whose expected values know an entry only by its position."""

    def seen(self, b, i, pos):
        j = OB.visible(pos, int(self.q_pos[b, i]), self.prefix[b] if self.prefix else 0)
        return j[pos[j] - 3 >= self.docs[b, i]] if self.docs is not None else j


class InUse(ByPosition, Cache):
    pass


CASES = {
    "last_tokens": dict(B=2, Tq=3, Hq=40, lens=(200, 333), shift=[50, 1], slopes=[0.01, 0.2]),
    "last_tokens_docs": dict(Tq=2, Hq=64, lens=(260,), shift=[30], docs=[[300, 801]], W=8),
    "one_token": dict(B=3, lens=(200, 65, 1000), shift=[10, 0, 777]),
    "older_tokens": dict(Tq=5, Hq=64, lens=(250,), shift=[50], q_pos=[[2, 3, 400, 900, 1199]], window=False),
    "older_tokens_hq8": dict(B=2, Tq=40, Hq=8, lens=(700, 90), shift=[100, 4], W=16),
    "hq128": dict(Tq=3, Hq=128, lens=(300,), shift=[20]),
    "prefix": dict(B=2, Tq=6, Hq=16, lens=(180,), shift=[20], prefix=[798, 40], q_pos=[list(range(787, 793))] * 2),
    "cap_one_head": dict(Tq=70, Hq=1, lens=(300,), shift=[12], cap=20.0, W=20),
    "before_the_first_token": dict(Tq=3, Hq=16, lens=(80,), shift=[5], q_pos=[[-1, 0, 339]], W=4),
    "many_chunks": dict(B=2, Tq=48, lens=(1500, 1100), shift=[300, 30]),
}
CASES.update({"d64_" + k: dict(CASES[k], d=64) for k in ("last_tokens", "last_tokens_docs", "older_tokens", "prefix")})


@pytest.mark.parametrize("name", CASES)
def test_attention_goes_by_position(name):
    c = ByPosition(seed=len(name) * 3 + 2, scrambled=True, **CASES[name])
    c.attend()
    assert status() == 0
    c.check_attention([(0, 0), (0, 47), (1, 20), (1, 47)] if name == "many_chunks" else None)


@pytest.mark.parametrize("name", CASES)
def test_weights_go_by_position(name):
    c = ByPosition(seed=len(name) * 3 + 3, scrambled=True, **CASES[name])
    c.attend()
    w_in = torch.rand(c.n_pages * 64, generator=torch.Generator().manual_seed(9)).cuda()
    out = torch.full_like(w_in, SENTINEL)
    c.weigh(c.lse, w_in, out, decay=0.75)
    assert status() == 0
    assert out.isfinite().all()
    owned = c.check_weights(c.lse, w_in, out, decay=0.75)
    assert torch.all(out.cpu()[torch.from_numpy(~owned)] == SENTINEL)


@pytest.mark.parametrize("d", [512, 64])
def test_drafted_tokens_right_after_an_eviction(d):
    """Compress, evict, then attend and weigh with tokens older than the newest entry, which may have moved."""
    c = InUse(31, Tq=8, Hq=24, d=d)
    c.compress(150)
    c.weight.copy_(torch.rand(c.weight.shape, generator=torch.Generator().manual_seed(32)))
    c.evict(120, 4, 16)
    assert status() == 0
    c.pull()
    assert c.lens == [120, 120] and c.shift == [30, 30]
    moved = [int(np.argmax(c.entry_pos[c.slots[b]].numpy())) for b in range(2)]
    assert min(moved) < 119                      # the newest entry lies in a hole
    c.q_pos = np.tile(np.arange(592, 600), (2, 1))
    c.t["q_pos"].copy_(torch.tensor(c.q_pos, dtype=torch.int32))
    c.attend()
    assert status() == 0
    c.check_attention()
    out = torch.zeros(c.n_pages * 64, device="cuda")
    c.weigh(c.lse, None, out)
    assert status() == 0 and out.isfinite().all()
    c.check_weights(c.lse, None, out)
    # a token's result does not change with what comes after it
    O, lse = c.O.clone(), c.lse.clone()
    for b in range(2):
        late = c.entry_pos[c.slots[b]].numpy() > 594
        c.t["scales"][torch.from_numpy(c.slots[b][late]).cuda()] = 0x7F
    c.attend()
    assert torch.equal(c.O[:, :3].view(torch.int16), O[:, :3].view(torch.int16)) and torch.equal(c.lse[:, :3], lse[:, :3])
