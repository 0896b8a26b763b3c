"""Calls at the edges of what the entry points of a bounded cache accept."""
import pytest
import torch

from bounded_case import Case
from compressed_sparse_attention_05_gb300 import abi, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def status():
    torch.cuda.synchronize()
    return abi.csa2_get_status()


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
